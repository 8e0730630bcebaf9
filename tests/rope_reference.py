"""Rotary positions in 64 bits, written from the formulas.  Test infrastructure only."""
import math

import torch

import gated_deltanet_linear_spec_gb300 as gdn


def frequencies(rotary, base=10000.0, scaling=gdn.GDN_ROPE_PLAIN, factor=1.0, original=4096.0, low=1.0, high=None):
    """(radians a position of each pair, magnitude), as Python floats."""
    out = []
    high = high or (32.0 if scaling == gdn.GDN_ROPE_RAMP else 4.0)
    if scaling == gdn.GDN_ROPE_NTK and rotary > 2:
        base = base * factor ** (rotary / (rotary - 2.0))
    for i in range(rotary // 2):
        f = base ** (-2.0 * i / rotary)
        if scaling == gdn.GDN_ROPE_LINEAR:
            f = f / factor
        if scaling == gdn.GDN_ROPE_BANDS:
            turns = original * f / (2 * math.pi)
            w = 1.0 if turns >= high else 0.0 if turns <= low else (turns - low) / (high - low)
            f = w * f + (1 - w) * f / factor
        if scaling == gdn.GDN_ROPE_RAMP:
            def pair(turns):
                return rotary * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rotary - 1)
            w = 1.0 - min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = w * f + (1 - w) * f / factor
        out.append(f)
    return out, 0.1 * math.log(factor) + 1.0 if scaling == gdn.GDN_ROPE_RAMP else 1.0


def turn(x, positions, freqs, magnitude, interleaved):
    """(out, tol) in 64 bits on the CPU: x [tokens, heads, d] turned, and how far a kernel's result may be off.

    A fraction of a turn is rounded to 2^-33 turns (2 pi 2^-33 radians) and, as at most a quarter of a half turn, to fp32
    (pi / 4 2^-24); sine and cosine are off by a step of fp32 below 1 (2^-24) and once more by the magnitude's product
    (2^-24): 3 2^-24 of the magnitude in all (2.8 of it used; the table's units of 2^-64 turns, 2 pi 2^-65 2^31 radians at the
    farthest position, are 0.01 more).  The table and the 64-bit reference hold frequencies to 2^-51 relative
    each, which positions multiply: 2^-50 of the angle.  x c - y s then rounds y s (2^-24 of it at most) and the sum."""
    x64, out = x.double().cpu(), x.double().cpu().clone()
    half = torch.finfo(x.dtype).eps / 2
    moved = torch.zeros_like(out)
    p = torch.tensor([int(v) for v in positions], dtype=torch.float64)
    r = 2 * len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        c, s = (magnitude * torch.cos(p * f))[:, None], (magnitude * torch.sin(p * f))[:, None]
        u, v = x64[..., a], x64[..., b]
        out[..., a], out[..., b] = u * c - v * s, v * c + u * s
        off = (u.abs() + v.abs()) * abs(magnitude) * (4 * 2.0 ** -24 + (p.abs() * f)[:, None] * 2.0 ** -50)
        moved[..., a], moved[..., b] = off, off
    tol = moved + out.abs() * half * 1.01 + 1e-30
    tol[..., r:] = 0.0
    return out, tol
