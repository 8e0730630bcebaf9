"""Cosine and sine that the kernels turn by, against whole-number products of the position and the stored fraction of a turn."""
import math

import pytest
import torch

import gated_deltanet_linear_spec_gb300 as gdn
from tests.test_gpu_attention import i32

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, -1, 2, 1000, 8191, 65536, 1000003, -999983, 4194301, 1 << 30, (1 << 31) - 1, -(1 << 31), 123456789, -987654321]


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("base", [10000.0, 10000000.0])
def test_the_angle_is_exact_modulo_a_turn(base, interleaved):
    """(1, 0) turns to (cos, sin): off by 2^-23 at most -- a rounding by 2^-33 of a turn, one to fp32 of at most an eighth of a turn
    (pi / 4 2^-24) and one step of fp32 below 1 in sincospi (2^-24)."""
    rope = gdn.Rope(128, base=base, layout=gdn.GDN_ROPE_INTERLEAVED if interleaved else gdn.GDN_ROPE_HALF)
    x = torch.zeros(len(POSITIONS), 1, 128)
    x[..., 0::2 if interleaved else 1][..., :64] = 1.0
    out = torch.empty_like(x, device="cuda")
    gdn.gdn_rope(rope, i32(POSITIONS), x.cuda(), out)
    out = out.cpu().double()
    cos, sin = (out[..., 0::2], out[..., 1::2]) if interleaved else (out[..., :64], out[..., 64:])
    for t, p in enumerate(POSITIONS):
        for i, f in enumerate(rope.turns.tolist()):
            angle = p * f % (1 << 64) / 2.0 ** 64 * 2 * math.pi
            for got, want in ((cos[t, 0, i], math.cos(angle)), (sin[t, 0, i], math.sin(angle))):
                assert abs(float(got) - want) <= 2.0 ** -23, (p, i)
