"""The operators of the paged key-value cache: what is timed, and their plain forms.

Three operators of the full-attention layers that sit between the GDN layers of a hybrid model:
  attend  attention of the new tokens of decode, verify and prompt rows over the paged cache
          (causal; optionally a sliding window with a few first tokens that stay visible);
  append  the new tokens' keys and values written into the rows' pages;
  pages   page management on the device: "fork" drops the rows of a search's losing branches,
          forks the winners and makes room for their next tokens; "compact" moves the live pages
          of a fragmented pool to its front.
With ``own`` false ``run`` computes them with elementary torch operations in 32 bits; with ``own``
true it calls the framework.  ``exact`` follows the definitions in 64 bits, row by row.
"""
import math
import random

import torch

own = False

GOLD = 0.6180339887498949
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attend(name, **kw):
    case = {"name": name, "op": "attend", "rows": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 1, "kv_hi": 1, "heads": 32,
            "kv_heads": 4, "dim": 128, "page": 16, "window": 0, "sinks": 0, "gather": False, "fused": False,
            "dtype": "bf16"}
    case.update(kw)
    return case


def listed():
    return [
        # one stream, one new token: the latency of a single call
        _attend("decode_one", kv_lo=777, kv_hi=777, heads=16, kv_heads=2),
        # 64 one-token rows, the framework's decode batch, over ragged contexts
        _attend("decode_64", rows=64, kv_lo=512, kv_hi=8192),
        # 64 rows of 3 drafts + 1, the framework's verify batch, q inside a fused q|k|v projection, tokens interleaved
        _attend("verify_64x4", rows=64, q_lo=4, q_hi=4, kv_lo=1000, kv_hi=16384, page=64, gather=True, fused=True),
        # a few very long contexts: the cache's length has to be split
        _attend("decode_long", rows=4, kv_lo=65536, kv_hi=131072, heads=16, kv_heads=2, dim=256, page=128),
        # ragged verify rows of up to 4 drafts + 1 under a sliding window whose old pages were released
        _attend("verify_window", rows=128, q_lo=1, q_hi=5, kv_lo=300, kv_hi=32768, heads=16, kv_heads=8, dim=64,
                page=32, window=1000, sinks=4, gather=True),
        # the framework's 32-bit activations: 2 drafts + 1
        _attend("verify_f32", rows=24, q_lo=3, q_hi=3, kv_lo=64, kv_hi=4096, heads=8, kv_heads=2, dim=64, dtype="f32"),
        # one 8192-token prompt, the framework's long row
        _attend("prompt_8192", q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, page=64, fused=True),
        # prompt pieces continuing earlier context, odd lengths, windowed
        _attend("prompts_window", rows=3, q_lo=333, q_hi=1024, kv_lo=1500, kv_hi=6001, heads=16, kv_heads=2, dim=256,
                window=2048, sinks=16),
        # the verify batch's new tokens into their pages
        {"name": "append_64x4", "op": "append", "rows": 64, "q_lo": 4, "q_hi": 4, "kv_lo": 100, "kv_hi": 2048,
         "kv_heads": 4, "dim": 128, "page": 16, "gather": True, "dtype": "bf16"},
        # the long prompt's tokens into its pages
        {"name": "append_prompt", "op": "append", "rows": 1, "q_lo": 8192, "q_hi": 8192, "kv_lo": 8192, "kv_hi": 8192,
         "kv_heads": 8, "dim": 128, "page": 64, "gather": False, "dtype": "bf16"},
        # a search step: 16 winners of 4 branches each, the losers' pages given back first
        {"name": "fork_16x4", "op": "fork", "parents": 16, "children": 4, "kv_lo": 200, "kv_hi": 8192, "grow": 64,
         "kv_heads": 4, "dim": 128, "page": 64, "dtype": "bf16"},
        # a pool whose finished rows left every other page free
        {"name": "compact_half", "op": "compact", "rows": 96, "kv_lo": 64, "kv_hi": 6000, "live": 0.5, "kv_heads": 4,
         "dim": 128, "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    return max(lo, min(hi, _log(rng, lo, hi)))


def draw(rng: random.Random):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    kind = rng.choice(["decode", "verify", "verify", "prompt", "append", "fork", "compact"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if kind in ("decode", "verify"):
        f32 = rng.random() < 0.15
        group = rng.choice([1, 2, 4, 8])
        rows = _size(rng, 1, 24 if f32 else 256)
        q_hi = 1 if kind == "decode" else rng.randint(2, 8)
        # the cache of one pass stays under that of the listed cases
        most = (1 << 24 if f32 else 1 << 29) // (rows * kv_heads * dim)
        kv_hi = max(q_hi, min(_size(rng, 16, 131072), most))
        kv_lo = max(q_hi, _size(rng, 1, kv_hi))
        windowed = rng.random() < 0.3
        return _attend("", rows=rows, q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=min(kv_lo, kv_hi), kv_hi=kv_hi,
                       heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page,
                       window=_size(rng, 16, 8192) if windowed else 0, sinks=rng.randint(0, 20) if windowed else 0,
                       gather=rng.random() < 0.5, fused=rng.random() < 0.5, dtype="f32" if f32 else "bf16")
    if kind == "prompt":
        group = rng.choice([1, 2, 4, 8])
        rows = rng.randint(1, 4)
        q_hi = _size(rng, 100, 4096 // rows)
        kv_hi = q_hi + rng.choice([0, _size(rng, 1, 4096)])
        kv_heads = min(kv_heads, (16 if dim == 256 else 32) // group)
        windowed = rng.random() < 0.4
        return _attend("", rows=rows, q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=q_hi, kv_hi=kv_hi,
                       heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page,
                       window=_size(rng, 64, 4096) if windowed else 0, sinks=rng.randint(0, 20) if windowed else 0,
                       gather=rng.random() < 0.5, fused=rng.random() < 0.5)
    if kind == "append":
        rows = _size(rng, 1, 128)
        q_hi = _size(rng, 1, max(1, 8192 // rows))
        return {"name": "", "op": "append", "rows": rows, "q_lo": rng.randint(1, q_hi), "q_hi": q_hi, "kv_lo": q_hi,
                "kv_hi": q_hi + _size(rng, 1, 1024), "kv_heads": kv_heads, "dim": dim, "page": page,
                "gather": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if kind == "fork":
        return {"name": "", "op": "fork", "parents": _size(rng, 1, 32), "children": rng.randint(1, 4), "kv_lo": 17,
                "kv_hi": _size(rng, 17, 8192), "grow": _size(rng, 1, 300), "kv_heads": kv_heads, "dim": dim,
                "page": page, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    return {"name": "", "op": "compact", "rows": _size(rng, 2, 128), "kv_lo": 16,
            "kv_hi": _size(rng, 100, 4096), "live": rng.uniform(0.2, 0.9), "kv_heads": min(kv_heads, 4), "dim": dim,
            "page": page, "dtype": rng.choice(["bf16", "bf16", "f32"])}


# ------------------------------------------------------------------------------------------
# Sizes that follow from a case alone

def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], even over the logarithm; always the same ones; the largest first."""
    at = [0.999] + [((i + 0.5) * GOLD) % 1.0 for i in range(1, n)]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** f)))) for f in at]


def _rows_of(case):
    """(new tokens, cache length with them) of each row."""
    n = case["rows"]
    new = _spread(case["q_lo"], case["q_hi"], n)
    return [(q, max(q, kv)) for q, kv in zip(new, _spread(case["kv_lo"], case["kv_hi"], n))]


def _first_seen(case, q, kv):
    """The first position behind the first tokens that some new token of the row sees."""
    return max(0, kv - q - case["window"] + 1) if case["window"] > 0 else 0


def _pages_held(case, q, kv):
    """The table entries of a row that hold a page: pages wholly out of sight were released."""
    ps = case["page"]
    first = _first_seen(case, q, kv) if case["op"] == "attend" else 0
    sinks = case.get("sinks", 0) if first else 0
    return [i for i in range(-(-kv // ps)) if (i + 1) * ps > first or i * ps < sinks]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attend":
        d, hq, hk = case["dim"], case["heads"], case["kv_heads"]
        keys = pairs = tokens = entries = 0
        for q, kv in _rows_of(case):
            first = _first_seen(case, q, kv)
            keys += kv - first + min(case["sinks"], first)
            entries += len(_pages_held(case, q, kv))
            tokens += q
            for p in range(kv - q, kv):
                at = max(0, p - case["window"] + 1) if case["window"] > 0 else 0
                pairs += p + 1 - at + min(case["sinks"], at)
        return {"bytes": 2 * keys * hk * d * es + 2 * tokens * hq * d * es + 4 * entries, "flops": 4 * pairs * hq * d}
    vec = case["kv_heads"] * case["dim"] * es
    if case["op"] == "append":
        return {"bytes": sum(q for q, _ in _rows_of(case)) * vec * 4, "flops": 0}
    ps = case["page"]
    if case["op"] == "fork":
        lens = _spread(case["kv_lo"], case["kv_hi"], case["parents"])
        data = sum(n % ps for n in lens) * case["children"] * vec * 4
        entries = sum(-(-(n + case["grow"]) // ps) for n in lens) * case["children"]
        return {"bytes": data + 4 * (4 * entries + _pool_pages(case)), "flops": 0}
    # compact: what moves is the live pages behind the live count, about live * (1 - live) of the pool
    pages = _pool_pages(case)
    moved = int(pages * case["live"] * (1 - case["live"]))
    return {"bytes": moved * ps * vec * 4 + 8 * pages, "flops": 0}


def _pool_pages(case):
    ps = case["page"]
    if case["op"] == "fork":
        lens = _spread(case["kv_lo"], case["kv_hi"], case["parents"])
        return 9 + sum(-(-n // ps) for n in lens) + sum(-(-case["grow"] // ps) + 2 for _ in lens) * case["children"]
    held = sum(len(_pages_held(case, q, kv)) for q, kv in _rows_of({"q_lo": 1, "q_hi": 1, **case}))
    return 9 + (int(held / case["live"]) if case["op"] == "compact" else held)


# ------------------------------------------------------------------------------------------
# Inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hk, d, ps = case["kv_heads"], case["dim"], case["page"]
    pages = _pool_pages(case)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt)

    s = {"case": case, "k_pool": rand(pages, hk, ps, d), "v_pool": rand(pages, hk, ps, d)}
    ids = list(range(1, pages))
    rng.shuffle(ids)
    if case["op"] == "fork":
        _prepare_fork(case, s, rng, ids)
    else:
        rows = _rows_of({"q_lo": 1, "q_hi": 1, **case})
        rng.shuffle(rows)
        n = len(rows)
        table_rows = list(range(n))
        rng.shuffle(table_rows)
        width = max(-(-kv // ps) for _, kv in rows)
        table, count = [[0] * width for _ in range(n)], [0] * pages
        for (q, kv), r in zip(rows, table_rows):
            for i in _pages_held(case, q, kv):
                table[r][i] = ids.pop()
                count[table[r][i]] = 1
        s.update(table=_i32(table), count=_i32(count), table_rows=_i32(table_rows), rows=rows)
        if case["op"] == "compact":
            s.update(table0=s["table"].clone(), count0=s["count"].clone(), live=_i32([0]))
        else:
            _prepare_tokens(case, s, rng, rand)
    if own:
        _prepare_handle(case, s)
    torch.cuda.synchronize()
    return s


def _prepare_tokens(case, s, rng, rand):
    rows = s["rows"]
    total = sum(q for q, _ in rows)
    starts = [0]
    for q, _ in rows:
        starts.append(starts[-1] + q)
    order = list(range(total))
    if case["gather"]:  # the rows lie in another order among the step's tokens
        by = list(range(len(rows)))
        rng.shuffle(by)
        at = 0
        for i in by:
            for t in range(rows[i][0]):
                order[starts[i] + t] = at + t
            at += rows[i][0]
    s.update(starts=_i32(starts), kv_lens=_i32([kv for _, kv in rows]), order=order, total=total,
             most=max(q for q, _ in rows), token_indx=_i32(order) if case["gather"] else None)
    hk, d = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        s["qkv"] = rand(total, 2 * hk, d)
        s["k"], s["v"] = s["qkv"][:, :hk], s["qkv"][:, hk:]
    else:
        s["qkv"] = rand(total, case["heads"] + (2 * hk if case["fused"] else 0), d)
        s["q"] = s["qkv"][:, :case["heads"]]
        s["out"] = torch.zeros(total, case["heads"], d, dtype=s["q"].dtype, device="cuda")


def _prepare_fork(case, s, rng, ids):
    """Parents with their pages; children that an earlier step forked from other parents."""
    ps, many = case["page"], case["children"]
    lens = _spread(case["kv_lo"], case["kv_hi"], case["parents"])
    rng.shuffle(lens)
    n = len(lens) * (1 + many)
    at = list(range(n))
    rng.shuffle(at)
    width = -(-(case["kv_hi"] + case["grow"]) // ps)
    table, count = [[0] * width for _ in range(n)], [0] * s["k_pool"].shape[0]
    for r, m in zip(at, lens):
        for i in range(-(-m // ps)):
            table[r][i] = ids.pop()
            count[table[r][i]] += 1
    src, dst, size = [], [], []
    for i, m in enumerate(lens):
        for j in range(many):
            src.append(at[i])
            dst.append(at[len(lens) + i * many + j])
            size.append(m)
    for i, r in enumerate(dst):  # the losers hold whole pages of some parent
        other = src[(i + many) % len(src)]
        for e in range(rng.randint(0, min(size[(i + many) % len(src)] // ps, width))):
            table[r][e] = table[other][e]
            count[table[r][e]] += 1
    s.update(table=_i32(table), count=_i32(count), src=_i32(src), dst=_i32(dst), lens=_i32(size),
             grown=_i32([m + case["grow"] for m in size]), first=_i32([0] * len(dst)), last=_i32([width] * len(dst)))


def _prepare_handle(case, s):
    """What a serving program keeps between its steps: descriptors over its tensors, and workspaces."""
    import gated_deltanet_linear_spec_gb300 as g
    s["cache"] = g.KvCache(s["k_pool"], s["v_pool"], s["table"], s["count"])
    if case["op"] in ("attend", "append"):
        s["kv_rows"] = g.KvRows(s["starts"], s["total"], s["kv_lens"], s["most"], s["table_rows"], s["token_indx"])
    if case["op"] == "attend":
        s["attn"] = g.Attention(case["heads"], window=case["window"], num_sinks=case["sinks"])
        need = g.gdn_attention_workspace_bytes(s["attn"], s["cache"], s["kv_rows"])
    else:
        need = g.gdn_kv_workspace_bytes(s["cache"], 0 if case["op"] != "fork" else s["src"].numel())
    s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------
# One pass

def run(s):
    op = s["case"]["op"]
    if own:
        import gated_deltanet_linear_spec_gb300 as g
        if op == "attend":
            g.gdn_paged_attention(s["attn"], s["cache"], s["kv_rows"], s["q"], s["out"], workspace=s["workspace"])
            return s["out"]
        if op == "append":
            g.gdn_kv_append(s["cache"], s["kv_rows"], s["k"], s["v"])
            return s["k_pool"], s["v_pool"]
        if op == "fork":
            g.gdn_kv_release(s["cache"], s["dst"], s["first"], s["last"])
            g.gdn_kv_fork(s["cache"], s["src"], s["dst"], s["lens"], workspace=s["workspace"])
            g.gdn_kv_reserve(s["cache"], s["dst"], s["lens"], s["grown"], workspace=s["workspace"])
            return s["k_pool"], s["v_pool"], s["table"], s["count"]
        s["table"].copy_(s["table0"])
        s["count"].copy_(s["count0"])
        g.gdn_kv_compact(s["cache"], s["live"], workspace=s["workspace"])
        return s["k_pool"], s["v_pool"], s["table"], s["count"], s["live"]
    if op == "attend":
        return _plain_attend(s)
    if op == "append":
        return _plain_append(s)
    if op == "fork":
        _plain_release(s)
        _plain_fork(s)
        _plain_reserve(s)
        return s["k_pool"], s["v_pool"], s["table"], s["count"]
    s["table"].copy_(s["table0"])
    s["count"].copy_(s["count0"])
    return _plain_compact(s)


def _plain_attend(s):
    case = s["case"]
    hq, hk, d, ps = case["heads"], case["kv_heads"], case["dim"], case["page"]
    n, most, total = len(s["rows"]), s["most"], s["total"]
    entries = s["table"][s["table_rows"].long()].long()                          # [n, width]
    length = entries.shape[1] * ps
    k = s["k_pool"][entries].transpose(1, 2).reshape(n, hk, length, d).float()   # [n, hk, length, d]
    v = s["v_pool"][entries].transpose(1, 2).reshape(n, hk, length, d).float()
    t = torch.arange(most, device="cuda")
    starts, kv = s["starts"].long(), s["kv_lens"].long()
    new = starts[1:] - starts[:-1]
    real = t[None] < new[:, None]                                                # [n, most]
    token = torch.where(real, starts[:-1, None] + t[None], 0)
    if s["token_indx"] is not None:
        token = s["token_indx"].long()[token]
    q = s["q"][token].float().reshape(n, most, hk, hq // hk, d).transpose(1, 2).reshape(n, hk, -1, d)
    pos = (kv - new)[:, None] + t[None]                                          # [n, most]
    key = torch.arange(length, device="cuda")
    seen = key[None, None] <= pos[..., None]                                     # [n, most, length]
    if case["window"] > 0:
        seen &= (key[None, None] > pos[..., None] - case["window"]) | (key < case["sinks"])
    seen &= (entries > 0).repeat_interleave(ps, 1)[:, None]
    seen = seen[:, None, :, None].expand(n, 1, most, hq // hk, length).reshape(n, 1, -1, length)
    w = q @ k.transpose(-1, -2)
    w *= 1.0 / math.sqrt(d)
    w.masked_fill_(~seen, -math.inf)
    w -= w.amax(-1, keepdim=True).clamp_min(-3e38)
    w.exp_()
    o = (w @ v) / w.sum(-1, keepdim=True).clamp_min(1e-38)
    o = o.reshape(n, hk, most, hq // hk, d).transpose(1, 2).reshape(n * most, hq, d)
    out = torch.zeros(total + 1, hq, d, dtype=s["q"].dtype, device="cuda")
    out[torch.where(real, token, total).reshape(-1)] = o.to(out.dtype)
    return out[:total]


def _plain_append(s):
    case = s["case"]
    hk, ps = case["kv_heads"], case["page"]
    i = torch.arange(s["total"], device="cuda")
    starts = s["starts"].long()
    row = torch.searchsorted(starts, i, right=True) - 1
    pos = s["kv_lens"].long()[row] - (starts[row + 1] - i)
    page = s["table"].long()[s["table_rows"].long()[row], pos // ps]
    token = i if s["token_indx"] is None else s["token_indx"].long()
    h = torch.arange(hk, device="cuda")[None]
    s["k_pool"][page[:, None], h, (pos % ps)[:, None]] = s["k"][token]
    s["v_pool"][page[:, None], h, (pos % ps)[:, None]] = s["v"][token]
    return s["k_pool"], s["v_pool"]


def _free_pages(count):
    """The pages in the order in which they are handed out, and how many there are to hand out."""
    used = count != 0
    used[0] = True
    return torch.sort(used.int(), stable=True).indices, (~used).sum()


def _plain_release(s):
    dst, width = s["dst"].long(), s["table"].shape[1]
    entries = s["table"][dst]
    e = torch.arange(width, device="cuda")[None]
    mine = (e >= s["first"][:, None]) & (e < s["last"][:, None])
    held = mine & (entries > 0)
    s["count"].index_add_(0, torch.where(held, entries, 0).reshape(-1).long(), -held.int().reshape(-1))
    s["table"][dst] = torch.where(mine, 0, entries)


def _plain_fork(s):
    ps, count = s["case"]["page"], s["count"]
    src, dst, lens = s["src"].long(), s["dst"].long(), s["lens"].long()
    from_, to = s["table"][src], s["table"][dst]
    full, part = lens // ps, lens % ps
    last = from_.gather(1, full.clamp_max(from_.shape[1] - 1)[:, None])[:, 0].long()
    need = (part > 0) & (last > 0)
    order, free = _free_pages(count)
    at = need.long().cumsum(0)
    ok = at <= free
    page = torch.where(need & ok, order[(at - 1).clamp_min(0)], 0)
    e = torch.arange(from_.shape[1], device="cuda")[None]
    whole = (e < full[:, None]) & ok[:, None]
    entry = torch.where(whole, from_, to)
    entry = torch.where((e == full[:, None]) & (part > 0)[:, None] & ok[:, None], page[:, None].int(), entry)
    held = whole & (from_ > 0)
    count.index_add_(0, torch.where(held, from_, 0).reshape(-1).long(), held.int().reshape(-1))
    count.index_add_(0, page, (page > 0).int())
    old = torch.where(page > 0, last, 0)
    copied = (torch.arange(ps, device="cuda")[None] < part[:, None])[:, None, :, None]
    s["k_pool"][page] = torch.where(copied & (page > 0)[:, None, None, None], s["k_pool"][old], s["k_pool"][page])
    s["v_pool"][page] = torch.where(copied & (page > 0)[:, None, None, None], s["v_pool"][old], s["v_pool"][page])
    s["table"][dst] = entry


def _plain_reserve(s):
    ps, count = s["case"]["page"], s["count"]
    dst = s["dst"].long()
    entries = s["table"][dst]
    e = torch.arange(entries.shape[1], device="cuda")[None]
    lo, hi = (s["lens"] + ps - 1) // ps, (s["grown"] + ps - 1) // ps
    need = (e >= lo[:, None]) & (e < hi[:, None]) & (entries <= 0)
    order, free = _free_pages(count)
    at = need.reshape(-1).long().cumsum(0).reshape(need.shape)
    ok = need & (at[:, -1:] <= free)
    page = torch.where(ok, order[(at - 1).clamp_min(0).clamp_max(order.numel() - 1)], 0)
    count.index_add_(0, page.reshape(-1), ok.int().reshape(-1))
    s["table"][dst] = torch.where(ok, page.int(), entries)


def _plain_compact(s):
    count, table = s["count"], s["table"].long()
    page = torch.arange(count.numel(), device="cuda")
    live = (count > 0) & (page > 0)
    many = live.sum()
    src = (live & (page > many)).nonzero()[:, 0]
    dst = (~live & (page > 0) & (page <= many)).nonzero()[:, 0]
    s["k_pool"][dst] = s["k_pool"][src]
    s["v_pool"][dst] = s["v_pool"][src]
    to = page.clone()
    to[src] = dst
    count[dst] = count[src]
    count[src] = 0
    s["table"].copy_(to[table.clamp_min(0)])
    s["live"][0] = many
    return s["k_pool"], s["v_pool"], s["table"], s["count"], s["live"]


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    return None  # pages move as they are: equal bits are asked for


def _row_keys(case, s, n):
    """Row n's pages as positions: the pool index (page, slot) of each position below its length, and whether it is held."""
    kv, ps = s["rows"][n][1], case["page"]
    j = torch.arange(kv, device="cuda")
    page = s["table"][int(s["table_rows"][n])].long()[torch.div(j, ps, rounding_mode="floor")]
    return j, page, j % ps


def _exact_attend(case, s):
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group = hq // hk
    out = torch.zeros(s["total"], hq, d, dtype=torch.float64, device="cuda")
    order = torch.tensor(s["order"], device="cuda")
    at = 0
    for n, (new, kv) in enumerate(s["rows"]):
        token = order[at:at + new]
        at += new
        j, page, slot = _row_keys(case, s, n)
        first = _first_seen(case, new, kv)
        use = (page > 0) & ((j >= first) | (j < case["sinks"]))
        j, page, slot = j[use], page[use], slot[use]
        where = torch.arange(kv - new, kv, device="cuda")[:, None]
        hidden = j[None] > where
        if case["window"] > 0:
            hidden |= (j[None] <= where - case["window"]) & (j[None] >= case["sinks"])
        for h in range(hk):
            k, v = s["k_pool"][page, h, slot].double(), s["v_pool"][page, h, slot].double()
            for a in range(0, new, 2048):  # pieces of a long prompt
                b = min(new, a + 2048)
                q = s["q"][token[a:b], h * group:(h + 1) * group].double()
                score = torch.einsum("tgd,jd->tgj", q, k) * d ** -0.5
                score = score.masked_fill(hidden[a:b, None], -math.inf)
                out[token[a:b], h * group:(h + 1) * group] = torch.einsum("tgj,jd->tgd", torch.softmax(score, -1), v)
    return out


def _exact_append(case, s):
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    order = torch.tensor(s["order"], device="cuda")
    at = 0
    for n, (new, kv) in enumerate(s["rows"]):
        _, page, slot = _row_keys(case, s, n)
        token = order[at:at + new]
        at += new
        k_pool[page[kv - new:], :, slot[kv - new:]] = s["k"][token].double()
        v_pool[page[kv - new:], :, slot[kv - new:]] = s["v"][token].double()
    return k_pool, v_pool
