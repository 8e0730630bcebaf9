"""Rotary positions and shared prefixes of the paged cache's attention layers: what is timed, and the plain forms.

  rope    heads turned by their tokens' positions (half and interleaved pairs, part of a head, scaled for long contexts);
  append  a step's new tokens: queries and keys turned, keys and values into the rows' pages, in one call;
  common  how many leading pages the rows of each group hold in common;
  attend  attention of groups of rows over a prefix that each group shares, and over every row's own tokens behind it.
With ``own`` false ``run`` computes them with elementary torch operations in 32 bits (angles in 64); with ``own`` true it
calls the framework.  ``exact`` follows the definitions in 64 bits, head by head and row by row.
"""
import math
import random

import torch

own = False

GOLD = 0.6180339887498949
EARLY = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCALINGS = ("plain", "linear", "ntk", "bands", "ramp")


def _turning(kw, dim):
    case = {"rotary": dim, "base": 10000.0, "interleaved": False, "scaling": "plain", "factor": 1.0, "original": 4096}
    case.update(kw)
    return case


def _rope(name, **kw):
    case = {"name": name, "op": "rope", "tokens": 1, "heads": 16, "dim": 128, "pos_hi": 8192, "fused": False,
            "dtype": "bf16"}
    case.update(_turning(kw, kw.get("dim", 128)))
    return case


def _append(name, **kw):
    case = {"name": name, "op": "append", "rows": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 1, "kv_hi": 1, "heads": 32,
            "kv_heads": 4, "dim": 128, "page": 16, "gather": False, "dtype": "bf16"}
    case.update(_turning(kw, kw.get("dim", 128)))
    return case


def _common(name, **kw):
    case = {"name": name, "op": "common", "groups": 1, "rows_lo": 2, "rows_hi": 2, "q_lo": 1, "q_hi": 1, "prefix_lo": 64,
            "prefix_hi": 64, "tail_lo": 1, "tail_hi": 64, "page": 16}
    case.update(kw)
    return case


def _attend(name, **kw):
    case = {"name": name, "op": "attend", "groups": 1, "rows_lo": 2, "rows_hi": 2, "q_lo": 1, "q_hi": 1, "prefix_lo": 64,
            "prefix_hi": 64, "tail_lo": 1, "tail_hi": 64, "heads": 32, "kv_heads": 4, "dim": 128, "page": 16, "window": 0,
            "sinks": 0, "gather": False, "fused": False, "dtype": "bf16"}
    case.update(kw)
    return case


def listed():
    return [
        # one stream, one new token: the latency of a single call
        _rope("rope_one"),
        # the queries of one long prompt, q inside a fused q|k|v projection
        _rope("rope_prompt", tokens=8192, heads=32, fused=True),
        # part of a wide head, interleaved pairs, 32 bits, positions far behind the length that was trained on
        _rope("rope_far", tokens=777, heads=8, dim=256, rotary=64, interleaved=True, scaling="ramp", factor=40.0,
              base=1000000.0, pos_hi=1000000, dtype="f32"),
        # the verify batch: 64 rows of 3 drafts + 1, tokens interleaved
        _append("append_64x4", rows=64, q_lo=4, q_hi=4, kv_lo=100, kv_hi=2048, gather=True),
        # one 8192-token prompt, a quarter of every head turned
        _append("append_prompt", q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, heads=16, kv_heads=2, dim=256, page=64,
                rotary=64, base=10000000.0),
        # four branches of one sequence
        _common("common_4", rows_lo=4, rows_hi=4, prefix_lo=777, prefix_hi=777),
        # a full batch over a few very long documents
        _common("common_256", groups=16, rows_lo=9, rows_hi=24, q_hi=4, prefix_lo=20000, prefix_hi=131072, tail_hi=2000),
        # four branches of one sequence, one new token each: the latency of a call
        _attend("shared_4", rows_lo=4, rows_hi=4, prefix_lo=777, prefix_hi=777, tail_hi=100, heads=16, kv_heads=2),
        # the decode batch behind one system prompt
        _attend("shared_64", rows_lo=64, rows_hi=64, prefix_lo=8200, prefix_hi=8200, tail_hi=1024),
        # the verify batch over one long document, q inside a fused projection, tokens interleaved
        _attend("shared_64x4", rows_lo=64, rows_hi=64, q_lo=4, q_hi=4, prefix_lo=32768, prefix_hi=32768, tail_lo=16,
                tail_hi=1024, page=64, gather=True, fused=True),
        # ragged groups (sampled continuations of several prompts), ragged verify rows, wide heads, some under a window
        _attend("shared_groups", groups=12, rows_lo=2, rows_hi=16, q_lo=1, q_hi=5, prefix_lo=500, prefix_hi=20000,
                tail_hi=300, heads=16, kv_heads=2, dim=256, page=32, window=6000, sinks=4, gather=True),
        # the framework's 32-bit activations: 2 drafts + 1
        _attend("shared_f32", groups=3, rows_lo=5, rows_hi=8, q_lo=3, q_hi=3, prefix_lo=300, prefix_hi=4096, tail_hi=200,
                heads=8, kv_heads=2, dim=64, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    return max(lo, min(hi, _log(rng, lo, hi)))


def draw(rng: random.Random):
    case = _draw(rng)
    del case["name"]
    return case


def _draw_turning(rng, dim):
    scaling = rng.choice(SCALINGS)
    return {"rotary": 2 * rng.randint(1, dim // 2) if rng.random() < 0.3 else dim // rng.choice([1, 2, 4]),
            "base": rng.choice([10000.0, 500000.0, 10000000.0]), "interleaved": rng.random() < 0.5, "scaling": scaling,
            "factor": 1.0 if scaling == "plain" else rng.choice([2.0, 8.0, 40.0])}


def _draw(rng):
    kind = rng.choice(["rope", "append", "common", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    if kind == "rope":
        dim = rng.choice([dim, 16 * rng.randint(1, 16)])
        heads = _size(rng, 1, 64)
        tokens = _size(rng, 1, (1 << 24) // (heads * dim))
        return _rope("", tokens=tokens, heads=heads, dim=dim, pos_hi=_size(rng, 1000, 4000000),
                     fused=rng.random() < 0.5, dtype=dtype, **_draw_turning(rng, dim))
    if kind == "append":
        rows = _size(rng, 1, 128)
        q_hi = _size(rng, 1, max(1, min(8192, (1 << 24) // (kv_heads * group * dim)) // rows))
        return _append("", rows=rows, q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=q_hi, kv_hi=q_hi + _size(rng, 1, 1024),
                       heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, gather=rng.random() < 0.5,
                       dtype=dtype, **_draw_turning(rng, dim))
    groups = _size(rng, 1, 16)
    rows_hi = _size(rng, 2, max(2, 256 // groups))
    rows_lo = rng.randint(1, rows_hi)
    q_hi = rng.choice([1, 1, 2, 3, 4, 5, 8])
    q_lo = rng.randint(1, q_hi)
    if kind == "common":
        prefix_lo = 100 * page
        prefix_hi = _size(rng, prefix_lo, 131072)
        return _common("", groups=groups, rows_lo=rows_lo, rows_hi=rows_hi, q_lo=q_lo, q_hi=q_hi,
                       prefix_lo=_size(rng, prefix_lo, prefix_hi), prefix_hi=prefix_hi, tail_hi=_size(rng, q_hi, 2000),
                       page=page)
    f32 = dtype == "f32"
    tail_hi = _size(rng, q_hi, 1024)
    # the plain form goes over rows x (prefix + tail) keys: no more of them, and of products, than in the listed cases
    most = min((1 << 25 if f32 else 1 << 30) // (groups * rows_hi * kv_heads * dim),
               (1 << 28 if f32 else 1 << 35) // (groups * rows_hi * q_hi * kv_heads * group * dim))
    prefix_hi = max(1, min(_size(rng, 16, 65536), most - tail_hi))
    windowed = rng.random() < 0.25
    return _attend("", groups=groups, rows_lo=rows_lo, rows_hi=rows_hi, q_lo=q_lo, q_hi=q_hi,
                   prefix_lo=_size(rng, 1, prefix_hi), prefix_hi=prefix_hi, tail_hi=tail_hi, heads=kv_heads * group,
                   kv_heads=kv_heads, dim=dim, page=page, window=_size(rng, 16, 8192) if windowed else 0,
                   sinks=rng.randint(0, 20) if windowed else 0, gather=rng.random() < 0.5, fused=rng.random() < 0.5,
                   dtype=dtype)


# ------------------------------------------------------------------------------------------
# Sizes that follow from a case alone

def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], even over the logarithm; always the same ones; the largest first."""
    at = [0.999] + [((i + 0.5) * GOLD) % 1.0 for i in range(1, n)]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** f)))) for f in at]


def _rows_of(case):
    """(new tokens, tokens with them) of each row."""
    n = case["rows"]
    new = _spread(case["q_lo"], case["q_hi"], n)
    return [(q, max(q, kv)) for q, kv in zip(new, _spread(case["kv_lo"], case["kv_hi"], n))]


def _groups_of(case):
    """Per group: the tokens that its rows were forked at, and (new tokens, tokens with them) of each row."""
    sizes = _spread(case["rows_lo"], case["rows_hi"], case["groups"])
    forks = _spread(case["prefix_lo"], case["prefix_hi"], case["groups"])
    total = sum(sizes)
    new, tails = _spread(case["q_lo"], case["q_hi"], total), _spread(case["tail_lo"], case["tail_hi"], total)
    out, at = [], 0
    for size, fork in zip(sizes, forks):
        out.append((fork, [(q, fork + max(q, tail)) for q, tail in zip(new[at:at + size], tails[at:at + size])]))
        at += size
    return out


def _seen(case, pos, until):
    """How many positions below ``until`` a query at ``pos`` sees."""
    until = min(until, pos + 1)
    first = max(0, pos - case["window"] + 1) if case["window"] > 0 else 0
    return max(0, until - first) + min(case["sinks"], first, until)


def work(case):
    es = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "rope":
        values = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * values * es + 4 * case["tokens"], "flops": 3 * case["tokens"] * case["heads"] * case["rotary"]}
    if case["op"] == "append":
        tokens = sum(q for q, _ in _rows_of(case))
        return {"bytes": 2 * tokens * (case["heads"] + 2 * case["kv_heads"]) * case["dim"] * es,
                "flops": 3 * tokens * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    if case["op"] == "common":
        # every row's entries up to the first that differs, or up to where the shortest row's new tokens begin
        entries = sum(len(rows) * min(fork // case["page"] + 1, -(-min(kv - q for q, kv in rows) // case["page"]))
                      for fork, rows in _groups_of(case))
        return {"bytes": 4 * entries, "flops": 0}
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    keys = pairs = tokens = 0
    for fork, rows in _groups_of(case):
        shared = fork // case["page"] * case["page"]
        keys += _seen(case, min(kv - q for q, kv in rows), shared)
        for q, kv in rows:
            tokens += q
            below = _seen(case, kv - q, kv - q) - _seen(case, kv - q, shared)  # the row's own, seen by its first query
            keys += below + q
            pairs += sum(_seen(case, p, p + 1) for p in range(kv - q, kv))
    return {"bytes": 2 * keys * hk * d * es + 2 * tokens * hq * d * es, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------------------------------
# Inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    dt = DTYPES[case.get("dtype", "bf16")]

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt)

    s = {"case": case}
    if case["op"] == "rope":
        n, h, d = case["tokens"], case["heads"], case["dim"]
        s["x"] = rand(n, h + (max(1, h // 4) if case["fused"] else 0), d)[:, :h]
        s["out"] = torch.zeros(n, h, d, dtype=dt, device="cuda")
        # a prompt's positions run on from some place
        s["positions"] = _i32([rng.randrange(case["pos_hi"])]) if n == 1 else \
            (torch.arange(n, device="cuda") + rng.randrange(max(1, case["pos_hi"] - n))).int()
    elif case["op"] == "append":
        _prepare_append(case, s, rng, host, rand)
    else:
        _prepare_groups(case, s, rng, host, rand)
    if own:
        _prepare_handle(case, s)
    torch.cuda.synchronize()
    return s


def _order(case, lens, rng):
    """The rows' first local tokens, and the global token of each local one."""
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    order = list(range(starts[-1]))
    if case.get("gather"):  # the rows lie in another order among the step's tokens
        by = list(range(len(lens)))
        rng.shuffle(by)
        at = 0
        for i in by:
            for t in range(lens[i]):
                order[starts[i] + t] = at + t
            at += lens[i]
    return starts, order


def _prepare_rows(case, s, rows, rng):
    lens = [q for q, _ in rows]
    starts, order = _order(case, lens, rng)
    s.update(rows=rows, starts=_i32(starts), kv_lens=_i32([kv for _, kv in rows]), order=order, total=starts[-1],
             most=max(lens), token_indx=_i32(order) if case.get("gather") else None)


def _shuffled_pages(pages, host):
    return (1 + torch.randperm(pages - 1, generator=host)).int()


def _prepare_append(case, s, rng, host, rand):
    rows, ps = _rows_of(case), case["page"]
    rng.shuffle(rows)
    _prepare_rows(case, s, rows, rng)
    held = [-(-kv // ps) for _, kv in rows]
    pages = 9 + sum(held)
    ids = _shuffled_pages(pages, host)
    table = torch.zeros(len(rows), max(held), dtype=torch.int32)
    at = 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    s.update(table=table.cuda(), table_rows=_i32(list(range(len(rows)))), k_pool=rand(pages, hk, ps, d),
             v_pool=rand(pages, hk, ps, d), qkv=rand(s["total"], hq + 2 * hk, d))
    s["q"], s["k"], s["v"] = s["qkv"].split([hq, hk, hk], 1)
    s["q_out"] = torch.zeros(s["total"], hq, d, dtype=s["q"].dtype, device="cuda")


def _prepare_groups(case, s, rng, host, rand):
    """Rows forked from one another: the pages that their common tokens fill are shared, the rest is every row's own."""
    ps, groups = case["page"], _groups_of(case)
    rng.shuffle(groups)
    rows = [row for _, of_group in groups for row in of_group]
    _prepare_rows(case, s, rows, rng)
    n = len(rows)
    table_rows = torch.randperm(n, generator=host)
    table = torch.zeros(n, max(-(-kv // ps) for _, kv in rows), dtype=torch.int32)
    pages = 9 + EARLY * len(groups) + sum(fork // ps + sum(-(-kv // ps) - fork // ps for _, kv in of_group) for fork, of_group in groups)
    ids = _shuffled_pages(pages, host)
    at, first, bounds = 0, 0, [0]
    for fork, of_group in groups:
        shared = fork // ps
        members = table_rows[first:first + len(of_group)]
        table[members, :shared] = ids[at:at + shared]
        at += shared
        # where pages are compared, one of the rows left the others up to EARLY pages before
        early = 1 + rng.randrange(len(of_group) - 1) if case["op"] == "common" and len(of_group) > 1 else -1
        for i, (r, (_, kv)) in enumerate(zip(members.tolist(), of_group)):
            own_from = shared - rng.randrange(min(shared, EARLY) + 1) if i == early else shared
            m = -(-kv // ps) - own_from
            table[r, own_from:own_from + m] = ids[at:at + m]
            at += m
        first += len(of_group)
        bounds.append(first)
    s.update(groups=groups, table=table.cuda(), table_rows=table_rows.int().cuda(), bounds=_i32(bounds))
    if case["op"] == "common":
        s["k_pool"] = torch.zeros(pages, 1, ps, 16, dtype=torch.bfloat16, device="cuda")
        s["v_pool"] = s["k_pool"]
        s["prefix"] = _i32([0] * len(groups))
        return
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    s.update(k_pool=rand(pages, hk, ps, d), v_pool=rand(pages, hk, ps, d), prefix=_i32([fork for fork, _ in groups]),
             qkv=rand(s["total"], hq + (2 * hk if case["fused"] else 0), d))
    s["q"] = s["qkv"][:, :hq]
    s["out"] = torch.zeros(s["total"], hq, d, dtype=s["q"].dtype, device="cuda")


def _prepare_handle(case, s):
    """What a serving program keeps between its steps: descriptors over its tensors, and workspaces."""
    import gated_deltanet_linear_spec_gb300 as g
    if case["op"] in ("rope", "append"):
        kind = {"plain": g.GDN_ROPE_PLAIN, "linear": g.GDN_ROPE_LINEAR, "ntk": g.GDN_ROPE_NTK, "bands": g.GDN_ROPE_BANDS,
                "ramp": g.GDN_ROPE_RAMP}[case["scaling"]]
        s["rope"] = g.Rope(case["rotary"], base=case["base"],
                           layout=g.GDN_ROPE_INTERLEAVED if case["interleaved"] else g.GDN_ROPE_HALF, scaling=kind,
                           factor=case["factor"], original_len=case["original"])
    if case["op"] == "rope":
        return
    s["cache"] = g.KvCache(s["k_pool"], s["v_pool"], s["table"])
    s["kv_rows"] = g.KvRows(s["starts"], s["total"], s["kv_lens"], s["most"], s["table_rows"], s["token_indx"])
    if case["op"] in ("common", "attend"):
        s["kv_groups"] = g.KvGroups(s["bounds"], s["prefix"])
    if case["op"] == "attend":
        s["attn"] = g.Attention(case["heads"], window=case["window"], num_sinks=case["sinks"])
        need = g.gdn_shared_attention_workspace_bytes(s["attn"], s["cache"], s["kv_rows"], s["kv_groups"])
        s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------
# One pass

def run(s):
    op = s["case"]["op"]
    if own:
        import gated_deltanet_linear_spec_gb300 as g
        if op == "rope":
            g.gdn_rope(s["rope"], s["positions"], s["x"], s["out"])
            return s["out"]
        if op == "append":
            g.gdn_kv_append_rope(s["cache"], s["kv_rows"], s["rope"], s["k"], s["v"], s["q"], s["q_out"])
            return s["k_pool"], s["v_pool"], s["q_out"]
        if op == "common":
            g.gdn_kv_common_prefix(s["cache"], s["kv_rows"], s["kv_groups"])
            return s["prefix"]
        g.gdn_shared_attention(s["attn"], s["cache"], s["kv_rows"], s["kv_groups"], s["q"], s["out"],
                               workspace=s["workspace"])
        return s["out"]
    if op == "rope":
        return _plain_rope(s["case"], s["positions"], s["x"])
    if op == "append":
        return _plain_append(s)
    if op == "common":
        return _plain_common(s)
    return _plain_attend(s)


def _frequencies(case):
    """Radians a position of each pair, in 64 bits, and the factor of cosine and sine."""
    r, factor, length = case["rotary"], case["factor"], case["original"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    base = case["base"]
    if case["scaling"] == "ntk" and r > 2:
        base *= factor ** (r / (r - 2))
    f = torch.exp(i * (-2.0 / r * math.log(base)))
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "bands":  # by how often a pair turns over the original length: from 1 to 4 times
        keep = ((length * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / factor), 1.0
    if case["scaling"] == "ramp":  # by the pair's number, between the pairs that turn 32 times and once
        def pair_of(turns):
            return r * math.log(length / (2 * math.pi * turns)) / (2 * math.log(case["base"]))
        lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), r - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _plain_rope(case, positions, x):
    r = case["rotary"]
    f, magnitude = _frequencies(case)
    angle = positions.double()[:, None] * f
    cos, sin = (magnitude * torch.cos(angle)).float()[:, None], (magnitude * torch.sin(angle)).float()[:, None]
    out = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:r:2].float(), x[..., 1:r:2].float()
        out[..., 0:r:2] = (a * cos - b * sin).to(x.dtype)
        out[..., 1:r:2] = (b * cos + a * sin).to(x.dtype)
    else:
        a, b = x[..., :r // 2].float(), x[..., r // 2:r].float()
        out[..., :r // 2] = (a * cos - b * sin).to(x.dtype)
        out[..., r // 2:r] = (b * cos + a * sin).to(x.dtype)
    return out


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
    s["k_pool"][page[:, None], h, (pos % ps)[:, None]] = _plain_rope(case, pos, s["k"][token])
    s["v_pool"][page[:, None], h, (pos % ps)[:, None]] = s["v"][token]
    s["q_out"][token] = _plain_rope(case, pos, s["q"][token])
    return s["k_pool"], s["v_pool"], s["q_out"]


def _plain_common(s):
    bounds = s["bounds"].long()
    entries = s["table"][s["table_rows"].long()].clamp_min(0)                    # [rows, width]
    row = torch.arange(entries.shape[0], device="cuda")
    group = torch.searchsorted(bounds, row, right=True) - 1
    differs = entries != entries[bounds[group]]
    e = torch.arange(entries.shape[1], device="cuda")
    first = torch.where(differs, e, entries.shape[1]).amin(1)
    starts = s["starts"].long()
    whole = (s["kv_lens"].long() - (starts[1:] - starts[:-1])) // s["case"]["page"]
    agree = torch.minimum(first, whole)
    out = torch.full((bounds.numel() - 1,), entries.shape[1], dtype=torch.long, device="cuda")
    out.scatter_reduce_(0, group, agree, "amin")
    s["prefix"].copy_(out * s["case"]["page"])
    return s["prefix"]


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


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(case, s["positions"].double(), s["x"].double())
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "common":
        return None  # whole numbers: equal ones are asked for
    return _exact_attend(case, s)


def _exact_turn(case, positions, x):
    """Pairs as complex numbers, pair by pair."""
    r, out = case["rotary"], x.clone()
    for i in range(r // 2):
        f = case["base"] ** (-2.0 * i / r)
        often = case["original"] * f / (2 * math.pi)  # turns over the original length
        size = 1.0
        if case["scaling"] == "linear":
            f /= case["factor"]
        elif case["scaling"] == "ntk":
            f *= case["factor"] ** (-2.0 * i / (r - 2)) if r > 2 else 1.0
        elif case["scaling"] == "bands":
            if often <= 1.0:
                f /= case["factor"]
            elif often < 4.0:
                part = (often - 1.0) / 3.0
                f = part * f + (1.0 - part) * f / case["factor"]
        elif case["scaling"] == "ramp":
            per = r / (2 * math.log(case["base"]))
            lo = max(math.floor(per * math.log(case["original"] / (64 * math.pi))), 0)
            hi = min(math.ceil(per * math.log(case["original"] / (2 * math.pi))), r - 1)
            part = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = (1.0 - part) * f + part * f / case["factor"]
            size = 0.1 * math.log(case["factor"]) + 1.0
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
        turn = torch.polar(torch.full_like(positions, size), positions * f)
        z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _row_keys(case, s, n):
    """Of row n's positions: the page and slot of each."""
    kv, ps = s["rows"][n][1], case["page"]
    j = torch.arange(kv, device="cuda")
    page = s["table"][int(s["table_rows"][n])].long()[torch.div(j, ps, rounding_mode="floor")]
    return j, page, j % ps


def _exact_append(case, s):
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
    order = torch.tensor(s["order"], device="cuda")
    at = 0
    for n, (new, kv) in enumerate(s["rows"]):
        j, page, slot = _row_keys(case, s, n)
        token, where = order[at:at + new], j[kv - new:].double()
        at += new
        k_pool[page[kv - new:], :, slot[kv - new:]] = _exact_turn(case, where, s["k"][token].double())
        v_pool[page[kv - new:], :, slot[kv - new:]] = s["v"][token].double()
        q_out[token] = _exact_turn(case, where, s["q"][token].double())
    return k_pool, v_pool, q_out


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
        where = torch.arange(kv - new, kv, device="cuda")[:, None]
        hidden = (j[None] > where) | (page <= 0)[None]
        if case["window"] > 0:
            hidden |= (j[None] <= where - case["window"]) & (j[None] >= case["sinks"])
        for h in range(hk):
            k, v = s["k_pool"][page, h, slot].double(), s["v_pool"][page, h, slot].double()
            q = s["q"][token, h * group:(h + 1) * group].double()
            score = torch.einsum("tgd,jd->tgj", q, k) * d ** -0.5
            score = score.masked_fill(hidden[:, None], -math.inf)
            out[token, h * group:(h + 1) * group] = torch.einsum("tgj,jd->tgd", torch.softmax(score, -1), v)
    return out
