"""Speculative decoding of a small hybrid model: one GDN layer, one full-attention layer.

    python examples/hybrid_decode.py [--dtype f32|bf16] [--steps 24]

Weights are random, drafts come from looking up the last token earlier in the sequence.  A step is what a server's
step is: verify rows of 3 drafts + 1 and newly come prompts in one batch, through ``gdn_mixed_batch`` and, per subset,
``gdn_kv_append`` and ``gdn_paged_attention``, after ``gdn_kv_reserve`` has given every row the pages for its new
tokens.  On the way a sequence is forked (``gdn_kv_fork`` for its pages, ``gdn_copy_slots`` for its GDN state), another
one ends (``gdn_kv_release``) and the pool is compacted (``gdn_kv_compact``); rejected drafts need nothing, as a
row's length alone says what counts.  At the end every sequence runs once more as one prompt, and the logits of its
generated tokens are compared.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import gated_deltanet_linear_spec_gb300 as gdn  # noqa: E402

VOCAB, WIDTH, DRAFTS = 24, 128, 3
ROWS, PAGE, PAGES_PER_ROW, PAGES = 8, 16, 24, 96
HQ, HKV, DIM = 4, 2, 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Model:
    def __init__(self, dtype, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(dtype)

        self.dtype = dtype
        self.layer = gdn.Layer(2, 4, 32, 32, 4, 3 + DRAFTS, dtype)
        C, hv = self.layer.channels, self.layer.num_v_heads
        self.params = gdn.Params(weight(C, 4), torch.rand(hv, generator=gen, device="cuda"),
                                 torch.randn(hv, generator=gen, device="cuda"))
        self.attn = gdn.Attention(HQ)
        self.embed = torch.randn(VOCAB, WIDTH, generator=gen, device="cuda").to(dtype)
        self.w_qkv, self.w_a, self.w_b = weight(C, WIDTH), weight(hv, WIDTH), weight(hv, WIDTH)
        self.w_out = weight(WIDTH, hv * self.layer.head_v_dim)
        self.w_attn, self.w_attn_out = weight((HQ + 2 * HKV) * DIM, WIDTH), weight(WIDTH, HQ * DIM)
        self.w_logits = weight(VOCAB, WIDTH)


def norm(x):
    return torch.nn.functional.rms_norm(x.float(), (WIDTH,)).to(x.dtype)


class Engine:
    """The device state of ROWS sequences, and one step over some of them."""

    def __init__(self, model):
        self.model, dtype, layer = model, model.dtype, model.layer
        pool = torch.zeros(PAGES, 2, HKV, PAGE, DIM, dtype=dtype, device="cuda")
        self.cache = gdn.KvCache(pool[:, 0], pool[:, 1], torch.zeros(ROWS, PAGES_PER_ROW, dtype=torch.int32, device="cuda"),
                                 torch.zeros(PAGES, dtype=torch.int32, device="cuda"))
        # slot 0 is NULL; row r's state after each of its tokens of a verify step is in slots[r]
        count = 1 + ROWS * (DRAFTS + 1)
        self.pools = gdn.Pools(torch.zeros(count, layer.conv_state_len, layer.channels, dtype=dtype, device="cuda"),
                               torch.zeros(count, layer.num_v_heads, layer.head_v_dim, layer.head_k_dim, device="cuda"))
        self.slots = torch.arange(1, count, dtype=torch.int32, device="cuda").view(ROWS, DRAFTS + 1)
        self.lens = [0] * ROWS       # tokens that count
        self.accepted = [1] * ROWS   # tokens of the last verify step that count
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, prompts, verify):
        """prompts, verify: {row: tokens}.  Returns {row: logits of its tokens}."""
        m, order = self.model, {**verify, **prompts}
        starts, total = {}, 0
        for r, tokens in order.items():
            starts[r], total = total, total + len(tokens)
        x = m.embed[torch.tensor([t for tokens in order.values() for t in tokens], device="cuda")]

        def subset(group):
            rows = list(group)
            first = i32([0] + torch.tensor([len(group[r]) for r in rows]).cumsum(0).tolist())
            index = i32([starts[r] + t for r in rows for t in range(len(group[r]))])
            return rows, first, index

        spec = non_spec = None
        attends = []
        if verify:
            rows, first, index = subset(verify)
            spec = gdn.Rows(first, index.numel(), index, spec_state_indices=self.slots[rows].contiguous(),
                            num_accepted_tokens=i32([self.accepted[r] for r in rows]))
            attends.append((spec, rows, verify))
        if prompts:
            rows, first, index = subset(prompts)
            non_spec = gdn.Rows(first, index.numel(), index, state_indices=self.slots[rows, 0].contiguous(),
                                has_initial_state=i32([0] * len(rows)))
            attends.append((non_spec, rows, prompts))

        # the GDN layer
        h = norm(x)
        out = torch.empty(total, m.layer.num_v_heads, m.layer.head_v_dim, dtype=m.dtype, device="cuda")
        gdn.gdn_mixed_batch(m.layer, m.params, self.pools, h @ m.w_qkv.T, h @ m.w_a.T, h @ m.w_b.T, non_spec, 0,
                            len(prompts), spec, out, status=self.status)
        x = x + out.flatten(1) @ m.w_out.T

        # the attention layer, q | k | v from one projection
        q, k, v = (norm(x) @ m.w_attn.T).view(total, HQ + 2 * HKV, DIM).split([HQ, HKV, HKV], 1)
        out = torch.empty(total, HQ, DIM, dtype=m.dtype, device="cuda")
        rows = list(order)
        gdn.gdn_kv_reserve(self.cache, i32(rows), i32([self.lens[r] for r in rows]),
                           i32([self.lens[r] + len(order[r]) for r in rows]), status=self.status)
        for of_gdn, rows, group in attends:
            kv_rows = gdn.KvRows.from_rows(of_gdn, i32([self.lens[r] + len(group[r]) for r in rows]),
                                           max(len(group[r]) for r in rows), i32(rows))
            gdn.gdn_kv_append(self.cache, kv_rows, k, v, status=self.status)
            gdn.gdn_paged_attention(m.attn, self.cache, kv_rows, q, out, status=self.status)
        x = x + out.flatten(1) @ m.w_attn_out.T
        logits = (norm(x) @ m.w_logits.T).float()
        return {r: logits[starts[r]:starts[r] + len(order[r])] for r in order}

    def fork(self, src, dst):
        gdn.gdn_kv_fork(self.cache, i32([src]), i32([dst]), i32([self.lens[src]]), status=self.status)
        gdn.gdn_copy_slots(self.model.layer, self.pools, self.slots[src].contiguous(), self.slots[dst].contiguous(),
                           status=self.status)
        self.lens[dst], self.accepted[dst] = self.lens[src], self.accepted[src]

    def end(self, row):
        gdn.gdn_kv_release(self.cache, i32([row]), status=self.status)
        self.lens[row], self.accepted[row] = 0, 1


def draft(tokens):
    """DRAFTS tokens: what followed the last token where it stood before."""
    for at in range(len(tokens) - 2, -1, -1):
        if tokens[at] == tokens[-1]:
            found = tokens[at + 1:at + 1 + DRAFTS]
            return found + [found[-1]] * (DRAFTS - len(found))
    return [tokens[-1]] * DRAFTS


def run(dtype, steps=24, seed=0):
    """Returns (sequences, tokens accepted per verify row and step, largest difference to the replay)."""
    model = Model(dtype, seed)
    engine = Engine(model)
    gen = torch.Generator().manual_seed(seed)

    def text(n):
        return torch.randint(0, VOCAB, (n,), generator=gen).tolist()

    waiting = {0: {0: text(37), 1: text(90)}, 3: {2: text(5)}, 6: {3: text(64)}}  # prompts, by the step they come at
    tokens, logits = {}, {}  # of every live row; logits[r][i]: those behind token i, from the prompt's last on
    done, given, verified = [], 0, 0
    for step in range(steps):
        prompts = waiting.get(step, {})
        verify = {r: [tokens[r][-1]] + draft(tokens[r]) for r in tokens}
        got = engine.step(prompts, verify)
        for r, prompt in prompts.items():
            tokens[r] = list(prompt) + [int(got[r][-1].argmax())]
            logits[r] = [got[r][-1]]
            engine.lens[r] = len(prompt)
        for r, fed in verify.items():
            best = got[r].argmax(-1).tolist()
            n = 1
            while n <= DRAFTS and fed[n] == best[n - 1]:
                n += 1
            tokens[r] += best[:n]
            logits[r] += list(got[r][:n])
            engine.lens[r] += n
            engine.accepted[r] = n
            given, verified = given + n, verified + 1
        if step == steps // 3:  # a second continuation of row 0
            engine.fork(0, 5)
            tokens[5], logits[5] = tokens[0][:-1] + [int(logits[0][-1].topk(2).indices[1])], list(logits[0])
        if step == steps // 2:  # row 1 ends; what stays moves to the front of the pool
            done.append((tokens.pop(1), logits.pop(1)))
            engine.end(1)
            live = i32([0])
            gdn.gdn_kv_compact(engine.cache, live, status=engine.status)
            held = engine.cache.block_table
            assert int(held.max()) == int(live) == int((engine.cache.refcount > 0).sum())
    done += [(tokens[r], logits[r]) for r in tokens]
    assert int(engine.status) == 0, int(engine.status)

    worst = 0.0
    replay = Engine(model)
    for seq, want in done:
        got = replay.step({0: seq[:-1]}, {})[0]
        worst = max(worst, float((got[-len(want):] - torch.stack(want)).abs().max()))
        replay.end(0)
    return [seq for seq, _ in done], given / max(verified, 1), worst


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--dtype", choices=DTYPES, default="bf16")
    parser.add_argument("--steps", type=int, default=24)
    args = parser.parse_args()
    sequences, per_step, difference = run(DTYPES[args.dtype], args.steps)
    for sequence in sequences:
        print(len(sequence), "tokens, the last:", sequence[-16:])
    print(f"{per_step:.2f} tokens a step and row; logits differ from one prompt's by {difference:.2e} at most")
