"""Plain implementations of the paged key-value cache's operators, on the CPU: attention in 64 bits
row by row, the page calls as sequential loops over Python lists.  Test infrastructure only."""
import math

import torch

ROW_RANGE, PAGE_RANGE, PAGE_SHARED, NO_PAGES, TOKEN_RANGE, SLOT_RANGE = 0x8, 0x20, 0x40, 0x80, 0x4, 0x1


def seen_keys(table_row, page_size, num_pages, pos, window, sinks):
    """Positions that a query at ``pos`` sees."""
    keys = []
    for j in range(pos + 1):
        page = table_row[j // page_size]
        if window > 0 and j <= pos - window and j >= sinks:
            continue
        if 0 < page < num_pages:
            keys.append(j)
    return keys


def attention(q, k_pool, v_pool, table, rows, table_rows, token_indx, kv_lens, scale, window, sinks):
    """(out, spread, logits) in float64: out[token, head]; spread = sum_j p_j |v_j|, what one relative
    error of the weights moves; logits = the largest sum |q_i k_i| scale of a query.  ``rows`` lists
    (first local token, new tokens)."""
    T, Hq, d = q.shape
    Hkv, ps = k_pool.shape[1], k_pool.shape[2]
    G = Hq // Hkv
    scale = scale if scale > 0 else 1.0 / math.sqrt(d)
    out = torch.zeros(T, Hq, d, dtype=torch.float64)
    spread = torch.zeros(T, Hq, d, dtype=torch.float64)
    logits = torch.zeros(T, Hq, 1, dtype=torch.float64)
    tab = table.tolist()
    for n, (bos, new) in enumerate(rows):
        row = tab[table_rows[n]]
        for t in range(new):
            g = token_indx[bos + t]
            pos = kv_lens[n] - new + t
            keys = seen_keys(row, ps, k_pool.shape[0], pos, window, sinks)
            if not keys:
                continue
            page = torch.tensor([row[j // ps] for j in keys])
            slot = torch.tensor([j % ps for j in keys])
            k, v = k_pool[page, :, slot].double(), v_pool[page, :, slot].double()  # [keys, Hkv, d]
            qq = q[g].double().reshape(Hkv, G, d)
            s = torch.einsum("hgd,jhd->hgj", qq, k) * scale
            p = torch.softmax(s, -1)
            out[g] = torch.einsum("hgj,jhd->hgd", p, v).reshape(Hq, d)
            spread[g] = torch.einsum("hgj,jhd->hgd", p, v.abs()).reshape(Hq, d)
            logits[g] = (torch.einsum("hgd,jhd->hgj", qq.abs(), k.abs()) * scale).amax(-1).reshape(Hq, 1)
    return out, spread, logits


def attention_tolerance(ref, spread, logits, keys, dim, dtype, weight_bits):
    """Half a step of the output's type, and what the 32-bit arithmetic and the weights' rounding can move.

    A score is a sum of dim products in fp32: off by at most (dim + 2) 2^-24 sum|q k| scale, and by
    2^-24 |s| again where it is scaled for the exponential.  A weight e^s is off by that and by
    2^-22 of its own (exponential and rescaling); numerator and denominator both carry it and sums of
    ``keys`` terms, at 2^-24 a term.  The products may take the weights rounded to ``weight_bits``
    bits: 2^-weight_bits relative, half a step."""
    half = torch.finfo(dtype).eps / 2
    weight = 2.0 ** -24 * (dim + 6) * logits + 2.0 ** -22 + keys * 2.0 ** -24
    return half * ref.abs() * 1.01 + (2 * weight + 2.0 ** -weight_bits) * spread + 1e-30


class Pages:
    """The page state as lists, and the calls one row after the other."""

    def __init__(self, table, refcount, page_size):
        self.table = [list(r) for r in table]
        self.count = list(refcount)
        self.ps = page_size
        self.status = 0

    def free(self):
        return [p for p in range(1, len(self.count)) if self.count[p] == 0]

    def _ceil(self, n):
        return -(-n // self.ps)

    def _row_ok(self, r):
        return 0 <= r < len(self.table)

    def reserve(self, rows, from_lens, to_lens):
        free, used = self.free(), 0
        for r, a, b in zip(rows, from_lens, to_lens):
            if not self._row_ok(r) or a < 0 or b < 0 or b > len(self.table[0]) * self.ps:
                self.status |= PAGE_RANGE
                continue
            need = [e for e in range(self._ceil(a), self._ceil(b)) if self.table[r][e] <= 0]
            if not need:
                continue
            used += len(need)
            if used > len(free):
                self.status |= NO_PAGES
                continue
            for e, p in zip(need, free[used - len(need):used]):
                self.table[r][e] = p
                self.count[p] = 1

    def release(self, rows, first, last):
        for r, a, b in zip(rows, first, last):
            if not self._row_ok(r) or a < 0 or b > len(self.table[0]):
                self.status |= PAGE_RANGE
                continue
            for e in range(a, b):
                p, self.table[r][e] = self.table[r][e], 0
                if p >= len(self.count) or (p > 0 and self.count[p] <= 0):
                    self.status |= PAGE_RANGE
                elif p > 0:
                    self.count[p] -= 1

    def fork(self, src, dst, lens):
        """Also returns the (old page, new page, tokens) copies."""
        free, used, copies = self.free(), 0, []
        for s, t, n in zip(src, dst, lens):
            ok = self._row_ok(s) and self._row_ok(t) and 0 <= n <= len(self.table[0]) * self.ps
            if ok:
                for e in range(self._ceil(n)):
                    ok = ok and self.table[t][e] <= 0 and self.table[s][e] < len(self.count)
            if not ok:
                self.status |= PAGE_RANGE
                continue
            full, part = divmod(n, self.ps)
            old = self.table[s][full] if part else 0
            used += 1 if old > 0 else 0
            if used > len(free):
                self.status |= NO_PAGES
                continue
            for e in range(full):
                p = max(self.table[s][e], 0)
                self.table[t][e] = p
                if p:
                    self.count[p] += 1
            if part:
                new = free[used - 1] if old > 0 else 0
                self.table[t][full] = new
                if new:
                    self.count[new] = 1
                    copies.append((old, new, part))
        return copies

    def compact(self):
        """Also returns the (from, to) moves and the number of live pages."""
        live = [p for p in range(1, len(self.count)) if self.count[p] > 0]
        m = len(live)
        holes = [p for p in range(1, m + 1) if self.count[p] <= 0]
        moves = list(zip([p for p in live if p > m], holes))
        to = dict(moves)
        for a, b in moves:
            self.count[b], self.count[a] = self.count[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return moves, m
