"""Plain implementations, in 64 bits and on the host, of the calls on sequences in pages, with the error
bounds that the CUDA calls are held to. They share no code with the library: records are decoded by the
oracle, attention is the softmax definition, the page operations are loops over lists."""
import numpy as np

import oracle
import synth


def random_batch(rng, lens, page_size, spare=3, width=None, h_q=16, s_q=1, R=352, blk=False, scale=1.0):
    """Records, a shuffled page table and queries for sequences of the given lengths (numpy / torch CPU)."""
    lens = np.asarray(lens, dtype=np.int32)
    counts = -(-lens.astype(np.int64) // page_size)
    pages = int(counts.sum()) + spare
    width = max(1, int(counts.max(initial=0))) if width is None else width
    order = rng.permutation(pages)
    table = np.full((lens.size, width), -1, dtype=np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    n = pages * page_size
    lat = synth.bf16_from_f32(scale * rng.standard_normal((n, 512)).astype(np.float32))
    rope = synth.bf16_from_f32(rng.standard_normal((n, 64)).astype(np.float32))
    recs = oracle.quantize_records(synth.bf16_bits(lat), synth.bf16_bits(rope), R, blk)
    q = synth.bf16_from_f32(rng.standard_normal((lens.size, s_q, h_q, 576)).astype(np.float32))
    return recs, table, lens, q


def slots_of(table_row, n, page_size):
    pos = np.arange(n)
    return table_row[pos // page_size].astype(np.int64) * page_size + pos % page_size


def attention(q, recs, blk, table, lens, page_size, sm_scale, sink=None):
    """out, lse in fp64, and the bounds on the library's results.

    Bounds. Keys are exact. A score is an fp32 sum of 576 products: with at most 128 roundings on any path,
    it is off by d = 2^-17 sm_scale sum|q||k|, and exp2 and its argument add 2^-20; a weight p is therefore
    off by e = 2 (d + 2^-20) relative to the row's sum, and by 2^-11 from its rounding to f16. A part of a
    cut row is rounded to f16 (2^-11 of it) and out to bf16 (2^-8 of it). With A = sum p|V| / sum p:
        |out - ref| <= 2^-8 |ref| + (2^-11 + 2^-11 + e) A + 2^-25 (1 + sum|V| / sum p),
        |lse - ref| <= d + 2^-19 + 2^-22 |ref|.
    The last term: below 2^-14 f16 has steps of 2^-24, so a weight 2^(z - m) there is off by up to 2^-25 of itself
    held against its reference m, whatever its size. The reference is some earlier largest score, so m is at most
    the row's (or part's) largest, the weights held against it add up to S' >= S = sum p with p held against the
    largest score, and the quotient moves by at most 2^-25 sum|V| / S' <= 2^-25 sum|V| / S (for parts: the weighted
    mean of the parts' moves, which adds up to the same). A part's f16 output likewise: 2^-25. It matters where one
    key outweighs the others by more than 2^14 and its own V is 0 in a dim."""
    qf = q.float().numpy().astype(np.float64)
    B, s_q, h_q, _ = qf.shape
    out = np.zeros((B, s_q, h_q, 512))
    lse = np.full((B, s_q, h_q), -np.inf)
    tol_out, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    keys = oracle.dequant_records(recs, blk)
    for b in range(B):
        n = int(min(max(lens[b], 0), table.shape[1] * page_size))
        for i in range(s_q):
            seen = n - s_q + i + 1
            if seen <= 0:
                continue
            slots = slots_of(table[b], seen, page_size)
            slots = slots[(slots >= 0) & (slots < recs.shape[0])]
            if slots.size == 0:
                continue
            k = keys[slots]
            z = sm_scale * (qf[b, i] @ k.T)                       # [h_q, n]
            m = z.max(axis=1, keepdims=True)
            p = np.exp(z - m)
            total = p.sum(axis=1, keepdims=True)
            lse[b, i] = (m + np.log(total))[:, 0]
            denom = total if sink is None else total + np.exp(sink[:, None].astype(np.float64) - m)
            v = k[:, :512]
            out[b, i] = p @ v / denom
            d = 2.0 ** -17 * abs(sm_scale) * (np.abs(qf[b, i]) @ np.abs(k).T).max(axis=1)
            A = p @ np.abs(v) / denom
            tol_out[b, i] = 2.0 ** -8 * np.abs(out[b, i]) + (2.0 ** -10 + 2 * (d[:, None] + 2.0 ** -20)) * A
            tol_out[b, i] += 2.0 ** -25 * (1 + np.abs(v).sum(axis=0)[None, :] / denom)
            tol_lse[b, i] = d + 2.0 ** -19 + 2.0 ** -22 * np.abs(lse[b, i])
    return out, lse, tol_out, tol_lse


def check_attention(out, lse, ref):
    r_out, r_lse, t_out, t_lse = ref
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(r_lse)
    assert np.array_equal(np.isneginf(l), empty), "rows without a visible key"
    assert np.all(o[empty] == 0.0)
    err = np.abs(o - r_out)
    assert np.all(err <= t_out), f"out: {np.max(err / np.maximum(t_out, 1e-300)):.3g} times its bound"
    e = np.abs(l - r_lse)[~empty]
    assert np.all(e <= t_lse[~empty]), f"lse: {np.max(e / t_lse[~empty]):.3g} times its bound"


class Pages:
    """The page operations on Python lists: sequences as lists of pages, counts as a list."""

    def __init__(self, table, lens, refs, page_size):
        self.table = [list(map(int, row)) for row in table]
        self.lens = [int(n) for n in lens]
        self.refs = [int(r) for r in refs]
        self.ps = page_size

    def count(self, n):
        return -(-n // self.ps)

    def fork(self, src, dst):
        old = [list(r) for r in self.table], list(self.lens)
        pairs = [(s, d) for s, d in zip(src, dst) if 0 <= s < len(self.lens) and 0 <= d < len(self.lens)]
        last = {d: s for s, d in pairs}
        for d, s in last.items():
            if s == d:
                continue
            for p in old[0][s][:self.count(old[1][s])]:
                self.refs[p] += 1
            for p in old[0][d][:self.count(old[1][d])]:
                self.refs[p] -= 1
            n = self.count(old[1][s])
            self.table[d] = old[0][s][:n] + [-1] * (len(old[0][s]) - n)
            self.lens[d] = old[1][s]

    def resize(self, new, max_new, pool=None):
        """Returns (slots, exhausted). pool: list of [num_pages, page_size, R] arrays."""
        width = len(self.table[0])
        want = [n if 0 <= n <= width * self.ps else self.lens[b] for b, n in enumerate(new)]
        for b, n in enumerate(want):
            if n < self.lens[b]:
                for j in range(self.count(n), self.count(self.lens[b])):
                    self.refs[self.table[b][j]] -= 1
                    self.table[b][j] = -1
                self.lens[b] = n
        free = [p for p, r in enumerate(self.refs) if r == 0]
        slots = [[-1] * max_new for _ in want]
        plan = []
        for b, n in enumerate(want):
            if n > self.lens[b]:
                old = self.lens[b]
                cow = old % self.ps != 0 and self.refs[self.table[b][old // self.ps]] > 1
                plan.append((b, n, cow, self.count(n) - self.count(old) + int(cow)))
        if sum(p[3] for p in plan) > len(free):
            return slots, True
        shared = []
        for b, n, cow, need in plan:
            mine, free = free[:need], free[need:]
            old = self.lens[b]
            if cow:
                p, to = self.table[b][old // self.ps], mine.pop(0)
                shared.append(p)
                if pool is not None:
                    for c in pool:
                        c[to, :old % self.ps] = c[p, :old % self.ps]
                self.table[b][old // self.ps] = to
                self.refs[to] = 1
            for j in range(self.count(old), self.count(n)):
                self.table[b][j] = mine.pop(0)
                self.refs[self.table[b][j]] = 1
            for j in range(min(max_new, n - old)):
                pos = old + j
                slots[b][j] = self.table[b][pos // self.ps] * self.ps + pos % self.ps
            self.lens[b] = n
        for p in shared:
            self.refs[p] -= 1
        return slots, False

    def compact(self, pool=None):
        n = sum(r > 0 for r in self.refs)
        movers = [p for p, r in enumerate(self.refs) if r > 0 and p >= n]
        holes = [p for p, r in enumerate(self.refs) if r <= 0 and p < n]
        to = {p: p for p, r in enumerate(self.refs) if r > 0}
        to.update(zip(movers, holes))
        refs = [0] * len(self.refs)
        for p, t in to.items():
            refs[t] = self.refs[p]
        if pool is not None:
            for c in pool:
                for p, h in zip(movers, holes):
                    c[h] = c[p]
        self.refs = refs
        for b, row in enumerate(self.table):
            k = self.count(self.lens[b])
            self.table[b] = [to[p] for p in row[:k]] + [-1] * (len(row) - k)
        return [to.get(p, -1) for p in range(len(refs))], n
