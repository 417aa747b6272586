"""The page operations on the GPU against the plain ones on lists, and a run of all calls on sequences in
pages together, as a serving loop makes them."""
import numpy as np
import pytest
import torch

import nvfp4_kv_cache_sparse_gb300 as lib
import oracle
import paged_reference as ref
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


class State:
    """Device tensors and their plain counterpart, kept in step."""

    def __init__(self, batch, width, pages, ps, layers=2, R=352, seed=0):
        rng = np.random.default_rng(seed)
        self.ps, self.pages = ps, pages
        self.pool = [rng.integers(0, 256, (pages, ps, R), dtype=np.uint8) for _ in range(layers)]
        self.caches = [torch.from_numpy(c.reshape(pages * ps, R).copy()).to(DEV) for c in self.pool]
        self.plain = ref.Pages([[-1] * width for _ in range(batch)], [0] * batch, [0] * pages, ps)
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def check(self, status=0):
        torch.cuda.synchronize()
        assert self.table.tolist() == self.plain.table
        assert self.lens.tolist() == self.plain.lens
        assert self.refs.tolist() == self.plain.refs
        for c, p in zip(self.caches, self.pool):
            assert np.array_equal(c.cpu().numpy().reshape(p.shape), p)
        assert int(self.status.item()) == status
        self.status.zero_()

    def resize(self, new, max_new=0, status=0):
        slots, exhausted = self.plain.resize(new, max_new, self.pool)
        got = lib.resize_sequences(self.caches, self.table, self.lens, self.refs, torch.tensor(new, dtype=torch.int32, device=DEV), max_new,
                                   page_size=self.ps, dev_status=self.status)
        self.check(status | (lib.DEV_PAGES_EXHAUSTED if exhausted else 0))
        assert got.tolist() == slots

    def fork(self, src, dst, status=0):
        self.plain.fork(src, dst)
        lib.fork_sequences(self.table, self.lens, self.refs, torch.tensor(src, dtype=torch.int32, device=DEV),
                           torch.tensor(dst, dtype=torch.int32, device=DEV), page_size=self.ps, dev_status=self.status)
        self.check(status)

    def compact(self, in_place=True):
        page_map, n = self.plain.compact(self.pool)
        kw = {} if in_place else {"table_out": torch.empty_like(self.table), "refs_out": torch.empty_like(self.refs)}
        old = self.table.clone(), self.refs.clone()
        table, refs, pm, live = lib.compact_pages(self.caches, self.table, self.lens, self.refs, page_size=self.ps, dev_status=self.status, **kw)
        if not in_place:
            assert torch.equal(old[0], self.table) and torch.equal(old[1], self.refs)
        self.table, self.refs = table, refs
        self.check()
        assert pm.tolist() == page_map and live.tolist() == [n]


def test_growing_shrinking_freeing():
    s = State(5, 9, 30, 16)
    s.resize([20, 0, 33, 16, 1], 3)
    s.resize([21, 5, 33, 17, 1], 4)      # inside a page, a new sequence, unchanged, over a page's edge
    s.resize([0, 5, 15, 144, 0], 2)      # freed pages are taken by the same call
    s.resize([144, 144, 144, 0, 0], 1)   # 27 of 30 pages
    s.resize([144, 144, 100, 50, 50], 5, 0)   # too few: the one that shrinks does, no other changes
    s.resize([-1, 145, 100, 3, 0], 1, lib.DEV_LENGTH_OUT_OF_RANGE)
    s.resize([0] * 5)
    assert not s.refs.any()


@pytest.mark.parametrize("R,layers,ps", [(352, 1, 64), (432, 3, 16), (656, 2, 4)])
def test_forks_share_and_copy_on_write(R, layers, ps):
    s = State(6, 8, 40, ps, layers, R)
    s.resize([3 * ps + 1, 2 * ps, ps + ps // 2, 0, 0, 0])
    s.fork([0, 1, 2], [3, 4, 5])
    s.resize([3 * ps + 2, 2 * ps + 1, ps + ps // 2, 3 * ps + 2, 2 * ps + 1, ps + ps // 2 + 1], 2)
    s.fork([3, 0, 5, 2, 1, 4], [0, 3, 2, 5, 4, 1])            # a permutation
    s.resize([0, 1, 2, 3, 4, 5])                               # into shared pages
    s.resize([ps + 1] * 6, 7)
    s.fork([1, 1, 1, 1, 1], [0, 2, 3, 4, 5])
    s.resize([ps + 2] * 6, 1)                                  # every holder copies, the shared page is free afterwards


def test_pairs_that_do_not_count():
    s = State(4, 4, 20, 16)
    s.resize([17, 40, 5, 0])
    s.fork([0, 1, 2], [3, 3, 3])              # the last one counts
    s.fork([0, -1, 2, 1], [1, 0, -7, 1])      # skipped ones; the last pair for 1 leaves it as it is
    s.fork([4, 0], [0, 4], lib.DEV_INDEX_OUT_OF_RANGE)
    s.fork([2, 9], [0, 0], lib.DEV_INDEX_OUT_OF_RANGE)   # an invalid later pair does not cancel a valid one


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("pages,ps", [(1, 16), (37, 16), (150, 1), (64, 64)])
def test_compact(in_place, pages, ps):
    rng = np.random.default_rng(pages)
    s = State(7, 6, pages, ps, 2)
    for k in range(4):
        new = rng.integers(0, 6 * ps + 1, 7)
        while sum(-(-int(n) // ps) for n in new) > pages:
            new = new // 2
        s.resize([int(n) for n in new])
        s.resize([int(n) * (i % 2 == k % 2) for i, n in enumerate(new)])
        if k == 2:
            s.fork([0, 2], [1, 3])
        s.compact(in_place)
        s.compact(in_place)                    # nothing left to move


def test_random_calls():
    rng = np.random.default_rng(3)
    for ps, pages in ((1, 60), (16, 45)):
        s = State(8, 7, pages, ps, 1)
        for _ in range(40):
            what = rng.integers(3)
            if what == 0:
                s.resize([int(n) for n in rng.integers(0, 7 * ps + 1, 8)], 3)
            elif what == 1:
                n = int(rng.integers(1, 9))
                s.fork([int(v) for v in rng.integers(0, 8, n)], [int(v) for v in rng.integers(-1, 8, n)])
            else:
                s.compact(bool(rng.integers(2)))


def test_large_pool_and_many_sequences():
    # more pages and sequences than one pass of the cluster covers (8 x 4096 pages, 8 x 1024 sequences)
    rng = np.random.default_rng(4)
    batch, width, pages, ps = 9000, 12, 70_003, 4
    s = State(batch, width, pages, ps, 1, 352)
    s.resize([int(n) for n in rng.integers(0, width * ps // 2, batch)], 1)
    order = rng.permutation(batch)
    s.fork([int(v) for v in order[:3000]], [int(v) for v in order[3000:6000]])
    s.resize([min(n + int(rng.integers(0, 6)), width * ps) if rng.random() < 0.7 else 0 for n in s.plain.lens], 2)
    s.compact()


def test_tables_with_a_stride():
    s = State(3, 4, 16, 16)
    wide = torch.full((3, 9), 77, dtype=torch.int32, device=DEV)
    wide[:, :4] = -1
    s.table = wide[:, :4]
    s.resize([20, 33, 0], 2)
    s.fork([1], [2])
    s.resize([0, 34, 34], 2)
    s.compact()
    assert torch.all(wide[:, 4:] == 77)


def test_copy_pages():
    rng = np.random.default_rng(6)
    for R, ps, layers, n in ((352, 64, 3, 10), (432, 1, 1, 7), (656, 128, 2, 1), (352, 4096, 1, 2)):
        pages = 40 if ps < 4096 else 6
        pool = rng.integers(0, 256, (layers, pages, ps, R), dtype=np.uint8)
        caches = [torch.from_numpy(c.reshape(pages * ps, R)).to(DEV) for c in pool]
        order = rng.permutation(pages)
        src, dst = [int(v) for v in order[:n]], [int(v) for v in order[n:2 * n]]
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
        lib.copy_pages(caches, t(src + [-1, pages, src[0]]), t(dst + [dst[0], dst[0], -3]), page_size=ps, dev_status=status)
        pool[:, dst] = pool[:, src]
        for c, p in zip(caches, pool):
            assert np.array_equal(c.cpu().numpy().reshape(p.shape), p)
        assert int(status.item()) == lib.DEV_INDEX_OUT_OF_RANGE
    lib.copy_pages(caches, t([]), t([]), page_size=ps)


def test_pages_outside_the_pool():
    s = State(2, 4, 8, 16)
    s.resize([40, 20])
    bad = s.table.clone()
    bad[0, 1] = 8
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens, refs = s.lens.clone(), s.refs.clone()
    lib.fork_sequences(bad, lens, refs, torch.tensor([0], dtype=torch.int32, device=DEV), torch.tensor([1], dtype=torch.int32, device=DEV),
                       page_size=16, dev_status=status)
    assert int(status.item()) == lib.DEV_INDEX_OUT_OF_RANGE
    assert bad[1].tolist() == bad[0].tolist() and refs.tolist() == [2, 1, 2, 0, 0, 0, 0, 0]
    status.zero_()
    slots = lib.resize_sequences([], bad, lens, refs, torch.tensor([0, 20], dtype=torch.int32, device=DEV), 1, page_size=16, dev_status=status)
    assert int(status.item()) == lib.DEV_INDEX_OUT_OF_RANGE and slots.tolist() == [[-1], [-1]]
    # row 0 gave back pages 0 and 2, row 1 (shared pages 0, 8, 2; now 20 tokens) its third page, 2
    assert refs.tolist() == [1, 1, 0, 0, 0, 0, 0, 0]


def test_calls_in_a_graph_and_on_another_stream():
    s = State(4, 8, 32, 16)
    s.resize([20, 30, 40, 5])
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    src, dst, up = t([0, 1]), t([2, 3]), t([21, 31, 21, 31])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.fork_sequences(s.table, s.lens, s.refs, src, dst, page_size=16)
        slots = lib.resize_sequences(s.caches, s.table, s.lens, s.refs, up, 1, page_size=16)
        _, _, page_map, live = lib.compact_pages(s.caches, s.table, s.lens, s.refs, page_size=16)
    for n in (21, 25, 33):
        up.copy_(t([n, n + 10, n, n + 10]))
        g.replay()
        s.plain.fork([0, 1], [2, 3])
        want, _ = s.plain.resize([n, n + 10, n, n + 10], 1, s.pool)
        pm, used = s.plain.compact(s.pool)
        s.check()
        assert slots.tolist() == want and page_map.tolist() == pm and live.tolist() == [used]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for n in (40, 48, 50):
        got = lib.resize_sequences(s.caches, s.table, s.lens, s.refs, t([n] * 4), 2, page_size=16, stream=stream)
        stream.synchronize()
        assert got.tolist() == s.plain.resize([n] * 4, 2, s.pool)[0]
    s.check()


def test_a_serving_loop():
    """Prompts are admitted and appended, sequences fork, decode step by step, finish, and the pool is
    compacted: after every step the decode equals attention over the tokens that were appended."""
    rng = np.random.default_rng(7)
    batch, width, pages, ps, R, h_q = 4, 6, 20, 16, 352, 16
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    cache = torch.full((pages * ps, R), 0xAB, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    history = [[] for _ in range(batch)]                       # records of each sequence's tokens
    sizes = [0] * batch

    def step(new, s_q):
        grow = [n - m for n, m in zip(new, sizes)]
        m = max(grow)
        slots = lib.resize_sequences([cache], table, lens, refs, t(new), m, page_size=ps, dev_status=status)
        lat = synth.bf16_from_f32(rng.standard_normal((batch * m, 512)).astype(np.float32))
        rope = synth.bf16_from_f32(rng.standard_normal((batch * m, 64)).astype(np.float32))
        lib.quantize_append(lat.to(DEV), rope.to(DEV), slots.flatten(), cache)
        recs = oracle.quantize_records(synth.bf16_bits(lat), synth.bf16_bits(rope), R).reshape(batch, m, R)
        for b in range(batch):
            history[b] = (history[b] + list(recs[b, :max(0, grow[b])]))[:new[b]]
            sizes[b] = new[b]
        q = synth.bf16_from_f32(rng.standard_normal((batch, s_q, h_q, 576)).astype(np.float32))
        out, lse = lib.paged_mla_decode(q.to(DEV), cache, table, lens, 1 / 24, page_size=ps, dev_status=status)
        flat = np.array([r for h in history for r in h], dtype=np.uint8).reshape(-1, R)
        at = np.cumsum([0] + sizes)
        rows = np.full((batch, max(1, max(sizes))), -1, dtype=np.int32)
        for b in range(batch):
            rows[b, :sizes[b]] = np.arange(at[b], at[b + 1])
        ref.check_attention(out, lse, ref.attention(q, flat, False, rows, np.array(sizes), 1, 1 / 24))
        assert int(status.item()) == 0

    step([33, 50, 7, 0], 1)                                    # prompts
    step([34, 51, 8, 0], 1)
    lib.fork_sequences(table, lens, refs, t([1]), t([3]), page_size=ps)
    history[3], sizes[3] = list(history[1]), sizes[1]
    step([36, 53, 10, 53], 2)                                  # the fork and its source part ways
    step([35, 52, 11, 54], 1)                                  # a rejected draft
    step([0, 55, 12, 55], 1)                                   # one finishes
    lib.compact_pages([cache], table, lens, refs, page_size=ps)
    step([20, 56, 13, 56], 1)                                  # another takes its row
    lib.fork_sequences(table, lens, refs, t([1, 3, 0]), t([3, 0, 1]), page_size=ps)   # beams trade places
    history[3], history[0], history[1] = history[1], history[3], history[0]
    sizes[3], sizes[0], sizes[1] = sizes[1], sizes[3], sizes[0]
    step([57, 21, 14, 58], 1)


@pytest.mark.parametrize("pairs,width", [(3, 5000), (300, 6), (40, 700), (9, 4096), (256, 128), (257, 3)])
def test_forks_of_wide_rows_and_many_pairs(pairs, width):
    rng = np.random.default_rng(pairs)
    batch, ps = 2 * pairs + 1, 4
    s = State(batch, width, 400 + 2 * batch, ps, 1)
    lens = [int(n) for n in rng.integers(0, min(width * ps, 24) + 1, batch)]
    lens[0], lens[1] = min(width * ps, 1500), 0
    s.resize(lens)
    order = [int(v) for v in rng.permutation(batch)]
    s.fork(order[:pairs], order[pairs:2 * pairs])
    s.fork(order[pairs:2 * pairs], order[:pairs][::-1])
    s.fork([order[0]] * pairs, [order[1]] * (pairs - 1) + [order[2]])   # one target named many times


@pytest.mark.parametrize("batch,ps,layers", [(24, 64, 1), (90, 64, 2), (40, 256, 1), (1, 4096, 2), (700, 8, 1)])
def test_shared_last_pages_of_every_sequence_are_copied(batch, ps, layers):
    # few bytes: by the call's own cluster; more: by a grid of copies
    s = State(2 * batch, 2, 4 * batch + 3, ps, layers)
    s.resize([ps // 2 + i % (ps // 2) for i in range(batch)] + [0] * batch)
    s.fork(list(range(batch)), list(range(batch, 2 * batch)))
    s.resize([min(n + 1 + i % 3, 2 * ps) for i, n in enumerate(s.plain.lens)], 3)
    s.resize([0] * (2 * batch))
