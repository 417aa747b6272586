"""nvfp4_paged_mla_decode on the GPU against the softmax definition in 64 bits."""
import numpy as np
import pytest
import torch

import nvfp4_kv_cache_sparse_gb300 as lib
import oracle
import paged_reference as ref
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 576 ** -0.5


def run(recs, table, lens, q, page_size, sink=None, blk=False, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((*q.shape[:3], 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:3], float("nan"), device=DEV)
    lib.paged_mla_decode(q.to(DEV), torch.from_numpy(recs).to(DEV), torch.from_numpy(table).to(DEV), torch.from_numpy(lens).to(DEV),
                         SCALE, page_size=page_size, attn_sink=None if sink is None else torch.from_numpy(sink).to(DEV),
                         out=out, lse=lse, dev_status=status, block_scales=blk, **kw)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


EDGE_LENS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("h_q", [1, 16, 20, 64, 128])
@pytest.mark.parametrize("s_q", [1, 3])
def test_lengths_around_pages_and_tiles(h_q, s_q):
    rng = np.random.default_rng(h_q + 1000 * s_q)
    recs, table, lens, q = ref.random_batch(rng, EDGE_LENS, 64, h_q=h_q, s_q=s_q)
    out, lse, st = run(recs, table, lens, q, 64)
    assert st == 0
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 64, SCALE))


@pytest.mark.parametrize("R,blk", [(352, False), (352, True), (432, False)])
@pytest.mark.parametrize("page_size", [1, 4, 16, 64, 256])
@pytest.mark.parametrize("h_q,s_q", [(8, 1), (24, 1), (40, 2)])
def test_records_and_page_sizes(R, blk, page_size, h_q, s_q):
    rng = np.random.default_rng(R + page_size + h_q)
    sink = rng.standard_normal(h_q).astype(np.float32)
    recs, table, lens, q = ref.random_batch(rng, [777, 5, 260], page_size, h_q=h_q, s_q=s_q, R=R, blk=blk)
    out, lse, st = run(recs, table, lens, q, page_size, sink=sink, blk=blk)
    assert st == 0
    ref.check_attention(out, lse, ref.attention(q, recs, blk, table, lens, page_size, SCALE, sink))


@pytest.mark.parametrize("h_q,s_q,n", [(16, 1, 9000), (32, 1, 6000), (128, 1, 5000), (5, 7, 4001)])
def test_one_long_sequence_is_cut_over_all_ctas_and_joined(h_q, s_q, n):
    rng = np.random.default_rng(n)
    sink = 2 * rng.standard_normal(h_q).astype(np.float32)
    recs, table, lens, q = ref.random_batch(rng, [n], 64, h_q=h_q, s_q=s_q, scale=2.0)
    q = (q.float() * torch.linspace(0.1, 4.0, h_q)[None, None, :, None]).to(torch.bfloat16)   # flat to peaked rows
    out, lse, st = run(recs, table, lens, q, 64, sink=sink)
    assert st == 0
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 64, SCALE, sink))


def test_many_sequences_per_cta():
    rng = np.random.default_rng(5)
    recs, table, lens, q = ref.random_batch(rng, rng.integers(0, 200, 500), 16, h_q=2, s_q=2)
    out, lse, st = run(recs, table, lens, q, 16)
    assert st == 0
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 16, SCALE))


@pytest.mark.parametrize("h_q,s_q,n", [(16, 150, 400), (64, 37, 500), (128, 5, 130)])
def test_a_chunk_of_a_prompt_is_causal(h_q, s_q, n):
    rng = np.random.default_rng(s_q)
    recs, table, lens, q = ref.random_batch(rng, [n, s_q, s_q - 3, 1], 32, h_q=h_q, s_q=s_q)
    out, lse, st = run(recs, table, lens, q, 32)
    assert st == 0
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 32, SCALE))


def test_growing_scores_move_the_reference():
    # the scores rise along the sequence by far more than the rescale threshold per tile
    rng = np.random.default_rng(8)
    n = 1500
    lat = np.outer(np.linspace(-30, 30, n), np.ones(512)).astype(np.float32) + 0.1 * rng.standard_normal((n, 512)).astype(np.float32)
    _, table, lens, q = ref.random_batch(rng, [n], 4, spare=0, h_q=24)
    table[0] = np.arange(n // 4)
    recs = oracle.quantize_records(synth.bf16_bits(synth.bf16_from_f32(lat)),
                                   synth.bf16_bits(synth.bf16_from_f32(np.zeros((n, 64), np.float32))), 352)
    q = (q.float() * 0.05 + 0.05 * torch.tensor([1.0, -1.0, 0.0]).repeat(8)[None, None, :, None]).to(torch.bfloat16)
    out, lse, st = run(recs, table, lens, q, 4)
    assert st == 0
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 4, SCALE))


def test_pages_outside_the_pool_are_masked_and_reported():
    rng = np.random.default_rng(9)
    recs, table, lens, q = ref.random_batch(rng, [400, 300], 32, h_q=16)
    table[0, 3], table[1, 0] = recs.shape[0] // 32, -5
    out, lse, st = run(recs, table, lens, q, 32)
    assert st == lib.DEV_INDEX_OUT_OF_RANGE
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 32, SCALE))


def test_lengths_outside_the_table_are_clamped():
    rng = np.random.default_rng(10)
    recs, table, lens, q = ref.random_batch(rng, [256, 100, 64], 32, h_q=16)
    long = lens.copy()
    long[0], long[2] = 9999, -7
    out, lse, st = run(recs, table, long, q, 32)
    assert st == lib.DEV_INDEX_OUT_OF_RANGE
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, long, 32, SCALE))


def test_table_rows_with_a_stride_and_no_pages_behind():
    rng = np.random.default_rng(11)
    recs, table, lens, q = ref.random_batch(rng, [130, 70], 16, h_q=16)
    wide = torch.full((2, table.shape[1] + 7), 2 ** 30, dtype=torch.int32)
    wide[:, :table.shape[1]] = torch.from_numpy(np.where(table < 0, 2 ** 30, table))   # unread entries hold anything
    out, lse = lib.paged_mla_decode(q.to(DEV), torch.from_numpy(recs).to(DEV), wide.to(DEV)[:, :table.shape[1]],
                                    torch.from_numpy(lens).to(DEV), SCALE, page_size=16)
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 16, SCALE))


@pytest.mark.parametrize("h_q,s_q", [(16, 4), (20, 3), (16, 1)])
def test_nan_reaches_the_rows_that_see_it_and_no_other(h_q, s_q):
    rng = np.random.default_rng(12)
    recs, table, lens, q = ref.random_batch(rng, [200, 200, 60], 16, h_q=h_q, s_q=s_q)
    clean = ref.attention(q, recs, False, table, lens, 16, SCALE)
    bad = int(ref.slots_of(table[0], 200, 16)[198 if s_q > 1 else 50])     # seen by the last two queries only
    spare = sorted(set(range(recs.shape[0])) - {int(s) for b in range(3) for s in ref.slots_of(table[b], int(lens[b]), 16)})
    recs[bad, 320:352] = 0x7F
    recs[bad + (1 if s_q == 1 else 0), 256] = 0x7F                            # and one RoPE value
    recs[spare] = 0xFF                                                        # slots behind a sequence's end
    qn = q.clone()
    qn[1, 0, 1, 7] = float("nan")
    qn[1, 0, 2, 7] = float("inf")
    out, lse, st = run(recs, table, lens, qn, 16)
    assert st == 0
    nan = torch.isnan(out).all(-1) & torch.isnan(lse)
    want = torch.zeros_like(nan)
    want[0, max(0, s_q - 2):] = True
    want[1, 0, 1:3] = True
    assert torch.equal(nan, want) and torch.equal(torch.isnan(out).any(-1), want)
    keep = ~want.cpu().numpy()
    o, r = out.float().cpu().numpy()[keep], clean[0][keep]
    assert np.all(np.abs(o - r) <= clean[2][keep])


def test_equal_to_the_sparse_decode_over_the_same_tokens():
    rng = np.random.default_rng(13)
    for h_q in (64, 128):
        recs, table, lens, q = ref.random_batch(rng, [700, 333], 64, h_q=h_q)
        idx = np.full((2, 1, 700), -1, dtype=np.int32)
        for b in range(2):
            idx[b, 0, :lens[b]] = ref.slots_of(table[b], int(lens[b]), 64)
        out, lse, _ = run(recs, table, lens, q, 64)
        o2, l2 = lib.sparse_mla_decode(q.to(DEV), torch.from_numpy(recs).to(DEV), torch.from_numpy(idx).to(DEV), SCALE)
        _, _, t_out, t_lse = ref.attention(q, recs, False, table, lens, 64, SCALE)
        assert np.all((out.float() - o2.float()).abs().cpu().numpy() <= 2 * t_out)
        assert np.all((lse - l2).abs().cpu().numpy() <= 2 * t_lse)


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(14)
    recs, table, lens, q = ref.random_batch(rng, [3000, 10, 555], 64, h_q=48)
    first = run(recs, table, lens, q, 64)
    for _ in range(3):
        again = run(recs, table, lens, q, 64)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_captured_call_follows_the_lengths():
    rng = np.random.default_rng(15)
    recs, table, lens, q = ref.random_batch(rng, [500, 400, 300], 64, h_q=16, s_q=2)
    c, t, n, qd = (torch.from_numpy(recs).to(DEV), torch.from_numpy(table).to(DEV), torch.from_numpy(lens).to(DEV), q.to(DEV))
    lib.paged_mla_decode(qd, c, t, n, SCALE)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = lib.paged_mla_decode(qd, c, t, n, SCALE)
    for new in ([500, 400, 300], [1, 0, 300], [64, 399, 2]):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref.check_attention(out, lse, ref.attention(q, recs, False, table, np.array(new), 64, SCALE))


def test_calls_on_two_streams_with_their_own_workspaces():
    rng = np.random.default_rng(16)
    work = [ref.random_batch(rng, [4000 + 500 * k, 100], 64, h_q=16) for k in range(2)]
    dev = [tuple(torch.from_numpy(x).to(DEV) if isinstance(x, np.ndarray) else x.to(DEV) for x in w) for w in work]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for k in range(2):
            recs, table, lens, q = dev[k]
            outs.append((k, lib.paged_mla_decode(q, recs, table, lens, SCALE, stream=streams[k])))
    torch.cuda.synchronize()
    refs = [ref.attention(w[3], w[0], False, w[1], w[2], 64, SCALE) for w in work]
    for k, (out, lse) in outs:
        ref.check_attention(out, lse, refs[k])


def test_a_pool_past_four_gigabytes():
    # the sequence's pages lie behind the 32-bit offsets of the pool
    pages, ps = 210_000, 64                                # 4.7 GB of 352-byte records
    rng = np.random.default_rng(17)
    recs, table, lens, q = ref.random_batch(rng, [300, 130], ps, h_q=16)
    pool = torch.zeros((pages * ps, 352), dtype=torch.uint8, device=DEV)
    n = recs.shape[0] // ps
    pool[-n * ps:] = torch.from_numpy(recs).to(DEV)
    far = np.where(table < 0, -1, table + pages - n).astype(np.int32)
    out, lse = lib.paged_mla_decode(q.to(DEV), pool, torch.from_numpy(far).to(DEV), torch.from_numpy(lens).to(DEV), SCALE, page_size=ps)
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, ps, SCALE))


def uneven(rng, n, lo, hi, empty=0.0, long=()):
    lens = rng.integers(lo, hi + 1, n)
    lens[rng.random(n) < empty] = 0
    lens[:len(long)] = long
    return lens


@pytest.mark.parametrize("name,h_q,s_q,lens", [
    ("more jobs than the plan has threads, a third of them empty", 17, 2, uneven(np.random.default_rng(20), 300, 1, 260, 0.33)),
    ("one long sequence among short ones", 33, 1, uneven(np.random.default_rng(21), 71, 1, 130, 0.0, (7000, 2500))),
    ("a wave and a little more", 64, 1, uneven(np.random.default_rng(22), 80, 500, 700)),
    ("few sequences, all cut", 128, 1, uneven(np.random.default_rng(23), 5, 1500, 3000)),
    ("many row tiles of one sequence", 128, 90, np.array([700])),
    ("all empty but one", 20, 3, np.array([0, 0, 0, 2, 0, 900, 0])),
    ("nothing at all", 40, 1, np.zeros(9, dtype=np.int64)),
])
def test_plans_of_the_pairs(name, h_q, s_q, lens):
    rng = np.random.default_rng(len(name))
    sink = rng.standard_normal(h_q).astype(np.float32)
    recs, table, lens, q = ref.random_batch(rng, lens, 32, h_q=h_q, s_q=s_q, scale=1.5)
    out, lse, st = run(recs, table, lens, q, 32, sink=sink)
    assert st == 0
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 32, SCALE, sink))


@pytest.mark.parametrize("h_q,s_q", [(16, 1), (24, 1), (64, 2)])
@pytest.mark.parametrize("places", [[(0, 0)], [(0, 3), (1, 9)], [(0, 40), (1, 12)], [(0, k) for k in range(44)]])
def test_pages_outside_the_pool_anywhere(h_q, s_q, places):
    rng = np.random.default_rng(30 + len(places))
    recs, table, lens, q = ref.random_batch(rng, [1400, 410], 32, h_q=h_q, s_q=s_q)
    for b, k in places:
        table[b, k] = recs.shape[0] // 32 + k if k % 2 else -1 - k
    out, lse, st = run(recs, table, lens, q, 32)
    assert st == lib.DEV_INDEX_OUT_OF_RANGE
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 32, SCALE))


@pytest.mark.parametrize("h_q", [16, 48])
def test_references_that_move_in_every_order(h_q):
    # the largest score of a row lies in any tile, also far above or below all others: rows of one call move
    # their references in different tiles, and in both groups of softmax warps
    rng = np.random.default_rng(31)
    recs, table, lens, q = ref.random_batch(rng, [3000, 1000], 64, h_q=h_q, scale=1.0)
    keys = oracle.dequant_records(recs, False)
    for b in range(2):
        slots = ref.slots_of(table[b], int(lens[b]), 64)
        for h in range(h_q):                       # a query along one of the sequence's own keys
            k = keys[slots[(977 * h + 31 * b) % slots.size]]
            q[b, 0, h] = torch.from_numpy(((2.0 - 4.0 * (h % 2)) * (0.2 + h % 5) * k).astype(np.float32)).to(torch.bfloat16)
    out, lse, st = run(recs, table, lens, q, 64)
    assert st == 0
    ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 64, SCALE))


@pytest.mark.parametrize("h_q,s_q", [(16, 1), (64, 3)])
def test_two_graphs_share_a_workspace_and_follow_the_lengths(h_q, s_q):
    rng = np.random.default_rng(32)
    recs, table, lens, q = ref.random_batch(rng, [2000, 300, 0, 700], 64, h_q=h_q, s_q=s_q)
    dev = [torch.from_numpy(x).to(DEV) for x in (recs, table, lens)]
    qs = [q.to(DEV), (0.5 * q.float()).to(torch.bfloat16).to(DEV)]
    ws = torch.empty(lib.paged_workspace_size(4, s_q, h_q), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for x in qs:
        lib.paged_mla_decode(x, dev[0], dev[1], dev[2], SCALE, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lib.paged_mla_decode(x, dev[0], dev[1], dev[2], SCALE, workspace=ws))
        graphs.append(g)
    for now in ([2000, 300, 0, 700], [1, 300, 0, 64], [0, 0, 0, 0], [1999, 299, 5, 699]):
        now = np.minimum(np.array(now, dtype=np.int32), np.maximum(lens, 0))
        dev[2].copy_(torch.from_numpy(now))
        ws.fill_(0xFF)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, (out, lse) in zip(qs, outs):
            ref.check_attention(out, lse, ref.attention(x.cpu(), recs, False, table, now, 64, SCALE))


@pytest.mark.parametrize("h_q", [16, 64, 128])
def test_a_negative_scale_and_none(h_q):
    rng = np.random.default_rng(33)
    recs, table, lens, q = ref.random_batch(rng, [700, 90], 16, h_q=h_q)
    for scale in (-0.04, 0.0):
        out, lse = lib.paged_mla_decode(q.to(DEV), torch.from_numpy(recs).to(DEV), torch.from_numpy(table).to(DEV),
                                        torch.from_numpy(lens).to(DEV), scale, page_size=16)
        ref.check_attention(out, lse, ref.attention(q, recs, False, table, lens, 16, scale))
