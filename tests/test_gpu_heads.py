"""The calls around the latent attention on the GPU against their formulas in 64 bits: products per head, the
expansion of pages and the attention of packed chunks."""
import numpy as np
import pytest
import torch

import heads_reference as ref
import nvfp4_kv_cache_sparse_gb300 as lib
import paged_reference as pages
from heads_reference import bf16, starts, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5


def zero_status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def tables(n, rng):
    angle = rng.uniform(-np.pi, np.pi, (n, 32))
    return torch.from_numpy(np.cos(angle).astype(np.float32)), torch.from_numpy(np.sin(angle).astype(np.float32))


@pytest.mark.parametrize("h", [1, 3, 16, 64, 128])
@pytest.mark.parametrize("T", [1, 5, 127, 128, 129, 300])
def test_absorb_and_project(T, h):
    rng = np.random.default_rng(1000 * h + T)
    kv_b = weights(rng, h)
    half = bool(T & 1)
    q, pos, (cos, sin) = bf16(rng, T, h, 192), torch.from_numpy(rng.integers(0, 500, T)), tables(500, rng)
    st = zero_status()
    got = lib.mla_absorb_query(q.to(DEV), kv_b.to(DEV), pos.to(DEV), cos.to(DEV), sin.to(DEV), half, dev_status=st)
    ref.check(got, *ref.absorb(q, kv_b, pos, cos, sin, half))
    latent = bf16(rng, T, h, 512)
    back = lib.mla_project_values(latent.to(DEV), kv_b.to(DEV), dev_status=st)
    ref.check(back, *ref.project(latent, kv_b))
    assert int(st.item()) == 0


@pytest.mark.parametrize("h", [5, 128])
def test_products_of_many_tokens_over_several_heads_per_cta(h):
    rng = np.random.default_rng(h)
    T = 1100 if h == 5 else 520
    kv_b = weights(rng, h)
    q = bf16(rng, T, h, 192)
    got = lib.mla_absorb_query(q.to(DEV), kv_b.to(DEV))
    ref.check(got, *ref.absorb(q, kv_b))
    assert torch.equal(got[..., 512:].cpu(), q[..., 128:])           # without positions the RoPE dims are copied
    latent = bf16(rng, T, h, 512)
    ref.check(lib.mla_project_values(latent.to(DEV), kv_b.to(DEV)), *ref.project(latent, kv_b))


def test_products_of_strided_inputs():
    rng = np.random.default_rng(2)
    T, h = 150, 6
    kv_b = weights(rng, 2 * h).view(h, 2, 256, 512)[:, 1]             # every other head's weights
    q = bf16(rng, h, T, 200).transpose(0, 1)[..., 8:]                 # heads outermost, rows with a gap
    wide = bf16(rng, T, h, 520)
    dev_q = torch.empty(h, T, 200, dtype=torch.bfloat16, device=DEV).transpose(0, 1)[..., 8:]
    dev_q.copy_(q)
    dev_b = weights(rng, 2 * h).to(DEV).view(h, 2, 256, 512)[:, 1]
    dev_b.copy_(kv_b)
    dev_wide = wide.to(DEV)
    assert not dev_q.is_contiguous() and not dev_b.is_contiguous()
    ref.check(lib.mla_absorb_query(dev_q, dev_b), *ref.absorb(q, kv_b))
    ref.check(lib.mla_project_values(dev_wide[..., 8:], dev_b), *ref.project(wide[..., 8:], kv_b))


def test_absorb_reports_positions_outside_the_tables():
    rng = np.random.default_rng(3)
    T, h = 140, 4
    kv_b, q, (cos, sin) = weights(rng, h), bf16(rng, T, h, 192), tables(50, rng)
    pos = torch.from_numpy(rng.integers(0, 50, T))
    bad = pos.clone()
    bad[7], bad[139] = 50, -1
    out, st = torch.full((T, h, 576), 7.0, dtype=torch.bfloat16, device=DEV), zero_status()
    lib.mla_absorb_query(q.to(DEV), kv_b.to(DEV), bad.to(DEV), cos.to(DEV), sin.to(DEV), True, out=out, dev_status=st)
    assert int(st.item()) == lib.DEV_POSITION_OUT_OF_RANGE
    r, tol = ref.absorb(q, kv_b, pos, cos, sin, True)
    r[[7, 139], :, 512:], tol[[7, 139], :, 512:] = 7.0, 0.0           # left as they were
    ref.check(out, r, tol)


@pytest.mark.parametrize("R,blk", [(352, False), (352, True), (432, False)])
@pytest.mark.parametrize("page_size", [1, 16, 64, 256])
@pytest.mark.parametrize("h", [1, 7])
def test_expand_records_and_page_sizes(R, blk, page_size, h):
    rng = np.random.default_rng(R + page_size + h)
    recs, table, lens, _ = pages.random_batch(rng, [300, 0, 1, 255, 64], page_size, R=R, blk=blk)
    kv_b, st = weights(rng, h), zero_status()
    n = int(lens.sum())
    kv = torch.full((n + 9, h, 256), 5.0, dtype=torch.bfloat16, device=DEV)
    pe = torch.full((n + 9, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    lib.paged_mla_expand(torch.from_numpy(recs).to(DEV), torch.from_numpy(table).to(DEV), starts(lens).to(DEV), kv_b.to(DEV), n + 9,
                         page_size=page_size, kv=kv, k_pe=pe, dev_status=st, block_scales=blk)
    r, tol, r_pe = ref.expand(recs, blk, table, lens, page_size, kv_b)
    ref.check(kv[:n], r, tol)
    assert np.array_equal(ref.f64(pe[:n]), r_pe)
    assert torch.all(kv[n:] == 5.0) and torch.all(pe[n:] == 5.0)      # rows behind the last sequence
    assert int(st.item()) == 0


@pytest.mark.parametrize("h,lens", [(128, [200]), (128, [700, 513]), (3, [40000]), (16, [0, 0, 0]), (16, [1] * 300), (64, [1300, 257])])
def test_expand_runs_over_tiles_and_heads(h, lens):
    rng = np.random.default_rng(h + len(lens))
    recs, table, lens, _ = pages.random_batch(rng, lens, 64)
    kv_b = weights(rng, h)
    n = int(lens.sum())
    kv, pe = lib.paged_mla_expand(torch.from_numpy(recs).to(DEV), torch.from_numpy(table).to(DEV), starts(lens).to(DEV), kv_b.to(DEV), n)
    if n == 0:
        assert kv.shape == (0, h, 256) and pe.shape == (0, 64)
        return
    r, tol, r_pe = ref.expand(recs, False, table, lens, 64, kv_b)
    ref.check(kv, r, tol)
    assert np.array_equal(ref.f64(pe), r_pe)


def test_expand_reports_pages_outside_the_pool():
    rng = np.random.default_rng(4)
    recs, table, lens, _ = pages.random_batch(rng, [400, 300], 32)
    table[0, 3], table[1, 0] = recs.shape[0] // 32, -5
    long = np.array([400, table.shape[1] * 32 + 3])                   # the second one goes on behind the table's last entry
    table[1, 10:] = table[1, 9]
    kv_b, st = weights(rng, 3), zero_status()
    n = int(long.sum())
    kv, pe = lib.paged_mla_expand(torch.from_numpy(recs).to(DEV), torch.from_numpy(table).to(DEV), starts(long).to(DEV), kv_b.to(DEV), n,
                                  page_size=32, dev_status=st)
    assert int(st.item()) == lib.DEV_INDEX_OUT_OF_RANGE
    r, tol, r_pe = ref.expand(recs, False, table, long, 32, kv_b)
    ref.check(kv, r, tol)
    assert np.array_equal(ref.f64(pe), r_pe)


def attend(rng, q_lens, k_lens, h, scale=SCALE, sink=None, pad=0, q=None, kv=None, pe=None):
    q = bf16(rng, sum(q_lens) + pad, h, 192) if q is None else q
    kv = bf16(rng, sum(k_lens) + pad, h, 256) if kv is None else kv
    pe = bf16(rng, sum(k_lens) + pad, 64) if pe is None else pe
    out = torch.full((q.shape[0], h, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((q.shape[0], h), 3.0, device=DEV)
    st = zero_status()
    lib.ragged_mla_attention(q.to(DEV), kv.to(DEV), pe.to(DEV), starts(q_lens).to(DEV), starts(k_lens).to(DEV), scale,
                             attn_sink=None if sink is None else torch.from_numpy(sink).to(DEV), out=out, lse=lse, dev_status=st)
    assert int(st.item()) == 0
    n = sum(q_lens)
    assert torch.all(out[n:] == 3.0) and torch.all(lse[n:] == 3.0)    # rows behind the last sequence
    used = sum(k_lens)
    ref.check_attention(out[:n], lse[:n], ref.attention(q[:n], kv[:used], pe[:used], q_lens, k_lens, scale, sink))


@pytest.mark.parametrize("h", [1, 3, 16])
@pytest.mark.parametrize("lq,lk", [(1, 1), (1, 127), (1, 128), (1, 129), (2, 700), (127, 127), (128, 128), (129, 129), (255, 300), (256, 256),
                                   (257, 257), (300, 1000), (5, 4), (300, 20), (400, 129), (7, 0)])
def test_one_sequence(lq, lk, h):
    attend(np.random.default_rng(lq * 7 + lk), [lq], [lk], h)


@pytest.mark.parametrize("h", [1, 5, 64, 128])
def test_packed_sequences_of_all_kinds(h):
    q_lens = [0, 1, 300, 0, 128, 2, 65, 129, 4]
    k_lens = [5, 1, 300, 0, 500, 0, 64, 1, 260]
    rng = np.random.default_rng(h)
    attend(rng, q_lens, k_lens, h, sink=rng.standard_normal(h).astype(np.float32), pad=70)


def test_many_short_sequences():
    rng = np.random.default_rng(6)
    q_lens = list(map(int, rng.integers(0, 9, 400)))
    k_lens = [n + int(e) for n, e in zip(q_lens, rng.integers(0, 40, 400))]
    attend(rng, q_lens, k_lens, 2)


def test_padding_between_two_sequences():
    rng = np.random.default_rng(14)
    gap = [0] * 50000
    attend(rng, gap + [130, 3] + gap + [40] + gap, gap + [200, 3] + [7] * 50000 + [41] + gap, 3)


@pytest.mark.parametrize("h,lq,lk", [(1, 3, 9001), (2, 256, 6000), (5, 700, 3333)])
def test_tiles_that_several_ctas_share(h, lq, lk):
    rng = np.random.default_rng(lk)
    attend(rng, [lq, 1], [lk, 40], h, sink=2 * rng.standard_normal(h).astype(np.float32))


# (long sequences whose rows fill tiles of 512 go to CTA pairs)
@pytest.mark.parametrize("h,q_lens,k_lens", [(1, [512], [4000]), (3, [512, 384], [3500, 4001]), (2, [1000, 40, 500], [5000, 3000, 4000]), (5, [2048], [2500]),
                                             (4, [511, 0, 513, 640], [3000, 7000, 2900, 640]), (2, [400, 400], [9000, 130])])
def test_long_sequences(h, q_lens, k_lens):
    rng = np.random.default_rng(sum(k_lens))
    attend(rng, q_lens, k_lens, h, sink=rng.standard_normal(h).astype(np.float32), pad=0)


def test_scores_that_jump_far_above_the_reference():
    # within a block, and between blocks, by more than the 2^64 that the reference may lag behind
    rng = np.random.default_rng(12)
    for lq, lk in ((130, 700), (512, 3000)):
        kv = bf16(rng, lk, 2, 256)
        jump = torch.zeros(lk)
        jump[20], jump[100:110], jump[300], jump[lk // 2:] = 90.0, 200.0, 420.0, 600.0
        kv[:, :, 0] = jump[:, None].to(torch.bfloat16)
        q = (0.05 * bf16(rng, lq, 2, 192).float()).to(torch.bfloat16)
        q[..., 0] = torch.tensor([1.0, -1.0], dtype=torch.bfloat16)
        attend(rng, [lq], [lk], 2, scale=1.0, q=q, kv=kv)


def test_rising_and_falling_scores_move_the_reference():
    rng = np.random.default_rng(8)
    n, h = 1200, 4
    ramp = torch.linspace(-30, 30, n)[:, None, None]
    kv = bf16(rng, n, h, 256)
    kv[..., :128] = (0.05 * kv[..., :128].float() + ramp).to(torch.bfloat16)
    q = (0.02 * bf16(rng, 300, h, 192).float() + 0.05 * torch.tensor([1.0, -1.0, 0.0, 3.0])[None, :, None]).to(torch.bfloat16)
    attend(rng, [300], [n], h, scale=1.0, q=q, kv=kv)


@pytest.mark.parametrize("scale", [0.0, -0.07, 3.0])
def test_scales(scale):
    rng = np.random.default_rng(9)
    attend(rng, [140, 3], [300, 2], 3, scale=scale)


def test_what_lies_behind_a_sequence_does_not_reach_it():
    # the keys and values behind a sequence's last one are another's, or nobody's, and not numbers
    rng = np.random.default_rng(10)
    h, q_lens, k_lens = 4, [130, 70, 9], [200, 140, 77]
    clean = bf16(rng, sum(k_lens), h, 256), bf16(rng, sum(k_lens), 64)
    q = bf16(rng, sum(q_lens), h, 192)
    kv, pe, dq = (torch.cat([t, torch.full_like(t[:150], float("nan"))]) for t in (*clean, q))
    kv[200:340], pe[200:340] = float("nan"), float("inf")            # the second sequence's
    out, lse = lib.ragged_mla_attention(dq.to(DEV), kv.to(DEV), pe.to(DEV), starts(q_lens).to(DEV), starts(k_lens).to(DEV), SCALE)
    r = ref.attention(q, *clean, q_lens, k_lens, SCALE)
    for a, b in ((0, 130), (200, 209)):
        ref.check_attention(out[a:b], lse[a:b], tuple(x[a:b] for x in r))
    assert torch.isnan(out[130:200].float()).all()


@pytest.mark.parametrize("lq,lk", [(300, 300), (140, 500), (600, 3100), (1100, 4000)])   # (the last two on CTA pairs)
def test_values_that_are_not_finite_reach_the_rows_that_see_them_only(lq, lk):
    rng = np.random.default_rng(lk)
    h, odd = 3, lk - lq + 2 * lq // 3                                  # a key that the last third of the rows sees
    q, kv, pe = bf16(rng, lq + 50, h, 192), bf16(rng, lk + 80, h, 256), bf16(rng, lk + 80, 64)
    dirty = kv.clone()
    dirty[odd, 0, 133], dirty[odd + 1, 0, 250], dirty[odd + 2, 1, 255], dirty[odd + 9, 1, 128] = float("nan"), float("inf"), -float("inf"), float("nan")
    st = zero_status()
    out, lse = lib.ragged_mla_attention(q.to(DEV), dirty.to(DEV), pe.to(DEV), starts([lq, 50]).to(DEV), starts([lk, 80]).to(DEV), SCALE, dev_status=st)
    assert int(st.item()) == 0
    r = ref.attention(q, kv, pe, [lq, 50], [lk, 80], SCALE)
    first = odd - (lk - lq)                                            # the first row that sees the NaN
    ref.check_attention(out[:first], lse[:first], tuple(x[:first] for x in r))
    ref.check_attention(out[lq:], lse[lq:], tuple(x[lq:] for x in r))  # another sequence
    ref.check_attention(out[:, 2], lse[:, 2], tuple(x[:, 2] for x in r))   # another head
    assert torch.isnan(out[first:lq, 0, 5].float()).all() and not torch.isfinite(out[first + 1:lq, 0, 122].float()).any()
    assert not torch.isfinite(out[first + 2:lq, 1, 127].float()).any() and torch.isnan(out[first + 9:lq, 1, 0].float()).all()
    ref.check_attention(out[:first + 2, 1], lse[:first + 2, 1], tuple(x[:first + 2, 1] for x in r))
    ref.check(lse.cpu().numpy().astype(np.float64), r[1], r[3], "lse")  # the weights are what they are


def test_attention_of_strided_inputs():
    rng = np.random.default_rng(11)
    h, q_lens, k_lens = 3, [150, 20], [180, 90]
    q, kv, pe = bf16(rng, 170, h, 192), bf16(rng, 270, h, 256), bf16(rng, 270, 64)
    dq = torch.zeros(h, 170, 208, dtype=torch.bfloat16, device=DEV).transpose(0, 1)[..., 16:]
    dkv = torch.zeros(270, 2 * h, 256, dtype=torch.bfloat16, device=DEV)[:, ::2]
    dpe = torch.zeros(270, 576, dtype=torch.bfloat16, device=DEV)[:, 512:]
    for d, s in ((dq, q), (dkv, kv), (dpe, pe)):
        d.copy_(s)
    out, lse = lib.ragged_mla_attention(dq, dkv, dpe, starts(q_lens).to(DEV), starts(k_lens).to(DEV), SCALE)
    ref.check_attention(out, lse, ref.attention(q, kv, pe, q_lens, k_lens, SCALE))


def test_offsets_beyond_32_bits():
    # 128 heads: the queries' results and the keys pass 2^31 elements; a few rows at the end are looked at
    rng = np.random.default_rng(13)
    h, T, last = 128, 30000, 3
    kv_b = weights(rng, h)
    q = bf16(rng, last, h, 192)
    dq = torch.zeros(T, h, 192, dtype=torch.bfloat16, device=DEV)
    dq[-last:] = q.to(DEV)
    out = lib.mla_absorb_query(dq, kv_b.to(DEV))
    assert out.numel() > 2 ** 31
    ref.check(out[-last:], *ref.absorb(q, kv_b))
    assert torch.all(out[-200:-last] == 0)
    del out, dq
    lat = torch.zeros(36000, h, 512, dtype=torch.bfloat16, device=DEV)
    assert lat.numel() > 2 ** 31
    o = bf16(rng, last, h, 512)
    lat[-last:] = o.to(DEV)
    ref.check(lib.mla_project_values(lat, kv_b.to(DEV))[-last:], *ref.project(o, kv_b))
    del lat
    # the last of many sequences in pages, and attention over its keys
    recs, table, lens, _ = pages.random_batch(rng, [130], 64)
    n = 66000
    starts_k = torch.tensor([0] + [n - 130] * 1 + [n], dtype=torch.int32, device=DEV)
    wide = torch.full((2, -(-n // 64)), 0, dtype=torch.int32, device=DEV)
    wide[1, :table.shape[1]] = torch.from_numpy(table[0]).to(DEV)
    kv, pe = lib.paged_mla_expand(torch.from_numpy(recs).to(DEV), wide, starts_k, kv_b.to(DEV), n)
    assert kv.numel() > 2 ** 31
    r, tol, r_pe = ref.expand(recs, False, table, lens, 64, kv_b)
    ref.check(kv[-130:], r, tol)
    assert np.array_equal(ref.f64(pe[-130:]), r_pe)
    q = bf16(rng, 5, h, 192)
    out, lse = lib.ragged_mla_attention(q.to(DEV), kv, pe, torch.tensor([0, 0, 5], dtype=torch.int32, device=DEV), starts_k, SCALE)
    ref.check_attention(out, lse, ref.attention(q, kv[-130:].cpu(), pe[-130:].cpu(), [5], [130], SCALE))
