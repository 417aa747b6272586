"""The attention of packed chunks on the GPU at the ends of what its arguments may be, on one CTA each and on CTA pairs, against its
formula in 64 bits."""
import numpy as np
import pytest
import torch

import heads_reference as ref
import nvfp4_kv_cache_sparse_gb300 as lib
from heads_reference import bf16, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5
SHAPES = [(140, 300), (512, 3000)]   # the second one on CTA pairs


def takes_pairs(rows, keys, batch):
    """The kernels' rule, by the tensors' rows and the batch"""
    r, k = -(-rows // batch), keys // batch
    blocks = max(k - r // 2, 0) // 128
    return 12 * -(-r // 512) * (blocks + 3) < 7 * -(-r // 256) * (blocks + 1)


def call(q, kv, pe, q_lens, k_lens, scale=SCALE, **more):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = lib.ragged_mla_attention(q.to(DEV), kv.to(DEV), pe.to(DEV), starts(q_lens).to(DEV), starts(k_lens).to(DEV), scale, dev_status=st, **more)
    assert int(st.item()) == 0
    return out, lse


@pytest.mark.parametrize("lq,lk", SHAPES)
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_a_scale_of_zero_weighs_all_keys_alike(lq, lk, scale):
    # scores of up to some 2^124 before the scale
    rng = np.random.default_rng(lk)
    assert takes_pairs(lq, lk, 1) == (lq == 512)
    q, kv, pe = bf16(rng, lq, 2, 192, scale=2.0 ** 58), bf16(rng, lk, 2, 256), bf16(rng, lk, 64, scale=2.0 ** 58)
    kv[..., :128] = bf16(rng, lk, 2, 128, scale=2.0 ** 58)
    out, lse = call(q, kv, pe, [lq], [lk], scale)
    ref.check_attention(out, lse, ref.attention(q, kv, pe, [lq], [lk], scale))


@pytest.mark.parametrize("lq,lk", SHAPES)
def test_scores_that_are_infinite(lq, lk):
    # a key that all rows see, infinite in one dim: a score of -infinity weighs nothing, one of +infinity makes its row NaN
    rng = np.random.default_rng(lk + 1)
    odd = (lk - lq) // 2
    q, kv, pe = bf16(rng, lq, 2, 192), bf16(rng, lk, 2, 256), bf16(rng, lk, 64)
    sign = torch.where(torch.arange(lq) % 3 == 0, -1.0, 1.0)
    q[..., 3] = sign[:, None].to(torch.bfloat16)
    dirty = kv.clone()
    dirty[odd, :, 3] = -float("inf")
    out, lse = call(q, dirty, pe, [lq], [lk])
    rest = torch.arange(lk) != odd
    r = ref.attention(q, kv[rest], pe[rest], [lq], [lk - 1], SCALE)
    fine = (sign > 0).numpy()
    ref.check_attention(out[sign.to(DEV) > 0], lse[sign.to(DEV) > 0], tuple(x[fine] for x in r))
    assert torch.isnan(out[sign.to(DEV) < 0].float()).all() and torch.isnan(lse[sign.to(DEV) < 0]).all()


def test_what_is_not_finite_on_cta_pairs_reaches_the_rows_that_see_it_only():
    # Keys and values behind the sequences' ends and behind the batch are NaN or infinite, and so are single values that some rows see: one for the first
    # rows of a tile's second half, one in the other CTA's columns, one in the last block
    rng = np.random.default_rng(21)
    h, q_lens, k_lens = 3, [700, 211], [6003, 5100]
    n, m = sum(q_lens), sum(k_lens)
    assert takes_pairs(n + 70, m + 300, 2)
    q, kv, pe = bf16(rng, n + 70, h, 192), bf16(rng, m + 300, h, 256), bf16(rng, m + 300, 64)
    dirty, dirty_pe = kv.clone(), pe.clone()
    dirty[m:], dirty_pe[m:] = float("nan"), float("inf")
    seen = [(0, 6003 - 700 + 250, 0, 130), (0, 6003 - 700 + 400, 1, 129), (0, 6003 - 700 + 401, 1, 255), (0, 6002, 2, 200),
            (1, 5100 - 211 + 60, 0, 190), (1, 5100 - 211 + 210, 1, 250)]   # sequence, key, head, dim
    nan = np.zeros((n, h), dtype=bool)
    for i, (b, key, head, dim) in enumerate(seen):
        dirty[key + b * 6003, head, dim] = (float("nan"), float("inf"), -float("inf"))[i % 3]
        row = b * 700 + key - (k_lens[b] - q_lens[b])                  # the first one that sees it
        nan[row:700 + b * 211, head] = True
    out, lse = call(q, dirty, dirty_pe, q_lens, k_lens)
    r = ref.attention(q[:n], kv[:m], pe[:m], q_lens, k_lens, SCALE)
    ref.check(lse[:n].cpu().numpy().astype(np.float64), r[1], r[3], "lse")
    got = ref.f64(out[:n])
    assert np.all(np.abs(got - r[0])[~nan] <= r[2][~nan])
    for b, key, head, dim in seen:
        first = b * 700 + key - (k_lens[b] - q_lens[b])
        assert not np.isfinite(got[first:700 + b * 211, head, dim - 128]).any()


def test_strided_inputs_and_a_queue_of_calls_on_cta_pairs():
    rng = np.random.default_rng(22)
    h, q_lens, k_lens = 5, [512, 384], [4000, 3501]
    n, m = sum(q_lens), sum(k_lens)
    assert takes_pairs(n, m, 2)
    q, kv, pe = bf16(rng, n, h, 192), bf16(rng, m, h, 256), bf16(rng, m, 64)
    dq = torch.zeros(h, n, 208, dtype=torch.bfloat16, device=DEV).transpose(0, 1)[..., 16:]
    dkv = torch.zeros(h, m, 256, dtype=torch.bfloat16, device=DEV).transpose(0, 1)   # heads outermost
    dpe = torch.zeros(m, 576, dtype=torch.bfloat16, device=DEV)[:, 512:]
    for d, s in ((dq, q), (dkv, kv), (dpe, pe)):
        d.copy_(s)
    sink = rng.standard_normal(h).astype(np.float32)
    ws = torch.empty(lib.ragged_workspace_size(), dtype=torch.uint8, device=DEV)
    got = [call(dq, dkv, dpe, q_lens, k_lens, attn_sink=torch.from_numpy(sink).to(DEV), workspace=ws)]
    for _ in range(20):   # nothing waits between these, and short sequences come between (one CTA each, the same workspace)
        got.append(lib.ragged_mla_attention(dq, dkv, dpe, starts(q_lens).to(DEV), starts(k_lens).to(DEV), SCALE, attn_sink=torch.from_numpy(sink).to(DEV), workspace=ws))
        lib.ragged_mla_attention(dq[:90], dkv[:90], dpe[:90], starts([90]).to(DEV), starts([90]).to(DEV), SCALE, workspace=ws)
    ref.check_attention(*got[0], ref.attention(q, kv, pe, q_lens, k_lens, SCALE, sink))
    for g in got[1:]:
        assert torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


def test_a_captured_call_on_cta_pairs_follows_the_lengths_of_its_replay():
    rng = np.random.default_rng(23)
    h, n, m = 4, 1024, 9000
    assert takes_pairs(n, m, 2)
    q, kv, pe = bf16(rng, n, h, 192), bf16(rng, m, h, 256), bf16(rng, m, 64)
    dq, dkv, dpe = q.to(DEV), kv.to(DEV), pe.to(DEV)
    cq, ck = starts([512, 512]).to(DEV), starts([4500, 4500]).to(DEV)
    out, lse = torch.empty(n, h, 128, dtype=torch.bfloat16, device=DEV), torch.empty(n, h, device=DEV)
    ws = torch.empty(lib.ragged_workspace_size(), dtype=torch.uint8, device=DEV)
    lib.ragged_mla_attention(dq, dkv, dpe, cq, ck, SCALE, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.ragged_mla_attention(dq, dkv, dpe, cq, ck, SCALE, out=out, lse=lse, workspace=ws)
    for q_lens, k_lens in (([512, 512], [4500, 4500]), ([1, 1000], [8000, 1000]), ([0, 0], [0, 0]), ([300, 3], [100, 70]), ([0, 1], [9000, 0]), ([257, 600], [700, 5])):
        cq.copy_(starts(q_lens))
        ck.copy_(starts(k_lens))
        out.fill_(3.0)
        lse.fill_(3.0)
        graph.replay()
        used, keys = sum(q_lens), sum(k_lens)
        assert torch.all(out[used:] == 3.0) and torch.all(lse[used:] == 3.0)
        ref.check_attention(out[:used], lse[:used], ref.attention(q[:used], kv[:keys], pe[:keys], q_lens, k_lens, SCALE))
