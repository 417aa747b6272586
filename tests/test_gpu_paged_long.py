"""nvfp4_paged_mla_decode over long sequences, where small weights add up: one early key outweighs the others and has the
value 0 (an attention sink), so that the output consists of the others. All other keys are alike, and the sequences share
their pages, so that the softmax has a closed form."""
import numpy as np
import pytest
import torch

import nvfp4_kv_cache_sparse_gb300 as lib
import oracle
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
PS = 64
SINK_ROPE = 16.0          # the first key: RoPE dim 0, no NoPE dims; the others: no RoPE dims


def shared_pool(R, tail):
    """Page 0: the sink and 63 other keys; page 1: 64 other keys. Returns the records and the others' dequantized values."""
    lat = np.tile(tail.astype(np.float32), (2 * PS, 1))
    rope = np.zeros((2 * PS, 64), dtype=np.float32)
    lat[0], rope[0, 0] = 0.0, SINK_ROPE
    recs = oracle.quantize_records(synth.bf16_bits(synth.bf16_from_f32(lat)), synth.bf16_bits(synth.bf16_from_f32(rope)), R)
    keys = oracle.dequant_records(recs)
    assert np.all(keys[0, :512] == 0) and keys[0, 512] == SINK_ROPE and np.all(keys[1:] == keys[1]) and np.all(keys[1:, 512:] == 0)
    return recs, keys[1, :512]


def call(recs, batch, n, q):
    table = torch.ones((batch, -(-n // PS)), dtype=torch.int32)
    table[:, 0] = 0
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = lib.paged_mla_decode(q.to(DEV).expand(batch, -1, -1, -1).contiguous(), torch.from_numpy(recs).to(DEV), table.to(DEV),
                                    torch.full((batch,), n, dtype=torch.int32, device=DEV), 1.0, page_size=PS, dev_status=status)
    assert int(status.item()) == 0
    return out.double().cpu().numpy()[:, 0], lse.double().cpu().numpy()[:, 0]


def queries(h_q, gaps):
    """Rows that see the sink `gaps` nats above the other keys, whose score is 0."""
    q = torch.zeros(1, 1, h_q, 576)
    for h in range(h_q):
        q[0, 0, h, 512] = gaps[h % len(gaps)] / SINK_ROPE
    q = q.to(torch.bfloat16)
    return q, q[0, 0, :, 512].double().numpy() * SINK_ROPE


@pytest.mark.parametrize("R", [352, 432])
@pytest.mark.parametrize("h_q,batch,n", [(16, 304, 2048), (16, 152, 131072), (16, 3, 1_000_000), (3, 70, 20000),
                                         (64, 152, 2048), (128, 76, 16384), (40, 40, 131072)])
def test_keys_far_below_the_first_one_keep_their_share(R, h_q, batch, n):
    """With N = n - 1 other keys of weight p = e^-gap and value v: out = N p v / (1 + N p), lse = gap + ln(1 + N p).

    Bounds. A score and its exp2 are off by 2^-17 (the argument, at most 2^5, by four roundings of 2^-24 of it, and 2^-22
    of exp2), which the weights are relative to 1, and lse. A weight is rounded to f16: by 2^-11 of itself, at least by
    2^-25 against a reference at most 2^k below the first key, k = gap / ln 2 - 14 within [3, 12] (every other quarter of the
    first tile holds scores of 0 only). Adding one value per tile of 128 keys to a row sum rounds 2^-24 of it each time,
    16 keys to an output 2^-23 of it. Parts of a cut row are f16 (2^-11 of it, at least 2^-25), out is bf16 (2^-8)."""
    recs, v = shared_pool(R, np.where(np.arange(512) % 3 == 0, -1.0, 1.0) * (1 + np.arange(512) % 5))
    q, gap = queries(h_q, [8.0, 12.0, 14.0, 17.0, 18.0, 20.0])
    out, lse = call(recs, batch, n, q)
    N, p = n - 1, np.exp(-gap)
    S = 1 + N * p
    want = (N * p / S)[:, None] * v
    k = np.clip(gap / np.log(2) - 14, 3, 12)
    sums = n / 128 * 2.0 ** -24
    rel = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -16 + sums + n / 16 * 2.0 ** -23
    tol = rel * np.abs(want) + (2.0 ** -25 * 2.0 ** -k * N / S)[:, None] * np.abs(v) + 2.0 ** -25
    err = np.abs(out - want)
    assert np.all(err <= tol), f"{np.max(err / tol):.3g} times the bound"
    assert np.all(np.abs(lse - (gap + np.log(S))) <= 2.0 ** -16 + sums + 2.0 ** -22 * gap)


@pytest.mark.parametrize("R", [352, 432])
@pytest.mark.parametrize("h_q,batch,n", [(16, 76, 2048), (16, 1, 9000), (64, 20, 2048), (128, 3, 5000)])
def test_small_outputs_of_cut_rows(R, h_q, batch, n):
    """The bounds of the test above with the smallest value other than 0, 2^-10, and rows that are cut: a part is held in f16
    after a scale of 16, so that it is off by 2^-11 of itself and at least by 2^-29."""
    recs, _ = shared_pool(R, np.ones(512))
    recs[1:, :256] = 0x91                            # codes 0.5 and -0.5
    recs[1:, 320 if R == 352 else 256:][:, :32] = 0x01   # scales 2^-9
    v = oracle.dequant_records(recs)[1, :512]
    assert np.all(np.abs(v) == 2.0 ** -10)
    q, gap = queries(h_q, [12.0, 13.0, 14.0, 15.0, 16.0, 17.0])
    out, lse = call(recs, batch, n, q)
    N, p = n - 1, np.exp(-gap)
    S = 1 + N * p
    want = (N * p / S)[:, None] * v
    k = np.clip(gap / np.log(2) - 14, 3, 12)
    rel = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -16 + n / 128 * 2.0 ** -24 + n / 16 * 2.0 ** -23
    tol = rel * np.abs(want) + (2.0 ** -25 * 2.0 ** -k * N / S)[:, None] * np.abs(v) + 2.0 ** -29
    err = np.abs(out - want)
    assert np.all(err <= tol), f"{np.max(err / tol):.3g} times the bound"


@pytest.mark.parametrize("h_q,batch", [(1, 40_000), (16, 40_000), (24, 40_000), (1, 10_000_000)])
def test_padding_between_two_sequences(h_q, batch):
    # a CTA's run spans the gap; read one length at a time, the largest took longer than the waits of its other warps last
    rng = np.random.default_rng(batch)
    ps, n0, n1 = 4096, 169 * 64, 151 * 64 - 5
    lat = synth.bf16_from_f32(rng.standard_normal((ps, 512)).astype(np.float32))
    recs = oracle.quantize_records(synth.bf16_bits(lat), synth.bf16_bits(synth.bf16_from_f32(np.zeros((ps, 64), np.float32))), 352)
    v = oracle.dequant_records(recs)[:, :512]
    lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
    lens[0], lens[-1] = n0, n1
    table = torch.zeros((batch, 3), dtype=torch.int32, device=DEV)     # one page, named by every entry
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.zeros((batch, 1, h_q, 576), dtype=torch.bfloat16, device=DEV)
    out, lse = lib.paged_mla_decode(q, torch.from_numpy(recs).to(DEV), table, lens, 1.0, page_size=ps, dev_status=status)
    assert int(status.item()) == 0
    assert not out[1:-1].any() and bool(torch.isneginf(lse[1:-1]).all())
    for b, n in ((0, n0), (-1, n1)):                                   # scores 0: means over the tokens
        seen = np.bincount(np.arange(n) % ps, minlength=ps) / n
        want, size = seen @ v, seen @ np.abs(v)
        assert np.all(np.abs(out[b, 0].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * size + 2.0 ** -28)
        assert np.all(np.abs(lse[b, 0].double().cpu().numpy() - np.log(n)) <= 2.0 ** -18)
