"""The calls around the latent attention as a serving loop makes them: both forms of the attention over the same cache, from
graphs, on other streams and with shared buffers."""
import numpy as np
import pytest
import torch

import heads_reference as ref
import nvfp4_kv_cache_sparse_gb300 as lib
import oracle
import synth
from heads_reference import bf16, starts, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rotation(n):
    angle = np.arange(n)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    return torch.from_numpy(np.cos(angle).astype(np.float32)), torch.from_numpy(np.sin(angle).astype(np.float32))


def serve(h, k_lens, q_lens, R=352, page_size=16, seed=0):
    """Pages taken, tokens appended with norm and rotation, and the queries of each sequence's last tokens"""
    rng = np.random.default_rng(seed)
    batch, total = len(k_lens), sum(k_lens)
    pages = sum(-(-n // page_size) for n in k_lens) + 5
    width = max(-(-n // page_size) for n in k_lens)
    pool = torch.zeros(pages * page_size, R, dtype=torch.uint8, device=DEV)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    lens, refs = torch.zeros(batch, dtype=torch.int32, device=DEV), torch.zeros(pages, dtype=torch.int32, device=DEV)
    slots = lib.resize_sequences([pool], table, lens, refs, i32(*k_lens), max(k_lens), page_size=page_size)
    slots = torch.cat([slots[b, :n] for b, n in enumerate(k_lens)])
    cos, sin = rotation(max(k_lens) + 1)
    pos_k = torch.cat([torch.arange(n) for n in k_lens])
    pos_q = torch.cat([torch.arange(k - q, k) for q, k in zip(q_lens, k_lens)])
    lib.norm_rope_quantize_append(bf16(rng, total, 512).to(DEV), torch.ones(512, dtype=torch.bfloat16, device=DEV), 1e-6, bf16(rng, total, 64).to(DEV),
                                  pos_k.to(DEV), cos.to(DEV), sin.to(DEV), True, slots, pool)
    q = bf16(rng, sum(q_lens), h, 192)
    return dict(pool=pool, table=table, lens=lens, page_size=page_size, cos=cos, sin=sin, pos_q=pos_q, q=q, kv_b=weights(rng, h), R=R)


def truth(s, q_lens, k_lens):
    """Attention in the expanded form in 64 bits over the records in the cache, nothing rounded on the way"""
    recs, table = s["pool"].cpu().numpy(), s["table"].cpu().numpy()
    kv, _, k_pe = ref.expand(recs, False, table, k_lens, s["page_size"], s["kv_b"])
    q = ref.f64(s["q"])
    pe, _ = ref.rotate(q[..., 128:], s["cos"].numpy().astype(np.float64)[s["pos_q"]], s["sin"].numpy().astype(np.float64)[s["pos_q"]], True)
    q = np.concatenate([q[..., :128], pe], -1)
    out, lse = [], []
    spread, q0, k0 = [], 0, 0
    for lq, lk in zip(q_lens, k_lens):
        for i in range(lq):
            n = lk - lq + i + 1
            keys = np.concatenate([kv[k0:k0 + n, :, :128], np.repeat(k_pe[k0:k0 + n, None], q.shape[1], 1)], -1)
            z = SCALE * np.einsum("hd,nhd->hn", q[q0 + i], keys)
            mass = SCALE * np.einsum("hd,nhd->hn", np.abs(q[q0 + i]), np.abs(keys)).max(-1)
            m = z.max(-1, keepdims=True)
            p = np.exp(z - m)
            total = p.sum(-1)
            v = kv[k0:k0 + n, :, 128:]
            out.append(np.einsum("hn,nhv->hv", p, v) / total[:, None])
            lse.append(m[:, 0] + np.log(total))
            spread.append((np.einsum("hn,nhv->hv", p, np.abs(v)) / total[:, None], mass))
        q0, k0 = q0 + lq, k0 + lk
    return np.stack(out), np.stack(lse), np.stack([x for x, _ in spread]), np.stack([x for _, x in spread])


@pytest.mark.parametrize("h,R", [(16, 352), (3, 432), (64, 352)])
def test_both_forms_give_the_attention_of_the_cache(h, R):
    # Roundings to bf16 (2^-8 each) of the rotated or absorbed query and of keys and values move a score by up to 2^-8 sum|q||k| each and so a weight by
    # e = 2 x 2 x 2^-8 of the row's sum (as |sum p (e_i - mean e)| <= 2 max|e| sum p) times that; an output then moves by e A, by 3 x 2^-8 A for
    # values, weights and the latent output (for the latter A is taken over the latent: sum |W| |o| is bounded below), and by 2^-8 |out|.
    q_lens, k_lens = [7, 40, 1], [120, 40, 33]
    s = serve(h, k_lens, q_lens, R)
    dev = {k: v.to(DEV) for k, v in s.items() if isinstance(v, torch.Tensor)}
    r_out, r_lse, A, mass = truth(s, q_lens, k_lens)
    # expanded: the rotation of the queries is taken from the absorbing call
    turned = lib.mla_absorb_query(dev["q"], dev["kv_b"], dev["pos_q"], dev["cos"], dev["sin"], True)
    kv, k_pe = lib.paged_mla_expand(dev["pool"], dev["table"], starts(k_lens).to(DEV), dev["kv_b"], sum(k_lens), page_size=s["page_size"])
    q = torch.cat([dev["q"][..., :128], turned[..., 512:]], -1)
    out, lse = lib.ragged_mla_attention(q, kv, k_pe, starts(q_lens).to(DEV), starts(k_lens).to(DEV), SCALE)
    d = 2 * 2.0 ** -8 * mass[..., None]
    ref.check(out, r_out, 2.0 ** -8 * np.abs(r_out) + (2 * 2.0 ** -8 + 2 * d * np.exp(2 * d)) * A, "expanded")
    assert np.all(np.abs(lse.cpu().numpy() - r_lse) <= d[..., 0] + 1e-5)
    # absorbed, sequence by sequence
    recs = oracle.dequant_records(s["pool"].cpu().numpy(), False)
    w = ref.f64(s["kv_b"])
    q0 = 0
    for b, (lq, lk) in enumerate(zip(q_lens, k_lens)):
        o, l = lib.paged_mla_decode(turned[q0:q0 + lq].view(1, lq, h, 576), dev["pool"], dev["table"][b:b + 1], dev["lens"][b:b + 1], SCALE,
                                    page_size=s["page_size"])
        back = lib.mla_project_values(o[0], dev["kv_b"])
        row = s["table"][b].cpu().numpy()
        c = recs[[row[t // s["page_size"]] * s["page_size"] + t % s["page_size"] for t in range(lk)]]
        most = np.abs(c[:, :512]).max(0)                              # |latent output| and A of the latents are at most this
        wide = np.einsum("hvc,c->hv", np.abs(w[:, 128:]), most)[None]
        qm = np.abs(ref.f64(turned[q0:q0 + lq])) @ np.abs(c).T        # [lq, h, lk]
        da = 2.0 ** -8 * SCALE * qm.max(-1)[..., None]
        tol = 2.0 ** -8 * np.abs(r_out[q0:q0 + lq]) + (2 * 2.0 ** -8 + 2 * da * np.exp(2 * da)) * wide
        ref.check(back, r_out[q0:q0 + lq], tol, "absorbed")
        assert np.all(np.abs(l[0].cpu().numpy() - r_lse[q0:q0 + lq]) <= da[..., 0] + 1e-3)
        # the two forms differ by far less than those bounds
        assert (back.float() - out[q0:q0 + lq].float()).norm() <= 0.03 * out[q0:q0 + lq].float().norm()
        q0 += lq


def buffers(rng, h, q_lens, k_lens):
    return [t.to(DEV) for t in (bf16(rng, sum(q_lens), h, 192), bf16(rng, sum(k_lens), h, 256), bf16(rng, sum(k_lens), 64), starts(q_lens), starts(k_lens))]


def test_a_captured_chunk_follows_the_lengths_of_its_replay():
    rng = np.random.default_rng(1)
    h, page_size, cap = 8, 16, 700
    s = serve(h, [300, 250, 90], [60, 50, 90], page_size=page_size)
    dev = {k: v.to(DEV) for k, v in s.items() if isinstance(v, torch.Tensor)}
    cq, ck = i32(0, 60, 110, 200), i32(0, 300, 550, 640)
    q = bf16(rng, cap, h, 192).to(DEV)
    kv, pe = torch.zeros(cap, h, 256, dtype=torch.bfloat16, device=DEV), torch.zeros(cap, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.zeros(cap, h, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(cap, h, device=DEV)
    ws = torch.empty(lib.ragged_workspace_size(), dtype=torch.uint8, device=DEV)

    def step(n_kv, n_pe, n_out, n_lse):
        lib.paged_mla_expand(dev["pool"], dev["table"], ck, dev["kv_b"], cap, page_size=page_size, kv=n_kv, k_pe=n_pe)
        lib.ragged_mla_attention(q, n_kv, n_pe, cq, ck, SCALE, out=n_out, lse=n_lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kv, pe, out, lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kv, pe, out, lse)
    for new_q, new_k in (([0, 60, 110, 200], [0, 300, 550, 640]), ([0, 1, 2, 2], [0, 17, 260, 261]), ([0, 0, 0, 0], [0, 0, 0, 0]), ([0, 0, 250, 340], [0, 5, 255, 345])):
        cq.copy_(i32(*new_q))
        ck.copy_(i32(*new_k))
        for t in (kv, pe, out, lse):
            t.fill_(2.0)
        graph.replay()
        eager = [torch.full_like(t, 2.0) for t in (kv, pe, out, lse)]
        step(*eager)
        for a, b in zip((kv, pe, out, lse), eager):
            assert torch.equal(a, b)
        assert torch.all(out[new_q[-1]:] == 2.0) and torch.all(kv[new_k[-1]:] == 2.0)


def test_calls_on_two_streams_and_the_same_bits_again():
    rng = np.random.default_rng(2)
    h = 16
    sets = [buffers(rng, h, ql, kl) for ql, kl in (([300, 20], [900, 25]), ([64] * 6, [500] * 6))]
    kv_b = weights(rng, h).to(DEV)
    latent = bf16(rng, 260, h, 512).to(DEV)
    first = [lib.ragged_mla_attention(*b, SCALE) for b in sets]
    a0, p0 = lib.mla_absorb_query(sets[0][0], kv_b), lib.mla_project_values(latent, kv_b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        again, more = [None, None], []
        for k, st in enumerate(streams):
            again[k] = lib.ragged_mla_attention(*sets[k], SCALE, stream=st)       # a workspace of its own each
            more.append((lib.mla_absorb_query(sets[0][0], kv_b, stream=st), lib.mla_project_values(latent, kv_b, stream=st)))
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(x, y) for x, y in zip(first[k], again[k]))
            assert torch.equal(more[k][0], a0) and torch.equal(more[k][1], p0)


def test_a_chain_without_waits_gives_the_same_bits():
    # every kernel starts its prologue while the one before it still runs: what it reads has to be there
    q_lens, k_lens, h = [30, 100], [200, 160], 16
    s = serve(h, k_lens, q_lens, seed=3)
    dev = {k: v.to(DEV) for k, v in s.items() if isinstance(v, torch.Tensor)}
    cq, ck = starts(q_lens).to(DEV), starts(k_lens).to(DEV)

    def chain(wait):
        got = []
        for _ in range(3):
            x = lib.mla_absorb_query(dev["q"], dev["kv_b"], dev["pos_q"], dev["cos"], dev["sin"], True)
            wait()
            kv, pe = lib.paged_mla_expand(dev["pool"], dev["table"], ck, dev["kv_b"], sum(k_lens), page_size=s["page_size"])
            wait()
            out, lse = lib.ragged_mla_attention(torch.cat([dev["q"][..., :128], x[..., 512:]], -1), kv, pe, cq, ck, SCALE)
            wait()
            o, l = lib.paged_mla_decode(x[-100:].view(1, 100, h, 576), dev["pool"], dev["table"][1:], dev["lens"][1:], SCALE, page_size=s["page_size"])
            wait()
            back = lib.mla_project_values(o[0], dev["kv_b"])
            wait()
            got += [x, kv, pe, out, lse, o, l, back]
        torch.cuda.synchronize()
        return got

    slow = chain(torch.cuda.synchronize)
    for a, b in zip(slow, chain(lambda: None)):
        assert torch.equal(a, b)


def test_a_shared_workspace_in_stream_order():
    rng = np.random.default_rng(4)
    ws = torch.empty(lib.ragged_workspace_size(), dtype=torch.uint8, device=DEV)
    sets = [buffers(rng, h, [lq], [lk]) for h, lq, lk in ((4, 300, 2000), (2, 5, 4000), (8, 256, 700))]
    want = [lib.ragged_mla_attention(*b, SCALE) for b in sets]
    torch.cuda.synchronize()
    ws.fill_(0xFF)
    got = [lib.ragged_mla_attention(*b, SCALE, workspace=ws) for b in sets * 3]
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[k % 3]))
