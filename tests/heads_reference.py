"""Plain implementations, in 64 bits and on the host, of the calls around the latent attention, with the error
bounds that the CUDA calls are held to.

A sum of n products in fp32, in any order and whatever the tree, is off by at most (n + 1) 2^-24 sum|a||b|, twice that where the
accumulator truncates; the result's rounding to bf16 adds 2^-8 of it at most (half a step of
8 significant bits). Denormal results may be flushed: 2^-126."""
import numpy as np
import torch

import oracle

TINY = 2.0 ** -126


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(scale * rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def weights(rng, h):
    return bf16(rng, h, 256, 512, scale=512 ** -0.5)


def product(spec, a, b, n):
    """einsum and its bound: n products a value"""
    ref = np.einsum(spec, a, b, optimize=True)
    mass = np.einsum(spec, np.abs(a), np.abs(b), optimize=True)
    return ref, 2.0 ** -8 * np.abs(ref) + 2 * (n + 1) * 2.0 ** -24 * mass + TINY


def rotate(x, cos, sin, half):
    """x [T, h, 64]; three fp32 roundings of terms no larger than |a| + |b|, then bf16"""
    a, b = (x[..., :32], x[..., 32:]) if half else (x[..., 0::2], x[..., 1::2])
    c, s = cos[:, None], sin[:, None]
    u, v = a * c - b * s, b * c + a * s
    mu, mv = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    join = (lambda p, q: np.concatenate([p, q], -1)) if half else (lambda p, q: np.stack([p, q], -1).reshape(*p.shape[:-1], 64))
    ref, mass = join(u, v), join(mu, mv)
    return ref, 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -24 * mass + TINY


def absorb(q, kv_b, positions=None, cos=None, sin=None, half=True):
    x, w = f64(q), f64(kv_b)
    nope, tol = product("thd,hdc->thc", x[..., :128], w[:, :128], 128)
    if positions is None:
        pe, tol_pe = x[..., 128:], np.zeros_like(x[..., 128:])
    else:
        at = positions.numpy()
        pe, tol_pe = rotate(x[..., 128:], cos.numpy().astype(np.float64)[at], sin.numpy().astype(np.float64)[at], half)
    return np.concatenate([nope, pe], -1), np.concatenate([tol, tol_pe], -1)


def project(latent, kv_b):
    return product("thc,hvc->thv", f64(latent), f64(kv_b)[:, 128:], 512)


def expand(recs, blk, table, lens, page_size, kv_b):
    """kv and its bound, k_pe (exact); tokens whose page lies outside the pool are zeros"""
    keys = np.concatenate([oracle.dequant_records(recs, blk), np.zeros((1, 576))])
    rows = []
    for b, n in enumerate(lens):
        for t in range(int(n)):
            page = int(table[b, t // page_size]) if t // page_size < table.shape[1] else -1
            slot = page * page_size + t % page_size
            rows.append(slot if page >= 0 and slot < recs.shape[0] else recs.shape[0])
    c = keys[np.asarray(rows, dtype=np.int64)]
    kv, tol = product("tc,hvc->thv", c[:, :512], f64(kv_b), 512)
    return kv, tol, c[:, 512:]


def starts(lens):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))


def attention(q, kv, k_pe, q_lens, k_lens, scale, sink=None):
    """out, lse and their bounds.

    A score is a sum of 192 products: off by d = 2 * 193 * 2^-24 |scale| sum|q||k|; exp2 and its argument add 2^-20 (the argument's
    rounding is 2^-24 of up to 2^4 and more of it only where the weight has vanished). A weight is off by e = 2 (d + 2^-20) of the row's
    sum and by 2^-8 of itself (bf16: half of a step of 2^-7 at 1); sums of n weights and products add 2 (n + 1) 2^-24; out is rounded to bf16:
        |out - ref| <= 2^-8 |ref| + (2^-8 + e + 4 (n + 1) 2^-24) A,  A = sum p|V| / sum p,
        |lse - ref| <= d + 2^-19 + 2 (n + 1) 2^-24 + 2^-22 |ref|."""
    x, k, pe = f64(q), f64(kv), f64(k_pe)
    h = x.shape[1]
    out, lse = np.zeros((x.shape[0], h, 128)), np.full((x.shape[0], h), -np.inf)
    tol_out, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    q0 = k0 = 0
    for lq, lk in zip(q_lens, k_lens):
        keys = np.concatenate([k[k0:k0 + lk, :, :128], np.repeat(pe[k0:k0 + lk, None], h, 1)], -1)
        v = k[k0:k0 + lk, :, 128:]
        if lq and lk:
            rows = x[q0:q0 + lq]
            z = scale * np.einsum("ihd,nhd->hin", rows, keys, optimize=True)
            mass = abs(scale) * np.einsum("ihd,nhd->hin", np.abs(rows), np.abs(keys), optimize=True)
            seen = np.arange(lk)[None, :] <= lk - lq + np.arange(lq)[:, None]
            z = np.where(seen[None], z, -np.inf)
            m = z.max(-1, keepdims=True)
            some = np.isfinite(m)
            p = np.exp(z - np.where(some, m, 0.0))
            total = p.sum(-1)
            denom = total if sink is None else total + np.exp(sink[:, None].astype(np.float64) - np.where(some, m, 0.0)[..., 0])
            safe = np.where(some[..., 0], denom, 1.0)
            n = seen.sum(-1)[None, :, None]
            d = 2 * 193 * 2.0 ** -24 * np.where(seen[None], mass, 0.0).max(-1)
            ref = np.einsum("hin,nhv->hiv", p, v, optimize=True) / safe[..., None]
            A = np.einsum("hin,nhv->hiv", p, np.abs(v), optimize=True) / safe[..., None]
            t = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * (d[..., None] + 2.0 ** -20) + 4 * (n + 1) * 2.0 ** -24) * A + TINY
            with np.errstate(divide="ignore"):
                ls = np.where(some[..., 0], np.where(some, m, 0.0)[..., 0] + np.log(total), -np.inf)
            tl = d + 2.0 ** -19 + 2 * (n[..., 0] + 1) * 2.0 ** -24 + 2.0 ** -22 * np.where(some[..., 0], np.abs(ls), 0.0)
            out[q0:q0 + lq], lse[q0:q0 + lq] = ref.transpose(1, 0, 2), ls.T
            tol_out[q0:q0 + lq], tol_lse[q0:q0 + lq] = t.transpose(1, 0, 2), tl.T
        q0, k0 = q0 + lq, k0 + lk
    return out, lse, tol_out, tol_lse


def check(got, ref, tol, name="out"):
    g = f64(got) if isinstance(got, torch.Tensor) else got
    err = np.abs(g - ref)
    assert np.all(err <= tol), f"{name}: {np.max(err / np.maximum(tol, 1e-300)):.3g} times its bound"


def check_attention(out, lse, ref):
    r_out, r_lse, t_out, t_lse = ref
    l = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(r_lse)
    assert np.array_equal(np.isneginf(l), empty), "rows without a visible key"
    assert np.all(f64(out)[empty] == 0.0)
    check(out, r_out, t_out)
    check(l[~empty], r_lse[~empty], t_lse[~empty], "lse")
