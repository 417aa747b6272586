"""What is measured of the operators around the latent attention: the query's absorption into the latent
space and the values' projection out of it (the absorbed form, beside the attention over pages), the
expansion of records in pages into per-head keys and values, and the attention of chunks of new tokens over
them (the expanded form). Each case is one call as a serving program makes it; ``run`` computes it with
elementary torch operations, or with the framework's call where ``own`` is set."""
import math

import torch

own = False

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
POSITIONS = 65536  # rows of the rotation tables


def listed():
    return [
        # one chat turn on a tensor-parallel rank with 16 heads: the query of one token, its latency counts
        {"name": "absorb_t1_h16", "kind": "absorb", "t": 1, "h": 16, "half": False},
        # a decode batch of 64 requests with all 128 heads: the weights' bytes count
        {"name": "absorb_t64_h128", "kind": "absorb", "t": 64, "h": 128, "half": False},
        # chunks of prompts for the absorbed form, an odd number of tokens: the queries' bytes count
        {"name": "absorb_t4001_h128", "kind": "absorb", "t": 4001, "h": 128, "half": True},
        # the way back of the same three calls
        {"name": "values_t1_h16", "kind": "values", "t": 1, "h": 16},
        {"name": "values_t64_h128", "kind": "values", "t": 64, "h": 128},
        {"name": "values_t4001_h128", "kind": "values", "t": 4001, "h": 128},
        # the prefix of one request on a rank with 16 heads
        {"name": "expand_b1_h16", "kind": "expand", "b": 1, "h": 16, "lo": 1500, "hi": 1500, "rec": 352, "blk": False, "page": 64},
        # ragged prefixes of eight requests on such a rank, 432-byte records
        {"name": "expand_b8_h16", "kind": "expand", "b": 8, "h": 16, "lo": 1000, "hi": 16384, "rec": 432, "blk": False, "page": 64},
        # two long prefixes, all 128 heads on one GPU
        {"name": "expand_b2_h128", "kind": "expand", "b": 2, "h": 128, "lo": 12345, "hi": 16640, "rec": 352, "blk": True, "page": 64},
        # short new prompts without a prefix, packed
        {"name": "attend_b16_new_h16", "kind": "attend", "b": 16, "h": 16, "qlo": 30, "qhi": 700, "plo": 0, "phi": 0, "sink": False},
        # chunks of 512 tokens over prefixes of very different lengths on a rank with 16 heads
        {"name": "attend_b4_chunk_h16", "kind": "attend", "b": 4, "h": 16, "qlo": 512, "qhi": 512, "plo": 500, "phi": 16000, "sink": False},
        # a long chunk over a long prefix with 64 heads: the products count
        {"name": "attend_b1_long_h64", "kind": "attend", "b": 1, "h": 64, "qlo": 2048, "qhi": 2048, "plo": 14592, "phi": 14592, "sink": True},
    ]


def draw(rng):
    def span(lo, hi):  # spread over the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    kind = rng.choice(["absorb", "values", "expand", "attend", "attend"])
    h = rng.choice([1, 3, 8, 16, 20, 32, 48, 64, 96, 128])
    if kind in ("absorb", "values"):
        case = {"kind": kind, "t": span(1, min(20000, 4001 * 128 // h)), "h": h}
        return {**case, "half": rng.random() < 0.5} if kind == "absorb" else case
    if kind == "expand":
        most = min(100000, 28000 * 128 // h)  # tokens
        hi = span(1, min(32768, most))
        rec, blk = rng.choice([(352, False), (352, True), (432, False)])
        return {"kind": kind, "b": span(1, min(64, most // hi)), "h": h, "lo": int(hi * rng.uniform(0, 1)), "hi": hi, "rec": rec, "blk": blk,
                "page": rng.choice([16, 32, 64, 64, 128])}
    qhi = span(1, 4096)
    phi = rng.choice([0, span(1, 16384)])
    cost = h * qhi * (phi + qhi)  # pairs, an upper bound
    most = max(1, min(int(1.9e9) // cost, 6000000 // (h * (phi + qhi))))
    if cost > 1.9e9:
        h = max(1, int(1.9e9 / (qhi * (phi + qhi))))
    return {"kind": kind, "b": span(1, min(32, most)), "h": h, "qlo": int(qhi * rng.uniform(0, 1)), "qhi": qhi, "plo": int(phi * rng.uniform(0, 1)),
            "phi": phi, "sink": rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------------------------------


def _weights(h, gen):
    """The up-projection of the latent: per head 128 rows for the key and 128 for the value."""
    return (torch.randn(h, NOPE + VALUE, LATENT, generator=gen, device="cuda") * LATENT ** -0.5).to(torch.bfloat16)


def _records(n, rec, blk, gen):
    """n records of normal latents with 1% of outliers, quantized: codes, scales in the record's order, RoPE."""
    x = torch.randn(n, LATENT, generator=gen, device="cuda")
    x = torch.where(torch.rand(n, LATENT, generator=gen, device="cuda") < 0.01, 20 * x, x)
    g = x.view(n, 32, 16)
    sc = (g.abs().amax(2) / 6).to(torch.float8_e4m3fn)
    q = g / sc.float().clamp(min=1e-9)[:, :, None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = (torch.bucketize(q.abs().view(n, LATENT), mid) + 8 * (q.view(n, LATENT) < 0)).to(torch.uint8)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    sb = sc.view(torch.uint8)
    rope = torch.randn(n, ROPE, generator=gen, device="cuda")
    if rec == 352:
        order = torch.arange(32, device="cuda")
        if not blk:
            order = 4 * (order & 7) + (order >> 3)  # byte i of the field holds this block's scale
        return torch.cat([codes, rope.to(torch.float8_e4m3fn).view(torch.uint8), sb[:, order]], 1).contiguous()
    pad = torch.zeros(n, 16, dtype=torch.uint8, device="cuda")
    return torch.cat([codes, sb, pad, rope.to(torch.bfloat16).view(torch.uint8)], 1).contiguous()


def _spread(b, lo, hi):
    """b lengths from lo to hi, the longest one first; the same for every seed, which gives their order."""
    return [hi - int((hi - min(lo, hi)) * (i * 0.6180339887 % 1)) for i in range(b)]


def _lens(b, lo, hi, gen):
    order = torch.randperm(b, generator=gen, device="cuda")
    return torch.tensor(_spread(b, lo, hi), dtype=torch.int32, device="cuda")[order]


def _starts(lens):
    return torch.cat([lens.new_zeros(1), torch.cumsum(lens, 0).to(torch.int32)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    kind, h = case["kind"], case["h"]
    if kind == "absorb":
        s["q"] = torch.randn(case["t"], h, NOPE + ROPE, generator=gen, device="cuda").to(torch.bfloat16)
        s["kv_b"] = _weights(h, gen)
        s["positions"] = torch.randint(0, POSITIONS, (case["t"],), generator=gen, device="cuda")
        angle = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)
        s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
    elif kind == "values":
        s["latent"] = torch.randn(case["t"], h, LATENT, generator=gen, device="cuda").to(torch.bfloat16)
        s["kv_b"] = _weights(h, gen)
    elif kind == "expand":
        page, lens = case["page"], _lens(case["b"], case["lo"], case["hi"], gen)
        count = (lens + page - 1) // page
        width = max(1, -(-case["hi"] // page))
        pages = int(count.sum()) + 3
        used = torch.arange(width, device="cuda") < count[:, None]
        perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        s["table"] = torch.full((case["b"], width), -1, dtype=torch.int32, device="cuda")
        s["table"][used] = perm[:int(count.sum())]
        s["starts"], s["total"] = _starts(lens), int(lens.sum())
        s["cache"] = _records(pages * page, case["rec"], case["blk"], gen)
        s["kv_b"] = _weights(h, gen)
    else:
        q_lens = _lens(case["b"], case["qlo"], case["qhi"], gen)
        k_lens = q_lens + _lens(case["b"], case["plo"], case["phi"], gen)
        s["starts_q"], s["starts_k"] = _starts(q_lens), _starts(k_lens)
        s["spans"] = list(zip(*(x.tolist() for x in (s["starts_q"][:-1], s["starts_q"][1:], s["starts_k"][:-1], s["starts_k"][1:]))))
        s["q"] = torch.randn(int(q_lens.sum()), h, NOPE + ROPE, generator=gen, device="cuda").to(torch.bfloat16)
        s["kv"] = torch.randn(int(k_lens.sum()), h, NOPE + VALUE, generator=gen, device="cuda").to(torch.bfloat16)
        s["k_pe"] = torch.randn(int(k_lens.sum()), ROPE, generator=gen, device="cuda").to(torch.bfloat16)
        s["sinks"] = torch.randn(h, generator=gen, device="cuda") if case["sink"] else None
        s["scale"] = (NOPE + ROPE) ** -0.5
    return s


# ---- plain forms ------------------------------------------------------------------------------------


def _rotate(x, cos, sin, half):
    """Pairs (f, f + 32) of the last dimension's 64 where half, else (2f, 2f + 1)."""
    a, b = (x[..., :32], x[..., 32:]) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)


def _plain_absorb(s):
    q = s["q"].float()
    nope = torch.matmul(q[..., :NOPE].transpose(0, 1), s["kv_b"][:, :NOPE].float()).transpose(0, 1)
    cos, sin = s["cos"][s["positions"]][:, None], s["sin"][s["positions"]][:, None]
    return torch.cat([nope, _rotate(q[..., NOPE:], cos, sin, s["half"])], -1).to(torch.bfloat16)


def _plain_values(s):
    w = s["kv_b"][:, NOPE:].float().transpose(1, 2)
    return torch.matmul(s["latent"].float().transpose(0, 1), w).transpose(0, 1).to(torch.bfloat16).contiguous()


def _plain_expand(s):
    page, starts, rec = s["page"], s["starts"].long(), s["rec"]
    token = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(starts, token, right=True) - 1
    pos = token - starts[b]
    record = s["cache"][s["table"].long()[b, pos // page] * page + pos % page]
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    codes = record[:, :256]
    val = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).view(-1, 32, 16)
    at = 320 if rec == 352 else 256
    sc = record[:, at:at + 32].contiguous().view(torch.float8_e4m3fn).float()
    if rec == 352 and not s["blk"]:
        block = torch.arange(32, device="cuda")
        sc = sc[:, 8 * (block & 3) + (block >> 2)]
    latent = (val * sc[..., None]).view(-1, LATENT)
    kv = torch.matmul(latent, s["kv_b"].float().view(-1, LATENT).t()).to(torch.bfloat16).view(-1, s["h"], NOPE + VALUE)
    if rec == 352:
        k_pe = record[:, 256:320].contiguous().view(torch.float8_e4m3fn).to(torch.bfloat16)
    else:
        k_pe = record[:, 304:432].contiguous().view(torch.bfloat16)
    return kv, k_pe


def _plain_attend(s):
    q, kv, k_pe = s["q"], s["kv"], s["k_pe"]
    out = torch.zeros(q.shape[0], s["h"], VALUE, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], s["h"]), float("-inf"), device="cuda")
    for q0, q1, k0, k1 in s["spans"]:
        if q1 == q0 or k1 == k0:
            continue
        x = q[q0:q1].float().transpose(0, 1)
        keys, values = kv[k0:k1, :, :NOPE].float().permute(1, 2, 0), kv[k0:k1, :, NOPE:].float().transpose(0, 1)
        z = (torch.matmul(x[..., :NOPE], keys) + torch.matmul(x[..., NOPE:], k_pe[k0:k1].float().t())) * s["scale"]
        last = k1 - k0 - (q1 - q0) + torch.arange(q1 - q0, device="cuda")  # each query's own position
        z = z.masked_fill(torch.arange(k1 - k0, device="cuda") > last[:, None], float("-inf"))
        m = z.amax(-1, keepdim=True)
        m = torch.where(m == float("-inf"), 0.0, m)
        p = torch.exp(z - m)
        total = p.sum(-1)
        denom = total if s["sinks"] is None else total + torch.exp(s["sinks"][:, None] - m[..., 0])
        o = torch.matmul(p, values) / torch.where(denom > 0, denom, 1.0)[..., None]
        out[q0:q1] = o.transpose(0, 1).to(torch.bfloat16)
        lse[q0:q1] = (m[..., 0] + torch.log(total)).t()
    return out, lse


# ---- one pass ---------------------------------------------------------------------------------------


def run(s):
    kind = s["kind"]
    if own:
        import nvfp4_kv_cache_sparse_gb300 as nv
    if kind == "absorb":
        if own:
            return nv.mla_absorb_query(s["q"], s["kv_b"], s["positions"], s["cos"], s["sin"], s["half"])
        return _plain_absorb(s)
    if kind == "values":
        if own:
            return nv.mla_project_values(s["latent"], s["kv_b"])
        return _plain_values(s)
    if kind == "expand":
        if own:
            kv, k_pe = nv.paged_mla_expand(s["cache"], s["table"], s["starts"], s["kv_b"], s["total"], page_size=s["page"], block_scales=s["blk"])
        else:
            kv, k_pe = _plain_expand(s)
        return {"kv": kv, "k_pe": k_pe}
    if own:
        out, lse = nv.ragged_mla_attention(s["q"], s["kv"], s["k_pe"], s["starts_q"], s["starts_k"], s["scale"], attn_sink=s["sinks"])
    else:
        out, lse = _plain_attend(s)
    return {"out": out, "lse": lse}


# ---- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    h = case["h"]
    if case["kind"] == "absorb":
        t = case["t"]
        return {"bytes": t * h * 2 * (NOPE + ROPE + LATENT + ROPE) + h * 2 * NOPE * LATENT + t * (8 + 8 * 32), "flops": 2 * t * h * NOPE * LATENT}
    if case["kind"] == "values":
        t = case["t"]
        return {"bytes": t * h * 2 * (LATENT + VALUE) + h * 2 * VALUE * LATENT, "flops": 2 * t * h * VALUE * LATENT}
    if case["kind"] == "expand":
        tokens = sum(_spread(case["b"], case["lo"], case["hi"]))
        return {"bytes": tokens * (case["rec"] + h * 2 * (NOPE + VALUE) + 2 * ROPE) + h * 2 * (NOPE + VALUE) * LATENT,
                "flops": 2 * tokens * h * (NOPE + VALUE) * LATENT}
    new, before = _spread(case["b"], case["qlo"], case["qhi"]), _spread(case["b"], case["plo"], case["phi"])
    pairs = sum(n * (sum(before) / case["b"] + (n + 1) / 2) for n in new)  # a chunk goes with any prefix
    return {"bytes": sum(new) * h * (2 * (NOPE + ROPE + VALUE) + 4) + (sum(new) + sum(before)) * 2 * (h * (NOPE + VALUE) + ROPE),
            "flops": 2 * h * pairs * (NOPE + ROPE + VALUE)}


# ---- the definition in 64 bits ------------------------------------------------------------------------


def _e4m3(byte):
    sign, expo, frac = 1.0 - 2.0 * (byte >> 7), (byte >> 3) & 15, (byte & 7).double()
    return sign * torch.where(expo > 0, (1 + frac / 8) * 2.0 ** (expo.double() - 7), frac * 2.0 ** -9)


def exact(case, seed):
    """Each operator's sums in 64 bits."""
    s = prepare(case, seed)
    kind, h = s["kind"], s["h"]
    if kind == "absorb":
        out = torch.empty(s["t"], h, LATENT + ROPE, dtype=torch.float64, device="cuda")
        out[..., :LATENT] = torch.einsum("thd,hdc->thc", s["q"][..., :NOPE].double(), s["kv_b"][:, :NOPE].double())
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"]][:, None]
        pe = s["q"][..., NOPE:].double()
        if s["half"]:
            z = torch.complex(pe[..., :32], pe[..., 32:]) * turn
            out[..., LATENT:LATENT + 32], out[..., LATENT + 32:] = z.real, z.imag
        else:
            z = torch.complex(pe[..., ::2].contiguous(), pe[..., 1::2].contiguous()) * turn
            out[..., LATENT::2], out[..., LATENT + 1::2] = z.real, z.imag
        return out
    if kind == "values":
        return torch.einsum("thc,hvc->thv", s["latent"].double(), s["kv_b"][:, NOPE:].double())
    if kind == "expand":
        page, rec, starts = s["page"], s["rec"], s["starts"].tolist()
        kv = torch.empty(s["total"], h, NOPE + VALUE, dtype=torch.float64, device="cuda")
        k_pe = torch.empty(s["total"], ROPE, dtype=torch.float64, device="cuda")
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        weight = s["kv_b"].double().view(-1, LATENT)
        for b in range(s["b"]):
            n, slots = starts[b + 1] - starts[b], s["cache"].view(-1, page, rec)
            if n == 0:
                continue
            r = slots[s["table"][b, :-(-n // page)].long()].view(-1, rec)[:n].long()
            x = torch.empty(n, LATENT, dtype=torch.float64, device="cuda")
            for parity in (0, 1):
                nibble = r[:, :256] >> 4 if parity else r[:, :256] & 15
                x[:, parity::2] = grid[nibble & 7] * torch.where(nibble >= 8, -1.0, 1.0)
            for block in range(32):
                at = 256 + block if rec == 432 else 320 + block if s["blk"] else 320 + 8 * (block & 3) + (block >> 2)
                x[:, 16 * block:16 * block + 16] *= _e4m3(r[:, at])[:, None]
            kv[starts[b]:starts[b + 1]] = (x @ weight.t()).view(n, h, -1)
            if rec == 352:
                k_pe[starts[b]:starts[b + 1]] = _e4m3(r[:, 256:320])
            else:
                k_pe[starts[b]:starts[b + 1]] = ((r[:, 304:432:2] + (r[:, 305:432:2] << 8)) << 16).to(torch.int32).view(torch.float32).double()
        return {"kv": kv, "k_pe": k_pe}
    out = torch.zeros(s["q"].shape[0], h, VALUE, dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], h), float("-inf"), dtype=torch.float64, device="cuda")
    for q0, q1, k0, k1 in s["spans"]:
        if k1 == k0:
            continue
        keys = torch.cat([s["kv"][k0:k1, :, :NOPE], s["k_pe"][k0:k1, None].expand(-1, h, -1)], -1).double()
        values = s["kv"][k0:k1, :, NOPE:].double()
        for j0 in range(q0, q1, 256):  # a few queries at a time
            j1 = min(q1, j0 + 256)
            z = torch.einsum("jhd,nhd->jhn", s["q"][j0:j1].double(), keys) * s["scale"]
            hidden = torch.arange(k1 - q1, k1 - q1 + j1 - j0, device="cuda")[:, None] + j0 < torch.arange(k0, k1, device="cuda")
            z = z.masked_fill(hidden[:, None, :], float("-inf"))
            part = torch.logsumexp(z, -1)
            whole = part if s["sinks"] is None else torch.logaddexp(part, s["sinks"].double().expand_as(part))
            weight = torch.where(torch.isinf(part)[..., None], 0.0, torch.exp(z - torch.where(torch.isinf(part), 0.0, whole)[..., None]))
            out[j0:j1] = torch.einsum("jhn,nhv->jhv", weight, values)
            lse[j0:j1] = part
    return {"out": out, "lse": lse}
