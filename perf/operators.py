"""What is measured of the paged-cache operators: attention over sequences whose NVFP4 records lie in
pages, and the page operations a serving loop makes between two decode calls (copying, forking, resizing
with freeing, compacting). Each case is one call (or the few calls of one step) as a serving program makes
it; ``run`` computes it with elementary torch operations, or with the framework's calls where ``own`` is
set."""
import math

import torch

own = False

LATENT, ROPE, QK = 512, 64, 576
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one chat turn on one tensor-parallel rank with 16 heads: the call whose latency a user waits for
        {"name": "decode_b1_h16", "kind": "decode", "b": 1, "sq": 1, "h": 16, "lo": 1500, "hi": 1500, "rec": 352, "blk": False, "page": 64, "sink": False},
        # a full decode batch of such a rank, prompts of very different lengths: the cache's bytes count
        {"name": "decode_b64_h16", "kind": "decode", "b": 64, "sq": 1, "h": 16, "lo": 1024, "hi": 32768, "rec": 352, "blk": False, "page": 64, "sink": False},
        # all 128 heads on one GPU, two tokens a step (multi-token prediction), 432-byte records, sinks
        {"name": "decode_b32_sq2_h128", "kind": "decode", "b": 32, "sq": 2, "h": 128, "lo": 1000, "hi": 8192, "rec": 432, "blk": False, "page": 64, "sink": True},
        # a prompt's chunk of 256 tokens over a long prefix, two requests: the products count
        {"name": "extend_b2_sq256_h64", "kind": "decode", "b": 2, "sq": 256, "h": 64, "lo": 12345, "hi": 16640, "rec": 352, "blk": True, "page": 64, "sink": False},
        # a few pages moved for one request, in the caches of eight layers
        {"name": "copy_n5_l8", "kind": "copy", "layers": 8, "pages": 64, "n": 5, "rec": 352, "page": 64},
        # a large prefix duplicated in every layer's cache
        {"name": "copy_n512_l16", "kind": "copy", "layers": 16, "pages": 2048, "n": 512, "rec": 432, "page": 64},
        # four beams that trade places
        {"name": "fork_b4", "kind": "fork", "b": 4, "width": 64, "lo": 1800, "hi": 2100, "page": 64, "pages": 512},
        # a large batch of long sequences, half of them forked into the other half
        {"name": "fork_b256", "kind": "fork", "b": 256, "width": 2048, "lo": 1024, "hi": 131072, "page": 64, "pages": 524288},
        # one speculative decode step: room for the drafts, then the rejected ones are given back
        {"name": "resize_b64", "kind": "resize", "b": 64, "width": 512, "lo": 1024, "hi": 32000, "new": 4, "page": 64, "pages": 32768, "layers": 1, "rec": 352, "branch": 0},
        # a step of a tree search: 32 sequences fork into eight, each branch gets a page of its own to write to
        {"name": "branch_b256_l8", "kind": "resize", "b": 256, "width": 256, "lo": 400, "hi": 1900, "new": 1, "page": 64, "pages": 8192, "layers": 8, "rec": 352, "branch": 8},
        # a small pool with holes in one layer
        {"name": "compact_p200_l1", "kind": "compact", "b": 8, "width": 64, "pages": 200, "live": 60, "layers": 1, "rec": 352, "page": 64},
        # a large pool, half of it freed, in the caches of sixteen layers
        {"name": "compact_p2048_l16", "kind": "compact", "b": 128, "width": 512, "pages": 2048, "live": 1024, "layers": 16, "rec": 352, "page": 64},
    ]


def draw(rng):
    def span(lo, hi):  # spread over the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    rec, blk = rng.choice([(352, False), (352, True), (432, False)])
    page = rng.choice([16, 32, 64, 64, 128])
    kind = rng.choice(["decode", "decode", "decode", "copy", "fork", "resize", "compact"])
    if kind == "decode":
        h = rng.choice([1, 3, 8, 16, 20, 32, 48, 64, 96, 128])
        sq = rng.choice([1, 1, 1, 2, 3, span(4, 200)])
        hi = min(span(1, 40000), 300000000 // (sq * h))
        most = int(min(300000000 / (sq * h), 1500000)) // hi  # sequences that the work and the cache allow
        b = max(1, min(span(1, 128), most))
        return {"kind": kind, "b": b, "sq": sq, "h": h, "lo": max(0, int(hi * rng.uniform(0, 1))), "hi": hi, "rec": rec, "blk": blk, "page": page,
                "sink": rng.random() < 0.5}
    if kind == "copy":
        pages, layers = span(8, 2048), span(1, 16)
        return {"kind": kind, "layers": layers, "pages": pages, "n": span(1, pages // 2), "rec": rng.choice([352, 432, 656]), "page": min(page, 64)}
    if kind == "fork":
        width = span(4, 2048)
        return {"kind": kind, "b": span(2, 255), "width": width, "lo": 0, "hi": rng.randint(page, width * page), "page": page, "pages": span(300, 2048) * 255}
    if kind == "resize":
        b = span(2, 256)
        width = span(8, max(8, min(512, int(1.2e9 / (b * page * rec)))))
        hi, most = max(1, width * page - 80), max(1, int(1.4e9 / (b * width * page * rec)))
        return {"kind": kind, "b": b, "width": width, "lo": int(0.2 * hi), "hi": hi, "new": span(1, 64), "page": page,
                "pages": b * (width + 1) + rng.randint(1, 1000), "layers": span(1, min(8, most)), "rec": rec, "branch": rng.choice([0, 2, 5])}
    pages = span(16, 2048)
    return {"kind": kind, "b": span(1, 128), "width": span(4, 512), "pages": pages, "live": rng.randint(1, pages - 1), "layers": span(1, 16),
            "rec": rng.choice([352, 432, 656]), "page": min(page, 64)}


# ---- inputs -----------------------------------------------------------------------------------------


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


def _lens(b, lo, hi, gen):
    n = torch.randint(min(lo, hi), hi + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = hi
    return n


def _table(lens, width, page, pages, gen):
    """Distinct pages for every sequence, in random places of the pool; -1 behind a sequence's last page."""
    count = (lens + page - 1) // page
    cols = torch.arange(width, device="cuda", dtype=torch.int32)
    used = cols[None, :] < count[:, None]
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = (torch.cumsum(used.flatten().to(torch.int64), 0) - 1).clamp(0, pages - 1).view(used.shape)
    table = torch.where(used, perm[at], torch.full_like(perm[at], -1))
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs.index_add_(0, table.clamp(min=0).flatten().long(), used.flatten().to(torch.int32))
    return table.contiguous(), refs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    page = case["page"]
    if case["kind"] == "decode":
        lens = _lens(case["b"], case["lo"], case["hi"], gen)
        width = max(1, -(-case["hi"] // page))
        pages = int(((lens + page - 1) // page).sum()) + 3
        s["table"], _ = _table(lens, width, page, pages, gen)
        s["lens"] = lens
        s["cache"] = _records(pages * page, case["rec"], case["blk"], gen)
        s["q"] = torch.randn(case["b"], case["sq"], case["h"], QK, generator=gen, device="cuda").to(torch.bfloat16)
        s["sinks"] = torch.randn(case["h"], generator=gen, device="cuda") if case["sink"] else None
        s["scale"] = QK ** -0.5
        s["refs"] = None
        return s
    pages = case["pages"]
    if case["kind"] in ("copy", "resize", "compact"):
        s["pool"] = torch.randint(0, 256, (case["layers"], pages, page, case["rec"]), generator=gen, device="cuda", dtype=torch.uint8)
        s["caches"] = list(s["pool"].view(case["layers"], pages * page, case["rec"]).unbind(0))
    if case["kind"] == "copy":
        perm = torch.randperm(pages, generator=gen, device="cuda")
        s["src"], s["dst"] = perm[:case["n"]].to(torch.int32), perm[pages // 2:pages // 2 + case["n"]].to(torch.int32)
        if case["n"] > pages // 2:
            raise ValueError("sources and targets overlap")
        return s
    if case["kind"] == "fork":
        b, width = case["b"], case["width"]
        lens = _lens(b, case["lo"], min(case["hi"], width * page, (pages // b) * page), gen)
        s["table"], s["refs"] = _table(lens, width, page, pages, gen)
        s["lens"] = lens
        perm = torch.randperm(b, generator=gen, device="cuda").to(torch.int32)
        half = max(1, b // 2)
        # the second half of a random order becomes copies of the first; a small batch trades places instead
        s["src"], s["dst"] = (perm[:half], perm[b - half:]) if b > 4 else (perm, perm.roll(1))
        return s
    if case["kind"] == "resize":
        b, width = case["b"], case["width"]
        lens = _lens(b, case["lo"], min(case["hi"], width * page - case["new"], (pages // b - 2) * page), gen).clamp(min=0)
        s["table"], s["refs"] = _table(lens, width, page, pages, gen)
        s["lens"] = lens
        if case["branch"]:
            rows = torch.arange(b, device="cuda", dtype=torch.int32)
            s["src"], s["dst"] = rows - rows % case["branch"], rows
            lens = lens[s["src"].long()]
        s["up"], s["down"] = lens + case["new"], lens.clone()
        return s
    lens = torch.zeros(case["b"], dtype=torch.int32, device="cuda")
    live = min(case["live"], case["b"] * case["width"])
    share = torch.arange(case["b"], device="cuda")
    count = (live // case["b"] + (share < live % case["b"])).to(torch.int32)
    lens += count * page - (torch.rand(case["b"], generator=gen, device="cuda") * (page - 1)).to(torch.int32) * (count > 0)
    s["lens"] = lens
    s["table"], s["refs"] = _table(lens, case["width"], page, pages, gen)
    s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    return s


# ---- plain forms ------------------------------------------------------------------------------------


def _keys(rec_bytes, rec, blk):
    """fp32 keys [..., 576] of records [..., rec]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rec_bytes.device)
    codes = rec_bytes[..., :256]
    val = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    at = 320 if rec == 352 else 256
    sc = rec_bytes[..., at:at + 32].contiguous().view(torch.float8_e4m3fn).float()
    if rec == 352 and not blk:
        block = torch.arange(32, device=rec_bytes.device)
        sc = sc[..., 8 * (block & 3) + (block >> 2)]
    val = (val.unflatten(-1, (32, 16)) * sc[..., None]).flatten(-2)
    if rec == 352:
        rope = rec_bytes[..., 256:320].contiguous().view(torch.float8_e4m3fn).float()
    else:
        rope = rec_bytes[..., 304:432].contiguous().view(torch.bfloat16).float()
    return torch.cat([val, rope], -1)


def _plain_decode(s):
    b, sq, h, page = s["b"], s["sq"], s["h"], s["page"]
    table, lens = s["table"], s["lens"]
    pos = torch.arange(table.shape[1] * page, device="cuda")
    slots = table.long().clamp(min=0)[:, pos // page] * page + pos % page
    keys = _keys(s["cache"][slots], s["rec"], s["blk"])
    keys = torch.where((pos < lens[:, None])[..., None], keys, 0.0)
    z = torch.matmul(s["q"].float().view(b, sq * h, QK), keys.transpose(1, 2)).view(b, sq, h, -1) * s["scale"]
    last = lens[:, None] - sq + torch.arange(sq, device="cuda")  # each query's own position
    seen = pos <= last[..., None]
    z = z.masked_fill(~seen[:, :, None, :], float("-inf"))
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(z - m)
    total = p.sum(-1)
    denom = total if s["sinks"] is None else total + torch.exp(s["sinks"] - m[..., 0])
    out = torch.matmul(p.view(b, sq * h, -1), keys[..., :LATENT]).view(b, sq, h, LATENT) / torch.where(denom > 0, denom, 1.0)[..., None]
    return {"out": out.to(torch.bfloat16), "lse": m[..., 0] + torch.log(total)}


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _plain_fork(table, lens, refs, src, dst, page):
    cols = torch.arange(table.shape[1], device="cuda")
    used = cols < _pages_of(lens, page)[:, None]
    src, dst = src.long(), dst.long()
    flat = table.clamp(min=0).long()
    refs.index_add_(0, flat[src].flatten(), used[src].flatten().to(torch.int32))
    refs.index_add_(0, flat[dst].flatten(), used[dst].flatten().to(torch.int32), alpha=-1)
    rows, n = torch.where(used[src], table[src], -1), lens[src]
    table[dst] = rows
    lens[dst] = n


def _plain_resize(pool, table, lens, refs, new, max_new, page):
    cols = torch.arange(table.shape[1], device="cuda")
    before, after = _pages_of(lens, page)[:, None], _pages_of(new, page)[:, None]
    gone = (cols >= after) & (cols < before)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), gone.flatten().to(torch.int32), alpha=-1)
    table.copy_(torch.where(gone, -1, table))
    last = (lens.long() // page).clamp(max=table.shape[1] - 1)[:, None]
    tail = table.gather(1, last)[:, 0].clamp(min=0).long()
    own_page = (new > lens) & (lens % page > 0) & (refs[tail] > 1)  # a shared page that gets its own records
    need = (after - before)[:, 0].clamp(min=0) + own_page
    at = torch.cumsum(need, 0) - need
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    free = torch.cat([free, free.new_zeros(1)])
    added = (cols >= before) & (cols < after)
    nth = (at + own_page)[:, None] + cols - before
    table.copy_(torch.where(added, free[nth.clamp(0, free.numel() - 1)], table))
    b = torch.nonzero(own_page)[:, 0]
    to = free[at[b].clamp(max=free.numel() - 1)].long()
    keep = (torch.arange(page, device="cuda") < (lens[b] % page)[:, None])[None, :, :, None]
    pool[:, to] = torch.where(keep, pool[:, tail[b]], pool[:, to])
    refs.index_add_(0, tail[b], torch.full_like(b, -1, dtype=torch.int32))
    table[b, last[b, 0]] = to.to(torch.int32)
    refs[to] = 1
    refs[table[added].long()] = 1
    pos = lens[:, None].long() + torch.arange(max_new, device="cuda")
    slot = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1)).long() * page + pos % page
    slots = torch.where(pos < new[:, None], slot, -1)
    lens.copy_(new)
    return slots


def _plain_compact(s):
    refs, table, lens, pool, page = s["refs"], s["table"], s["lens"], s["pool"], s["page"]
    index = torch.arange(refs.numel(), device="cuda", dtype=torch.int32)
    live = refs > 0
    n = live.sum()
    movers, holes = torch.nonzero(live & (index >= n))[:, 0], torch.nonzero(~live & (index < n))[:, 0]
    to = torch.where(live, index, -1)
    to[movers] = holes.to(torch.int32)
    pool[:, holes] = pool[:, movers]
    used = torch.arange(table.shape[1], device="cuda") < _pages_of(lens, page)[:, None]
    s["table_out"].copy_(torch.where(used, to[table.clamp(min=0).long()], -1))
    s["refs_out"].zero_()
    s["refs_out"][to[live].long()] = refs[live]
    return to, n.to(torch.int32).view(1)


# ---- one pass ---------------------------------------------------------------------------------------


def run(s):
    kind, page = s["kind"], s["page"]
    if own:
        import nvfp4_kv_cache_sparse_gb300 as nv
    if kind == "decode":
        if own:
            out, lse = nv.paged_mla_decode(s["q"], s["cache"], s["table"], s["lens"], s["scale"], page_size=page, attn_sink=s["sinks"], block_scales=s["blk"])
            return {"out": out, "lse": lse}
        return _plain_decode(s)
    if kind == "copy":
        if own:
            nv.copy_pages(s["caches"], s["src"], s["dst"], page_size=page)
        else:
            s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
        return s["pool"]
    table, lens, refs = s["table"], s["lens"], s["refs"]
    if kind == "fork":
        if own:
            nv.fork_sequences(table, lens, refs, s["src"], s["dst"], page_size=page)
        else:
            _plain_fork(table, lens, refs, s["src"], s["dst"], page)
        return [table, lens, refs]
    if kind == "resize":
        if own:
            if s["branch"]:
                nv.fork_sequences(table, lens, refs, s["src"], s["dst"], page_size=page)
            slots = nv.resize_sequences(s["caches"], table, lens, refs, s["up"], s["new"], page_size=page)
            grown = table.clone()
            nv.resize_sequences(s["caches"], table, lens, refs, s["down"], 0, page_size=page)
        else:
            if s["branch"]:
                _plain_fork(table, lens, refs, s["src"], s["dst"], page)
            slots = _plain_resize(s["pool"], table, lens, refs, s["up"], s["new"], page)
            grown = table.clone()
            _plain_resize(s["pool"], table, lens, refs, s["down"], 0, page)
        return [slots, grown, table, lens, refs, s["pool"]]
    if own:
        _, _, to, live = nv.compact_pages(s["caches"], table, lens, refs, page_size=page, table_out=s["table_out"], refs_out=s["refs_out"])
    else:
        to, live = _plain_compact(s)
    return [s["table_out"], s["refs_out"], to, live, s["pool"]]


# ---- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    page = case["page"]
    if case["kind"] == "decode":
        mean = (case["lo"] + case["hi"]) / 2 if case["b"] > 1 else case["hi"]
        tokens, rows = case["b"] * mean, case["b"] * case["sq"] * case["h"]
        seen = max(1.0, mean - (case["sq"] - 1) / 2 if mean >= case["sq"] else mean * mean / (2 * case["sq"]))  # keys of a query, on average
        return {"bytes": tokens * case["rec"] + rows * (2 * QK + 2 * LATENT + 4) + 4 * tokens / page, "flops": 2 * rows * seen * (QK + LATENT)}
    page_bytes = page * case.get("rec", 0) * case.get("layers", 0)
    if case["kind"] == "copy":
        return {"bytes": 2 * case["n"] * page_bytes + 8 * case["n"], "flops": 0}
    if case["kind"] == "fork":
        used = min(case["width"], (case["lo"] + case["hi"]) / 2 / page, case["pages"] / case["b"])
        pairs = case["b"] if case["b"] <= 4 else max(1, case["b"] // 2)
        # the parents' and the children's pages read, the children's rows written, the counts of both changed
        return {"bytes": pairs * (2 * 4 * used + 4 * case["width"] + 2 * 8 * used + 16), "flops": 0}
    if case["kind"] == "resize":
        # the counts read for free pages, lengths, slots; in a branch step the forked rows and the copied records
        pages_used = min(case["width"], (case["lo"] + case["hi"]) / 2 / page)
        forked = case["b"] * (16 * pages_used + page * case["rec"] * case["layers"]) if case["branch"] else 0
        return {"bytes": 4 * case["pages"] + case["b"] * (16 + 8 * case["new"]) + forked, "flops": 0}
    moved = case["live"] * (1 - case["live"] / case["pages"])
    return {"bytes": 2 * moved * page_bytes + 12 * case["pages"] + 8 * case["b"] * case["width"], "flops": 0}


# ---- the definition in 64 bits ------------------------------------------------------------------------


def exact(case, seed):
    """Softmax attention of each query over its own tokens, sequence by sequence, in 64 bits. The page operations give whole numbers only."""
    if case["kind"] != "decode":
        return None
    s = prepare(case, seed)
    b, sq, h, page, rec = s["b"], s["sq"], s["h"], s["page"], s["rec"]
    out = torch.zeros(b, sq, h, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((b, sq, h), float("-inf"), dtype=torch.float64, device="cuda")
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    byte = torch.arange(256, device="cuda")
    sign, expo, frac = 1.0 - 2.0 * (byte >> 7), (byte >> 3) & 15, (byte & 7).double()
    e4m3 = sign * torch.where(expo > 0, (1 + frac / 8) * 2.0 ** (expo.double() - 7), frac * 2.0 ** -9)
    for i in range(b):
        n = int(s["lens"][i])
        if n == 0:
            continue
        records = torch.cat([s["cache"][int(p) * page:int(p) * page + page] for p in s["table"][i, :-(-n // page)].tolist()])[:n].long()
        k = torch.empty(n, QK, dtype=torch.float64, device="cuda")
        for parity in (0, 1):
            nibble = records[:, :256] >> 4 if parity else records[:, :256] & 15
            k[:, parity:LATENT:2] = grid[nibble & 7] * torch.where(nibble >= 8, -1.0, 1.0)
        for block in range(32):
            at = 256 + block if rec == 432 else 320 + block if s["blk"] else 320 + 8 * (block & 3) + (block >> 2)
            k[:, 16 * block:16 * block + 16] *= e4m3[records[:, at]][:, None]
        if rec == 352:
            k[:, LATENT:] = e4m3[records[:, 256:320]]
        else:
            word = records[:, 304:432:2] + (records[:, 305:432:2] << 8)
            k[:, LATENT:] = (word << 16).to(torch.int32).view(torch.float32).double()
        first = n - sq
        for j0 in range(0, sq, 32):  # a few queries at a time
            j1 = min(sq, j0 + 32)
            z = torch.einsum("jhd,nd->jhn", s["q"][i, j0:j1].double(), k) * s["scale"]
            hidden = torch.arange(n, device="cuda") > first + torch.arange(j0, j1, device="cuda")[:, None]
            z = z.masked_fill(hidden[:, None, :], float("-inf"))
            part = torch.logsumexp(z, -1)
            whole = part if s["sinks"] is None else torch.logaddexp(part, s["sinks"].double().expand_as(part))
            weight = torch.where(torch.isinf(part)[..., None], 0.0, torch.exp(z - torch.where(torch.isinf(part), 0.0, whole)[..., None]))
            out[i, j0:j1] = torch.einsum("jhn,nd->jhd", weight, k[:, :LATENT])
            lse[i, j0:j1] = part
    return {"out": out, "lse": lse}
