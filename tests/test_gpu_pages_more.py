"""More of the page operations on the GPU: the smallest pools, pools that are exactly large enough, and long chains of
calls that start while the one before still runs."""
import numpy as np
import pytest
import torch

import nvfp4_kv_cache_sparse_gb300 as lib
from test_gpu_pages import State

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("pages", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 31, 32, 33, 63, 65])
def test_compaction_of_the_smallest_pools(pages):
    # a CTA of the cluster has four pages or none to count: it reaches the exchange of the sums at once
    rng = np.random.default_rng(pages)
    s = State(4, pages, pages, 2, 1, 352, pages)
    for k in range(3):
        new = [int(n) for n in rng.multinomial(2 * pages, [0.25] * 4)]
        while sum(-(-n // 2) for n in new) > pages:
            new[int(np.argmax(new))] -= 1
        s.resize(new)
        s.resize([n if i % 2 == k % 2 else 0 for i, n in enumerate(new)])
        s.compact(k != 1)


@pytest.mark.parametrize("spare,status", [(2, True), (3, False)])
def test_every_holder_of_a_shared_last_page_takes_one(spare, status):
    # three sequences share a page and grow at once: three pages, although the shared one is free afterwards
    s = State(3, 2, 1 + spare, 16)
    s.resize([5, 0, 0])
    s.fork([0, 0], [1, 2])
    before = list(s.plain.lens)
    s.resize([6, 7, 8], 2)     # (State checks DEV_PAGES_EXHAUSTED against the plain operation's answer)
    assert (s.plain.lens == before) == status
    assert s.plain.refs[0] == (3 if status else 0)


@pytest.mark.parametrize("h_q", [16, 64])
@pytest.mark.parametrize("seed", range(4))
def test_a_chain_of_calls_without_waits(h_q, seed):
    """Each call is launched as a programmatic dependent of the one before and reads what that one wrote (lengths, narrow
    table rows that share cache lines, counts, records): the same bits with a wait behind every call, without any, and
    from a replayed graph."""
    rng = np.random.default_rng(seed)
    batch, width, ps, pages, R, steps = 24, 5, 16, 200, 352, 12
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    plan, lens = [], np.zeros(batch, dtype=int)
    for _ in range(steps):
        new = np.where(rng.random(batch) < 0.15, 0, np.minimum(lens + rng.integers(0, 9, batch), width * ps))
        order = rng.permutation(batch)
        k = int(rng.integers(1, 8))
        lens = new.copy()
        lens[order[k:2 * k]] = new[order[:k]]
        plan.append((t(new), t(order[:k]), t(order[k:2 * k])))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    lat = torch.randn(steps, batch * 8, 512, generator=gen, device=DEV).to(torch.bfloat16)
    rope = torch.randn(steps, batch * 8, 64, generator=gen, device=DEV).to(torch.bfloat16)
    q = torch.randn(steps, batch, 1, h_q, 576, generator=gen, device=DEV).to(torch.bfloat16)

    def chain(wait):
        cache = torch.zeros((pages * ps, R), dtype=torch.uint8, device=DEV)
        table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
        n, refs = torch.zeros(batch, dtype=torch.int32, device=DEV), torch.zeros(pages, dtype=torch.int32, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        kw = {"page_size": ps, "dev_status": status}
        results = []
        for i, (new, src, dst) in enumerate(plan):
            slots = lib.resize_sequences([cache], table, n, refs, new, 8, **kw)
            wait()
            lib.quantize_append(lat[i], rope[i], slots.flatten(), cache)
            wait()
            results += [slots, *lib.paged_mla_decode(q[i], cache, table, n, 0.04, **kw)]
            wait()
            lib.fork_sequences(table, n, refs, src, dst, **kw)
            wait()
            results += lib.paged_mla_decode(q[i], cache, table, n, 0.04, **kw)
            wait()
            if i % 3 == 2:
                results += lib.compact_pages([cache], table, n, refs, **kw)[2:]
                wait()
        return results + [cache, table, n, refs, status]

    want = chain(torch.cuda.synchronize)
    torch.cuda.synchronize()
    assert int(want[-1].item()) == 0 and int(want[-3].sum().item()) > 100
    for _ in range(3):
        got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain(lambda: None)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
