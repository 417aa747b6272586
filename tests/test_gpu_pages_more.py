"""More of the page operations on the GPU: the smallest pools, pools that are exactly large enough."""
import numpy as np
import pytest

from test_gpu_pages import State

pytestmark = pytest.mark.gpu


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
