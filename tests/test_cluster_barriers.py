"""Reads the CUDA sources: a kernel that writes to the shared memory of other CTAs of its cluster first waits in a barrier
of the cluster, as a CTA's shared memory exists only once it runs. (No run shows the fault: CTAs of a cluster start
almost together.)"""
import os
import re

import pytest

import nvfp4_kv_cache_sparse_gb300.build as build

REMOTE = r"\b(publish|signal_leader|mapa_shared|st_async_\w+)\s*\("
BARRIER = r"\b(cluster_sync|cluster_wait)\s*\("


def body(text, at):
    """The braces' content from the first brace behind position at."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise ValueError("unbalanced braces")


def kernels():
    for name in sorted(f for f in os.listdir(build.CSRC) if f.endswith((".cu", ".cuh"))):
        with open(os.path.join(build.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
        for m in re.finditer(r"__global__[^{;]*?(\w+)\s*\(\s*const", text):
            code = body(text, m.end())
            if re.search(REMOTE, code):
                yield pytest.param(code, id=m.group(1))


@pytest.mark.parametrize("code", list(kernels()))
def test_a_barrier_precedes_the_first_remote_access(code):
    barrier = re.search(BARRIER, code)
    assert barrier is not None and barrier.start() < re.search(REMOTE, code).start()


def test_the_kernels_that_publish_are_found():
    found = [p.id for p in kernels()]
    assert {"resize_kernel", "compact_plan_kernel", "decode_pair_kernel"} <= set(found)
