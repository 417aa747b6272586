"""Reads the CUDA sources: before a CTA of a cluster leaves, every arrival that a commit or an asynchronous store of the peer sends
to one of its barriers has been waited for. No barrier of the cluster orders such an arrival, so one that nobody waits for may
reach the shared memory after the CTA is gone. (No run shows the fault: they are on their way for a short time only.)

A barrier is either one whose every phase some warp waits for in the course of its work (named here, with who), or its last phases are
waited for in the end, in a variable `landed`."""
import re

import pytest

from test_cluster_barriers import kernels

FOLLOWED = {
    "decode_pair_kernel": {"qkdone": "the softmax, each tile", "pvdone": "the softmax, the last tile, and converters, the others",
                           "kfull_a": "the QK issuer, each tile", "kfull_b": "the same", "vfull_a": "the PV issuer, each tile", "vfull_b": "the same",
                           "pfull_a": "the PV issuer, each tile", "pfull_b": "the same", "qready": "the QK issuer", "drain": "the issuers, in whose CTA alone it counts"},
    "paged_expand_kernel": {"acc_full": "the epilogue, each unit", "a_free": "the converters: it is sent only where another tile follows",
                            "drain": "the issuer, in whose CTA alone it counts"},
    "sparse_decode_kernel": {},
    "ragged_attention_kernel": {"s_full": "the softmax, each block", "o_done": "the softmax, each tile", "drain": "the issuers, in whose CTA alone it counts"},
}
SENDS = r"\b(?:mma_commit_cg2|mma_commit_multicast|commit)\s*\(([^;]*);", r"\bsignal_leader\s*\(([^;]*);"


def sent(code):
    return {b for pattern in SENDS for args in re.findall(pattern, code) for b in re.findall(r"ctl->(\w+)", args)}


def landed(code):
    return {b for text in re.findall(r"\blanded\s*=([^;]*);", code) for b in re.findall(r"ctl->(\w+)", text)}


CODE = {p.id: p.values[0] for p in kernels()}


@pytest.mark.parametrize("name", sorted(FOLLOWED))
def test_no_arrival_is_left_on_its_way(name):
    code = CODE[name]
    assert set(FOLLOWED[name]) <= sent(code)
    assert sent(code) - set(FOLLOWED[name]) == landed(code) != set()
