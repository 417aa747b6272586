"""Refusals of the calls on sequences in pages that need no GPU: the binding's ValueErrors and the C ABI's
status codes, and the plain page operations that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_kv_cache_sparse_gb300 as lib
import paged_reference as ref
from nvfp4_kv_cache_sparse_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def cdll():
    build.build()
    return lib.load()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_decode_refusals():
    ok = dict(q=torch.zeros(2, 1, 16, 576, dtype=torch.bfloat16), cache=u8(128, 352), page_table=i32(2, 2), seq_lens=i32(2), sm_scale=0.1)
    for change, match in (({"q": torch.zeros(2, 1, 16, 576)}, "q bf16"), ({"q": torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16)}, "q bf16"),
                          ({"cache": u8(128, 656)}, "cache"), ({"cache": torch.zeros(128, 352)}, "cache"),
                          ({"page_table": torch.zeros(2, 2, dtype=torch.int64)}, "page_table"), ({"page_table": i32(2, 4)[:, ::2]}, "page_table"),
                          ({"page_table": i32(3, 2), "seq_lens": i32(3)}, "batch"), ({"seq_lens": i32(3)}, "seq_lens"),
                          ({"seq_lens": torch.zeros(2)}, "seq_lens"), ({"attn_sink": torch.zeros(15)}, "attn_sink"),
                          ({"page_size": 0}, "page_size"), ({"cache": u8(128, 432), "block_scales": True}, "block_scales"),
                          ({}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            lib.paged_mla_decode(**{**ok, **change})


def test_page_call_refusals():
    table, lens, refs, idx = i32(2, 4), i32(2), i32(8), i32(2)
    with pytest.raises(ValueError, match="caches"):
        lib.copy_pages([], idx, idx)
    with pytest.raises(ValueError, match="caches"):
        lib.copy_pages([u8(512, 350)], idx, idx)
    with pytest.raises(ValueError, match="page_size"):
        lib.copy_pages([u8(512, 352)], idx, idx, page_size=0)
    with pytest.raises(ValueError, match="CUDA device"):
        lib.copy_pages([u8(512, 352)], idx, idx)
    with pytest.raises(ValueError, match="differ in length"):
        lib.fork_sequences(table, lens, refs, idx, i32(3))
    with pytest.raises(ValueError, match="int32"):
        lib.fork_sequences(table, lens, refs, idx.long(), idx)
    with pytest.raises(ValueError, match="CUDA device"):
        lib.fork_sequences(table, lens, refs, idx, idx)
    with pytest.raises(ValueError, match="new_lens"):
        lib.resize_sequences([], table, lens, refs, i32(3))
    with pytest.raises(ValueError, match="max_new"):
        lib.resize_sequences([], table, lens, refs, i32(2), -1)
    with pytest.raises(ValueError, match="page_refs"):
        lib.resize_sequences([], table, lens, refs.long(), i32(2))
    with pytest.raises(ValueError, match="fewer pages"):
        lib.resize_sequences([u8(511, 352)], table, lens, refs, i32(2))
    with pytest.raises(ValueError, match="overlap"):
        lib.fork_sequences(i32(1, 4).expand(2, 4), lens, refs, idx, idx)
    with pytest.raises(ValueError, match="table_out"):
        lib.compact_pages([], table, lens, refs, table_out=i32(2, 5))


def test_workspace_sizes(cdll):
    n16, n32, n64 = lib.paged_workspace_size(3, 1, 16), lib.paged_workspace_size(1, 2, 16), lib.paged_workspace_size(7, 1, 33)
    assert 0 < n16 < n32 < n64 < lib.paged_workspace_size(1, 500, 128)   # (grows with the 128-row tiles)
    assert lib.paged_workspace_size(0, 1, 16) == 0 and lib.paged_workspace_size(1, 0, 16) == 0
    assert lib.pages_workspace_size(2, 4, 100) >= 4 * 108
    assert lib.pages_workspace_size(2, 1000, 100, 50) >= 4 * 50 * 1001
    n = ctypes.c_size_t()
    ref_n = ctypes.byref(n)
    for args, st in (((1, 1, 129), lib.ERR_UNSUPPORTED), ((1, 1, 0), lib.ERR_UNSUPPORTED), ((-1, 1, 16), lib.ERR_INVALID_ARG),
                     ((2 ** 30, 2, 16), lib.ERR_INVALID_ARG)):
        assert cdll.nvfp4_paged_mla_decode_workspace_size(*args, ref_n) == st
    assert cdll.nvfp4_paged_mla_decode_workspace_size(1, 1, 16, None) == lib.ERR_INVALID_ARG
    assert cdll.nvfp4_mla_pages_workspace_size(1 << 16, 1 << 16, 10, 0, ref_n) == lib.ERR_INVALID_ARG
    assert cdll.nvfp4_mla_pages_workspace_size(1, 1, 1 << 31, 0, ref_n) == lib.ERR_INVALID_ARG
    assert cdll.nvfp4_mla_pages_workspace_size(1, 1, 1, -1, ref_n) == lib.ERR_INVALID_ARG


def test_c_status_codes_before_any_device_query(cdll):
    A, D, U, W = 4096, lib.ERR_INVALID_ARG, lib.ERR_UNSUPPORTED, lib.ERR_WORKSPACE   # A: an aligned non-null address, never read

    def decode(q=A, cache=A, pages=8, ps=64, rec=352, table=A, stride=4, width=4, lens=A, b=2, s_q=1, h=16, out=A, lse=A, ws=A, n=1 << 30):
        return cdll.nvfp4_paged_mla_decode(q, cache, pages, ps, rec, table, stride, width, lens, b, s_q, h, 1.0, None, out, lse, ws, n, None, None)

    for kw, st in (({"b": 0}, lib.OK), ({"s_q": 0}, lib.OK), ({"q": None}, D), ({"q": A + 8}, D), ({"cache": A + 8}, D), ({"lens": None}, D),
                   ({"table": None}, D), ({"out": A + 2}, D), ({"ps": 0}, D), ({"ps": 48}, D), ({"ps": 8192}, D), ({"stride": 3}, D),
                   ({"rec": 656}, U), ({"rec": 400}, U), ({"rec": 432 | lib.SCALES_BLOCK_ORDER}, U), ({"h": 0}, U), ({"h": 129}, U),
                   ({"width": 1 << 25, "stride": 1 << 25}, D), ({"pages": -1}, D), ({"ws": None}, W), ({"ws": A + 16}, W), ({"n": 1000}, W)):
        assert decode(**kw) == st, kw

    caches = (ctypes.c_void_p * 2)(A, A)
    bad = (ctypes.c_void_p * 2)(A, A + 4)

    def copy(c=caches, num=2, pages=8, ps=64, rec=656, src=A, dst=A, n=2):
        return cdll.nvfp4_mla_copy_pages(c, num, pages, ps, rec, src, dst, n, None, None)

    for kw, st in (({"n": 0}, lib.OK), ({"n": -1}, D), ({"num": 0}, D), ({"num": 257}, D), ({"c": bad}, D), ({"src": None}, D), ({"dst": A + 2}, D),
                   ({"rec": 100}, U), ({"ps": 3}, D)):
        assert copy(**kw) == st, kw

    def fork(table=A, stride=4, width=4, lens=A, b=2, refs=A, pages=8, ps=64, src=A, dst=A, n=2, ws=A, nb=1 << 20):
        return cdll.nvfp4_mla_fork_sequences(table, stride, width, lens, b, refs, pages, ps, src, dst, n, ws, nb, None, None)

    for kw, st in (({"n": 0}, lib.OK), ({"n": -1}, D), ({"table": None}, D), ({"refs": A + 4}, D), ({"stride": 2}, D), ({"src": None}, D), ({"nb": 4}, W)):
        assert fork(**kw) == st, kw

    def resize(table=A, stride=4, width=4, lens=A, new=A, b=2, refs=A, pages=8, ps=64, c=caches, num=2, rec=352, slots=A, m=3, ws=A, nb=1 << 20):
        return cdll.nvfp4_mla_resize_sequences(table, stride, width, lens, new, b, refs, pages, ps, c, num, rec, slots, m, ws, nb, None, None)

    for kw, st in (({"b": 0}, lib.OK), ({"new": None}, D), ({"slots": None}, D), ({"slots": A + 4}, D), ({"m": -1}, D), ({"c": bad}, D), ({"c": None}, D),
                   ({"rec": 1}, U), ({"ws": None}, W), ({"nb": 32}, W)):
        assert resize(**kw) == st, kw

    def compact(c=caches, num=2, rec=352, table=A, stride=4, tout=A, ostride=4, width=4, lens=A, b=2, refs=A, rout=A, pages=8, ps=64, pm=A, live=A,
                ws=A, nb=1 << 20):
        return cdll.nvfp4_mla_compact_pages(c, num, rec, table, stride, tout, ostride, width, lens, b, refs, rout, pages, ps, pm, live, ws, nb, None, None)

    for kw, st in (({"live": None}, D), ({"pm": None}, D), ({"ostride": 3}, D), ({"ostride": 5}, D), ({"rout": A + 4}, D), ({"refs": None}, D),
                   ({"table": None}, D), ({"rec": 0}, U), ({"nb": 0}, W)):
        assert compact(**kw) == st, kw


def test_the_plain_page_operations_keep_their_invariants():
    # counts equal the table's entries, whatever is called in whatever order
    rng = np.random.default_rng(0)
    for ps in (1, 4, 16):
        p = ref.Pages([[-1] * 8 for _ in range(6)], [0] * 6, [0] * 40, ps)
        for _ in range(200):
            what = rng.integers(3)
            if what == 0:
                p.resize([int(n) for n in rng.integers(-2, 8 * ps + 3, 6)], 2)
            elif what == 1:
                n = int(rng.integers(1, 7))
                p.fork(list(rng.integers(-1, 7, n)), list(rng.integers(-1, 7, n)))
            else:
                p.compact()
            used = [e for b, row in enumerate(p.table) for e in row[:p.count(p.lens[b])]]
            assert p.refs == list(np.bincount(used, minlength=40)) and all(e >= 0 for e in used)
            assert all(e == -1 for b, row in enumerate(p.table) for e in row[p.count(p.lens[b]):])
