"""Refusals of the calls around the latent attention that need no GPU: the binding's ValueErrors and the C ABI's
status codes."""
import ctypes

import pytest
import torch

import nvfp4_kv_cache_sparse_gb300 as lib
from nvfp4_kv_cache_sparse_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def cdll():
    build.build()
    return lib.load()


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(shape)


def refuse(call, ok, cases):
    for change, match in cases:
        with pytest.raises(ValueError, match=match):
            call(**{**ok, **change})


def test_absorb_refusals():
    refuse(lib.mla_absorb_query, dict(q=bf(4, 3, 192), kv_b=bf(3, 256, 512)),
           (({"q": f32(4, 3, 192)}, "q bf16"), ({"q": bf(4, 3, 576)}, "q bf16"), ({"q": bf(4, 3, 384)[..., ::2]}, "q bf16"), ({"q": bf(4, 192)}, "q bf16"),
            ({"kv_b": bf(2, 256, 512)}, "kv_b"), ({"kv_b": bf(3, 512, 256)}, "kv_b"), ({"kv_b": f32(3, 256, 512)}, "kv_b"),
            ({"cos_table": f32(9, 32)}, "go with positions"), ({"positions": torch.zeros(4, dtype=torch.int64)}, "cos_table"),
            ({"positions": i32(4)}, "positions"), ({"positions": torch.zeros(5, dtype=torch.int64)}, "positions"),
            ({"positions": torch.zeros(4, dtype=torch.int64), "cos_table": f32(9, 64), "sin_table": f32(9, 64)}, "cos_table"),
            ({"positions": torch.zeros(4, dtype=torch.int64), "cos_table": f32(9, 32), "sin_table": f32(8, 32)}, "cos_table"),
            ({"dev_status": f32(1)}, "dev_status"), ({}, "CUDA device")))


def test_project_refusals():
    refuse(lib.mla_project_values, dict(latent=bf(4, 3, 512), kv_b=bf(3, 256, 512)),
           (({"latent": bf(4, 3, 576)}, "latent"), ({"latent": bf(4, 3, 512).half()}, "latent"), ({"kv_b": bf(4, 256, 512)}, "kv_b"), ({}, "CUDA device")))


def test_expand_refusals():
    ok = dict(cache=torch.zeros(128, 352, dtype=torch.uint8), page_table=i32(2, 2), cu_seqlens=i32(3), kv_b=bf(3, 256, 512), num_rows=5)
    refuse(lib.paged_mla_expand, ok,
           (({"cache": torch.zeros(128, 656, dtype=torch.uint8)}, "cache"), ({"cache": f32(128, 352)}, "cache"), ({"page_table": i32(3, 2)}, "page_table"),
            ({"page_table": i32(2, 4)[:, ::2]}, "page_table"), ({"page_table": i32(1, 2).expand(2, 2)}, "overlap"), ({"cu_seqlens": i32(0)}, "cu_seqlens"),
            ({"cu_seqlens": torch.zeros(3, dtype=torch.int64)}, "cu_seqlens"), ({"kv_b": bf(256, 512)}, "kv_b"), ({"num_rows": -1}, "num_rows"),
            ({"page_size": 0}, "page_size"), ({"cache": torch.zeros(128, 432, dtype=torch.uint8), "block_scales": True}, "block_scales"), ({}, "CUDA device")))


def test_attention_refusals():
    ok = dict(q=bf(4, 3, 192), kv=bf(9, 3, 256), k_pe=bf(9, 64), cu_seqlens_q=i32(3), cu_seqlens_k=i32(3), sm_scale=0.1)
    refuse(lib.ragged_mla_attention, ok,
           (({"q": bf(4, 3, 576)}, "q bf16"), ({"kv": bf(9, 2, 256)}, "heads"), ({"kv": bf(9, 3, 320)}, "kv bf16"), ({"k_pe": bf(8, 64)}, "k_pe"),
            ({"k_pe": f32(9, 64)}, "k_pe"), ({"k_pe": bf(9, 128)[:, ::2]}, "k_pe"), ({"cu_seqlens_q": i32(4)}, "differ in length"),
            ({"cu_seqlens_k": torch.zeros(3)}, "cu_seqlens_k"), ({"attn_sink": f32(4)}, "attn_sink"), ({}, "CUDA device")))


def test_c_status_codes_before_any_device_query(cdll):
    A, D, U, W = 4096, lib.ERR_INVALID_ARG, lib.ERR_UNSUPPORTED, lib.ERR_WORKSPACE   # A: an aligned non-null address, never read
    big = 1 << 31

    def absorb(q=A, ts=576, hs=192, w=A, rs=512, ws=256 * 512, pos=A, cos=A, sin=A, P=9, half=1, T=4, h=3, out=A):
        return cdll.nvfp4_mla_absorb_query(q, ts, hs, w, rs, ws, pos, cos, sin, P, half, T, h, out, None, None)

    for change, st in (({"h": 0}, U), ({"h": 129}, U), ({"T": -1}, D), ({"T": big}, D), ({"half": 2}, D), ({"P": -1}, D), ({"q": None}, D), ({"q": A + 8}, D),
                       ({"ts": 190}, D), ({"hs": 0}, D), ({"hs": -8}, D), ({"ts": 1 << 40}, D), ({"w": A + 2}, D), ({"rs": 511}, D), ({"ws": 4}, D), ({"out": None}, D),
                       ({"out": A + 16}, D), ({"cos": None}, D), ({"sin": None}, D), ({"cos": A + 4}, D), ({"pos": A + 4}, D), ({"T": 0, "q": None, "out": None}, lib.OK)):
        assert absorb(**change) == st, change

    def project(x=A, ts=3 * 512, hs=512, w=A, rs=512, ws=256 * 512, T=4, h=3, out=A):
        return cdll.nvfp4_mla_project_values(x, ts, hs, w, rs, ws, T, h, out, None, None)

    for change, st in (({"h": 200}, U), ({"T": -1}, D), ({"x": None}, D), ({"x": A + 2}, D), ({"ts": 1}, D), ({"hs": 12}, D), ({"w": None}, D), ({"out": A + 4}, D),
                       ({"T": 0, "out": None}, lib.OK)):
        assert project(**change) == st, change

    def expand(cache=A, pages=8, ps=64, rec=352, table=A, ts=4, width=4, cu=A, b=2, w=A, h=3, kv=A, pe=A, rows=100):
        return cdll.nvfp4_paged_mla_expand(cache, pages, ps, rec, table, ts, width, cu, b, w, 512, 256 * 512, h, kv, pe, rows, None, None)

    for change, st in (({"rec": 656}, U), ({"rec": 400}, U), ({"rec": 432 | lib.SCALES_BLOCK_ORDER}, U), ({"h": 0}, U), ({"ps": 48}, D), ({"ps": 8192}, D), ({"ts": 3}, D),
                       ({"b": -1}, D), ({"pages": -1}, D), ({"pages": big}, D), ({"rows": -1}, D), ({"rows": big}, D), ({"cache": None}, D), ({"cache": A + 8}, D),
                       ({"table": None}, D), ({"cu": None}, D), ({"w": None}, D), ({"kv": A + 16}, D), ({"pe": None}, D), ({"pe": A + 8}, D),
                       ({"rows": 0, "kv": None, "pe": None}, lib.OK), ({"b": 0, "cu": None}, lib.OK)):
        assert expand(**change) == st, change

    size = lib.ragged_workspace_size()
    assert size > 0 and size % 256 == 0 and cdll.nvfp4_ragged_mla_attention_workspace_size(None) == D

    def attend(q=A, qt=576, qh=192, nq=4, kv=A, kt=768, kh=256, pe=A, ps=64, nk=9, cq=A, ck=A, b=2, h=3, sink=None, out=A, lse=A, ws=A, wb=size):
        return cdll.nvfp4_ragged_mla_attention(q, qt, qh, nq, kv, kt, kh, pe, ps, nk, cq, ck, b, h, 0.1, sink, out, lse, ws, wb, None, None)

    for change, st in (({"h": 0}, U), ({"h": 129}, U), ({"nq": -1}, D), ({"nk": -1}, D), ({"nq": big}, D), ({"nk": big}, D), ({"nk": 1 << 26}, D), ({"b": -1}, D), ({"b": (1 << 20) + 1}, D),
                       ({"q": None}, D), ({"q": A + 4}, D), ({"qt": 4}, D), ({"qh": 100}, D), ({"kv": None}, D), ({"kt": 0}, D), ({"kh": 4}, D), ({"pe": None}, D),
                       ({"ps": 60}, D), ({"cq": None}, D), ({"ck": A + 2}, D), ({"sink": A + 2}, D), ({"out": A + 16}, D), ({"lse": None}, D), ({"ws": None}, W),
                       ({"wb": size - 1}, W), ({"ws": A + 128}, W), ({"nq": 0, "q": None}, lib.OK), ({"b": 0, "cq": None}, lib.OK)):
        assert attend(**change) == st, change
