"""The attention of packed chunks on the GPU at the ends of what its arguments may be, against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import heads_reference as ref
import nvfp4_kv_cache_sparse_gb300 as lib
from heads_reference import bf16, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("lq,lk", [(140, 300), (600, 3100)])   # (the second one on CTA pairs)
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_a_scale_of_zero_weighs_all_keys_alike(lq, lk, scale):
    # scores of up to some 2^124 before the scale
    rng = np.random.default_rng(lk)
    q, kv, pe = bf16(rng, lq, 2, 192, scale=2.0 ** 58), bf16(rng, lk, 2, 256), bf16(rng, lk, 64, scale=2.0 ** 58)
    kv[..., :128] = bf16(rng, lk, 2, 128, scale=2.0 ** 58)
    out, lse = lib.ragged_mla_attention(q.to(DEV), kv.to(DEV), pe.to(DEV), starts([lq]).to(DEV), starts([lk]).to(DEV), scale)
    ref.check_attention(out, lse, ref.attention(q, kv, pe, [lq], [lk], scale))
