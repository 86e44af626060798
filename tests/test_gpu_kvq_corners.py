"""Corners of the quantised KV cache's value ranges on the GPU, against the fp64 oracle."""

import numpy as np
import pytest
import torch

import kv_cache_compression_lowram_b200 as K
from kvq_utils import DT, check_attention, config, fill, queries, to_device

pytestmark = pytest.mark.gpu
DEV = "cuda"
LOG2E = 1.4426950408889634


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------ attention

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group", [(64, 1), (64, 16), (128, 4), (128, 7), (128, 16), (256, 4), (256, 8)])
@pytest.mark.parametrize("sparse", [False, True])
def test_weights_at_the_top_of_their_range(bits, dtype, d, group, sparse):
    """Value scales of 1, then 16 times that with scores just as far above the first ones as they may be
    without a new maximum: the largest weights that are ever rounded to fp16."""
    n = 4096 if sparse else 512       # every warp meets both halves
    cfg = config(batch=1, kv_heads=1, q_heads=group, head_dim=d, page=64, max_pages=n // 64, bits=bits, dtype=dtype)
    arrays = fill(cfg, 30)
    late = arrays["table"][0, n // 128:]
    arrays["k_code"][:], arrays["k_scale"][:] = 0, 0
    arrays["k_scale"][0, late, 0, :, 0, 1] = 1.0       # khat = 1 in the first group
    arrays["v_scale"][..., 0] = 1.0
    arrays["v_scale"][0, late, ..., 0] = 16.0
    slack = 2.0 if dtype == "f32" else 4.0
    q = torch.zeros(1, 1, 1, group, d)
    q[..., 0] = (slack - 2.0 ** -13) * d ** 0.5 / LOG2E
    q = q.to(DT[dtype])
    cache = K.LowramKvq(cfg, to_device(arrays))
    out = cache.decode_sparse(q.to(DEV), i32([n]), n // 64) if sparse else cache.decode(q.to(DEV), i32([n]))
    assert torch.isfinite(out).all()
    check_attention(cfg, arrays, q, [n], out)
