"""fp32 attention of the quantised KV cache on the GPU against the tight bounds of kvq_tight."""

import pytest
import torch

import kv_cache_compression_lowram_b200 as K
import kvq_tight as T
from kvq_utils import to_device

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d,group,bits,n,lens", T.CASES + [(128, 4, 4, 1, [600, 2, 300]), (64, 16, 8, 2, [900, 4, 33])])
def test_queries_and_weights_keep_their_second_part(d, group, bits, n, lens):
    cfg, arrays, q = T.problem(d, group, bits, lens, 16, n=n)
    cache = K.LowramKvq(cfg, to_device(arrays), max_q=n)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for out in (cache.decode(q.to(DEV), at), cache.decode_sparse(q.to(DEV), at, cfg["max_pages"])):
        assert T.worst(cfg, arrays, q, lens, out.double().cpu().numpy()) <= 1.0
