"""Calls of the quantised KV cache on the GPU beside the ordinary ones: other streams, in place, several
threads."""

import numpy as np
import pytest
import torch

import kv_cache_compression_lowram_b200 as K
from kvq_utils import config, fill, queries, to_device

pytestmark = pytest.mark.gpu
DEV = "cuda"
LONG = 200_000_000      # cycles: about a tenth of a second


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_are_taken_on_the_stream_of_the_call(raw):
    """Without ``out``, a call on another stream gets memory that nothing on the current stream still
    writes, and that is not handed out again before the call is done."""
    cfg = config(batch=2, layers=2, kv_heads=2, q_heads=8, page=16, max_pages=20)
    cache = K.LowramKvq(cfg, to_device(fill(cfg, 40)))
    q, lens = queries(cfg).to(DEV), i32([300, 77])
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    calls = (lambda **kw: (cache.decode(q, lens, **kw),), lambda **kw: cache.decode_sparse(q, lens, 5, sel=True, **kw))
    for call in calls:
        want = [t.clone() for t in call()]
        for _ in range(2):
            torch.cuda.synchronize()
            junk = [torch.empty_like(t) for t in want]      # blocks of the current stream, freed before they are written
            torch.cuda._sleep(LONG)
            for t in junk:
                t.fill_(7)
            del junk, t
            got = call(stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            with torch.cuda.stream(side):
                torch.cuda._sleep(LONG)
            got = call(stream=stream)
            del got                                          # and what comes next on the current stream is its own
            other = [torch.full_like(t, 3) for t in want]
            torch.cuda.synchronize()
            assert all((t == 3).all() for t in other)
    with torch.cuda.stream(side):      # the current stream, named
        got = cache.decode(q, lens, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, cache.decode(q, lens))


def test_validate_waits_for_calls_on_other_streams():
    cfg = config(batch=2, kv_heads=2, q_heads=4, page=16, max_pages=4)
    cache = K.LowramKvq(cfg, to_device(fill(cfg, 41)))
    q, out, lens = queries(cfg).to(DEV), queries(cfg).to(DEV), i32([65, 3])
    side = torch.cuda.Stream()
    for call in (lambda: cache.decode(q, lens, out=out, stream=side), lambda: cache.decode_sparse(q, lens, 2, out=out, stream=side)):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(LONG)
        call()
        assert cache.validate() == 2 and cache.validate() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group,n,lens", [(128, 4, 1, [9000, 0, 33]), (64, 16, 4, [3000, 5, 700]), (256, 12, 3, [2000, 64, 1])])
def test_attention_in_place(dtype, d, group, n, lens):
    """out = q, also where several blocks share a sequence and where its rows take more than one tile."""
    cfg = config(batch=3, layers=2, kv_heads=2, q_heads=2 * group, head_dim=d, page=16, max_pages=-(-max(lens) // 16), n_pages=60, dtype=dtype)
    arrays = fill(dict(cfg, batch=1, max_pages=1), 42)
    arrays["table"] = np.random.default_rng(3).integers(0, 60, (3, cfg["max_pages"])).astype(np.int32)
    cache = K.LowramKvq(cfg, to_device(arrays), max_q=n)
    q, lens = queries(cfg, n).to(DEV), i32(lens)
    for call in (lambda q, out: cache.decode(q, lens, out=out), lambda q, out: cache.decode_sparse(q, lens, 40, out=out)):
        want = call(q, None)
        for _ in range(3):
            own = q.clone()
            assert call(own, own) is own and torch.equal(own, want)
