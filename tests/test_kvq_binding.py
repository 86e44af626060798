"""The Python side of the quantised KV cache without a GPU: tensors that only say they are on one."""

import pytest
import torch

import kv_cache_compression_lowram_b200 as K
from kvq_utils import config


class OnGpu(torch.Tensor):
    """A CPU tensor that calls itself one of a GPU."""

    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.index))


def on_gpu(index, *shape, dtype=torch.bfloat16):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)
    t.index = index
    return t


@pytest.fixture
def no_library(monkeypatch):
    """What reaches the library is a failure."""
    def reached(*_):
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(K, "_kvq_call", reached)


CFG = config(batch=2, layers=1, kv_heads=2, q_heads=4, page=16, max_pages=2)


def arrays(index):
    return {n: on_gpu(index, *shape, dtype=dtype) for n, (shape, dtype) in K._kvq_layouts(K.kvq_config_struct(CFG)).items()}


def calls(a, index):
    x, q = on_gpu(index, 1, 2, 3, 2, 128), on_gpu(index, 1, 2, 1, 4, 128)
    pos, ws = on_gpu(index, 2, dtype=torch.int32), on_gpu(index, 64, dtype=torch.uint8)
    return [lambda: K.lowram_kvq_write(CFG, a, 0, x, x, pos), lambda: K.lowram_kvq_read(CFG, a, 0, x, x, pos),
            lambda: K.lowram_kvq_decode_attn(CFG, a, 0, q, pos, q, ws), lambda: K.lowram_kvq_sparse_attn(CFG, a, 0, 2, q, pos, q)]


def test_data_on_another_device_than_the_arrays_is_refused(no_library):
    for call in calls(arrays(0), 1):
        with pytest.raises(ValueError, match="device"):
            call()
    for call in calls(arrays(1), 1):      # the same calls with everything on one device go on
        with pytest.raises(AssertionError, match="reached"):
            call()


@pytest.fixture
def no_gpu_needed(monkeypatch):
    """Allocations and waits of LowramKvq's constructor, without a GPU."""
    zeros = torch.zeros

    class Stream:
        def synchronize(self):
            pass

    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: on_gpu(0, *a, **k) if device is not None else zeros(*a, **k))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())


def test_arrays_of_a_cache_cannot_be_exchanged(no_library, no_gpu_needed):
    """Calls use the arrays that the cache was made with, so putting others in their place is refused."""
    mine = arrays(0)
    cache = K.LowramKvq(CFG, mine)
    assert cache.arrays["table"] is mine["table"] and cache.arrays["k_mean"] is mine["k_mean"]
    with pytest.raises(TypeError):
        cache.arrays["table"] = on_gpu(0, 2, 2, dtype=torch.int32)
    mine["table"] = None      # the caller's own dict is theirs
    assert cache.arrays["table"] is not None
    again = K.LowramKvq(CFG, cache.arrays)
    assert all(again.arrays[n] is cache.arrays[n] for n in cache.arrays)
    with pytest.raises(AssertionError, match="reached"):
        K.lowram_kvq_write(CFG, cache.arrays, 0, *[on_gpu(0, 1, 2, 3, 2, 128)] * 2, on_gpu(0, 2, dtype=torch.int32))


def test_table_beside_arrays(no_library, no_gpu_needed):
    """``table`` completes arrays that have none; beside one of theirs it is refused, not ignored."""
    table = on_gpu(0, 2, 2, dtype=torch.int32)
    bare = {n: t for n, t in arrays(0).items() if n != "table"}
    assert K.LowramKvq(CFG, bare, table=table).arrays["table"] is table
    assert K.LowramKvq(CFG, bare).arrays["table"] is None
    assert "table" not in bare
    with pytest.raises(ValueError, match="table"):
        K.LowramKvq(CFG, arrays(0), table=table)
