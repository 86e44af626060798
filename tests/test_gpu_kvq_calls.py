"""Calls of the quantised KV cache on the GPU beside the ordinary ones: other streams, in place, several
threads."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import kv_cache_compression_lowram_b200 as K
from kvq_utils import check_attention, config, fill, queries, to_device

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def test_first_calls_of_several_threads():
    """The first calls of a process, made by several threads at once, each with its cache and stream."""
    code = """
import threading, torch, kv_cache_compression_lowram_b200 as K
N = 6
cfg = dict(batch=2, n_layers=1, n_kv_heads=2, n_q_heads=8, head_dim=128, page=16, n_pages=64, max_pages=32, bits=4, dtype="bf16")
torch.manual_seed(1)
x = torch.randn(1, 2, 500, 2, 128, device="cuda").bfloat16()
q = torch.randn(1, 2, 1, 8, 128, device="cuda").bfloat16()
pos, lens = (torch.full((2,), n, dtype=torch.int32, device="cuda") for n in (0, 500))
caches, streams = [K.LowramKvq(cfg) for _ in range(N)], [torch.cuda.Stream() for _ in range(N)]
outs, gate = [None] * N, threading.Barrier(N)
torch.cuda.synchronize()
def work(i):
    gate.wait()
    with torch.cuda.stream(streams[i]):
        caches[i].write(x, x, pos)
        outs[i] = [caches[i].decode(q, lens), caches[i].decode_sparse(q, lens, 9)] + list(caches[i].read(pos, n=500))
threads = [threading.Thread(target=work, args=(i,)) for i in range(N)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert all(torch.equal(a, b) for o in outs for a, b in zip(o, outs[0])) and torch.isfinite(outs[0][0]).all()
assert (outs[0][2] - x).abs().max() < 0.5 and all(c.validate() == 0 for c in caches)
print("threads done")
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "threads done" in done.stdout, done.stderr[-2000:]


@pytest.mark.parametrize("batch,pages", [(1, 9000), (3, 9000), (24, 6000), (4, 5200)])
def test_sparse_clusters_of_every_size(batch, pages):
    """Tables so wide that an SM holds one block: clusters of 8, 4, 2 and 1 blocks, all with the same pages
    selected as among the same keys in the oracle."""
    r = np.random.default_rng(batch)
    lens = [pages * 16] + [int(x) for x in r.integers(1, 4000, batch - 1)]
    cfg = config(batch=batch, kv_heads=8, q_heads=16, head_dim=64, page=16, max_pages=pages, n_pages=200)
    arrays = fill(dict(cfg, batch=1, max_pages=1), 43)
    arrays["table"] = r.integers(0, 200, (batch, pages)).astype(np.int32)
    cache = K.LowramKvq(cfg, to_device(arrays))
    q = queries(cfg, seed=5)
    out, sel = cache.decode_sparse(q.to(DEV), i32(lens), 20, sel=True)
    check_attention(cfg, arrays, q, lens, out, top_k=20, sel=sel)
