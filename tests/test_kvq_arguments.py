"""What the C entry points of the quantised KV cache refuse before any CUDA call, beside the ordinary
arguments."""

import ctypes

import pytest

import kv_cache_compression_lowram_b200 as K
from kvq_utils import config
from test_kvq_host import PTR, attn_call, rows_call


@pytest.mark.parametrize("kw", [
    dict(batch=1, layers=1 << 15, kv_heads=1 << 15, q_heads=1 << 15, n_pages=1 << 30, page=16, max_pages=1),
    dict(batch=1, layers=1 << 15, kv_heads=1 << 14, q_heads=1 << 14, n_pages=1 << 30, page=32, max_pages=1)])
def test_pools_whose_rows_pass_64_bits(kw):
    """Products of sizes that are a multiple of 2^64 are not taken for a small pool."""
    assert K.lowram_kvq_token_bytes(config(**kw)) == 0
    with pytest.raises(K.LowramError):
        K.lowram_kvq_workspace_bytes(config(**kw), 1, 1)
    for fn in (K.lib().lowram_kvq_write, K.lib().lowram_kvq_read):
        assert rows_call(fn, config(**kw)) == 1


MISPLACED = ctypes.c_void_p((1 << 20) + 2)      # no address of an int32


def test_integers_at_odd_addresses():
    """pos, count, lens and sel hold 32-bit integers: an address that is not a multiple of 4 would fault."""
    for fn in (K.lib().lowram_kvq_write, K.lib().lowram_kvq_read):
        for kw in (dict(pos=MISPLACED), dict(count=MISPLACED)):
            assert rows_call(fn, **kw) == 1, kw
            assert b"misaligned" in K.lib().lowram_last_error_string()
    for sparse, kw in ((False, dict(lens=MISPLACED)), (True, dict(lens=MISPLACED)), (True, dict(sel=MISPLACED))):
        assert attn_call(sparse, **kw) == 1, kw
        assert b"misaligned" in K.lib().lowram_last_error_string()


def test_outputs_that_overlap_the_queries_in_part():
    """out may be q itself (a row is read before it is written), but not a shifted view of it."""
    size = 2 * 8 * 128 * 2      # config()'s batch, query heads, channels, bytes
    for sparse in (False, True):
        for shift in (16, 256, size - 16):
            for q, out in ((PTR.value, PTR.value + shift), (PTR.value + shift, PTR.value)):
                assert attn_call(sparse, q=ctypes.c_void_p(q), out=ctypes.c_void_p(out)) == 1
                assert b"overlaps" in K.lib().lowram_last_error_string()
        # itself, and neighbours: refused for something else
        for out in (PTR.value, PTR.value + size):
            kw = dict(top_k=0) if sparse else dict(ws=None)
            assert attn_call(sparse, out=ctypes.c_void_p(out), **kw) == 1
            assert b"overlaps" not in K.lib().lowram_last_error_string()
