"""The quantised KV cache without a GPU: its format in the oracle, and what its entry points refuse
before any CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

import kv_cache_compression_lowram_b200 as K
from kvq_utils import config
from oracle import kvq as O

PTR = ctypes.c_void_p(1 << 20)      # an aligned address that is never followed
ODD = ctypes.c_void_p((1 << 20) + 8)


def cache(**kw):
    c = K.LowramKvqCacheC()
    for n in ("k_code", "k_scale", "v_code", "v_scale", "k_mean", "table"):
        setattr(c, n, PTR.value)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def strides(*s):
    return (ctypes.c_int64 * 4)(*s)


OK_STRIDES = strides(4096, 2048, 256, 128)


def rows_call(fn, cfg=None, arr=None, layer0=0, n_layers=1, n=4, k=PTR, ks=OK_STRIDES, v=PTR, vs=OK_STRIDES, pos=PTR, count=None):
    c = K.kvq_config_struct(cfg or config())
    return fn(ctypes.byref(c), None if arr is False else ctypes.byref(arr or cache()), layer0, n_layers, n, k, ks, v, vs, pos, count, None)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_oracle_format(bits, d):
    r = np.random.default_rng(d + bits)
    n = r.integers(0, 1 << bits, (3, d))
    raw = O.pack(n, bits)
    assert raw.shape == (3, d * bits // 8) and np.array_equal(O.unpack(raw, bits), n)
    x = r.standard_normal((50, d)) * 10.0 ** r.integers(-3, 4, (50, 1))
    n, s = O.quantise(x, bits)
    back = O.dequantise(n, s)
    # half a step, the roundings of lo and s to fp16, and what fp16's smallest step leaves
    step = np.repeat(s[..., 0].astype(float), 64, -1)
    rng = np.abs(x).max(-1, keepdims=True) * 2
    assert (np.abs(back - x) <= step / 2 + rng * 2.0 ** -10 + 2.0 ** -24 * (1 << bits)).all()
    # worked example: 64 channels 0 .. 63 in 4 bits: s = 63 / 15 = 4.2, codes round(c / fp16(4.2))
    n, s = O.quantise(np.arange(64.0), 4)
    assert float(s[0, 0]) == float(np.float16(4.2)) and float(s[0, 1]) == 0.0
    assert n[[0, 2, 3, 6, 7, 62, 63]].tolist() == [0, 0, 1, 1, 2, 15, 15]


def test_code_places_are_a_permutation():
    for d in (64, 128, 256):
        for bits in (4, 8):
            assert len({O.code_place(c, d, bits) for c in range(d)}) == d
    # channel 64 g + 8 w + i is code i of cell w G + g
    assert O.code_place(64 + 8 * 3 + 5, 128, 4) == ((3 * 2 + 1) * 4 + 2, 4)
    assert O.code_place(64 + 8 * 3 + 5, 128, 8) == ((3 * 2 + 1) * 8 + 5, 0)


def test_oracle_selection():
    s = np.array([1.0, 5.0, np.nan, 5.0, -np.inf, 7.0])
    assert O.select(s, 5, 1) == [5]
    assert O.select(s, 5, 3) == [1, 3, 5]
    assert O.select(s, 5, 2) == [1, 5]
    assert O.select(s, 5, 5) == [0, 1, 2, 3, 5]
    assert O.select(s, 0, 4) == [0]


def test_token_bytes():
    for d, bits, want in ((64, 4, 72), (128, 4, 144), (128, 8, 272), (256, 8, 544)):
        assert K.lowram_kvq_token_bytes(config(head_dim=d, bits=bits)) == want
    assert K.lowram_kvq_token_bytes(config(bits=5)) == 0


BAD = [dict(batch=0), dict(layers=0), dict(kv_heads=3), dict(q_heads=34), dict(page=24), dict(page=8), dict(page=512),
       dict(max_pages=16385), dict(bits=3), dict(bits=16), dict(max_pages=0, n_pages=4), dict(batch=70000),
       dict(layers=64, kv_heads=8, n_pages=1 << 15, page=256)]   # 2^32 rows


@pytest.mark.parametrize("kw", BAD)
def test_bad_configs(kw):
    cfg = config(**kw)
    with pytest.raises(K.LowramError) as ei:
        K.lowram_kvq_workspace_bytes(cfg, 1, 1)
    assert ei.value.status == 1
    for fn in (K.lib().lowram_kvq_write, K.lib().lowram_kvq_read):
        assert rows_call(fn, cfg) == 1
    assert K.lib().lowram_last_error_string()


@pytest.mark.parametrize("d", [32, 96, 192, 512])
def test_unsupported_head_dim(d):
    for fn in (K.lib().lowram_kvq_write, K.lib().lowram_kvq_read):
        assert rows_call(fn, config(head_dim=d)) == 4


def test_rows_are_checked():
    for fn in (K.lib().lowram_kvq_write, K.lib().lowram_kvq_read):
        bad = [dict(arr=False), dict(arr=cache(k_code=None)), dict(arr=cache(v_scale=ODD.value)), dict(arr=cache(k_mean=ODD.value)),
               dict(arr=cache(table=PTR.value + 2)), dict(layer0=-1), dict(layer0=1), dict(n_layers=0), dict(n_layers=2), dict(n=-1),
               dict(n=8 * 32 + 1), dict(k=None), dict(k=ODD), dict(v=None), dict(ks=None), dict(vs=strides(0, -8, 256, 128)),
               dict(ks=strides(0, 2048, 257, 128)), dict(vs=strides(0, 2048, 256, 4)), dict(pos=None)]
        for kw in bad:
            assert rows_call(fn, **kw) == 1, kw
            assert K.lib().lowram_last_error_string()
        # without a table the pool has to hold every sequence's pages
        assert rows_call(fn, config(batch=4, max_pages=8, n_pages=31), cache(table=None)) == 1
        assert rows_call(fn, n=0) == 0
    # an output that two rows share is refused, a source may be broadcast
    assert rows_call(K.lib().lowram_kvq_read, vs=strides(0, 2048, 0, 128)) == 1
    # too many rows for one launch
    big = config(batch=30000, layers=500, kv_heads=500, q_heads=500, n_pages=2)
    assert rows_call(K.lib().lowram_kvq_write, big, n_layers=500) == 1


def attn_call(sparse, cfg=None, arr=None, layer0=0, n_layers=1, n=1, top_k=4, q=PTR, lens=PTR, out=PTR, ws=PTR, ws_bytes=1 << 40, sel=None):
    c = K.kvq_config_struct(cfg or config())
    a = ctypes.byref(arr or cache())
    if sparse:
        return K.lib().lowram_kvq_sparse_attn(ctypes.byref(c), a, layer0, n_layers, n, top_k, q, lens, out, sel, None)
    return K.lib().lowram_kvq_decode_attn(ctypes.byref(c), a, layer0, n_layers, n, q, lens, out, ws, ws_bytes, None)


def test_attention_arguments_are_checked():
    for sparse in (False, True):
        bad = [dict(n=0), dict(n=17), dict(q=None), dict(q=ODD), dict(out=None), dict(out=ODD), dict(lens=None), dict(layer0=1),
               dict(n_layers=0), dict(cfg=config(bits=2)), dict(arr=cache(v_code=None)),
               dict(cfg=config(batch=60000, layers=500, kv_heads=100, q_heads=100, n_pages=9), n_layers=500)]
        for kw in bad:
            assert attn_call(sparse, **kw) == 1, kw
        assert attn_call(sparse, config(head_dim=80)) == 4
    # 2^31 steps of 16 tokens and more in one call
    assert attn_call(False, config(batch=2048, layers=64, kv_heads=8, max_pages=16384, n_pages=9, page=16), n_layers=64) == 1
    need = K.lowram_kvq_workspace_bytes(config(), 1, 1)
    for kw in (dict(ws=None), dict(ws=ODD), dict(ws_bytes=need - 1)):
        assert attn_call(False, **kw) == 1
    for kw in (dict(top_k=0), dict(top_k=513), dict(arr=cache(k_mean=None))):
        assert attn_call(True, **kw) == 1


def test_workspace_grows_with_its_arguments():
    cfg = config(layers=4)
    sizes = [K.lowram_kvq_workspace_bytes(cfg, l, n) for l, n in ((1, 1), (4, 1), (4, 16))]
    assert sizes == sorted(sizes)
    for l, n in ((0, 1), (5, 1), (1, 0), (1, 17)):
        with pytest.raises(K.LowramError):
            K.lowram_kvq_workspace_bytes(cfg, l, n)


def test_binding_refuses_wrong_tensors():
    """Types, shapes, devices and layouts are refused before the library is called."""
    cfg = config(batch=2, layers=1, kv_heads=2, q_heads=4)
    ok = K.LowramKvqCacheC()
    pos = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(1, 2, 3, 2, 128, dtype=torch.bfloat16)
    for k in (x, x.float(), x[..., :64], x[:, :1], x[0]):
        with pytest.raises(ValueError):
            K.lowram_kvq_write(cfg, ok, 0, k, k, pos)
        with pytest.raises(ValueError):
            K.lowram_kvq_read(cfg, ok, 0, k, k, pos)
    q = torch.zeros(1, 2, 1, 4, 128, dtype=torch.bfloat16)
    for t in (q, q[0], q[:, :, :, :3], q.float()):
        with pytest.raises(ValueError):
            K.lowram_kvq_decode_attn(cfg, ok, 0, t, pos, torch.empty_like(t), x)
        with pytest.raises(ValueError):
            K.lowram_kvq_sparse_attn(cfg, ok, 0, 4, t, pos, torch.empty_like(t))
    arrays = {n: torch.zeros(s, dtype=t) for n, (s, t) in K._kvq_layouts(K.kvq_config_struct(cfg)).items()}
    with pytest.raises(ValueError):      # not on a GPU
        K.LowramKvq(cfg, arrays)
    with pytest.raises(ValueError):
        K.LowramKvq(cfg, {"k_code": None})
    with pytest.raises(K.LowramError):
        K.LowramKvq(config(page=20), arrays)
    with pytest.raises(K.LowramError):
        K.LowramKvq(cfg, arrays, max_q=17)
