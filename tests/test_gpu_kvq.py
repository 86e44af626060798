"""The quantised KV cache on the GPU against the fp64 oracle: writing, reading, attention over
whole sequences and over selected pages, and a run of them together.  The bounds of the attention
outputs are derived in kvq_utils."""

import numpy as np
import pytest
import torch

import kv_cache_compression_lowram_b200 as K
from kvq_utils import DT, U32, UBF, check_attention, config, fill, queries, spoil_behind, to_device
from oracle import kvq as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------ write and read

def written(cfg, arrays, k, v, pos, count, layer0=0):
    """The oracle's pool after a write (k, v float64 numpy [NL][B][n][H][d])."""
    a = {x: arrays[x].copy() for x in arrays}
    page = cfg["page"]
    for b in range(cfg["batch"]):
        for x, t in (("k", k), ("v", v)):
            for i in range(count[b]):
                p, s = arrays["table"][b, (pos[b] + i) // page], (pos[b] + i) % page
                n, sc = O.quantise(t[:, b, i], cfg["bits"])
                sl = slice(layer0, layer0 + t.shape[0])
                a[x + "_code"][sl, p, :, s], a[x + "_scale"][sl, p, :, s] = O.pack(n, cfg["bits"]), sc
        for c in range(pos[b] // page, (pos[b] + count[b]) // page):
            p, sl = arrays["table"][b, c], slice(layer0, layer0 + k.shape[0])
            a["k_mean"][sl, p] = O.rows(a["k_code"][sl, p], a["k_scale"][sl, p], cfg["bits"]).mean(2)
    return a


def check_pool(cfg, dev, want, exact_means=False):
    for n in ("k_code", "v_code"):
        assert np.array_equal(dev[n].cpu().numpy(), want[n]), n
    for n in ("k_scale", "v_scale"):
        assert np.array_equal(dev[n].cpu().numpy().view(np.uint16), want[n].view(np.uint16)), n
    got = dev["k_mean"].double().cpu().numpy()
    big = np.abs(O.dequantise(np.full(want["k_code"].shape[:-1] + (cfg["head_dim"],), (1 << cfg["bits"]) - 1), want["k_scale"])).max()
    assert (np.abs(got - want["k_mean"]) <= UBF * np.abs(want["k_mean"]) + cfg["page"] * U32 * big).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,n,pos,count", [
    (64, 16, 1, [0, 15, 16, 200], None),
    (128, 32, 1, [31, 0, 64, 255], [1, 1, 0, 1]),
    (128, 64, 150, [0, 63, 64, 10], [150, 129, 0, 1]),
    (256, 16, 37, [5, 0, 16, 91], None),
    (256, 256, 300, [200, 0, 255, 512], [300, 256, 2, 256]),
])
def test_write_and_read(bits, dtype, d, page, n, pos, count):
    cfg = config(batch=4, layers=3, kv_heads=3, q_heads=3, head_dim=d, page=page, max_pages=-(-(max(pos) + n) // page), bits=bits, dtype=dtype)
    arrays = fill(cfg, 3)
    dev = to_device(arrays)
    cache = K.LowramKvq(cfg, dev)
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn(2, 4, n, 3, d, generator=g).to(DT[dtype]) for _ in range(2))
    cnt = count or [n] * 4
    cache.write(k.to(DEV), v.to(DEV), i32(pos), None if count is None else i32(count), layer0=1)
    want = written(cfg, arrays, k.double().numpy(), v.double().numpy(), pos, cnt, 1)
    check_pool(cfg, dev, want)
    assert cache.validate() == 0
    ko, vo = (torch.full((2, 4, n, 3, d), 7.0, dtype=DT[dtype], device=DEV) for _ in range(2))
    cache.read(i32(pos), None if count is None else i32(count), out=(ko, vo), layer0=1)
    for x, o in (("k", ko), ("v", vo)):
        for b in range(4):
            p, s = arrays["table"][b, (pos[b] + np.arange(cnt[b])) // page], (pos[b] + np.arange(cnt[b])) % page
            ref = O.rows(want[x + "_code"][1:, p, :, s], want[x + "_scale"][1:, p, :, s], bits)   # [rows][NL][H][d]
            ref = torch.tensor(np.moveaxis(ref, 0, 1)).float().to(DT[dtype])   # exact in 64 bits, to fp32, to dt
            assert torch.equal(o[:, b, :cnt[b]].cpu(), ref)
            assert (o[:, b, cnt[b]:] == 7.0).all()


def test_write_takes_slices_and_any_axis_order():
    cfg = config(batch=3, layers=2, kv_heads=2, page=16, max_pages=4)
    arrays = fill(cfg, 4)
    qkv = torch.randn(3, 20, 2, 12, 128, dtype=torch.bfloat16, device=DEV)      # [B][n][L][heads][d]
    k, v = qkv[..., 4:6, :].permute(2, 0, 1, 3, 4), qkv[:, :, :, 10:, :].permute(2, 0, 1, 3, 4)
    devs = [to_device(arrays) for _ in range(2)]
    for dev, (x, y) in zip(devs, ((k, v), (k.contiguous(), v.contiguous()))):
        K.LowramKvq(cfg, dev).write(x, y, i32([0, 7, 40]))
    for n in devs[0]:
        assert torch.equal(devs[0][n].view(torch.uint8), devs[1][n].view(torch.uint8)), n
    cache = K.LowramKvq(cfg, devs[0])
    wide = torch.zeros(3, 20, 2, 12, 128, dtype=torch.bfloat16, device=DEV)
    out = wide[..., 4:6, :].permute(2, 0, 1, 3, 4), wide[:, :, :, 10:, :].permute(2, 0, 1, 3, 4)
    cache.read(i32([0, 7, 40]), out=out)
    ref = cache.read(i32([0, 7, 40]), n=20)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    assert (wide[..., :4, :] == 0).all() and (wide[..., 6:10, :] == 0).all()
    # one token for all: a broadcast source
    one = torch.randn(1, 1, 1, 1, 128, dtype=torch.bfloat16, device=DEV).expand(2, 3, 20, 2, 128)
    cache.write(one, one, i32([0, 0, 0]))
    ref = cache.read(i32([0, 0, 0]), n=20)[0]
    assert torch.equal(ref, ref[:1, :1, :1, :1].expand_as(ref).contiguous())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_how_tokens_arrive_does_not_matter(dtype):
    """All at once, in pieces and one by one, after a rollback too: the same pool, bit for bit."""
    cfg = config(batch=2, layers=2, kv_heads=1, head_dim=256, page=32, max_pages=4, dtype=dtype)
    arrays = fill(cfg, 5)
    k, v = (torch.randn(2, 2, 100, 1, 256, device=DEV).to(DT[dtype]) for _ in range(2))
    devs = []
    for cuts in ([100], [1] * 100, [31, 2, 30, 1, 36], [40, -20, 80]):
        dev = to_device(arrays)
        cache, at = K.LowramKvq(cfg, dev), 0
        for c in cuts:
            if c < 0:      # tokens dropped from the end, other ones written over them first
                cache.write(v[:, :, at:at + 20], k[:, :, at:at + 20], i32([at, at]))
                at += c
                continue
            cache.write(k[:, :, at:at + c], v[:, :, at:at + c], i32([at, at]))
            at += c
        devs.append(dev)
    for dev in devs[1:]:
        used = dev["table"][:, :3].long().flatten()
        for n in ("k_code", "v_code", "k_scale", "v_scale", "k_mean"):
            assert torch.equal(dev[n][:, used].view(torch.uint8), devs[0][n][:, used].view(torch.uint8)), n


@pytest.mark.parametrize("bits", [4, 8])
def test_write_odd_values(bits):
    """Constant groups, ranges that are small beside the values, tiny and large values, exact half
    steps; a group with NaN or infinity reads back non-finite and disturbs no other."""
    d, n = 128, 64
    cfg = config(batch=1, kv_heads=1, q_heads=1, head_dim=d, page=64, max_pages=1, bits=bits, dtype="f32")
    x = torch.randn(n, d, generator=torch.Generator().manual_seed(1)).double()
    q = (1 << bits) - 1
    x[0] = 0
    x[1] = 1.2345678
    x[2] = 1000 + 0.01 * x[2]
    x[3] = -1000 + 1e-3 * x[3]
    x[4] *= 1e-7
    x[5] *= 1e-5
    x[6] *= 1e4
    x[7] = torch.arange(d) % (q + 1) * 0.5          # codes exactly
    x[8] = (torch.arange(d) % q + 0.5) * 0.25       # half steps ...
    x[8, ::64] = 0.0                                # ... between 0
    x[8, 1::64] = q * 0.25                          # and q steps of 0.25
    x[9] = x[9].abs() * 1e-41
    x[10] = -6e4
    x[10, 5::64] = 6e4
    x = x.float()
    v = x.clone()
    v[20, 3], v[21, 70], v[22, 9], v[23, 65] = float("nan"), float("inf"), -float("inf"), 3e38
    dev = to_device(fill(cfg, 1))
    cache = K.LowramKvq(cfg, dev)
    cache.write(x.view(1, 1, n, 1, d).to(DEV), v.view(1, 1, n, 1, d).to(DEV), i32([0]))
    codes, scale = O.quantise(x.numpy(), bits)
    p = int(dev["table"][0, 0])
    assert np.array_equal(dev["k_scale"][0, p, 0].cpu().numpy().view(np.uint16), scale.view(np.uint16))
    assert np.array_equal(O.unpack(dev["k_code"][0, p, 0].cpu().numpy(), bits), codes)
    got = cache.read(i32([0]), n=n)[1][0, 0, :, 0].cpu()
    clean = torch.ones(n, d, dtype=torch.bool)
    for r, c in ((20, 0), (21, 64), (22, 0), (23, 64)):
        clean[r, c:c + 64] = False
        assert not torch.isfinite(got[r, c:c + 64]).all()
    assert torch.equal(got[clean], torch.tensor(O.dequantise(codes, scale)).float()[clean])


def test_long_pool_offsets_pass_32_bits():
    """Rows behind 4 GB of codes: write, read and both attentions at the end of a large pool."""
    cfg = config(batch=1, layers=2, kv_heads=8, q_heads=8, head_dim=256, page=256, max_pages=3, bits=8, n_pages=4600)
    shapes = dict(k_code=(2, 4600, 8, 256, 256), v_code=(2, 4600, 8, 256, 256))
    dev = {n: torch.empty(s, dtype=torch.uint8, device=DEV) for n, s in shapes.items()}
    for n in ("k_scale", "v_scale"):
        dev[n] = torch.empty(2, 4600, 8, 256, 4, 2, dtype=torch.float16, device=DEV)
    dev["k_mean"] = torch.empty(2, 4600, 8, 256, dtype=torch.bfloat16, device=DEV)
    dev["table"] = i32([[4599, 4597, 4598]])
    cache = K.LowramKvq(cfg, dev)
    k, v = (torch.randn(1, 1, 700, 8, 256, device=DEV).bfloat16() for _ in range(2))
    cache.write(k, v, i32([0]), layer0=1)
    small = {n: (dev[n][1:, 4597:].double() if n == "k_mean" else dev[n][1:, 4597:]).cpu().numpy() for n in dev if n != "table"}
    small["table"] = np.array([[2, 0, 1]], np.int32)
    q = queries(cfg, layers=1)
    out = cache.decode(q.to(DEV), i32([700]), layer0=1)
    check_attention(cfg, small, q, [700], out)
    out, sel = cache.decode_sparse(q.to(DEV), i32([700]), 2, sel=True, layer0=1)
    check_attention(cfg, small, q, [700], out, top_k=2, sel=sel)
    ko, vo = cache.read(i32([0]), n=700, layer0=1)
    for x, o in (("k", ko), ("v", vo)):
        ref = O.rows(small[x + "_code"][0, [2, 0, 1]], small[x + "_scale"][0, [2, 0, 1]], 8)
        ref = np.moveaxis(ref, 1, 2).reshape(-1, 8, 256)[:700]
        assert torch.equal(o[0, 0].cpu(), torch.tensor(ref).float().bfloat16())


# ------------------------------------------------------------------------ attention

CASES = [  # d, kv_heads, group, page, n, lens
    (64, 1, 1, 16, 1, [1]),
    (128, 2, 4, 64, 1, [1, 16, 17, 300]),
    (128, 1, 8, 16, 1, [0, 31, 32, 33, 511]),
    (128, 2, 3, 32, 2, [1, 2, 0, 95]),
    (128, 1, 16, 128, 1, [640, 5]),
    (64, 3, 7, 32, 3, [100, 2, 257]),
    (64, 2, 2, 256, 16, [700, 16, 3]),
    (256, 1, 4, 16, 1, [77, 0, 160]),
    (256, 2, 12, 64, 5, [200, 64]),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads,group,page,n,lens", CASES)
def test_decode(bits, dtype, d, heads, group, page, n, lens):
    cfg = config(batch=len(lens), layers=2, kv_heads=heads, q_heads=heads * group, head_dim=d, page=page,
                 max_pages=-(-max(lens) // page) + 1, bits=bits, dtype=dtype)
    arrays = fill(cfg, 11)
    spoil_behind(cfg, arrays, lens)
    cache = K.LowramKvq(cfg, to_device(arrays), max_q=n)
    q = queries(cfg, n, 1)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV)
    cache.decode(q.to(DEV), i32(lens), out=out, layer0=1)
    check_attention(cfg, arrays, q, lens, out, 1)
    again = cache.decode(q.to(DEV), i32(lens), layer0=1)
    assert torch.equal(out, again) and cache.validate() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,layers,heads,ctx,page", [(1, 1, 1, 20000, 64), (2, 1, 2, 9001, 16), (40, 2, 2, 130, 16), (150, 1, 1, 700, 128)])
def test_decode_split_and_batched(dtype, batch, layers, heads, ctx, page):
    """Long sequences that many CTAs share, and many sequences of every length."""
    r = np.random.default_rng(2)
    lens = [ctx] + [int(x) for x in r.integers(0, ctx + 1, batch - 1)]
    cfg = config(batch=batch, layers=layers, kv_heads=heads, q_heads=4 * heads, page=page, max_pages=-(-ctx // page), dtype=dtype,
                 n_pages=-(-ctx // page) + 7)
    arrays = fill(cfg, 12) if batch == 1 else None
    if arrays is None:      # sequences share pages: a small pool, tables drawn from it
        arrays = fill(dict(cfg, batch=1), 12)
        arrays["table"] = r.integers(0, cfg["n_pages"], (batch, cfg["max_pages"])).astype(np.int32)
    cache = K.LowramKvq(cfg, to_device(arrays))
    q = queries(cfg)
    check_attention(cfg, arrays, q, lens, cache.decode(q.to(DEV), i32(lens)))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["small_v", "large_v", "zero_q", "large_q", "peak_last", "peak_first", "offset_v", "rising_v"])
def test_decode_ranges(bits, dtype, what):
    """Values far from one, one token far above the rest, value scales that grow along the sequence."""
    cfg = config(batch=2, kv_heads=1, q_heads=4, page=16, max_pages=40, bits=bits, dtype=dtype)
    arrays = fill(cfg, 13, v_std={"small_v": 1e-4, "large_v": 3e3}.get(what, 1.0), v_bias=30.0 if what == "offset_v" else 0.0)
    lens = [600, 333]
    q = queries(cfg, std={"zero_q": 0.0, "large_q": 12.0}.get(what, 1.0))
    if what.startswith("peak"):
        for b in range(2):
            t = 0 if what == "peak_first" else lens[b] - 1
            n, s = O.quantise(3.0 * q[0, b, 0, :1].double().numpy(), bits)
            p = arrays["table"][b, t // 16]
            arrays["k_code"][0, p, 0, t % 16], arrays["k_scale"][0, p, 0, t % 16] = O.pack(n, bits)[0], s[0]
    if what == "rising_v":
        for b in range(2):
            for i in range(40):
                arrays["v_scale"][:, arrays["table"][b, i]] *= np.float16(2.0 ** (i // 3 - 8))
    cache = K.LowramKvq(cfg, to_device(arrays))
    check_attention(cfg, arrays, q, lens, cache.decode(q.to(DEV), i32(lens)))
    out = cache.decode_sparse(q.to(DEV), i32(lens), 5)
    check_attention(cfg, arrays, q, lens, out, top_k=5)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top_k", [1, 2, 5, 64])
@pytest.mark.parametrize("d,heads,group,page,n,lens", CASES)
def test_sparse(bits, dtype, top_k, d, heads, group, page, n, lens):
    cfg = config(batch=len(lens), layers=2, kv_heads=heads, q_heads=heads * group, head_dim=d, page=page,
                 max_pages=-(-max(lens) // page) + 1, bits=bits, dtype=dtype)
    arrays = fill(cfg, 14)
    spoil_behind(cfg, arrays, lens)
    cache = K.LowramKvq(cfg, to_device(arrays), max_q=n)
    q = queries(cfg, n, 1, seed=3)
    out, sel = cache.decode_sparse(q.to(DEV), i32(lens), top_k, sel=True, layer0=1)
    check_attention(cfg, arrays, q, lens, out, 1, top_k, sel)
    assert torch.equal(out, cache.decode_sparse(q.to(DEV), i32(lens), top_k, layer0=1)) and cache.validate() == 0


@pytest.mark.parametrize("batch,heads,ctx,page,top_k", [(1, 1, 16384 * 16, 16, 32), (1, 2, 50000, 16, 512), (3, 2, 30000, 32, 17), (64, 2, 900, 16, 9)])
def test_sparse_many_pages(batch, heads, ctx, page, top_k):
    r = np.random.default_rng(3)
    lens = [ctx] + [int(x) for x in r.integers(0, ctx + 1, batch - 1)]
    n_pages = 500
    cfg = config(batch=batch, kv_heads=heads, q_heads=4 * heads, head_dim=64, page=page, max_pages=-(-ctx // page), n_pages=n_pages)
    arrays = fill(dict(cfg, batch=1, max_pages=1), 15)
    arrays["table"] = r.integers(0, n_pages, (batch, cfg["max_pages"])).astype(np.int32)   # equal pages: ties everywhere
    cache = K.LowramKvq(cfg, to_device(arrays))
    q = queries(cfg, seed=4)
    out, sel = cache.decode_sparse(q.to(DEV), i32(lens), top_k, sel=True)
    check_attention(cfg, arrays, q, lens, out, top_k=top_k, sel=sel)


def test_decode_many_short_and_one_long():
    """More sequences than a warp has lanes, nearly all empty or of a few tokens."""
    lens = [0, 1, 2, 5, 33] * 8 + [700] + [3] * 30
    cfg = config(batch=len(lens), kv_heads=1, q_heads=4, page=16, max_pages=44, n_pages=50)
    arrays = fill(dict(cfg, batch=1, max_pages=1), 20)
    arrays["table"] = np.random.default_rng(6).integers(0, 50, (len(lens), 44)).astype(np.int32)
    cache = K.LowramKvq(cfg, to_device(arrays))
    q = queries(cfg)
    check_attention(cfg, arrays, q, lens, cache.decode(q.to(DEV), i32(lens)))
    out, sel = cache.decode_sparse(q.to(DEV), i32(lens), 6, sel=True)
    check_attention(cfg, arrays, q, lens, out, top_k=6, sel=sel)


def test_calls_of_several_kinds_share_a_workspace():
    """Layers, query tokens and lengths change from call to call; the counters end at zero each time."""
    cfg = config(batch=3, layers=3, kv_heads=2, q_heads=6, page=32, max_pages=200, n_pages=210)
    arrays = fill(dict(cfg, batch=1, max_pages=1), 21)
    arrays["table"] = np.random.default_rng(8).integers(0, 210, (3, 200)).astype(np.int32)
    cache = K.LowramKvq(cfg, to_device(arrays), max_q=5)
    for n, layers, lens in ((5, 3, [6400, 3000, 17]), (1, 1, [6400, 1, 0]), (2, 2, [600, 5000, 6000]), (5, 1, [6400, 6400, 6400]), (1, 3, [90, 80, 70])):
        q = queries(cfg, n, layers, seed=n + layers)
        check_attention(cfg, arrays, q, lens, cache.decode(q.to(DEV), i32(lens)))
    assert not cache._workspace[-4 * 3 * 3 * 2 * 2:].any()


@pytest.mark.parametrize("bits", [4, 8])
def test_nan_in_a_token_that_an_earlier_query_does_not_see(bits):
    cfg = config(batch=1, kv_heads=1, q_heads=4, page=16, max_pages=4, bits=bits)
    arrays = fill(cfg, 22)
    p = arrays["table"][0, 39 // 16]
    for x in "kv":
        arrays[x + "_scale"][0, p, 0, 39 % 16] = np.float16(np.nan)
    cache = K.LowramKvq(cfg, to_device(arrays), max_q=3)
    q = queries(cfg, 3)
    for out in (cache.decode(q.to(DEV), i32([40])), cache.decode_sparse(q.to(DEV), i32([40]), 4)):
        assert torch.isnan(out[0, 0, 2]).all()
        arrays["k_scale"][0, p, 0, 39 % 16] = arrays["v_scale"][0, p, 0, 39 % 16] = 0      # for the oracle: not seen
        check_attention(cfg, arrays, q[:, :, :2], [39], out[:, :, :2].contiguous())
        arrays["k_scale"][0, p, 0, 39 % 16] = arrays["v_scale"][0, p, 0, 39 % 16] = np.float16(np.nan)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_and_infinite_queries_spoil_their_own_rows(bits, dtype):
    """Also where every token's score is NaN, and in a sequence whose keys all are."""
    cfg = config(batch=2, kv_heads=2, q_heads=8, page=16, max_pages=40, bits=bits, dtype=dtype)
    arrays = fill(cfg, 26)
    cache = K.LowramKvq(cfg, to_device(arrays))
    q = queries(cfg)
    lens = [600, 35]
    q[0, 0, 0, 1, 5], q[0, 0, 0, 6, 7], q[0, 1, 0, 3, 0] = float("nan"), float("inf"), float("-inf")
    clean = torch.ones(2, 8, dtype=torch.bool)
    clean[0, 1] = clean[0, 6] = clean[1, 3] = False
    ref = q.clone()
    ref[0, :, 0][~clean] = 0
    got = cache.decode(q.to(DEV), i32(lens))
    assert torch.isnan(got[0, :, 0].cpu()[~clean]).all()
    got[0, :, 0][~clean.to(DEV)] = cache.decode(ref.to(DEV), i32(lens))[0, :, 0][~clean.to(DEV)]
    check_attention(cfg, arrays, ref, lens, got)
    out = cache.decode_sparse(q.to(DEV), i32(lens), 3)
    assert torch.isnan(out[0, :, 0].cpu()[~clean]).all() and torch.isfinite(out[0, :, 0].cpu()[clean]).all()
    arrays["k_scale"][:, arrays["table"][1]] = np.nan
    bad = K.LowramKvq(cfg, to_device(arrays))
    for out in (bad.decode(ref.to(DEV), i32(lens)), bad.decode_sparse(ref.to(DEV), i32(lens), 3)):
        assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[0, 0]).all()


def test_refusals_on_the_device():
    cfg = config(batch=2, kv_heads=2, q_heads=4)
    cache = K.LowramKvq(cfg, to_device(fill(cfg, 23)))
    q, lens = queries(cfg).to(DEV), i32([20, 30])
    odd = torch.empty(q.numel() + 1, dtype=q.dtype, device=DEV)[1:].view(q.shape)
    x = torch.zeros(1, 2, 3, 2, 128, dtype=torch.bfloat16, device=DEV)
    wide = torch.zeros(1, 2, 3, 2, 130, dtype=torch.bfloat16, device=DEV)[..., :128]
    for call in (lambda: cache.decode(odd, lens), lambda: cache.decode(q, lens, out=odd), lambda: cache.decode_sparse(odd, lens, 2),
                 lambda: cache.write(wide, x, lens), lambda: cache.decode(q, lens, layer0=1), lambda: cache.decode_sparse(q, lens, 0),
                 lambda: cache.read(lens, out=(x, x[:, :, :1].expand_as(x))),
                 lambda: cache.decode(torch.zeros(1, 2, 2, 4, 128, dtype=q.dtype, device=DEV), lens, out=None, layer0=-1)):
        with pytest.raises(K.LowramError) as ei:
            call()
        assert ei.value.status == 1
    for call in (lambda: cache.decode(q, lens.long()), lambda: cache.decode(q, lens[:1]), lambda: cache.decode(q.float(), lens),
                 lambda: cache.decode(q, lens.cpu()), lambda: cache.decode(q.transpose(2, 3), lens), lambda: cache.write(x, x, None and lens, lens.cpu()),
                 lambda: cache.read(lens, n=None), lambda: cache.read(lens, n=3, stream=torch.cuda.Stream())):
        with pytest.raises((ValueError, K.LowramError)):
            call()
    none = torch.zeros(1, 2, 0, 2, 128, dtype=torch.bfloat16, device=DEV)
    cache.write(none, none, lens)      # nothing to do is not an error
    few = K.LowramKvq(cfg, cache.arrays, max_q=1)
    assert few.validate() == 0


@pytest.mark.parametrize("kind", ["equal", "two_values", "last_bits", "tiny_means", "tiny_queries", "large_means"])
@pytest.mark.parametrize("heads", [1, 40])
def test_sparse_scores_too_near_for_fp32(kind, heads):
    """More pages near the border than are ranked by comparison: equal means, two values, and means whose
    scores differ in the last bits of 64 only."""
    pages = 700
    cfg = config(batch=1, kv_heads=heads, q_heads=heads, head_dim=64, page=16, max_pages=pages, n_pages=pages)
    arrays = fill(dict(cfg, n_pages=2, max_pages=1), 24)
    arrays = {n: (np.repeat(v[:, :1], pages, 1) if n != "table" else np.arange(pages, dtype=np.int32)[None]) for n, v in arrays.items()}
    r = np.random.default_rng(9)
    m = arrays["k_mean"]
    m[:] = 0
    m[..., 0] = 1.0
    if kind == "two_values":
        m[0, r.permutation(pages)[:300], :, 0] = 1.5
    if kind == "last_bits":      # a channel whose product is 2^-40 of the score
        m[..., 1] = r.integers(0, 200, (1, pages, 1))
    if kind in ("tiny_means", "tiny_queries", "large_means"):      # squares and products that leave fp32's range
        m[:] = torch.tensor(r.standard_normal(m.shape) * {"tiny_means": 1e-22, "tiny_queries": 1e-3, "large_means": 1e22}[kind]).bfloat16().double().numpy()
    q = torch.ones(1, 1, 1, heads, 64, dtype=torch.bfloat16) * (1e-37 if kind == "tiny_queries" else 1.0)
    if kind == "last_bits":
        q[..., 1] = 2.0 ** -40
    cache = K.LowramKvq(cfg, to_device(arrays))
    for k in (1, 2, 30, 299, 302, 500):
        out, sel = cache.decode_sparse(q.to(DEV), i32([pages * 16]), k, sel=True)
        check_attention(cfg, arrays, q, [pages * 16], out, top_k=k, sel=sel)


@pytest.mark.parametrize("dtype,bits,d,group,batch", [("bf16", 4, 64, 1, 450), ("f32", 8, 256, 8, 1), ("bf16", 8, 128, 16, 300)])
def test_sparse_with_the_longest_table(dtype, bits, d, group, batch):
    """16384 pages a sequence and top_k = 512: the most shared memory a call asks for."""
    r = np.random.default_rng(10)
    lens = [int(x) for x in r.integers(0, 200, batch)]
    lens[0] = 16384 * 16 if batch == 1 else 9000
    cfg = config(batch=batch, kv_heads=1, q_heads=group, head_dim=d, page=16, max_pages=16384, n_pages=40, bits=bits, dtype=dtype)
    arrays = fill(dict(cfg, batch=1, max_pages=1), 25)
    arrays["table"] = r.integers(0, 40, (batch, 16384)).astype(np.int32)
    cache = K.LowramKvq(cfg, to_device(arrays))
    q = queries(cfg)
    out, sel = cache.decode_sparse(q.to(DEV), i32(lens), 512, sel=True)
    check_attention(cfg, arrays, q, lens, out, top_k=512, sel=sel)


def test_sparse_ties_and_nan_means():
    cfg = config(batch=1, kv_heads=1, q_heads=2, head_dim=64, page=16, max_pages=40)
    arrays = fill(cfg, 16)
    q = queries(cfg)
    arrays["k_mean"][:] = 0.0                                   # all scores equal: the lowest pages
    for k in (1, 7, 39, 40):
        out, sel = K.LowramKvq(cfg, to_device(arrays)).decode_sparse(q.to(DEV), i32([640]), k, sel=True)
        assert sel.flatten().tolist() == list(range(k - 1)) + [39]
    arrays["k_mean"][0, arrays["table"][0, :3]] = np.nan          # NaN is behind every number ...
    arrays["k_mean"][0, arrays["table"][0, 5], 0, 0] = np.inf * np.sign(float(q[0, 0, 0, :, 0].double().sum()))
    out, sel = K.LowramKvq(cfg, to_device(arrays)).decode_sparse(q.to(DEV), i32([640]), 4, sel=True)
    assert sel.flatten().tolist() == [3, 4, 5, 39]
    out, sel = K.LowramKvq(cfg, to_device(arrays)).decode_sparse(q.to(DEV), i32([640]), 38, sel=True)   # ... but chosen when needed
    assert sel.flatten().tolist() == [0] + list(range(3, 40))


# ------------------------------------------------------------------------ tables, streams, graphs

def test_identity_table_and_shared_pages():
    cfg = config(batch=2, kv_heads=2, page=16, max_pages=5, n_pages=10)
    arrays = fill(cfg, 17)
    q = queries(cfg)
    lens = [80, 47]
    for tab in (None, np.array([[3, 3, 1, 0, 9], [3, 1, 1, 2, 4]], np.int32)):
        arrays["table"] = np.arange(10, dtype=np.int32).reshape(2, 5) if tab is None else tab
        dev = to_device(arrays)
        if tab is None:
            del dev["table"]
        cache = K.LowramKvq(cfg, dev)
        check_attention(cfg, arrays, q, lens, cache.decode(q.to(DEV), i32(lens)))
        out, sel = cache.decode_sparse(q.to(DEV), i32(lens), 3, sel=True)
        check_attention(cfg, arrays, q, lens, out, top_k=3, sel=sel)


def test_bad_tables_and_lengths_are_masked_and_reported():
    cfg = config(batch=3, kv_heads=2, page=16, max_pages=6)
    arrays = fill(cfg, 18)
    dev = to_device(arrays)
    cache = K.LowramKvq(cfg, dev)
    q = queries(cfg).to(DEV)
    before = {n: t.clone() for n, t in dev.items()}
    x = torch.randn(1, 3, 40, 2, 128, device=DEV).bfloat16()
    # lengths outside the table's room count as none and as all
    out = cache.decode(q, i32([-5, 1000, 96]))
    assert cache.validate() == 2
    assert torch.equal(out, cache.decode(q, i32([0, 96, 96]))) and cache.validate() == 0
    out = cache.decode_sparse(q, i32([-5, 1000, 96]), 3)
    assert cache.validate() == 2
    assert torch.equal(out, cache.decode_sparse(q, i32([0, 96, 96]), 3)) and cache.validate() == 0
    # tokens in front of and behind the room are dropped; the others are written
    cache.write(x, x, i32([-30, 80, 2**31 - 10]), i32([30, 40, 40]))
    assert cache.validate() == 2
    p = arrays["table"][1, 5]
    for n in ("k_code", "v_code", "k_scale", "v_scale", "k_mean"):
        same = (dev[n] == before[n]).flatten(2).all(-1)[0]
        assert not same[p] and same.sum() == cfg["n_pages"] - 1, n
    ko, vo = cache.read(i32([-30, 80, 2**31 - 10]), n=40)
    assert cache.validate() == 2
    assert (ko[:, 0, :30] == 0).all() and (ko[:, 1, 16:] == 0).all() and (ko[:, 2] == 0).all()
    ref, _ = cache.read(i32([0, 80, 0]), i32([10, 16, 0]), n=40)
    assert torch.equal(ko[:, 0, 30:], ref[:, 0, :10]) and torch.equal(ko[:, 1, :16], ref[:, 1, :16])
    cache.write(x, x, i32([0, 0, 0]), i32([-1, 0, 0]))
    assert cache.validate() == 2
    # pages outside the pool
    for n, t in before.items():
        dev[n].copy_(t)
    bad = arrays["table"].copy()
    bad[0, 1], bad[1, 0], bad[2, 5] = -7, cfg["n_pages"], 2**31 - 1
    dev["table"].copy_(torch.from_numpy(bad))
    out, sel = cache.decode_sparse(q, i32([96, 60, 96]), 6, sel=True)
    assert cache.validate() == 1
    dense = cache.decode(q, i32([96, 60, 96]))
    assert cache.validate() == 1 and torch.isfinite(dense).all()
    # all pages of sequence 0 fit top_k: both attend what is left of it
    d = dict(cfg, batch=1)
    left = dict(arrays, table=np.delete(arrays["table"][:1], 1, 1))
    check_attention(d, left, q[:, :1].cpu(), [80], dense[:, :1])
    check_attention(d, left, q[:, :1].cpu(), [80], out[:, :1])
    ko, _ = cache.read(i32([0, 0, 80]), i32([40, 40, 16]), n=40)   # 80 + 16 is all a table row holds
    assert cache.validate() == 1 and (ko[:, 0, 16:32] == 0).all() and (ko[:, 1, :16] == 0).all() and (ko[:, 2] == 0).all()
    cache.write(x, x, i32([16, 0, 80]), i32([16, 16, 16]))
    assert cache.validate() == 1
    for n in ("k_code", "v_code", "k_scale", "v_scale", "k_mean"):
        assert torch.equal(dev[n].view(torch.uint8), before[n].view(torch.uint8))


def test_streams_and_graphs():
    """A whole step on another stream, captured twice into graphs that share the cache's workspace,
    and replayed in turn on new data."""
    cfg = config(batch=3, layers=2, kv_heads=2, q_heads=8, page=16, max_pages=64)
    cache = K.LowramKvq(cfg)
    eager = K.LowramKvq(cfg)
    g = torch.Generator(device=DEV).manual_seed(3)
    pos, lens = i32([500, 16, 0]), i32([501, 17, 1])
    k, v = (torch.randn(2, 3, 1, 2, 128, device=DEV, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(2, 3, 1, 8, 128, device=DEV, generator=g).bfloat16()
    hist = [torch.randn(2, 3, 500, 2, 128, device=DEV, generator=g).bfloat16() for _ in range(2)]
    for c in (cache, eager):
        c.write(*hist, i32([0, 0, 0]))

    def step(c):
        c.write(k, v, pos)
        return c.decode(q, lens), c.decode_sparse(q, lens, 4)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step(cache)
    torch.cuda.current_stream().wait_stream(side)
    want = step(eager)
    assert all(torch.equal(a, b) for a, b in zip(first, want))
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(cache))
        graphs.append(graph)
    for r in range(4):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, device=DEV, generator=g))
        lens.copy_(pos + 1)
        graphs[r % 2].replay()
        want = step(eager)
        assert all(torch.equal(a, b) for a, b in zip(outs[r % 2], want)), r
        pos += 1
    assert cache.validate() == 0


def test_two_streams_at_once():
    """Two caches over the same arrays, each with its workspace, attend and read at the same time on the
    streams that their calls are given."""
    cfg = config(batch=4, layers=2, kv_heads=4, q_heads=16, page=32, max_pages=130)
    arrays = fill(dict(cfg, n_pages=200, batch=1, max_pages=1), 27)
    cfg["n_pages"] = 200
    arrays["table"] = np.random.default_rng(12).integers(0, 200, (4, 130)).astype(np.int32)
    dev = to_device(arrays)
    lens = i32([4100, 77, 3000, 1])
    q = queries(cfg, 2).to(DEV)
    one = K.LowramKvq(cfg, dev, max_q=2)
    want = one.decode(q, lens), one.decode_sparse(q, lens, 9), one.read(i32([0, 7, 64, 0]), n=64)[0]
    caches, streams = [one, K.LowramKvq(cfg, dev, max_q=2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    rounds = 8
    outs = [[(torch.empty_like(q), torch.empty_like(q), torch.empty_like(want[2]), torch.empty_like(want[2])) for _ in range(rounds)] for _ in caches]
    pos = i32([0, 7, 64, 0])
    torch.cuda.synchronize()
    for r in range(rounds):
        for c, s, o in zip(caches, streams, outs):
            c.decode(q, lens, out=o[r][0], stream=s)
            c.decode_sparse(q, lens, 9, out=o[r][1], stream=s)
            c.read(pos, out=o[r][2:], stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for r in o:
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1]) and torch.equal(r[2], want[2])


def test_first_calls_may_be_captured():
    """A process whose first calls of the quantised cache are captured, and replayed on new data."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, kv_cache_compression_lowram_b200 as K
c = K.LowramKvq(dict(batch=2, n_layers=1, n_kv_heads=2, n_q_heads=8, head_dim=128, page=16, n_pages=16, max_pages=8, bits=4, dtype="bf16"))
x = torch.randn(1, 2, 100, 2, 128, device="cuda").bfloat16()
q = torch.randn(1, 2, 1, 8, 128, device="cuda").bfloat16()
pos, lens = (torch.full((2,), n, dtype=torch.int32, device="cuda") for n in (0, 100))
out = [torch.zeros_like(x), torch.zeros_like(x)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c.write(x, x, pos)
    c.read(pos, out=out)
    a, b = c.decode(q, lens), c.decode_sparse(q, lens, 7)
x.normal_()
g.replay()
torch.cuda.synchronize()
assert torch.equal(a, c.decode(q, lens)) and torch.equal(b, c.decode_sparse(q, lens, 7)) and c.validate() == 0
assert (out[0] - x).abs().max() < 0.5 and torch.equal(*out) and a.abs().max() > 0 and (a - b).abs().max() < 0.02
print("captured")
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-2000:]


@pytest.mark.parametrize("bits", [4, 8])
def test_a_run_together(bits):
    """Prompts written, then tokens appended and attended step by step, as a decode loop does; the
    cache is then moved to another one through a read and a write."""
    cfg = config(batch=2, layers=2, kv_heads=2, q_heads=8, page=16, max_pages=8, bits=bits)
    cache = K.LowramKvq(cfg, table=i32(np.random.default_rng(1).permutation(18)[:16].reshape(2, 8)))
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(2, 2, 100, 2, 128, generator=g).bfloat16() for _ in range(2))
    lens = [70, 41]
    cache.write(k[:, :, :70].to(DEV), v[:, :, :70].to(DEV), i32([0, 0]), i32(lens))
    for step in range(20):
        new = [torch.stack([x[:, b, lens[b]:lens[b] + 1] for b in range(2)], 1).to(DEV) for x in (k, v)]
        cache.write(*new, i32(lens))
        lens = [n + 1 for n in lens]
        if step % 6 and step != 19:
            continue
        q = queries(cfg, seed=step)
        arrays = {n: (t.double() if n == "k_mean" else t).cpu().numpy() for n, t in cache.arrays.items() if n != "err"}
        check_attention(cfg, arrays, q, lens, cache.decode(q.to(DEV), i32(lens)))
        out, sel = cache.decode_sparse(q.to(DEV), i32(lens), 3, sel=True)
        check_attention(cfg, arrays, q, lens, out, top_k=3, sel=sel)
        for b in range(2):      # the pool holds what the oracle quantises
            ref = O.dequantise(*O.quantise(k[:, b, :lens[b]].double().numpy(), bits))
            got = O.rows(arrays["k_code"][:, arrays["table"][b]], arrays["k_scale"][:, arrays["table"][b]], bits)
            got = np.moveaxis(got, 2, 3).reshape(2, -1, 2, 128)[:, :lens[b]]
            assert np.array_equal(got, ref)
    assert cache.validate() == 0
    ko, vo = cache.read(i32([0, 0]), i32(lens), n=96)
    assert torch.equal(ko[:, 0, :lens[0]].cpu(), torch.tensor(O.dequantise(*O.quantise(k[:, 0, :lens[0]].double().numpy(), bits))).float().bfloat16())
    other = K.LowramKvq(cfg)
    other.write(ko, vo, i32([0, 0]), i32(lens))
    assert other.validate() == 0
