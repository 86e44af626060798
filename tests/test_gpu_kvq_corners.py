"""Corners of the quantised KV cache's value ranges on the GPU, against the fp64 oracle."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import kv_cache_compression_lowram_b200 as K
from kvq_utils import DT, U16, UBF, check_attention, config, fill, queries, to_device
from oracle import kvq as O

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


def check_one_token(bits, dtype, d, group, q_log2, k_log2):
    """Scores so far apart that the softmax is one token's value: |o - v| is at most the rounding of the
    weight (fp16 in BF16 calls) and of the output."""
    lens = [700, 90]
    cfg = config(batch=2, kv_heads=1, q_heads=group, head_dim=d, page=16, max_pages=44, bits=bits, dtype=dtype)
    arrays = fill(cfg, 31, k_std=2.0 ** k_log2)
    q = queries(cfg, std=2.0 ** q_log2)
    assert torch.isfinite(q).all()
    cache = K.LowramKvq(cfg, to_device(arrays))
    outs = [cache.decode(q.to(DEV), i32(lens))] + [cache.decode_sparse(q.to(DEV), i32(lens), 44)]
    checked = 0
    for b in range(2):
        k, v = (O.rows(arrays[x + "_code"][0, arrays["table"][b], 0], arrays[x + "_scale"][0, arrays["table"][b], 0], bits).reshape(-1, d)[:lens[b]]
                for x in "kv")
        x = q[0, b, 0].double().numpy() @ k.T / d ** 0.5
        for j in range(group):
            best, second = np.sort(x[j])[[-1, -2]]
            # scores are sums in fp32 (d + 12 roundings): the best is the best, and the rest is nothing
            if best - second < 80 + 4 * (d + 12) * 2.0 ** -24 * np.abs(q[0, b, 0, j].double().numpy()) @ np.abs(k).max(0) / d ** 0.5:
                continue
            checked += 1
            ref, M = v[x[j].argmax()], np.abs(v[x[j].argmax()]).max() + 16
            for out in outs:
                got = out[0, b, 0, j].double().cpu().numpy()
                tol = 2.0 ** -20 * M + (U16 * M + UBF * np.abs(ref) if dtype == "bf16" else 0.0)
                assert (np.abs(got - ref) <= tol).all(), (b, j, got[:4], ref[:4])
    assert checked >= group


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group", [(64, 2), (128, 4), (128, 16), (256, 8)])
@pytest.mark.parametrize("q_log2,k_log2", [(12, 10), (15, 10), (17, 11), (20, 12), (30, 12), (100, 0), (112, -4)])
def test_large_scores_choose_one_token(bits, dtype, d, group, q_log2, k_log2):
    check_one_token(bits, dtype, d, group, q_log2, k_log2)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group", [(64, 2), (128, 4), (128, 16), (256, 8)])
@pytest.mark.parametrize("q_log2,k_log2", [(118, -10), (122, -12), (126, -14)])
def test_queries_near_the_largest_number(bits, dtype, d, group, q_log2, k_log2):
    check_one_token(bits, dtype, d, group, q_log2, k_log2)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group", [(64, 2), (128, 4), (128, 16), (256, 8)])
def test_nan_spoils_its_row_however_large_the_other_scores(bits, dtype, d, group):
    """A token of NaN among scores that lie thousands apart: the part of the sequence that holds it has no
    weight against the others, and the row (for a key) or the group (for a value) is NaN all the same."""
    lens = [700, 300]
    cfg = config(batch=2, kv_heads=1, q_heads=group, head_dim=d, page=16, max_pages=44, bits=bits, dtype=dtype)
    arrays = fill(cfg, 34)
    q = queries(cfg, std=2.0 ** 12)
    k = O.rows(arrays["k_code"][0, arrays["table"][0], 0], arrays["k_scale"][0, arrays["table"][0], 0], bits).reshape(-1, d)[:700]
    low = int((q[0, 0, 0].double().numpy() @ k.T).max(0).argmin())
    for x, spoilt in (("k", d), ("v", 64)):
        bad = dict(arrays, **{x + "_scale": arrays[x + "_scale"].copy()})
        bad[x + "_scale"][0, arrays["table"][0, low // 16], 0, low % 16, 0, 1] = np.nan
        cache = K.LowramKvq(cfg, to_device(bad))
        for out in (cache.decode(q.to(DEV), i32(lens)), cache.decode_sparse(q.to(DEV), i32(lens), 44)):
            assert torch.isnan(out[0, 0, ..., :spoilt]).all() and torch.isfinite(out[0, 0, ..., spoilt:]).all()
            assert torch.isfinite(out[0, 1]).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group", [(128, 3), (128, 8), (128, 16), (256, 4), (256, 8)])
@pytest.mark.parametrize("small_first", [False, True])
def test_groups_of_unlike_scale(bits, dtype, d, group, small_first):
    """Value groups 2^28 apart: every channel is as near to its own group's values as if it were alone."""
    lens = [300, 41]
    cfg = config(batch=2, kv_heads=1, q_heads=group, head_dim=d, page=16, max_pages=20, bits=bits, dtype=dtype)
    arrays = fill(cfg, 32)
    G = d // 64
    std = np.array([2.0 ** (13 if (g % 2 == 0) != small_first else -15) for g in range(G)])
    v = np.random.default_rng(33).standard_normal((1, cfg["n_pages"], 1, 16, d)) * np.repeat(std, 64)
    n, s = O.quantise(v, bits)
    arrays["v_code"], arrays["v_scale"] = O.pack(n, bits), s
    q = queries(cfg)
    cache = K.LowramKvq(cfg, to_device(arrays))
    for out in (cache.decode(q.to(DEV), i32(lens)), cache.decode_sparse(q.to(DEV), i32(lens), 20)):
        for g in range(G):      # one group at a time, the others' values taken out of the bound
            one = dict(arrays, v_scale=arrays["v_scale"].copy())
            one["v_scale"][..., [x for x in range(G) if x != g], :] = 0
            got = out.clone()
            got.view(*got.shape[:-1], G, 64)[..., [x for x in range(G) if x != g], :] = 0
            check_attention(cfg, one, q, lens, got)


# ------------------------------------------------------------------------ writing

def written_rows(x, bits, d, dtype):
    """(codes, scales, read back) of rows x [n][d] after a write as keys and values."""
    n = x.shape[0]
    page = 256
    cfg = config(batch=1, kv_heads=1, q_heads=1, head_dim=d, page=page, max_pages=-(-n // page), bits=bits, dtype=dtype)
    cache = K.LowramKvq(cfg)
    t = x.to(DT[dtype]).view(1, 1, n, 1, d).to(DEV)
    cache.write(t, t, i32([0]))
    back = cache.read(i32([0]), n=n)
    assert torch.equal(cache.arrays["k_code"], cache.arrays["v_code"]) and torch.equal(back[0].view(torch.uint8), back[1].view(torch.uint8))
    code, scale = (cache.arrays[k].cpu().numpy()[0, :-(-n // page), 0] for k in ("k_code", "k_scale"))
    return code.reshape(-1, code.shape[-1])[:n], scale.reshape(-1, d // 64, 2)[:n], back[0][0, 0, :, 0].cpu()


def check_rows(x, bits, d, dtype):
    x = x.to(DT[dtype])
    code, scale, back = written_rows(x, bits, d, dtype)
    n, s = O.quantise(x.double().numpy(), bits)
    bad = np.argwhere(scale.view(np.uint16) != s.view(np.uint16))
    assert not len(bad), (len(bad), bad[:4].tolist())
    bad = np.argwhere(O.unpack(code, bits) != n)
    assert not len(bad), (len(bad), bad[:4].tolist())
    assert torch.equal(back, torch.tensor(O.dequantise(n, s)).float().to(DT[dtype]))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_groups_without_a_scale(bits, dtype, d):
    """Constant groups and ranges below fp16's smallest scale: s = 0 and every code 0."""
    x = torch.zeros(40, d)
    for i, c in enumerate((1e-8, -1e-8, 1e-6, 1.5e-7, 3.3e-5, 1.2345678, -777.7, 6e4, 2.0 ** -24, 2.0 ** -25, 1e-41)):
        x[i] = c
    g = torch.Generator().manual_seed(1)
    x[20:30] = 1e-8 * torch.randn(10, d, generator=g)
    x[30:40] = 2.0 ** -24 * (1 + torch.rand(10, d, generator=g)) * ((1 << bits) - 1) / 8
    check_rows(x, bits, d, dtype)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_beside_a_half_step(bits, dtype):
    """Offset and step put a half step at 0: tiny values on both sides of it, and 0 itself."""
    d, q = 128, (1 << bits) - 1
    tiny = [sign * 2.0 ** -e for e in (10, 17, 20, 24, 25, 30, 60, 100, 126, 133) for sign in (1, -1)] + [0.0]
    rows = []
    for step in (1.0, 0.25, 2.0 ** -9):
        for first in range(0, len(tiny), 8):
            r = torch.zeros(d)
            r[0::64], r[1::64] = -q / 2 * step, q / 2 * step
            for i, t in enumerate(tiny[first:first + 8]):
                r[2 + 7 * i::64] = t
            rows.append(r)
    x = torch.stack(rows).to(DT[dtype])
    code, scale, _ = written_rows(x, bits, d, dtype)
    for r in range(len(rows)):      # in fractions: the smallest of these are below 2^-53 of the offset
        s, lo = (Fraction(float(y)) for y in scale[r, 0])
        assert (scale[r] == scale[r, 0]).all() and lo == -q * s / 2
        want = [min(max(round((Fraction(float(y)) - lo) / s), 0), q) for y in x[r]]
        assert O.unpack(code[r], bits).tolist() == want, r


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ranges_that_fp32_rounds(bits, dtype):
    """One end of the range is so small beside the other that their distance has more than 24 bits: the
    scale is still the format's, fp16 of fp32 of the exact quotient."""
    d = 64
    rows = [(1.8671875, -1.8477439880371094e-06), (1.6171875, -5.781650543212891e-06), (1.1171875, -1.341104507446289e-05),
            (1.3671875, -9.47713851928711e-06)]
    rows += [(-b, -a) for a, b in rows]
    r = np.random.default_rng(4)
    for _ in range(500):
        a, b = (1 + r.integers(0, 128, 2) / 128) * 2.0 ** np.array([0, -r.integers(8, 40)])
        rows.append((a, -b) if r.random() < 0.5 else (b, -a))
    x = torch.zeros(len(rows), d, dtype=torch.float64)
    for i, (hi, lo) in enumerate(rows):
        x[i, 0::2], x[i, 1::2] = hi, lo
    x = torch.cat([x * 2.0 ** e for e in (0, 14, -9)])
    check_rows(x, bits, d, dtype)


@pytest.mark.parametrize("bits", [4, 8])
def test_write_odd_values_bf16(bits):
    """Small ranges beside large values, tiny and large values, codes and half steps exactly; a group with
    NaN or infinity reads back non-finite and disturbs no other."""
    d, n, q = 128, 64, (1 << bits) - 1
    x = torch.randn(n, d, generator=torch.Generator().manual_seed(1)).double()
    x[2] = 1000 + 8 * x[2].round()
    x[3] = -1000 + 4 * x[3]
    x[4] *= 1e-7
    x[5] *= 1e-5
    x[6] *= 1e4
    x[7] = torch.arange(d) % (q + 1) * 0.5
    x[8] = (torch.arange(d) % q + 0.5) * 0.25
    x[8, ::64], x[8, 1::64] = 0.0, q * 0.25
    x[9] = x[9].abs() * 1e-38
    x[10] = -6e4
    x[10, 5::64] = 6e4
    check_rows(x, bits, d, "bf16")
    x[20, 3], x[21, 70], x[22, 9], x[23, 65] = float("nan"), float("inf"), -float("inf"), 3e38
    got = written_rows(x, bits, d, "bf16")[2]
    clean = torch.ones(n, d, dtype=torch.bool)
    for r, c in ((20, 0), (21, 64), (22, 0), (23, 64)):
        clean[r, c:c + 64] = False
        assert not torch.isfinite(got[r, c:c + 64]).all()
    x[~clean] = 0
    codes, scale = O.quantise(x.bfloat16().double().numpy(), bits)
    assert torch.equal(got[clean], torch.tensor(O.dequantise(codes, scale)).float().bfloat16()[clean])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_beyond_fp16(bits, dtype):
    """A group's largest value may pass fp16's range as long as its offset and step do not; where one of
    them does, the whole group is non-finite, and the next one is not."""
    d, q = 128, (1 << bits) - 1
    r = torch.rand(4, d, generator=torch.Generator().manual_seed(2))
    r[:, ::64] = 0      # the smallest value of each group
    check_rows(torch.stack([r[0] * 60000.0 * q, 6.5e4 * (2 * r[1] - 1), r[2] * 6.5e4 * q - 6.5e4]), bits, d, dtype)
    x = torch.stack([r[0] * 90000.0 * q, r[1] - 7e4, -1e6 * r[2], 1e5 + r[3]])
    x[:, 64:] = r[:, 64:]
    back = written_rows(x, bits, d, dtype)[2]
    assert not torch.isfinite(back[:, :64]).any() and torch.isfinite(back[:, 64:]).all()
