"""Shared by the tests of the quantised KV cache: caches filled by the oracle, error bounds.

Bounds, derived before the first run.  Let u16 = 2^-11, ubf = 2^-8, u32 = 2^-24 be half steps, and
X = max_t sum_c |q_c khat_tc| / sqrt(d).
* Logits: d products summed in fp32 and two or three more roundings: off by at most
  e = (d + 8) u32 X (tensor-core sums may truncate: twice that).  The exponential adds 4 u32 and
  its argument's own rounding, u32 X log2(e).  A weight is then off by a factor 1 +- w,
  w = 2 (d + 12) u32 (1 + X); BF16 calls round weight times value scale to fp16 once, adding u16.
* An output is a weighted mean of values in [-M, M]: numerator and denominator are each off by w M
  (sums over T tokens in fp32 pieces: + T^(1/2) u32 M), so |o - ref| <= 2 w M, plus the last
  rounding ubf |ref| or u32 |ref|.  M = max |lo| + s * (2^bits - 1) over the rows.
"""

from __future__ import annotations

import numpy as np
import torch

from oracle import kvq as O

U16, UBF, U32 = 2.0 ** -11, 2.0 ** -8, 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def config(batch=2, layers=1, kv_heads=2, q_heads=8, head_dim=128, page=32, max_pages=8, bits=4, dtype="bf16", n_pages=None):
    return dict(batch=batch, n_layers=layers, n_kv_heads=kv_heads, n_q_heads=q_heads, head_dim=head_dim, page=page,
                n_pages=n_pages or batch * max_pages + 2, max_pages=max_pages, bits=bits, dtype=dtype)


def fill(cfg, seed=0, k_std=1.0, v_std=1.0, v_bias=0.0):
    """numpy arrays of a whole pool (every page quantised random rows, means of the rows) and a
    shuffled table."""
    r = np.random.default_rng(seed)
    L, P, H, page, d, bits = (cfg[k] for k in ("n_layers", "n_pages", "n_kv_heads", "page", "head_dim", "bits"))
    out = {}
    for x, std, bias in (("k", k_std, 0.0), ("v", v_std, v_bias)):
        t = r.standard_normal((L, P, H, page, d)) * std + bias
        if x == "k":
            t += r.standard_normal((L, P, H, 1, d)) * 0.5 * std
        n, s = O.quantise(t, bits)
        out[x + "_code"], out[x + "_scale"] = O.pack(n, bits), s
        if x == "k":
            m = O.dequantise(n, s).mean(3)
            out["k_mean"] = torch.tensor(m).bfloat16().double().numpy()
    out["table"] = r.permutation(P)[:cfg["batch"] * cfg["max_pages"]].astype(np.int32).reshape(cfg["batch"], -1)
    return out


def to_device(arrays, device="cuda"):
    out = {}
    for k, v in arrays.items():
        t = torch.from_numpy(np.ascontiguousarray(v))
        out[k] = (t.bfloat16() if k == "k_mean" else t).to(device)
    return out


def queries(cfg, n=1, layers=None, seed=1, std=1.0):
    r = np.random.default_rng(seed)
    q = r.standard_normal((layers or cfg["n_layers"], cfg["batch"], n, cfg["n_q_heads"], cfg["head_dim"])) * std
    return torch.tensor(q, dtype=torch.float32).to(DT[cfg["dtype"]])


def spoil_behind(cfg, arrays, lens):
    """NaN scales and random codes in every slot behind each sequence's last token."""
    r = np.random.default_rng(5)
    page = cfg["page"]
    for b, length in enumerate(lens):
        for i in range(cfg["max_pages"]):
            first = min(max(int(length) - i * page, 0), page)
            p = arrays["table"][b, i]
            for x in "kv":
                arrays[x + "_scale"][:, p, :, first:] = np.float16(np.nan)
                arrays[x + "_code"][:, p, :, first:] = r.integers(0, 256, arrays[x + "_code"][:, p, :, first:].shape, dtype=np.uint8)
            if first < page:
                arrays["k_mean"][:, p] = np.nan


def check_attention(cfg, arrays, q, lens, out, layer0=0, top_k=0, sel=None):
    qf = q.detach().cpu().double().numpy()
    ref, rsel = O.attention(cfg, arrays, qf, lens, layer0, top_k, arrays["table"])
    got = out.detach().cpu().double().numpy()
    if top_k and sel is not None:
        assert np.array_equal(sel.cpu().numpy(), rsel)
    d, qm = cfg["head_dim"], (1 << cfg["bits"]) - 1
    with np.errstate(invalid="ignore"):
        ks, vs = (np.abs(arrays[x + "_scale"].astype(np.float64)) for x in "kv")
        kmax = np.nanmax(ks[..., 1] + ks[..., 0] * qm)
        M = np.nanmax(vs[..., 1] + vs[..., 0] * qm)
    X = np.abs(qf).sum(-1, keepdims=True) * kmax / np.sqrt(d)
    T = max(1, int(max(lens)))
    w = 2 * (d + 12) * U32 * (1 + X) + (U16 if cfg["dtype"] == "bf16" else 0.0)
    tol = 2 * w * M + np.sqrt(T) * U32 * M + (UBF if cfg["dtype"] == "bf16" else U32) * np.abs(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)), np.argwhere(bad)[:4].tolist())
    return float((np.abs(got - ref) / tol).max())
