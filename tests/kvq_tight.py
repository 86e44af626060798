"""Bounds of the quantised KV cache's fp32 attention that see the second fp16 part of the queries and of the
weights.  Row by row and token by token, instead of the largest key and value of the whole pool.

Derived before the first run, with u = 2^-24 (half a step of fp32).  Per group a key is
s (n - mid) + (lo + mid s), mid = (2^bits - 1) / 2, and a value likewise.
* A score.  Let a_t = sum_c |q_c| (s |n - mid| + |lo + mid s|) / sqrt(d).  q in two fp16 parts keeps
  2^-22 of each entry (and 2^-38 of the largest one, where the second part is subnormal).  A product of
  the tensor core adds 16 exact products to its sum, 17 numbers cut off at 2^-23 of the largest: a group
  has 8 such steps (4, for two parts), 8 * 17 * 2^-23.  In fp32: the group sums of q (64), two fused
  operations a group, scaling (8).  So it is off by at most
      e_t = a_t (2^-22 + 136 * 2^-23 + (72 + 2 G) u) + 2^-38 max|q| sum_c s |n - mid| / sqrt(d).
* A weight p_t = exp(x_t - max) is off by e_t, the exponential's own 2^-21 and the rounding of its
  argument, 2^-23 |x_t - max|: a factor 1 +- d_t, and 1 +- 2 d_t covers the squares.
* An output o = sum p v / sum p.  Errors of weights move it by sum p d |v - o| / sum p.  The products:
  w = p s in two fp16 parts keeps 2^-22 of it, and 2^-33 of a weight of one with the group's largest
  scale; two steps of 17 numbers cut off at 2^-23, then sums over T / 16 steps, over the lanes and over
  the parts of a sequence (T / 16 + 24 roundings): relative to S = sum p (s |n - mid| + |lo + mid s|) / sum p.
  Numerator and denominator both: twice the roundings.  The quotient: 2 u |o|.
"""

from __future__ import annotations

import numpy as np

from oracle import kvq as O

U = 2.0 ** -24


def parts(raw, scale, bits):
    """[t][d] code - mid, step, centre (lo + mid s)."""
    mid = ((1 << bits) - 1) / 2
    s = np.repeat(scale.astype(np.float64), O.GROUP, axis=-2)
    return O.unpack(raw, bits) - mid, s[..., 0], s[..., 1] + mid * s[..., 0]


def softmax(x):
    p = np.exp(x - x.max())
    return p, p.sum()


def row(q, k, v, d):
    """(output, bound) of one query row over k, v: parts() of its tokens."""
    x = (k[0] * k[1] + k[2]) @ q / np.sqrt(d)
    p, total = softmax(x)
    val = v[0] * v[1] + v[2]
    o = p @ val / total
    G, T = d // O.GROUP, len(x)
    a = (np.abs(k[0]) * k[1] + np.abs(k[2])) @ np.abs(q) / np.sqrt(d)
    e = a * (2.0 ** -22 + 136 * 2.0 ** -23 + (72 + 2 * G) * U) + 2.0 ** -38 * np.abs(q).max() * (np.abs(k[0]) * k[1]).sum(1) / np.sqrt(d)
    dt = 2 * (e + 2.0 ** -21 + 2.0 ** -23 * (x.max() - x))
    size = p @ (np.abs(v[0]) * v[1] + np.abs(v[2])) / total
    floor = 2.0 ** -33 * v[1].max(0) * np.abs(v[0]).sum(0) / total
    bound = (p * dt) @ np.abs(val - o) / total + floor + size * (2.0 ** -22 + 34 * 2.0 ** -23 + 2 * (T / 16 + 24) * U) + 2 * U * np.abs(o)
    return o, bound


def f16(x):
    return x.astype(np.float16).astype(np.float64)


def row_in_one_part(q, k, v, d, what):
    """The same row with only one fp16 part of the queries ("q") or of the weights ("w")."""
    sigma = 2.0 ** (13 - np.floor(np.log2(np.abs(q).max())))
    q1 = f16(q * sigma) / sigma if what == "q" else q
    x = ((k[0] * k[1]) @ q1 + k[2] @ q) / np.sqrt(d)
    p, total = softmax(x)
    if what == "q":
        return p @ (v[0] * v[1] + v[2]) / total
    top = 2.0 ** np.floor(np.log2(v[1].max(0)))
    w = f16(p[:, None] * v[1] * 512 / top) * top / 512
    return ((w * v[0]).sum(0) + p @ v[2]) / total


def problem(d, group, bits, lens, page, seed=0, n=1):
    """(config, arrays, q): keys along one direction, so that the scores are coherent sums, and queries whose
    entries all lie just below half a step beside an fp16 number."""
    from kvq_utils import config, fill
    import torch
    cfg = config(batch=len(lens), kv_heads=2, q_heads=2 * group, head_dim=d, page=page, max_pages=-(-max(lens) // page) + 1, bits=bits, dtype="f32")
    arrays = fill(cfg, seed)
    r = np.random.default_rng(seed + 1)
    base = f16(r.standard_normal((2, d)))
    shape = (1, cfg["n_pages"], 2, page)
    k = r.uniform(-1, 1, shape + (1,)) * base[:, None] + 0.02 * r.standard_normal(shape + (d,))
    code, scale = O.quantise(k, bits)
    arrays["k_code"], arrays["k_scale"] = O.pack(code, bits), scale
    # (k_mean stays as it is: what is selected does not matter here)
    q = np.repeat(base[None, None, None], len(lens), 1).repeat(n, 2)[..., None, :] * r.choice([-0.25, 0.25, 0.5], (1, len(lens), n, 2, group, 1))
    q = q * (1 + 0.98 * 2.0 ** -12)
    return cfg, arrays, torch.tensor(q.reshape(1, len(lens), n, 2 * group, d), dtype=torch.float32)


def rows_of(cfg, arrays, q, lens):
    """Every query row with tokens: (index into q, query, parts of its keys, parts of its values)."""
    qf = q.double().numpy()
    n, H, d, bits = q.shape[2], cfg["n_kv_heads"], cfg["head_dim"], cfg["bits"]
    g = cfg["n_q_heads"] // H
    for b, length in enumerate(lens):
        pids = arrays["table"][b]
        for h in range(H):
            k, v = ([y.reshape(-1, d) for y in parts(arrays[x + "_code"][0, pids, h], arrays[x + "_scale"][0, pids, h], bits)] for x in "kv")
            for i in range(n):
                lim = length - n + 1 + i
                if lim <= 0:
                    continue
                for j in range(g):
                    at = (0, b, i, h * g + j)
                    yield at, qf[at], [y[:lim] for y in k], [y[:lim] for y in v]


def worst(cfg, arrays, q, lens, out):
    """The largest error of out [like q] over its bound."""
    most = 0.0
    for at, qi, k, v in rows_of(cfg, arrays, q, lens):
        o, bound = row(qi, k, v, cfg["head_dim"])
        most = max(most, float((np.abs(out[at] - o) / bound).max()))
    return most


CASES = [  # d, group, bits, n, lens
    (64, 1, 4, 1, [2, 3, 17]), (64, 8, 8, 1, [2, 5, 33]), (128, 4, 4, 1, [2, 3, 40]), (128, 3, 8, 2, [3, 9, 20]), (128, 16, 4, 1, [2, 7, 64]),
    (128, 7, 8, 1, [2, 4, 100]), (64, 5, 4, 6, [8, 30, 3]), (256, 4, 4, 1, [2, 3, 50]), (256, 8, 8, 1, [2, 6, 31]), (256, 12, 4, 3, [5, 4, 18]),
]
