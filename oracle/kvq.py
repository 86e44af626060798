"""fp64 oracle of the quantised KV cache: format, writing, attention, page selection (numpy).

Arrays have the layouts of ``lowram.h`` (codes uint8, scales float16 (s, lo) pairs, page means
float64 here).  Nothing is shared with the library."""

from __future__ import annotations

import numpy as np

GROUP = 64


def code_place(c: int, d: int, bits: int):
    """(byte, shift) of channel c in a row of codes: cell (c % 64) / 8 * G + c / 64, code c % 8."""
    cell, i = c % GROUP // 8 * (d // GROUP) + c // GROUP, c % 8
    return (cell * bits + i * bits // 8, 4 * (i % 2) if bits == 4 else 0)


def unpack(raw: np.ndarray, bits: int) -> np.ndarray:
    d = raw.shape[-1] * 8 // bits
    place = [code_place(c, d, bits) for c in range(d)]
    at, sh = np.array([p for p, _ in place]), np.array([s for _, s in place])
    return (raw[..., at].astype(np.int64) >> sh) & ((1 << bits) - 1)


def pack(codes: np.ndarray, bits: int) -> np.ndarray:
    d = codes.shape[-1]
    out = np.zeros(codes.shape[:-1] + (d * bits // 8,), np.uint8)
    for c in range(d):
        at, sh = code_place(c, d, bits)
        out[..., at] |= (codes[..., c].astype(np.uint8) << sh)
    return out


def quantise(x: np.ndarray, bits: int):
    """x [..., d] -> (codes [..., d], scales [..., G, 2] float16)."""
    q = (1 << bits) - 1
    t = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, GROUP))
    mn, mx = t.min(-1), t.max(-1)
    with np.errstate(over="ignore"):
        s = ((mx - mn) / q).astype(np.float32).astype(np.float16)
        lo = mn.astype(np.float32).astype(np.float16)
    sd, ld = s.astype(np.float64)[..., None], lo.astype(np.float64)[..., None]
    n = np.where(sd > 0, np.rint((t - ld) / np.where(sd > 0, sd, 1.0)), 0.0)
    return np.clip(n, 0, q).astype(np.int64).reshape(x.shape), np.stack((s, lo), -1)


def dequantise(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    s = np.repeat(scale.astype(np.float64), GROUP, axis=-2)
    return s[..., 0] * codes + s[..., 1]


def rows(raw, scale, bits):
    return dequantise(unpack(raw, bits), scale)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray):
    """q [g][d], k, v [t][d] -> [g][d]; zeros without a token."""
    if k.shape[0] == 0:
        return np.zeros_like(q)
    x = q @ k.T / np.sqrt(q.shape[-1])
    p = np.exp(x - x.max(-1, keepdims=True))
    return p @ v / p.sum(-1, keepdims=True)


def select(score: np.ndarray, newest: int, top_k: int):
    """Pages of a query, ascending: the newest and the best top_k - 1 before it (ties to the lower)."""
    s = np.where(np.isnan(score[:newest]), -np.inf, score[:newest])
    best = sorted(range(newest), key=lambda c: (-s[c], c))[:top_k - 1]
    return sorted(best) + [newest]


def attention(cfg: dict, arrays: dict, q: np.ndarray, lens, layer0: int = 0, top_k: int = 0, table=None, n_pages=None):
    """(out, sel): q [n_layers][B][n][Hq][d]; top_k = 0 attends over whole sequences (sel None).
    ``arrays``: k_code, k_scale, v_code, v_scale, k_mean as numpy; table [B][max_pages]."""
    H, page, bits = cfg["n_kv_heads"], cfg["page"], cfg["bits"]
    NL, B, n, Hq, d = q.shape
    g = Hq // H
    out = np.zeros(q.shape)
    sel = np.full((NL, B, n, H, max(top_k, 1)), -1, np.int64)
    for li in range(NL):
        layer = layer0 + li
        for b in range(B):
            length = int(np.clip(lens[b], 0, table.shape[1] * page))
            used = -(-length // page)
            pids = table[b, :used]
            for h in range(H):
                if used:
                    k, v = (rows(arrays[x + "_code"][layer, pids, h], arrays[x + "_scale"][layer, pids, h], bits).reshape(-1, d)
                            for x in "kv")
                for i in range(n):
                    lim = length - n + 1 + i
                    if lim <= 0:
                        continue
                    qi = q[li, b, i, h * g:(h + 1) * g].astype(np.float64)
                    if not top_k:
                        out[li, b, i, h * g:(h + 1) * g] = attend(qi, k[:lim], v[:lim])
                        continue
                    newest = (lim - 1) // page
                    pick = select(arrays["k_mean"][layer, pids[:newest], h].astype(np.float64) @ qi.sum(0), newest, top_k)
                    sel[li, b, i, h, :len(pick)] = pick
                    at = (np.array(pick)[:, None] * page + np.arange(page)).reshape(-1)
                    at = at[at < lim]
                    out[li, b, i, h * g:(h + 1) * g] = attend(qi, k[at], v[at])
    return out, (sel if top_k else None)
