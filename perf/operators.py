"""Cases for the quantised KV cache: writing and reading it, attention over it, and attention over selected pages.

The cache holds keys and values in 4 or 8 bits.  Every token row of a (layer, page, KV head) is cut
into groups of 64 channels; a group is codes n in [0, 2^bits - 1] with an fp16 (scale s, offset lo)
and stands for lo + s * n.  Arrays (P pages in a pool, G = head_dim / 64):

  k_code, v_code   [L][P][Hkv][page][head_dim * bits / 8] uint8: 8 cells w, each [G] x 8 codes, so the
                   codes of channel 64 g + 8 w + i lie in cell w * G + g (4 bits: byte i / 2, low nibble first)
  k_scale, v_scale [L][P][Hkv][page][G][2] fp16 (s, lo)
  k_mean           [L][P][Hkv][head_dim] bf16: the mean of a full page's dequantised keys
  table            [B][max_pages] int32: pages of each sequence

Operators: "roundtrip" writes new tokens into the cache and reads them back, "read" reads a range of a
filled cache, "decode" attends over whole sequences, "sparse" over the newest page and the top_k - 1
best-scoring older ones.
"""

import math
import random

import torch

own = False
GROUP = 64
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases

def _case(name, op, **kw):
    c = dict(op=op, bits=4, dtype="bf16", layers=1, batch=1, kv_heads=8, q_heads=32, head_dim=128, page=64, ctx=1024,
             n=1, ragged=False, top_k=0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's keys and values of every layer of a small batch
        _case("append_step", "roundtrip", layers=32, batch=4, ctx=509, n=1, ragged=True),
        # a batch of prompts written after a short shared prefix
        _case("append_prompts", "roundtrip", batch=8, ctx=40, n=8192),
        # fp32 activations, 8 bits, odd head count, small pages, every sequence another length
        _case("append_ragged_f32", "roundtrip", bits=8, dtype="f32", layers=2, batch=5, kv_heads=3, q_heads=6,
              head_dim=64, page=16, ctx=333, n=777, ragged=True),
        # whole contexts read back (moving a sequence to another cache)
        _case("read_contexts", "read", batch=4, ctx=32768, n=32768),
        # a short ragged window in 8 bits, wide heads
        _case("read_window", "read", bits=8, batch=6, kv_heads=2, q_heads=8, head_dim=256, page=32, ctx=1500, n=129,
              ragged=True),
        # one short conversation: latency
        _case("decode_short", "decode", ctx=301),
        # the 32K shape of the compressed cache's benchmark, batch 4, several layers in a call
        _case("decode_32k", "decode", layers=4, batch=4, ctx=32768),
        # four tokens verified at once, 8 bits, ragged batch with an empty slot
        _case("decode_verify_int8", "decode", bits=8, batch=16, q_heads=64, head_dim=64, page=16, ctx=8191, n=4,
              ragged=True),
        # long contexts at full size
        _case("decode_128k", "decode", batch=8, ctx=131072, page=128, ragged=True),
        # one long conversation, 32 pages of 2048
        _case("sparse_single", "sparse", ctx=131072, top_k=32),
        # a batch of 64K contexts
        _case("sparse_batch", "sparse", layers=2, batch=16, ctx=65536, top_k=32, ragged=True),
        # fp32, 8 bits, wide heads, three tokens at once
        _case("sparse_f32", "sparse", bits=8, dtype="f32", batch=3, kv_heads=2, q_heads=16, head_dim=256, page=32,
              ctx=5003, n=3, ragged=True, top_k=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["roundtrip", "read", "decode", "decode", "sparse", "sparse"])
    bits, dtype = rng.choice([4, 4, 4, 8]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128, 128, 256])
    heads = rng.choice([1, 2, 3, 4, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    batch, layers = _log(rng, 1, 32), rng.choice([1, 1, 1, 2, 4])
    row = 2 * layers * batch * heads * (d * bits // 8 + d // 16)   # cache bytes of one position
    vals = 2 * layers * batch * heads * d * (2 if dtype == "bf16" else 4)
    kw = dict(bits=bits, dtype=dtype, layers=layers, batch=batch, kv_heads=heads, q_heads=heads * group, head_dim=d, page=page,
              ragged=rng.random() < 0.5)
    if op in ("roundtrip", "read"):
        n = _log(rng, 1, max(2, min(32768, int(3.0e8 / vals))))
        ctx = _log(rng, 1, max(2, min(4096, int(3.0e8 / row)))) + (n if op == "read" else 0)
        return _case(None, op, ctx=ctx, n=n, **kw)
    n = rng.choice([1, 1, 1, 2, 4, 5])
    ctx = max(n, _log(rng, 16, max(32, min(131072, int(4.0e8 / (row * n))))))
    top_k = rng.choice([1, 4, 8, 16, 32, 64]) if op == "sparse" else 0
    while layers * batch * n * heads * min(top_k, -(-ctx // page)) * page * d > 2.5e8:   # rows the plain form gathers
        top_k //= 2
    return _case(None, op, ctx=ctx, n=n, top_k=top_k, **kw)


def _lens(case):
    """Tokens held by each sequence: all ctx, or ragged with one full, one empty and the rest in between."""
    B, ctx = case["batch"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * B
    r = random.Random(ctx * 1009 + B * 31 + case["page"])
    out = [ctx] + [r.randint(1, ctx) for _ in range(B - 1)]
    if B >= 4:
        out[B // 2] = 0
    return out


def _spans(case):
    """(start, count) of the tokens each sequence writes or reads."""
    r = random.Random(case["ctx"] * 7 + case["n"] * 131 + case["batch"])
    out = []
    for length in _lens(case):
        n = r.randint(0, case["n"]) if case["ragged"] and out else case["n"]
        if case["op"] == "read":
            n = min(n, length)
            out.append((length - n, n))
        else:
            out.append((length, n))
    return out


def _max_pages(case):
    most = case["ctx"] + (case["n"] if case["op"] == "roundtrip" else 0)
    return -(-most // case["page"])


# ------------------------------------------------------------------------------- inputs

def _cells(x, groups):
    """[..., d] -> [..., 8, G, 8]: the order in which codes are stored."""
    return x.reshape(*x.shape[:-1], groups, 8, 8).transpose(-3, -2)


def _pack(codes, bits):
    """codes [..., d] (integers) -> [..., d * bits / 8] uint8"""
    c = _cells(codes, codes.shape[-1] // GROUP).to(torch.uint8)
    if bits == 4:
        c = c[..., 0::2] | (c[..., 1::2] << 4)
    return c.flatten(-3)


def _unpack(raw, bits):
    """[..., d * bits / 8] uint8 -> codes [..., d] uint8"""
    d = raw.shape[-1] * 8 // bits
    c = raw.reshape(*raw.shape[:-1], 8, d // GROUP, bits)
    if bits == 4:
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    return c.transpose(-3, -2).flatten(-3)


def _quantise(x, bits, wide):
    """x [..., d] -> packed codes and (scale, offset) pairs, computed in the type `wide`."""
    qmax = torch.tensor((1 << bits) - 1, dtype=wide, device=x.device)
    t = x.reshape(*x.shape[:-1], -1, GROUP).to(wide)
    low, high = t.amin(-1), t.amax(-1)
    lo, s = low.half(), ((high - low) / qmax).float().half()
    sw = s.to(wide)[..., None]
    n = torch.where(sw > 0, (t - lo.to(wide)[..., None]) / sw, torch.zeros_like(t)).round()
    n = torch.minimum(n.clamp_min(0), qmax)
    return _pack(n.flatten(-2), bits), torch.stack((s, lo), -1)


def _dequantise(raw, scale, bits, wide):
    n = _unpack(raw, bits).to(wide)
    s = scale.to(wide).repeat_interleave(GROUP, dim=-2)
    return n * s[..., 0] + s[..., 1]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    L, B, H, d, page, bits = (case[k] for k in ("layers", "batch", "kv_heads", "head_dim", "page", "bits"))
    dt, mp, G = _DT[case["dtype"]], _max_pages(case), case["head_dim"] // GROUP
    P = B * mp + 3
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    st = dict(case=case,
              k_code=torch.empty(L, P, H, page, d * bits // 8, dtype=torch.uint8, device="cuda"),
              v_code=torch.empty(L, P, H, page, d * bits // 8, dtype=torch.uint8, device="cuda"),
              k_scale=torch.empty(L, P, H, page, G, 2, dtype=torch.float16, device="cuda"),
              v_scale=torch.empty(L, P, H, page, G, 2, dtype=torch.float16, device="cuda"),
              k_mean=torch.empty(L, P, H, d, dtype=torch.bfloat16, device="cuda"),
              table=torch.randperm(P, device="cuda", generator=g)[:B * mp].to(torch.int32).reshape(B, mp))
    # keys of a page lie around a centre of their own, with a constant part in a few channels
    part = max(1, (1 << 26) // (H * page * d))
    bias = 2.0 * rand(H, 1, d) * (torch.rand(H, 1, d, device="cuda", generator=g) < 0.05)
    for layer in range(L):
        for p in range(0, P, part):
            n = min(part, P - p)
            x = 0.6 * rand(n, H, page, d) + 0.6 * rand(n, H, 1, d) + bias
            st["k_code"][layer, p:p + n], st["k_scale"][layer, p:p + n] = _quantise(x, bits, torch.float32)
            st["k_mean"][layer, p:p + n] = x.mean(2).bfloat16()
            x = rand(n, H, page, d)
            st["v_code"][layer, p:p + n], st["v_scale"][layer, p:p + n] = _quantise(x, bits, torch.float32)
    st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    if case["op"] in ("roundtrip", "read"):
        spans = _spans(case)
        st["pos"] = torch.tensor([p for p, _ in spans], dtype=torch.int32, device="cuda")
        st["count"] = torch.tensor([n for _, n in spans], dtype=torch.int32, device="cuda")
        st["k_out"] = torch.zeros(L, B, case["n"], H, d, dtype=dt, device="cuda")
        st["v_out"] = torch.zeros(L, B, case["n"], H, d, dtype=dt, device="cuda")
        # the plain form's index lists: (sequence, token) of every row, (sequence, page) of every page filled
        seq, tok, done = [], [], []
        for b, (p, n) in enumerate(spans):
            seq.append(torch.full((n,), b))
            tok.append(torch.arange(n))
            done += [(b, c) for c in range(p // page, (p + n) // page)]
        st["seq"], st["tok"] = torch.cat(seq).cuda(), torch.cat(tok).cuda()
        st["done"] = torch.tensor(done, dtype=torch.long).reshape(-1, 2).cuda()
        if case["op"] == "roundtrip":
            # keys and values are slices of one projection, as a model has them
            kv = rand(L, B, case["n"], 2 * H, d).to(dt)
            kv[..., :H, :] += bias[:, 0].to(dt)
            st["k"], st["v"] = kv[..., :H, :], kv[..., H:, :]
    else:
        st["q"] = (1.5 * rand(L, B, case["n"], case["q_heads"], d)).to(dt)
    if own:
        import kv_cache_compression_lowram_b200 as K
        st["cache"] = K.LowramKvq(dict(batch=B, n_layers=L, n_kv_heads=H, n_q_heads=case["q_heads"], head_dim=d, page=page, n_pages=P,
                                       max_pages=mp, bits=bits, dtype=case["dtype"]),
                                  {k: st[k] for k in ("k_code", "k_scale", "v_code", "v_scale", "k_mean", "table")},
                                  max_q=case["n"] if "q" in st else 1)
    return st


# ------------------------------------------------------------------------------- plain forms

def _plain_write(st):
    case = st["case"]
    page, bits, seq, tok = case["page"], case["bits"], st["seq"], st["tok"]
    at = st["pos"][seq] + tok
    pid, slot = st["table"][seq, at // page].long(), at % page
    for x, code, scale in ((st["k"], st["k_code"], st["k_scale"]), (st["v"], st["v_code"], st["v_scale"])):
        c, s = _quantise(x[:, seq, tok], bits, torch.float64)      # [L][rows][H][...]
        code[:, pid, :, slot] = c.transpose(0, 1)
        scale[:, pid, :, slot] = s.transpose(0, 1)
    pid = st["table"][st["done"][:, 0], st["done"][:, 1]].long()
    st["k_mean"][:, pid] = _dequantise(st["k_code"][:, pid], st["k_scale"][:, pid], bits, torch.float64).mean(3).float().bfloat16()


def _plain_read(st):
    case = st["case"]
    page, seq, tok = case["page"], st["seq"], st["tok"]
    at = st["pos"][seq] + tok
    pid, slot = st["table"][seq, at // page].long(), at % page
    for out, code, scale in ((st["k_out"], st["k_code"], st["k_scale"]), (st["v_out"], st["v_code"], st["v_scale"])):
        x = _dequantise(code[:, pid, :, slot], scale[:, pid, :, slot], case["bits"], torch.float32)   # [rows][L][H][d]
        out[:, seq, tok] = x.transpose(0, 1).to(out.dtype)


def _attend(q, k, v, mask):
    """q [..., r, d], k, v [..., s, d] fp32, mask [..., r, s] -> [..., r, d]; rows without a token give 0."""
    x = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    x = x.masked_fill(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _limits(st):
    n = st["case"]["n"]
    return st["lens"].long()[:, None] - n + 1 + torch.arange(n, device="cuda")      # [B][n]


def _plain_decode(st):
    case = st["case"]
    L, B, n, H, d, page = (case[k] for k in ("layers", "batch", "n", "kv_heads", "head_dim", "page"))
    g, tab = case["q_heads"] // H, st["table"].long()
    k, v = (_dequantise(st[c][:, tab].transpose(2, 3).flatten(3, 4), st[s][:, tab].transpose(2, 3).flatten(3, 4), case["bits"], torch.float32)
            for c, s in (("k_code", "k_scale"), ("v_code", "v_scale")))                    # [L][B][H][S][d]
    q = st["q"].float().reshape(L, B, n, H, g, d).permute(0, 1, 3, 2, 4, 5).flatten(3, 4)    # [L][B][H][n g][d]
    mask = torch.arange(k.shape[3], device="cuda") < _limits(st)[..., None]                # [B][n][S]
    o = _attend(q, k, v, mask.repeat_interleave(g, dim=1)[None, :, None])
    return o.reshape(L, B, H, n, g, d).permute(0, 1, 3, 2, 4, 5).reshape(st["q"].shape).to(st["q"].dtype)


def _plain_sparse(st):
    case = st["case"]
    L, B, n, H, d, page, top = (case[k] for k in ("layers", "batch", "n", "kv_heads", "head_dim", "page", "top_k"))
    g, tab, lim = case["q_heads"] // H, st["table"].long(), _limits(st)
    mp = tab.shape[1]
    mean = st["k_mean"][:, tab].double().transpose(2, 3)                                     # [L][B][H][mp][d]
    q = st["q"].reshape(L, B, n, H, g, d)
    score = torch.einsum("lbnhd,lbhpd->lbnhp", q.double().sum(4), mean)
    last = torch.where(lim > 0, (lim - 1) // page, lim.new_full((), -1))[None, :, :, None, None]
    ids = torch.arange(mp, device="cuda")
    score = torch.where((ids < last) & ~score.isnan(), score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :min(top - 1, mp)]
    pick = torch.cat((best, last.expand(L, B, n, H, 1).clamp_min(0)), -1)                    # [L][B][n][H][k]
    use = torch.cat((best < last, last.expand(L, B, n, H, 1) >= 0), -1)
    li, bi = torch.arange(L, device="cuda").view(L, 1, 1, 1, 1), torch.arange(B, device="cuda").view(1, B, 1, 1, 1)
    hi, pid = torch.arange(H, device="cuda").view(1, 1, 1, H, 1), tab[bi, pick]
    k, v = (_dequantise(st[c][li, pid, hi].flatten(4, 5), st[s][li, pid, hi].flatten(4, 5), case["bits"], torch.float32)
            for c, s in (("k_code", "k_scale"), ("v_code", "v_scale")))                    # [L][B][n][H][k page][d]
    at = (pick[..., None] * page + torch.arange(page, device="cuda")).flatten(4)
    mask = (at < lim[None, :, :, None, None]) & use.repeat_interleave(page, dim=-1)
    o = _attend(q.float(), k, v, mask[..., None, :])
    return o.reshape(st["q"].shape).to(st["q"].dtype)


def run(st):
    op = st["case"]["op"]
    if own:
        c = st["cache"]
        if op == "decode":
            return c.decode(st["q"], st["lens"])
        if op == "sparse":
            return c.decode_sparse(st["q"], st["lens"], st["case"]["top_k"])
        if op == "roundtrip":
            c.write(st["k"], st["v"], st["pos"], st["count"])
        c.read(st["pos"], st["count"], out=(st["k_out"], st["v_out"]))
    elif op in ("decode", "sparse"):
        return _plain_decode(st) if op == "decode" else _plain_sparse(st)
    else:
        if op == "roundtrip":
            _plain_write(st)
        _plain_read(st)
    out = {"k": st["k_out"], "v": st["v_out"]}
    if op == "roundtrip":
        out["k_mean"] = st["k_mean"]
    return out


# ------------------------------------------------------------------------------- work and exact values

def work(case):
    L, H, d, page = (case[k] for k in ("layers", "kv_heads", "head_dim", "page"))
    elt = 2 if case["dtype"] == "bf16" else 4
    row = 2 * (d * case["bits"] // 8 + d // GROUP * 4)            # a token's K and V in the cache
    if case["op"] in ("roundtrip", "read"):
        rows = L * H * sum(n for _, n in _spans(case))
        full = L * H * sum((p + n) // page - p // page for p, n in _spans(case))
        if case["op"] == "read":
            return {"bytes": rows * (row + 2 * d * elt), "flops": rows * 4 * d}
        return {"bytes": rows * (row + 4 * d * elt) + full * 2 * d, "flops": rows * 16 * d}
    g, n = case["q_heads"] // H, case["n"]
    qo = 2 * L * case["batch"] * n * case["q_heads"] * d * elt
    if case["op"] == "decode":
        tokens = sum(_lens(case))
        return {"bytes": L * H * tokens * row + qo, "flops": L * H * tokens * n * g * 4 * d}
    means = tokens = reads = 0
    for length in _lens(case):
        kept = []
        for i in range(n):
            lim = length - n + 1 + i
            last = (lim - 1) // page if lim > 0 else -1
            older = min(case["top_k"] - 1, max(last, 0))
            kept.append(older * page + (lim - last * page if last >= 0 else 0))
        means += (length - 1) // page if length > 0 else 0
        tokens += sum(kept)
        reads += max(kept)                                        # the queries may all pick the same pages
    return {"bytes": L * H * (means * d * 2 + reads * row) + qo,
            "flops": L * H * (means * n * 2 * d + tokens * g * 4 * d)}


def _rows64(raw, scale, bits):
    """One (layer, page list, head)'s rows in 64 bits, channel by channel from the layout: [tokens][d]."""
    d = raw.shape[-1] * 8 // bits
    c = torch.arange(d, device=raw.device)
    cell = (c % 64) // 8 * (d // 64) + c // 64
    byte = cell * bits + (c % 8) * bits // 8
    n = raw[..., byte].double()
    if bits == 4:
        n = torch.where(c % 2 == 0, n % 16, torch.div(n, 16, rounding_mode="floor"))
    s = scale[..., c // 64, :].double()
    return (s[..., 0] * n + s[..., 1]).reshape(-1, d)


def exact(case, seed):
    st = prepare(case, seed)
    st.pop("cache", None)
    L, B, H, d, page, bits, n = (case[k] for k in ("layers", "batch", "kv_heads", "head_dim", "page", "bits", "n"))
    tab = st["table"].cpu()
    if case["op"] in ("roundtrip", "read"):
        k_out, v_out, mean = st["k_out"].double(), st["v_out"].double(), st["k_mean"].double()
        for b, (p, cnt) in enumerate(_spans(case)):
            if cnt == 0:
                continue
            pages = tab[b].cuda().long()
            for layer in range(L):
                for h in range(H):
                    old = [_rows64(st[x + "_code"][layer, pages, h], st[x + "_scale"][layer, pages, h], bits) for x in "kv"]
                    if case["op"] == "read":
                        k_out[layer, b, :cnt, h], v_out[layer, b, :cnt, h] = old[0][p:p + cnt], old[1][p:p + cnt]
                        continue
                    for x, rows, out in (("k", old[0], k_out), ("v", old[1], v_out)):
                        t = st[x][layer, b, :cnt, h].double().view(cnt, -1, 64)
                        lo = t.min(-1, keepdim=True).values.float().half().double()
                        s = ((t.max(-1, keepdim=True).values - t.min(-1, keepdim=True).values) / ((1 << bits) - 1)).float().half().double()
                        code = torch.where(s > 0, ((t - lo) / s).round().clamp(0, (1 << bits) - 1), 0.0)
                        out[layer, b, :cnt, h] = rows[p:p + cnt] = (lo + s * code).view(cnt, d)
                    for c in range(p // page, (p + cnt) // page):
                        mean[layer, int(tab[b, c]), h] = old[0][c * page:(c + 1) * page].mean(0)
        out = {"k": k_out, "v": v_out}
        if case["op"] == "roundtrip":
            out["k_mean"] = mean
        return out
    q, g = st["q"].double(), case["q_heads"] // H
    res = torch.zeros_like(q)
    means = st["k_mean"].double()
    for b, length in enumerate(_lens(case)):
        if length == 0:
            continue
        pages = tab[b].cuda().long()
        for layer in range(L):
            for h in range(H):
                if case["op"] == "decode":
                    k, v = (_rows64(st[x + "_code"][layer, pages, h], st[x + "_scale"][layer, pages, h], bits) for x in "kv")
                for i in range(n):
                    lim = length - n + 1 + i
                    if lim <= 0:
                        continue
                    qi = q[layer, b, i, h * g:(h + 1) * g]
                    if case["op"] == "decode":
                        kk, vv = k[:lim], v[:lim]
                    else:
                        last = (lim - 1) // page
                        score = (means[layer, pages[:last], h] @ qi.sum(0)).tolist()
                        keep = sorted(range(last), key=lambda c: (-score[c], c))[:case["top_k"] - 1]
                        keep = torch.tensor(sorted(keep) + [last], device="cuda")
                        some = (len(keep) - 1) * page + lim - last * page
                        kk, vv = (_rows64(st[x + "_code"][layer, pages[keep], h], st[x + "_scale"][layer, pages[keep], h], bits)[:some] for x in "kv")
                    res[layer, b, i, h * g:(h + 1) * g] = torch.softmax(qi @ kk.T / math.sqrt(d), -1) @ vv
    return res
