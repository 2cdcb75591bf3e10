"""Cases of the paged-cache operators: appending to and attending over paged quantized K/V caches.

Three operators, each in its plain form (elementary torch operations) and through the package:

  append   new keys and values of a ragged batch -- keys normalised per head and rotated by their
           position where the case says so -- quantized into the pages of a K and a V cache;
  attend   causal attention of each sequence's newest tokens (one token, or a chunk) over its pages;
  cross    attention of each sequence's tokens over all of its cached states, without a mask.

Formats: "prod3" is 2 Lloyd-Max bits and one QJL sign per coordinate, "mseB" is B Lloyd-Max bits.
"""

import functools
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
QJL = math.sqrt(math.pi / 2.0)
MAX_POS = 65536

# ------------------------------------------------------------------ cases


def listed():
    base = {"prep": "none", "window": 0, "singles": 0, "ragged": False, "mix": 1}
    append = {**base, "op": "append", "ctx": 0, "Hq": 0}
    attend = {**base, "op": "attend"}
    cross = {**base, "op": "cross"}
    return [
        # one new token for each of a few running sequences: the append of one decode step
        {**append, "name": "append_decode", "B": 4, "new": 1, "ctx": 4096, "Hkv": 8, "d": 128, "k": "prod3", "v": "prod3",
         "page": 64, "dtype": "bf16", "prep": "norm+half"},
        # a long prompt entering the cache
        {**append, "name": "append_prompt", "B": 1, "new": 16384, "Hkv": 8, "d": 128, "k": "prod3", "v": "prod3",
         "page": 64, "dtype": "bf16", "prep": "half"},
        # a batch of ragged prompts on small pages, half of each head rotated in neighbouring pairs
        {**append, "name": "append_ragged", "B": 24, "new": 701, "ctx": 333, "ragged": True, "Hkv": 4, "d": 128, "k": "mse4",
         "v": "mse4", "page": 16, "dtype": "fp16", "prep": "partial"},
        # an encoder's states entering the cache of a decoder's cross attention
        {**append, "name": "append_states", "B": 8, "new": 1200, "Hkv": 12, "d": 64, "k": "mse4", "v": "mse4", "page": 32,
         "dtype": "fp16"},
        # the first tokens of short conversations: latency alone
        {**attend, "name": "attend_short", "B": 2, "new": 1, "ctx": 200, "Hq": 32, "Hkv": 8, "d": 128, "k": "prod3",
         "v": "prod3", "page": 64, "dtype": "bf16", "prep": "half"},
        # one long conversation, one token
        {**attend, "name": "attend_token", "B": 1, "new": 1, "ctx": 32767, "Hq": 32, "Hkv": 8, "d": 128, "k": "prod3",
         "v": "prod3", "page": 64, "dtype": "bf16", "prep": "half"},
        # a full decode batch of conversations of all lengths
        {**attend, "name": "attend_tokens", "B": 32, "new": 1, "ctx": 16384, "ragged": True, "Hq": 32, "Hkv": 4, "d": 128,
         "k": "mse4", "v": "mse4", "page": 64, "dtype": "bf16", "prep": "norm+half"},
        # one chunk of a long prompt over what is cached of it
        {**attend, "name": "attend_chunk", "B": 1, "new": 1024, "ctx": 32768, "Hq": 32, "Hkv": 8, "d": 128, "k": "prod3",
         "v": "prod3", "page": 64, "dtype": "bf16", "prep": "half"},
        # whole prompts of several lengths, nothing cached before
        {**attend, "name": "attend_prompts", "B": 4, "new": 4096, "ragged": True, "ctx": 0, "Hq": 32, "Hkv": 8, "d": 128,
         "k": "mse4", "v": "mse4", "page": 128, "dtype": "fp16", "prep": "half"},
        # chunks and single tokens in one batch, a sliding window, fewer bits for the values
        {**attend, "name": "attend_mixed", "B": 14, "new": 513, "ctx": 8000, "ragged": True, "singles": 11, "Hq": 16, "Hkv": 2,
         "d": 128, "k": "mse4", "v": "mse2", "page": 16, "dtype": "bf16", "window": 4096},
        # decoder tokens, one for each sequence, over the states of an encoder
        {**cross, "name": "cross_tokens", "B": 16, "new": 1, "ctx": 1200, "Hq": 12, "Hkv": 12, "d": 64, "k": "mse4",
         "v": "mse4", "page": 32, "dtype": "fp16"},
        # whole targets over the states of an encoder, both of many lengths
        {**cross, "name": "cross_targets", "B": 8, "new": 449, "ctx": 1501, "ragged": True, "Hq": 12, "Hkv": 12, "d": 64,
         "k": "mse4", "v": "mse4", "page": 32, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("append", "attend", "attend", "cross"))
        d = 64 if op == "cross" else rng.choice((64, 128, 128))
        k, v = ("mse4", "mse4") if d == 64 else rng.choice((("prod3", "prod3"), ("mse4", "mse4"), ("mse4", "mse2")))
        G = 1 if op == "cross" else rng.choice((1, 2, 4, 8))
        Hkv = rng.choice((1, 2, 4, 8, 12))
        B = _log(rng, 1, 48)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        c = {"op": op, "B": B, "new": new, "ctx": _log(rng, 16, 2000 if op == "cross" else 32768),
             "ragged": rng.random() < 0.7, "singles": rng.randrange(B) if new > 1 and rng.random() < 0.3 else 0,
             "Hq": 0 if op == "append" else Hkv * G, "Hkv": Hkv, "d": d, "k": k, "v": v,
             "page": rng.choice((16, 32, 64, 128, 256)), "dtype": rng.choice(("bf16", "fp16")),
             "prep": "none" if op == "cross" else rng.choice(("none", "half", "norm+half", "partial")),
             "window": rng.choice((0, 0, 0, 512, 4096)) if op == "attend" else 0, "mix": rng.randrange(1 << 20)}
        n = [x[0] for x in lengths(c)]
        L = [x[1] for x in lengths(c)]
        slots = B * max(L) * Hkv
        if op == "append":
            fits = sum(n) * Hkv <= 16384 * 8 and slots <= 1 << 22
        else:
            fits = B * max(n) * max(L) * c["Hq"] <= 1.1e9 and slots <= 1 << 21 and sum(n) * c["Hq"] <= 1 << 19
        if fits:
            return c


def lengths(c):
    """[(new tokens, tokens in the cache after them)] of the sequences: fixed by the case."""
    r = random.Random(c["mix"])
    out = []
    for b in range(c["B"]):
        n = 1 if b < c["singles"] else c["new"]
        ctx = c["ctx"]
        if c["ragged"] and b != c["singles"]:  # one sequence has the full lengths
            n = r.randint(max(1, n // 8), n)
            ctx = r.randint(ctx // 8, ctx)
        out.append((n, max(1, ctx) if c["op"] == "cross" else ctx + n))
    return out


# ------------------------------------------------------------------ the quantizer's constants


@functools.lru_cache(maxsize=None)
def _rotation(d, m, seed):
    """Pi (the orthogonal factor of a seeded Gaussian matrix, diag(R) > 0) and the sign projections S, in 64 bits."""
    count = d * d + m * d
    i = np.arange(1, count + 2, dtype=np.uint64)
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + i * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    u = (z >> np.uint64(11)).astype(np.float64) * 2.0 ** -53
    a, b = u[0:count:2], u[1:count + 1:2]
    r = np.sqrt(-2.0 * np.log(1.0 - a))
    g = np.stack([r * np.cos(2 * np.pi * b), r * np.sin(2 * np.pi * b)], 1).reshape(-1)[:count]
    Q, R = np.linalg.qr(g[:d * d].reshape(d, d))
    return Q * np.sign(np.diag(R))[None, :], g[d * d:].reshape(m, d)


@functools.lru_cache(maxsize=None)
def _codebook(d, bits):
    """Lloyd-Max centroids and boundaries of one coordinate of a uniform unit vector, in 64 bits."""
    L, top = 1 << bits, min(1.0, 14.0 / math.sqrt(d))
    x, w = np.polynomial.legendre.leggauss(96)
    grid = np.linspace(-top, top, 200001)
    cum = np.cumsum((1 - grid ** 2) ** ((d - 3) / 2))
    c = np.interp((np.arange(L) + 0.5) / L, cum / cum[-1], grid)
    for _ in range(40000):
        e = np.concatenate([[-top], (c[1:] + c[:-1]) / 2, [top]])
        h, mid = (e[1:] - e[:-1]) / 2, (e[1:] + e[:-1]) / 2
        t = mid[:, None] + h[:, None] * x[None, :]
        p = (1 - t * t) ** ((d - 3) / 2) * w[None, :]
        c1 = (p * t).sum(1) / p.sum(1)
        c1 = (c1 - c1[::-1]) / 2
        moved = np.abs(c1 - c).max()
        c = c1
        if moved < 1e-16:
            break
    return c, (c[1:] + c[:-1]) / 2


def _format(fmt, d):
    return (2, d) if fmt == "prod3" else (int(fmt[3:]), 0)


@functools.lru_cache(maxsize=None)
def _constants(fmt, d, seed):
    """The constants of one quantizer on the GPU: Pi, S, M = S Pi^T, centroids, boundaries (64 bits)."""
    bits, m = _format(fmt, d)
    Pi, S = _rotation(d, m, seed)
    c, beta = _codebook(d, bits)
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return {"bits": bits, "m": m, "d": d, "Pi": on(Pi), "S": on(S), "M": on(S @ Pi.T), "c": on(c), "beta": on(beta)}


@functools.lru_cache(maxsize=None)
def _handle(fmt, d, seed):
    import embedding_vector_quantization_b200 as tq
    bits, m = _format(fmt, d)
    return tq.Handle(d, 3, seed, qjl_m=m) if m else tq.Handle(d, bits, seed, norm_dtype=tq.TQ_F16)


# ------------------------------------------------------------------ packed rows (LSB first)


def _pack(idx, bits):
    per = 8 // bits
    sh = torch.arange(per, device=idx.device, dtype=torch.int32) * bits
    return (idx.to(torch.int32).unflatten(-1, (-1, per)) << sh).sum(-1).to(torch.uint8)


def _unpack(codes, bits):
    sh = torch.arange(8 // bits, device=codes.device, dtype=torch.int32) * bits
    return ((codes.to(torch.int32).unsqueeze(-1) >> sh) & ((1 << bits) - 1)).flatten(-2)


# ------------------------------------------------------------------ state


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _heads(g, n, H, d, scale):
    """n vectors of H heads: log-normal channel scales and two outlier channels for each head."""
    return torch.randn(n, H, d, generator=g, device="cuda") * scale


def _scales(g, H, d):
    s = torch.exp(0.5 * torch.randn(H, d, generator=g, device="cuda"))
    at = torch.rand(H, d, generator=g, device="cuda").argsort(1)[:, :2]
    return s.scatter(1, at, s.gather(1, at) * 10)


def _quantize32(x, K):
    """Packed rows of vectors x [..., d] for a cache that is only read (32 bits are enough for its making)."""
    n = x.norm(dim=-1)
    y = (x @ K["Pi"].float().T) / n.unsqueeze(-1)
    idx = torch.bucketize(y, K["beta"].float())
    rows = {"codes": _pack(idx, K["bits"]), "norms": n.half()}
    if K["m"]:
        e = y - K["c"].float()[idx]
        rows["signs"] = _pack((e @ K["M"].float().T >= 0).to(torch.int32), 1)
        rows["rnorms"] = (n * e.norm(dim=-1)).half()
    return rows


def prepare(case, seed):
    c = case
    g = _gen(seed)
    lens = lengths(c)
    B, Hkv, d, ps = c["B"], c["Hkv"], c["d"], c["page"]
    n = torch.tensor([x[0] for x in lens], dtype=torch.int32)
    L = torch.tensor([x[1] for x in lens], dtype=torch.int32)
    ntok, pages_of = int(n.sum()), [-(-x[1] // ps) for x in lens]
    max_pages, total = max(pages_of), sum(pages_of)
    num_pages = total + 3
    order = torch.randperm(num_pages, generator=g, device="cuda")[:total].to(torch.int32).cpu()
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    for b, (at, k) in enumerate(zip(np.cumsum([0] + pages_of[:-1]), pages_of)):
        table[b, :k] = order[int(at):int(at) + k]
    start = torch.cat([torch.zeros(1, dtype=torch.int32), n.cumsum(0).to(torch.int32)])
    s = {"case": c, "ntok": ntok, "max_q": int(n.max()), "max_len": int(L.max()), "num_pages": num_pages,
         "start": start.cuda(), "len": L.cuda(), "table": table.cuda(),
         "K": _constants(c["k"], d, 0), "V": _constants(c["v"], d, 1), "scale": 1.0 / math.sqrt(d)}
    if "half" in c["prep"] or c["prep"] == "partial":
        rot = d // 2 if c["prep"] == "partial" else d
        f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        angle = torch.arange(MAX_POS, dtype=torch.float64)[:, None] * f
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    if "norm" in c["prep"]:
        s["weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(DTYPES[c["dtype"]])
    for name in ("K", "V"):
        Q, scale = s[name], _scales(g, Hkv, d)
        if c["op"] == "append":
            fill = lambda *z: torch.randint(0, 256, z, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
            shape = (num_pages, Hkv, ps)
            s[name + "cache"] = {"codes": fill(*shape, d * Q["bits"] // 8),
                                 "norms": torch.rand(shape, generator=g, device="cuda").half()}
            if Q["m"]:
                s[name + "cache"] |= {"signs": fill(*shape, Q["m"] // 8),
                                      "rnorms": torch.rand(shape, generator=g, device="cuda").half()}
            s["k" if name == "K" else "v"] = _heads(g, ntok, Hkv, d, scale).to(DTYPES[c["dtype"]])
        else:
            x = torch.cat([_heads(g, min(1 << 17, num_pages * ps - i), Hkv, d, scale) for i in range(0, num_pages * ps, 1 << 17)])
            rows = _quantize32(x, Q)
            s[name + "cache"] = {k: t.unflatten(0, (num_pages, ps)).transpose(1, 2).contiguous() for k, t in rows.items()}
            del x
    if c["op"] != "append":
        s["q"] = torch.randn(ntok, c["Hq"], d, generator=g, device="cuda").to(DTYPES[c["dtype"]])
        s["out"] = torch.empty_like(s["q"])
    if own:
        import embedding_vector_quantization_b200 as tq
        hk, hv = _handle(c["k"], d, 0), _handle(c["v"], d, 1)
        s["hk"], s["hv"] = hk, hv
        s["kc"] = tq.PagedCache(hk, num_pages, Hkv, ps, tensors=s["Kcache"])
        s["vc"] = tq.PagedCache(hv, num_pages, Hkv, ps, tensors=s["Vcache"])
        s["batch"] = tq.PagedBatch(s["start"], s["len"], s["table"], ntok, s["max_q"])
        s["head_prep"] = None
        if "cos_sin" in s or "weight" in s:
            s["head_prep"] = tq.HeadPrep(cos_sin=s.get("cos_sin"), interleaved=c["prep"] == "partial", weight=s.get("weight"),
                                         eps=1e-6)
        if c["op"] != "append":
            s["workspace"] = torch.empty(tq.tq_attn_paged_workspace_bytes(hk.ptr, hv.ptr, s["batch"], c["Hq"], Hkv, s["kc"].struct),
                                         dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _places(s):
    """Sequence and position in the cache of each token of the batch."""
    t = torch.arange(s["ntok"], device="cuda")
    seq = torch.searchsorted(s["start"][1:].long(), t, right=True)
    return seq, t - s["start"][1:].long()[seq] + s["len"].long()[seq]


def _prep(x, s, pos):
    """RMS norm of each head, then the rotation by the position; x [n, H, d] in the type to compute in."""
    if "weight" in s:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["weight"].to(x.dtype)
    if "cos_sin" in s:
        t = s["cos_sin"][pos].to(x.dtype).unsqueeze(1)
        rot = t.shape[-1]
        co, si = t[..., :rot // 2], t[..., rot // 2:]
        if s["case"]["prep"] == "partial":
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            x = torch.cat([torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2), x[..., rot:]], -1)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            x = torch.cat([a * co - b * si, b * co + a * si, x[..., rot:]], -1)
    return x


def _append_plain(x, Q, cache, page, slot):
    """Quantizes x [n, H, d] (64 bits: an index turns on which side of a border its coordinate lies) into its rows."""
    n = x.square().sum(-1).sqrt()
    y = x @ Q["Pi"].T / n.unsqueeze(-1)
    y = torch.where(n.unsqueeze(-1) > 0, y, torch.zeros_like(y))
    idx = torch.bucketize(y, Q["beta"])
    cache["codes"][page, :, slot] = _pack(idx, Q["bits"])
    cache["norms"][page, :, slot] = n.to(cache["norms"].dtype)
    if Q["m"]:
        e = y - Q["c"][idx]
        e = torch.where(n.unsqueeze(-1) > 0, e, torch.zeros_like(e))
        cache["signs"][page, :, slot] = _pack((e @ Q["M"].T >= 0).to(torch.int32), 1)
        cache["rnorms"][page, :, slot] = (n * e.square().sum(-1).sqrt()).to(cache["rnorms"].dtype)


def _dequantize(rows, Q):
    """The vectors that packed rows stand for, in 32 bits."""
    x = (Q["c"].float()[_unpack(rows["codes"], Q["bits"])] * rows["norms"].float().unsqueeze(-1)) @ Q["Pi"].float()
    if Q["m"]:
        w = rows["rnorms"].float() * (QJL / Q["m"])
        x = x + ((2 * _unpack(rows["signs"], 1) - 1).float() * w.unsqueeze(-1)) @ Q["S"].float()
    return x


def _attend_plain(s):
    c = s["case"]
    B, Hq, Hkv, d, ps = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    seq, pos = _places(s)
    q = _prep(s["q"].float(), s, pos)
    first = torch.arange(s["ntok"], device="cuda") - s["start"].long()[seq]
    rows = torch.zeros(B, s["max_q"], Hq, d, device="cuda")
    rows[seq, first] = q
    at = torch.zeros(B, s["max_q"], dtype=torch.long, device="cuda")
    at[seq, first] = pos
    key = torch.arange(s["max_len"], device="cuda")
    page = s["table"].long()[:, key // ps].clamp(min=0)
    get = lambda cache, Q: _dequantize({k: t[page, :, key % ps] for k, t in cache.items()}, Q).transpose(1, 2)  # noqa: E731
    k, v = get(s["Kcache"], s["K"]), get(s["Vcache"], s["V"])  # [B, Hkv, L, d]
    rows = rows.unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G Q, d]
    score = (rows @ k.transpose(-1, -2)).mul_(s["scale"]).unflatten(2, (-1, s["max_q"]))  # [B, Hkv, G, Q, L]
    seen = (key < s["len"].long()[:, None])[:, None].expand(-1, s["max_q"], -1)
    if c["op"] == "attend":
        seen = seen & (key <= at[..., None])
        if c["window"]:
            seen = seen & (key > at[..., None] - c["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top.isfinite(), top, torch.zeros_like(top))).exp_()
    o = (p.flatten(2, 3) @ v).unflatten(2, (-1, s["max_q"])) / p.sum(-1, keepdim=True).clamp(min=1e-37)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, Q, Hq, d]
    return o[seq, first].to(s["q"].dtype)


def _rows_of(s):
    return {"k_" + k: t for k, t in s["Kcache"].items()} | {"v_" + k: t for k, t in s["Vcache"].items()}


def run(state):
    s, c = state, state["case"]
    if own:
        import embedding_vector_quantization_b200 as tq
        if c["op"] == "append":
            tq.append_paged(s["hk"], s["hv"], s["k"], s["v"], s["kc"], s["vc"], s["batch"], prep=s["head_prep"])
        else:
            return tq.attn_paged(s["hk"], s["hv"], s["q"], s["kc"], s["vc"], s["batch"], s["scale"], causal=c["op"] == "attend",
                                 window=c["window"], prep=s["head_prep"], out=s["out"], workspace=s["workspace"])
    elif c["op"] == "append":
        seq, pos = _places(s)
        page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
        _append_plain(_prep(s["k"].double(), s, pos), s["K"], s["Kcache"], page, slot)
        _append_plain(s["v"].double(), s["V"], s["Vcache"], page, slot)
    else:
        return _attend_plain(s)
    return _rows_of(s)  # packed indices are whole numbers: equal bit for bit, in the old rows too


# ------------------------------------------------------------------ work and exact values


def _row_bytes(fmt, d):
    bits, m = _format(fmt, d)
    return d * bits // 8 + 2 + (m // 8 + 2 if m else 0)


def work(case):
    c, d = case, case["d"]
    lens = lengths(c)
    tokens = sum(n for n, _ in lens)
    kb, vb = _row_bytes(c["k"], d), _row_bytes(c["v"], d)
    table = 4 * d if "half" in c["prep"] else 2 * d if c["prep"] == "partial" else 0
    width = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "append":
        m = _format(c["k"], d)[1] + _format(c["v"], d)[1]
        return {"bytes": tokens * (c["Hkv"] * (2 * d * width + kb + vb) + table), "flops": tokens * c["Hkv"] * 2 * d * (2 * d + m)}
    pairs = keys = 0
    for n, L in lens:
        if c["op"] == "cross":
            pairs, keys = pairs + n * L, keys + L
        else:
            W = c["window"] or L
            full = [min(W, p + 1) for p in (L - n, L - 1)]
            ramp = max(0, min(L, W) - (L - n))  # queries that still see all before them
            pairs += sum(range(L - n + 1, L - n + 1 + min(n, ramp))) + (n - min(n, ramp)) * full[1]
            keys += min(L, W + n - 1)
    rows = tokens * c["Hq"]
    return {"bytes": rows * d * width * 2 + keys * c["Hkv"] * (kb + vb) + tokens * table, "flops": 4 * d * pairs * c["Hq"] + 4 * d * d * rows}


def exact(case, seed):
    s, c = prepare(case, seed), case
    start, L, table, ps, d = s["start"].tolist(), s["len"].tolist(), s["table"].long(), c["page"], c["d"]

    def turned(x, pos):  # each head's norm and rotation, as a rotation of complex numbers
        x = x.double()
        if "weight" in s:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + 1e-6) * s["weight"].double()
        if "cos_sin" in s:
            t = s["cos_sin"].double()[pos][:, None]
            rot = t.shape[-1]
            z = torch.complex(t[..., :rot // 2].contiguous(), t[..., rot // 2:].contiguous())
            pairs = x[..., :rot].unflatten(-1, (-1, 2)) if c["prep"] == "partial" else x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
            y = y if c["prep"] == "partial" else y.transpose(-1, -2)
            x = torch.cat([y.flatten(-2), x[..., rot:]], -1)
        return x

    if c["op"] == "append":
        out = {}
        for name, x, Q in (("k", s["k"], s["K"]), ("v", s["v"], s["V"])):
            cache = s[name.upper() + "cache"]
            out |= {name + "_" + k: None for k in cache}
            norms = cache["norms"].double()
            rnorms = cache["rnorms"].double() if Q["m"] else None
            for b in range(c["B"]):
                pos = torch.arange(L[b] - (start[b + 1] - start[b]), L[b], device="cuda")
                z = x[start[b]:start[b + 1]].double()
                z = turned(z, pos) if name == "k" else z
                page, slot = table[b, pos // ps], pos % ps
                norms[page, :, slot] = torch.linalg.vector_norm(z, dim=-1)
                if Q["m"]:  # the distance of each coordinate, in the norm's units, to the nearest centroid
                    y = torch.einsum("nhi,ji->nhj", z, Q["Pi"])
                    grid = torch.linalg.vector_norm(z, dim=-1)[..., None, None] * Q["c"]
                    rnorms[page, :, slot] = (y[..., None] - grid).abs().amin(-1).square().sum(-1).sqrt()
            out[name + "_norms"] = norms
            if Q["m"]:
                out[name + "_rnorms"] = rnorms
        return out
    out = torch.zeros(s["ntok"], c["Hq"], d, dtype=torch.float64, device="cuda")
    G = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        key = torch.arange(L[b], device="cuda")
        page, slot = table[b, key // ps], key % ps
        pos = torch.arange(L[b] - (start[b + 1] - start[b]), L[b], device="cuda")
        q = s["q"][start[b]:start[b + 1]]
        q = turned(q, pos if c["op"] == "attend" else pos.clamp(min=0))
        for h in range(c["Hkv"]):
            x = []
            for Q, cache in ((s["K"], s["Kcache"]), (s["V"], s["Vcache"])):
                y = torch.take(Q["c"], _unpack(cache["codes"][page, h, slot], Q["bits"]).long())
                y = y * cache["norms"][page, h, slot].double()[:, None]
                z = y @ Q["Pi"]
                if Q["m"]:
                    sign = torch.where(_unpack(cache["signs"][page, h, slot], 1) > 0, 1.0, -1.0).double()
                    z = z + (math.sqrt(math.pi / 2) / Q["m"]) * cache["rnorms"][page, h, slot].double()[:, None] * (sign @ Q["S"])
                x.append(z)
            a = torch.einsum("ngi,li->gnl", q[:, h * G:(h + 1) * G], x[0]) / math.sqrt(d)
            if c["op"] == "attend":
                off = pos[:, None] - key[None, :]
                hide = (off < 0) | (off >= c["window"]) if c["window"] else off < 0
                a = a.masked_fill(hide, -math.inf)
            out[start[b]:start[b + 1], h * G:(h + 1) * G] = torch.einsum("gnl,li->ngi", torch.softmax(a, -1), x[1])
    return out
