"""Paged caches for the tests: random page orders, garbage in every slot that no sequence owns, and the operators'
definitions in 64 bits.

Tolerance of an attention output, from the roundings on its way (h: half a step of the operands' type relative to a
value; independent roundings, six standard deviations, each bounded by its largest size h instead of h / sqrt(3)):

* a score moves by d_j = scale h sqrt(sum_i k'_ji^2 (2 sum_l Pi_il^2 z_l^2 + 2 q'_i^2)): the prepared query, Pi, the
  rotated query and the key's operand are each rounded once (k', q' in the rotated domain, the sign part likewise with S);
* a weight moves by d_j + 2 h relative (its own rounding, the value's operand), so an output by
  sqrt(sum_j p_j^2 v_ji^2) (max_j d_j + 2 h);
* the mapped-back sum o = Pi^T acc + c S^T acc_s: acc, Pi (and S) rounded once: 2 h sqrt(sum_j Pi_ji^2 acc_j^2);
* the output's own rounding: eps / 2 |o|, not a matter of chance and outside the factor of six.

The kernels for chunks expand the keys and values to the original basis first and leave queries and outputs there. Their
roundings are as many and as large: centroid, Pi (S), the expanded row and the prepared query, once each, move a score by
the same four terms, because Pi keeps lengths; the weights and the expanded values by 2 h; nothing is mapped back.

The general kernels keep everything in fp32; sums of n <= 512 products grow a rounding by at most sqrt(n) < 23: h = 23 / 2^24.
"""

import numpy as np
import torch

from oracle import codebook, rotation

QJL = float(np.sqrt(np.pi / 2))


class Format:
    """(MSE bits, projections) of a handle, its 64-bit constants and the package's handle."""

    def __init__(self, tq, d, bits, m, seed, norm="f16"):
        self.d, self.bits, self.m, self.seed = d, bits, m, seed
        Pi, S = rotation.rotation(d, seed, m)
        self.Pi = torch.from_numpy(np.ascontiguousarray(Pi)).cuda()
        self.S = torch.from_numpy(np.ascontiguousarray(S)).cuda() if m else None
        if bits:
            c, beta = codebook.lloyd_max(d, bits)
        else:
            c, beta = np.zeros(1), np.zeros(0)
        self.c, self.beta = torch.from_numpy(np.ascontiguousarray(c)).cuda(), torch.from_numpy(np.ascontiguousarray(beta)).cuda()
        dt = tq.TQ_F16 if norm == "f16" else tq.TQ_F32
        self.handle = tq.Handle(d, bits + 1, seed, qjl_m=m, norm_dtype=dt) if m else tq.Handle(d, bits, seed, norm_dtype=dt)

    def quantize(self, x):
        """idx, sigma, norm, residual norm of x [..., d] (64 bits)."""
        n = x.square().sum(-1).sqrt()
        y = torch.where(n[..., None] > 0, (x @ self.Pi.T) / n[..., None].clamp(min=1e-300), torch.zeros_like(x))
        idx = torch.bucketize(y, self.beta) if self.bits else torch.zeros_like(y, dtype=torch.long)
        if not self.m:
            return idx, None, n, None
        e = torch.where(n[..., None] > 0, y - self.c[idx], torch.zeros_like(y))
        sigma = (e @ (self.S @ self.Pi.T).T >= 0).long()
        return idx, sigma, n, n * e.square().sum(-1).sqrt()

    def rotated(self, idx, sigma, n, rn):
        """Rows in the rotated domain: n c[idx] and, for sign rows, the weighted signs."""
        a = n[..., None] * self.c[idx] if self.bits else torch.zeros(idx.shape, dtype=torch.float64, device=idx.device)
        if not self.m:
            return a, None
        w = (rn if self.bits else n) * (QJL / self.m)
        return a, w[..., None] * (2.0 * sigma - 1.0)


def pack(idx, bits):
    """LSB-first rows of bytes."""
    b = ((idx.long()[..., None] >> torch.arange(bits, device=idx.device)) & 1).flatten(-2)
    b = b.unflatten(-1, (-1, 8)) << torch.arange(8, device=idx.device)
    return b.sum(-1).to(torch.uint8)


def make_batch(tq, news, lens, page, seed=0, spare=2, max_pages=None, pad=0):
    """Block tables of random pages for sequences of lens[b] cached tokens, news[b] of them new."""
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-L // page)) for L in lens]
    num_pages = sum(need) + spare
    order = torch.randperm(num_pages, generator=g).to(torch.int32)
    max_pages = max_pages or max(1, max(need))
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    start = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32)
    ntok = int(start[-1]) + pad
    bt = tq.PagedBatch(start.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), ntok,
                       max(news) if news else 0)
    bt.num_pages, bt.page = num_pages, page
    bt.news, bt.lens = list(news), list(lens)
    return bt


def garbage_cache(tq, f, bt, Hkv, seed=0):
    """A cache whose every slot holds random bytes and NaN norms."""
    g = torch.Generator().manual_seed(1000 + seed)
    pc = tq.PagedCache(f.handle, bt.num_pages, Hkv, bt.page)
    for t in (pc.codes, pc.signs):
        if t is not None:
            t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for t in (pc.norms, pc.rnorms):
        if t is not None:
            t.fill_(float("nan"))
    return pc


def slots(bt, b, lo, hi):
    pos = torch.arange(lo, hi, device="cuda")
    return bt.block_table[b].long()[pos // bt.page], pos % bt.page


def fill_cache(pc, f, bt, xs):
    """Writes the 64-bit quantization of xs[b] [len_b, Hkv, d] into the pages; returns each sequence's stored rows."""
    rows = []
    for b, x in enumerate(xs):
        idx, sigma, n, rn = f.quantize(x)
        page, slot = slots(bt, b, 0, x.shape[0])
        n = n.to(pc.norms.dtype)
        pc.norms[page, :, slot] = n
        if pc.codes is not None:
            pc.codes[page, :, slot] = pack(idx, f.bits)
        if f.m:
            pc.signs[page, :, slot] = pack(sigma, 1)
            if pc.rnorms is not None:
                rn = rn.half()
                pc.rnorms[page, :, slot] = rn
        rows.append((idx, sigma, n.double(), None if rn is None else rn.double()))
    return rows


def prep_ref(x, prep, pos):
    """RMS norm and rotation in 64 bits; x [n, H, d], pos [n]."""
    if prep is None:
        return x
    if prep.weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + prep.struct.eps) * prep.weight.double()
    if prep.cos_sin is not None:
        t = prep.cos_sin.double()[pos][:, None]
        rot = t.shape[-1]
        co, si = t[..., :rot // 2], t[..., rot // 2:]
        if prep.struct.interleaved:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * co - b * si, a * si + b * co], -1)
        x = torch.cat([y, x[..., rot:]], -1)
    return x


def rope_table(max_pos, rot, seed=0):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def attention_ref(bt, q, fk, fv, krows, vrows, scale, causal, window, prep, h):
    """(out, tolerance without the output's own rounding) [tokens, Hq, d] of the tokens that are not padding."""
    outs, tols = [], []
    for b, n in enumerate(bt.news):
        t0, L = sum(bt.news[:b]), bt.lens[b]
        Hq, d = q.shape[1], q.shape[2]
        out = torch.zeros(n, Hq, d, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        pos = torch.arange(L - n, L, device="cuda")
        if n == 0 or L <= 0:
            outs.append(out), tols.append(tol)
            continue
        rp = prep.pos[t0:t0 + n].long() if prep is not None and prep.pos is not None else pos
        z = prep_ref(q[t0:t0 + n].double(), prep, rp.clamp(min=0))
        ka, kb = fk.rotated(*krows[b])
        va, vb = fv.rotated(*vrows[b])
        G = Hq // ka.shape[1]
        key = torch.arange(L, device="cuda")
        seen = torch.ones(n, L, dtype=torch.bool, device="cuda")
        if causal:
            seen = key[None] <= pos[:, None]
            if window:
                seen &= key[None] > pos[:, None] - window
        for hq in range(Hq):
            hk = hq // G
            zz = z[:, hq]
            q1 = zz @ fk.Pi.T
            s = q1 @ ka[:, hk].T
            var = (2 * zz.square() @ fk.Pi.square().T + 2 * q1.square()) @ ka[:, hk].square().T
            if kb is not None:
                q2 = zz @ fk.S.T
                s = s + q2 @ kb[:, hk].T
                var = var + (2 * zz.square() @ fk.S.square().T + 2 * q2.square()) @ kb[:, hk].square().T
            s = (s * scale).masked_fill(~seen, -torch.inf)
            dev = (var.sqrt() * scale * h).masked_fill(~seen, 0).amax(1)
            top = s.amax(1, keepdim=True)
            p = torch.exp(s - torch.where(top.isfinite(), top, torch.zeros_like(top)))
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
            acc = p @ va[:, hk]
            v = va[:, hk] @ fv.Pi
            o = acc @ fv.Pi
            back = 2 * acc.square() @ fv.Pi.square()
            if vb is not None:
                acc_s = p @ vb[:, hk]
                v = v + vb[:, hk] @ fv.S
                o = o + acc_s @ fv.S
                back = back + 2 * acc_s.square() @ fv.S.square()
            out[:, hq] = o
            # the values' two parts are rounded apart: their spread is taken in the rotated domain
            spread = (p.square() @ va[:, hk].square()) @ fv.Pi.square()
            if vb is not None:
                spread = spread + (p.square() @ vb[:, hk].square()) @ fv.S.square()
            spread = torch.maximum(spread, p.square() @ v.square())
            tol[:, hq] = 6 * (spread.sqrt() * (dev[:, None] + 2 * h) + h * back.sqrt())
        outs.append(out), tols.append(tol)
    return torch.cat(outs), torch.cat(tols)


def check_attention(got, ref, tol, dtype):
    """Largest |got - ref| over its tolerance (at most 1 passes); prints nothing."""
    eps = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny
    room = tol + eps * (ref.abs() + tol) + tiny
    worst = ((got.double() - ref).abs() / room).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"largest error is {worst:.3g} of its tolerance"
    return worst
