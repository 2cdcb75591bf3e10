"""Paged caches: append of ragged batches and attention of chunks, single tokens and cross attention, against 64 bits."""

import numpy as np
import pytest
import torch

from conftest import build_lib
import paged_util as pu

pytestmark = pytest.mark.gpu

H_FP32 = 23 * 2.0 ** -24   # the general kernels, fp32 throughout
H_F16 = 2.0 ** -11         # half a step of the f16 operands

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tq():
    return build_lib()


_formats = {}


def fmt(tq, d, name, seed, norm="f16"):
    """"mseB", "prodB" (B - 1 MSE bits, d signs), "qjl" (signs alone), "prodBxM" (M signs)."""
    key = (d, name, seed, norm)
    if key not in _formats:
        if name == "qjl":
            bits, m = 0, d
        elif name.startswith("prod"):
            b, _, m = name[4:].partition("x")
            bits, m = int(b) - 1, int(m or d)
        else:
            bits, m = int(name[3:]), 0
        _formats[key] = pu.Format(tq, d, bits, m, seed, norm)
    return _formats[key]


def heads(seed, n, H, d, dtype=torch.float64, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, H, d, generator=g, dtype=torch.float64)
    if outliers:
        x = x * torch.exp(0.5 * torch.randn(H, d, generator=g, dtype=torch.float64))
    return x.to(dtype).cuda()


def make_prep(tq, kind, d, dtype, max_pos=4096, seed=0, pos=None):
    if kind == "none":
        return None
    w = None
    if "norm" in kind:
        w = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()
    rot = d // 2 if "partial" in kind else d
    table = pu.rope_table(max_pos, rot) if "half" in kind or "partial" in kind else None
    return tq.HeadPrep(cos_sin=table, interleaved="partial" in kind, weight=w, eps=1e-5, pos=pos)


# ------------------------------------------------------------------ append

APPEND = [
    # d, keys, values, Hkv, new tokens, cached after, page, dtype, prep
    (128, "prod3", "prod3", 8, [1], [1], 64, "bf16", "norm+half"),
    (128, "prod3", "prod3", 8, [1, 1, 1, 1], [7, 64, 65, 1000], 64, "bf16", "half"),
    (128, "prod3", "mse4", 2, [5, 0, 129, 1], [5, 9, 300, 17], 16, "fp16", "partial"),
    (128, "mse4", "mse2", 4, [33, 64, 31], [40, 64, 100], 32, "fp32", "norm"),
    (128, "mse3", "mse1", 3, [70], [71], 16, "bf16", "half"),
    (128, "qjl", "prod2", 1, [19, 2], [19, 2], 48, "bf16", "none"),
    (64, "mse4", "mse4", 12, [257, 3], [300, 3], 32, "fp16", "none"),
    (64, "prod4", "prod3", 2, [40], [41], 16, "bf16", "norm+partial"),
    (32, "mse2", "prod5x64", 1, [9], [9], 16, "fp32", "half"),
    (96, "prod3x32", "mse3", 2, [50, 1], [50, 1], 16, "bf16", "half"),
    (256, "mse4", "mse3", 2, [37], [90], 16, "bf16", "norm+half"),
    (160, "mse2", "mse4", 1, [8], [8], 1024, "fp16", "half"),
    (128, "prod3", "prod3", 4, [700, 413], [700, 1413], 64, "bf16", "norm+half"),
    (128, "mse4", "mse4", 4, [1000], [1000], 128, "fp16", "half"),
]


def run_append(tq, fk, fv, bt, k, v, prep, Hkv, stream=None, call=None):
    kc, vc = pu.garbage_cache(tq, fk, bt, Hkv, 1), pu.garbage_cache(tq, fv, bt, Hkv, 2)
    (call or tq.append_paged)(fk.handle, fv.handle, k, v, kc, vc, bt, prep=prep, stream=stream)
    return kc, vc


def expected_cache(tq, f, bt, Hkv, seed, x, prep):
    """The garbage cache with the batch's rows written by the 64-bit definition."""
    want = pu.garbage_cache(tq, f, bt, Hkv, seed)
    for b, n in enumerate(bt.news):
        t0, L = sum(bt.news[:b]), bt.lens[b]
        pos = torch.arange(L - n, L, device="cuda")
        rp = prep.pos[t0:t0 + n].long() if prep is not None and prep.pos is not None else pos
        z = pu.prep_ref(x[t0:t0 + n].double(), prep, rp)
        idx, sigma, nn, rn = f.quantize(z)
        page, slot = pu.slots(bt, b, L - n, L)
        want.norms[page, :, slot] = nn.to(want.norms.dtype)
        if want.codes is not None:
            want.codes[page, :, slot] = pu.pack(idx, f.bits)
        if f.m:
            want.signs[page, :, slot] = pu.pack(sigma, 1)
        if want.rnorms is not None:
            want.rnorms[page, :, slot] = rn.half()
    return want


def check_cache(got, want):
    """Indices and signs bit for bit; norms to one rounding (their sum may be one step off the exact one); the rest untouched."""
    for name in ("codes", "signs"):
        a, b = getattr(got, name), getattr(want, name)
        if b is not None:
            assert torch.equal(a, b), f"{name}: {(a != b).sum().item()} bytes differ"
    for name in ("norms", "rnorms"):
        a, b = getattr(got, name), getattr(want, name)
        if b is None:
            continue
        assert torch.equal(a.isnan(), b.isnan()), name
        ok = ~b.isnan()
        # half a step from the exact value on each side, so at most one step apart
        assert ((a[ok].double() - b[ok].double()).abs() <= torch.finfo(a.dtype).eps * b[ok].double().abs() + 1e-7).all(), name


@pytest.mark.parametrize("d,kf,vf,Hkv,news,lens,page,dtype,prep", APPEND)
def test_append(tq, d, kf, vf, Hkv, news, lens, page, dtype, prep):
    fk, fv = fmt(tq, d, kf, 0), fmt(tq, d, vf, 1, "f32" if vf == "mse2" else "f16")
    bt = pu.make_batch(tq, news, lens, page, seed=d)
    k, v = heads(2, bt.ntok, Hkv, d, DT[dtype]), heads(3, bt.ntok, Hkv, d, DT[dtype])
    pr = make_prep(tq, prep, d, DT[dtype])
    kc, vc = run_append(tq, fk, fv, bt, k, v, pr, Hkv)
    assert fk.handle.status() == tq.TQ_OK
    check_cache(kc, expected_cache(tq, fk, bt, Hkv, 1, k, pr))
    check_cache(vc, expected_cache(tq, fv, bt, Hkv, 2, v, None))


@pytest.mark.parametrize("d,kf,vf", [(64, "mse4", "prod3"), (128, "prod3", "mse4"), (256, "mse4", "mse2"), (96, "prod3x32", "mse3")])
@pytest.mark.parametrize("n", [73, 75, 147, 149])
def test_append_around_the_kernels_borders(tq, d, kf, vf, n):
    """One row to a CTA, eight, or tiles for the tensor cores: the same indices and signs."""
    fk, fv = fmt(tq, d, kf, 0), fmt(tq, d, vf, 1)
    bt = pu.make_batch(tq, [n], [n + 5], 32)
    k, v = heads(11, n, 1, d, torch.bfloat16), heads(12, n, 1, d, torch.bfloat16)
    pr = make_prep(tq, "norm+half", d, torch.bfloat16)
    kc, vc = run_append(tq, fk, fv, bt, k, v, pr, 1)
    assert fk.handle.status() == tq.TQ_OK
    check_cache(kc, expected_cache(tq, fk, bt, 1, 1, k, pr))
    check_cache(vc, expected_cache(tq, fv, bt, 1, 2, v, None))


def test_append_pieces_give_the_same_bytes(tq):
    """A prompt appended at once, in chunks and token by token: the same indices and signs; norms at most one step apart
    (the kernels sum their squares in different orders and precisions)."""
    fk, fv = fmt(tq, 128, "prod3", 0), fmt(tq, 128, "mse4", 1)
    n, Hkv, page = 300, 4, 64
    k, v = heads(5, n, Hkv, 128, torch.bfloat16), heads(6, n, Hkv, 128, torch.bfloat16)
    pr = make_prep(tq, "norm+half", 128, torch.bfloat16)
    whole = pu.make_batch(tq, [n], [n], page)
    kc, vc = run_append(tq, fk, fv, whole, k, v, pr, Hkv)
    for cuts in ([0, 129, 130, 300], list(range(0, 301, 1))):
        k2, v2 = pu.garbage_cache(tq, fk, whole, Hkv, 1), pu.garbage_cache(tq, fv, whole, Hkv, 2)
        for a, b in zip(cuts[:-1], cuts[1:]):
            bt = tq.PagedBatch(torch.tensor([0, b - a], dtype=torch.int32).cuda(), torch.tensor([b], dtype=torch.int32).cuda(),
                               whole.block_table, b - a)
            tq.append_paged(fk.handle, fv.handle, k[a:b], v[a:b], k2, v2, bt, prep=pr)
        for x, y in ((kc, k2), (vc, v2)):
            check_cache(x, y)


def test_append_zero_and_tiny_vectors(tq):
    """Zero vectors get norm 0, the lower middle cell and every sign set; vectors far from unit length keep their codes."""
    for kf in ("prod3", "mse4", "mse1"):
        fk, fv = fmt(tq, 128, kf, 0, "f32" if kf != "prod3" else "f16"), fmt(tq, 128, "prod3", 1)
        bt = pu.make_batch(tq, [6], [6], 16)
        k = heads(7, 6, 2, 128, torch.float32)
        k[0] = 0
        k[1] *= 1e-6
        k[2] *= 1e3
        k[3, :, 1:] = 0
        v = k.flip(0).contiguous()
        kc, vc = run_append(tq, fk, fv, bt, k, v, None, 2)
        check_cache(kc, expected_cache(tq, fk, bt, 2, 1, k, None))
        check_cache(vc, expected_cache(tq, fv, bt, 2, 2, v, None))


@pytest.mark.parametrize("n", [4, 1200])
def test_append_layouts_positions_padding(tq, n):
    """Slices of one projection's output, odd strides, explicit rotation positions, rows of padding."""
    fk, fv = fmt(tq, 128, "mse4", 0), fmt(tq, 128, "mse4", 1)
    Hkv, pad = 2, 3
    bt = pu.make_batch(tq, [n - 1, 1], [n + 4, 9], 32, pad=pad)
    qkv = heads(8, bt.ntok, 8 + 2 * Hkv, 128, torch.bfloat16)
    pos = torch.randint(0, 4096, (bt.ntok,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    pr = make_prep(tq, "half", 128, torch.bfloat16, pos=pos)
    pos[-pad:] = -5   # the padding's positions are not read
    k, v = qkv[:, 8:8 + Hkv], qkv[:, 8 + Hkv:]
    k[-pad:] = float("nan")
    kc, vc = run_append(tq, fk, fv, bt, k, v, pr, Hkv)
    assert fk.handle.status() == tq.TQ_OK
    check_cache(kc, expected_cache(tq, fk, bt, Hkv, 1, k, pr))
    check_cache(vc, expected_cache(tq, fv, bt, Hkv, 2, v, None))
    odd = torch.empty(bt.ntok, Hkv * 128 + 3, dtype=torch.bfloat16, device="cuda")[:, 1:1 + Hkv * 128].unflatten(1, (Hkv, 128))
    odd.copy_(k)
    k2, v2 = run_append(tq, fk, fv, bt, odd, v.transpose(0, 1).contiguous().transpose(0, 1), pr, Hkv)
    assert torch.equal(k2.codes, kc.codes) and torch.equal(v2.codes, vc.codes)


@pytest.mark.parametrize("n", [3, 1100])
def test_append_bad_places_are_skipped(tq, n):
    """Tokens past the table, on bad pages or without a rotation row are recorded and skipped; the others are written."""
    fk, fv = fmt(tq, 128, "prod3", 0), fmt(tq, 128, "prod3", 1)
    Hkv = 2
    bt = pu.make_batch(tq, [n, n], [n, n], 16)
    k, v = heads(9, bt.ntok, Hkv, 128, torch.bfloat16), heads(10, bt.ntok, Hkv, 128, torch.bfloat16)
    good = run_append(tq, fk, fv, bt, k, v, None, Hkv)
    assert fk.handle.status() == tq.TQ_OK
    for wrong in (-1, bt.num_pages, 2 ** 31 - 1):
        t = bt.block_table.clone()
        t[1, 0] = wrong
        bad = tq.PagedBatch(bt.q_start, bt.len, t, bt.ntok)
        bad.num_pages, bad.page = bt.num_pages, bt.page
        kc, vc = run_append(tq, fk, fv, bad, k, v, None, Hkv)
        assert fk.handle.status() == tq.TQ_EINVAL and fk.handle.status() == tq.TQ_OK
        page = int(bt.block_table[1, 0])
        for got, want, f, seed in ((kc, good[0], fk, 1), (vc, good[1], fv, 2)):
            old = pu.garbage_cache(tq, f, bt, Hkv, seed)
            keep = torch.arange(bt.num_pages, device="cuda") != page
            assert torch.equal(got.codes[keep], want.codes[keep]) and torch.equal(got.codes[~keep], old.codes[~keep])
            assert torch.equal(got.signs[keep], want.signs[keep]) and got.norms[~keep].isnan().all()
    long = tq.PagedBatch(bt.q_start, bt.len + 16 * bt.block_table.shape[1], bt.block_table, bt.ntok)
    long.num_pages, long.page = bt.num_pages, bt.page
    kc, vc = run_append(tq, fk, fv, long, k, v, None, Hkv)
    assert fk.handle.status() == tq.TQ_EINVAL and kc.norms.isnan().all() and vc.norms.isnan().all()
    short = make_prep(tq, "half", 128, torch.bfloat16, max_pos=2)
    kc, vc = run_append(tq, fk, fv, bt, k, v, short, Hkv)
    assert fk.handle.status() == tq.TQ_EINVAL
    assert int((~kc.norms.isnan()).sum()) == int((~vc.norms.isnan()).sum()) == 2 * 2 * Hkv
    negative = tq.PagedBatch(bt.q_start, bt.len - 1, bt.block_table, bt.ntok)
    negative.num_pages, negative.page = bt.num_pages, bt.page
    run_append(tq, fk, fv, negative, k, v, None, Hkv)
    assert fk.handle.status() == tq.TQ_EINVAL


# ------------------------------------------------------------------ attention


def attention_case(tq, d, kf, vf, Hkv, G, news, lens, page, dtype, prep="none", causal=True, window=0, seed=0, pad=0,
                   spread=True, **batch):
    fk, fv = fmt(tq, d, kf, 0), fmt(tq, d, vf, 1)
    bt = pu.make_batch(tq, news, lens, page, seed=seed, pad=pad, **batch)
    kc, vc = pu.garbage_cache(tq, fk, bt, Hkv, 1), pu.garbage_cache(tq, fv, bt, Hkv, 2)
    kr = pu.fill_cache(kc, fk, bt, [heads(100 + b, max(0, L), Hkv, d) for b, L in enumerate(lens)])
    vr = pu.fill_cache(vc, fv, bt, [heads(200 + b, max(0, L), Hkv, d) for b, L in enumerate(lens)])
    q = heads(seed + 300, bt.ntok, Hkv * G, d, DT[dtype], outliers=False)
    pr = make_prep(tq, prep, d, DT[dtype], max_pos=max(4096, max(lens) + 1))
    return fk, fv, bt, kc, vc, kr, vr, q, pr


def check_case(tq, c, scale, causal, window, h, **kw):
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, scale, causal=causal, window=window, prep=pr, **kw)
    assert fk.handle.status() == tq.TQ_OK
    ref, tol = pu.attention_ref(bt, q, fk, fv, kr, vr, scale, causal, window, pr, h)
    used = ref.shape[0]
    assert not got[:used].isnan().any()
    pu.check_attention(got[:used], ref, tol, q.dtype)
    return got


ATTN = [
    # d, keys, values, Hkv, G, new, cached, page, prep, causal, window
    (128, "prod3", "prod3", 2, 4, [1], [1], 16, "none", True, 0),
    (128, "prod3", "prod3", 2, 4, [1, 1, 1], [5, 64, 700], 64, "half", True, 0),
    (128, "prod3", "prod3", 1, 4, [1], [5000], 64, "half", True, 0),
    (128, "mse4", "mse4", 2, 8, [1, 1, 1, 1], [129, 1, 2048, 127], 16, "norm+half", True, 0),
    (128, "mse4", "mse4", 2, 1, [2, 1, 3], [129, 1, 200], 48, "half", True, 0),
    (128, "mse4", "mse2", 2, 4, [130, 0, 1, 33], [400, 10, 77, 33], 16, "none", True, 0),
    (128, "mse4", "mse2", 2, 8, [70, 1, 1], [1000, 600, 3], 16, "partial", True, 100),
    (128, "prod3", "prod3", 2, 4, [200, 1], [519, 300], 64, "norm+half", True, 0),
    (128, "prod3", "prod3", 1, 4, [64], [64], 128, "half", True, 16),
    (128, "mse2", "mse2", 1, 2, [300], [301], 256, "none", True, 0),
    (128, "mse3", "mse1", 1, 3, [17], [80], 16, "half", True, 0),
    (128, "prod3", "mse4", 2, 4, [40, 1], [600, 90], 32, "half", True, 0),
    (128, "mse4", "prod3", 2, 4, [40, 1], [600, 90], 32, "half", True, 0),
    (64, "mse4", "mse4", 3, 1, [1, 1], [60, 333], 32, "none", False, 0),
    (64, "mse4", "mse4", 3, 1, [100, 7, 1], [150, 444, 1], 32, "none", False, 0),
    (64, "mse4", "mse4", 2, 4, [100, 7], [150, 444], 32, "half", True, 0),
    (64, "prod3", "prod3", 1, 4, [30, 1], [200, 500], 16, "norm+half", True, 0),
    (128, "prod3", "prod3", 1, 4, [5, 300, 1], [0, 12, 700], 64, "none", False, 0),   # more queries than states; no states
    (128, "mse4", "mse4", 1, 4, [5, 30, 1], [2, 0, 0], 16, "none", True, 0),          # rows before the first position
    (128, "mse4", "mse4", 1, 1, [1], [9000], 1024, "none", True, 1),
    (32, "mse2", "prod2x64", 2, 2, [9, 1], [50, 70], 16, "half", True, 0),
    (96, "qjl", "mse3", 2, 1, [20], [33], 16, "none", True, 0),
    (256, "mse4", "mse4", 1, 4, [21, 1], [99, 400], 16, "half", True, 0),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("d,kf,vf,Hkv,G,news,lens,page,prep,causal,window", ATTN)
def test_attention(tq, d, kf, vf, Hkv, G, news, lens, page, prep, causal, window, dtype):
    c = attention_case(tq, d, kf, vf, Hkv, G, news, lens, page, dtype, prep, causal, window)
    check_case(tq, c, 1 / np.sqrt(d), causal, window, H_FP32 if dtype == "fp32" else H_F16)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_padding_keeps_out(tq, dtype):
    """Rows of padding are not written, whatever they held; workspaces may be larger than needed and hold anything."""
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, [3, 0, 140], [60, 5, 300], 16, dtype, "half", pad=5)
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    q[-5:] = float("nan")
    out = torch.full_like(q, float("nan"))
    size = tq.tq_attn_paged_workspace_bytes(fk.handle.ptr, fv.handle.ptr, bt.struct, 8, 2, kc.struct)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    got = check_case(tq, c, 0.09, True, 0, H_FP32 if dtype == "fp32" else H_F16, out=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr() and got[-5:].isnan().all()
    guard = torch.full((size + 256,), 77, dtype=torch.uint8, device="cuda")
    again = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, prep=pr, workspace=guard[:size])
    assert torch.equal(again[:-5], got[:-5]) and (guard[size:] == 77).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("news", [[1, 1], [150, 3]])
def test_attention_large_values(tq, news, dtype):
    """Norms and queries far from one: 1e-3, 1e3 and 3e4 times the usual; weights spread over the whole range."""
    for ks, qs, vs in ((1e-3, 1.0, 1e-3), (300.0, 0.01, 1e3), (1.0, 3e4, 100.0)):
        fk, fv = fmt(tq, 128, "prod3", 0), fmt(tq, 128, "mse4", 1)
        lens = [300, 77]
        bt = pu.make_batch(tq, news, lens, 32)
        kc, vc = pu.garbage_cache(tq, fk, bt, 2, 1), pu.garbage_cache(tq, fv, bt, 2, 2)
        kr = pu.fill_cache(kc, fk, bt, [heads(1 + b, L, 2, 128) * ks for b, L in enumerate(lens)])
        g = torch.Generator().manual_seed(4)
        vr = pu.fill_cache(vc, fv, bt, [heads(5 + b, L, 2, 128) * vs * torch.exp2(-8 * torch.rand(L, 2, 1, generator=g).double()).cuda()
                                        for b, L in enumerate(lens)])
        q = (heads(8, bt.ntok, 8, 128, outliers=False) * qs).to(DT[dtype])
        scale = 0.3 / (ks * qs * 128 ** 0.5)
        check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, None), scale, True, 0, H_FP32 if dtype == "fp32" else H_F16)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention_bad_pages(tq, dtype):
    """Keys on a page out of range are not seen; the call records it and the others stay right."""
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, [1, 40, 1], [100, 60, 90], 16, dtype)
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    want = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09)
    for wrong in (-1, bt.num_pages, -2 ** 31):
        t = bt.block_table.clone()
        t[0, 2] = wrong
        bad = tq.PagedBatch(bt.q_start, bt.len, t, bt.ntok)
        got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bad, 0.09)
        assert fk.handle.status() == tq.TQ_EINVAL and fk.handle.status() == tq.TQ_OK
        assert torch.equal(got[1:], want[1:])
        # the first sequence without those sixteen keys
        keep = [i for i in range(100) if i // 16 != 2]
        cut = pu.make_batch(tq, [1], [84], 16)
        k2, v2 = pu.garbage_cache(tq, fk, cut, 2, 1), pu.garbage_cache(tq, fv, cut, 2, 2)
        page, slot = pu.slots(cut, 0, 0, 84)
        src, sl = pu.slots(bt, 0, 0, 100)
        for a, b in ((k2, kc), (v2, vc)):
            a.codes[page, :, slot] = b.codes[src, :, sl][keep]
            a.norms[page, :, slot] = b.norms[src, :, sl][keep]
        cutq = tq.attn_paged(fk.handle, fv.handle, q[:1].contiguous(), k2, v2, cut, 0.09)
        tol = 1e-5 if dtype == "fp32" else 2.0 ** -7   # the same roundings in another order
        assert (got[:1].double() - cutq.double()).abs().max() <= tol * want[:1].double().abs().max()
    over = tq.PagedBatch(bt.q_start, bt.len + 16 * bt.block_table.shape[1], bt.block_table, bt.ntok)
    tq.attn_paged(fk.handle, fv.handle, q, kc, vc, over, 0.09)   # lengths past the table: what the table has is seen
    fk.handle.status()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("news", [[1, 2], [60, 1]])
def test_attention_rotation_out_of_range(tq, news, dtype):
    """A query whose rotation position is not in the table gets zeros (recorded); the others are untouched."""
    c = attention_case(tq, 128, "mse4", "mse4", 1, 4, news, [100, 90], 16, dtype, "half")
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    pos = torch.randint(0, 4096, (bt.ntok,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    good = tq.HeadPrep(cos_sin=pr.cos_sin, pos=pos)
    want = check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, good), 0.09, False, 0, H_FP32 if dtype == "fp32" else H_F16)
    for wrong in (-1, 4096, 2 ** 31 - 1, -2 ** 31):
        p2 = pos.clone()
        p2[1] = wrong
        got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, causal=False, prep=tq.HeadPrep(cos_sin=pr.cos_sin, pos=p2))
        assert fk.handle.status() == tq.TQ_EINVAL and fk.handle.status() == tq.TQ_OK
        keep = torch.arange(bt.ntok) != 1
        assert (got[1] == 0).all() and torch.equal(got[keep.cuda()], want[keep.cuda()])


@pytest.mark.parametrize("kf,vf,kn,vn", [("mse4", "mse4", "f32", "f32"), ("prod3", "prod3", "f32", "f32"), ("mse4", "mse2", "f32", "f16"),
                                         ("prod3", "prod3", "f16", "f32"), ("mse2", "mse2", "f32", "f32")])
def test_attention_norm_types(tq, kf, vf, kn, vn):
    """fp32 norms, and keys' and values' norms of different types."""
    fk, fv = fmt(tq, 128, kf, 0, kn), fmt(tq, 128, vf, 1, vn)
    for news, lens in (([1, 2, 1], [300, 77, 1700]), ([130, 1], [400, 900])):
        bt = pu.make_batch(tq, news, lens, 48)
        kc, vc = pu.garbage_cache(tq, fk, bt, 2, 1), pu.garbage_cache(tq, fv, bt, 2, 2)
        kr = pu.fill_cache(kc, fk, bt, [heads(1 + b, L, 2, 128) for b, L in enumerate(lens)])
        vr = pu.fill_cache(vc, fv, bt, [heads(9 + b, L, 2, 128) for b, L in enumerate(lens)])
        q = heads(8, bt.ntok, 8, 128, torch.bfloat16, outliers=False)
        check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, None), 0.09, True, 0, H_F16)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [-0.08, 0.0])
def test_attention_scale(tq, scale, dtype):
    """A negative scale turns the order of the scores round, a scale of zero averages."""
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, [1, 70], [200, 150], 16, dtype)
    check_case(tq, c, scale, True, 0, H_FP32 if dtype == "fp32" else H_F16)


@pytest.mark.parametrize("G", [3, 16, 40])
def test_attention_group_sizes(tq, G):
    for news, lens in (([1, 1], [77, 300]), ([50, 1], [60, 300])):
        c = attention_case(tq, 128, "mse4", "mse4", 1, G, news, lens, 16, "bf16", "half")
        check_case(tq, c, 0.09, True, 0, H_F16)


EIGHTS = [
    # d, keys, values, Hkv, G, new, cached, page, prep, causal, window: 9 to 32 (16 with signs) rows for some sequences
    (128, "mse4", "mse4", 2, 4, [4, 1, 8, 3], [40, 700, 3000, 3], 16, "half", True, 0),
    (128, "mse4", "mse2", 2, 8, [2, 4, 1], [1500, 1537, 129], 64, "norm+half", True, 0),
    (128, "mse2", "mse2", 1, 3, [7, 10, 2], [900, 2500, 64], 32, "none", True, 50),
    (128, "prod3", "prod3", 2, 16, [1, 1], [77, 2000], 32, "half", True, 0),
    (128, "prod3", "prod3", 2, 5, [3, 2, 1], [300, 1700, 9], 16, "partial", True, 200),
    (64, "prod3", "prod3", 1, 4, [4, 3], [90, 4000], 256, "half", True, 0),
    (64, "mse4", "mse4", 3, 1, [32, 9, 17, 33, 200], [1500, 16, 444, 800, 1000], 32, "none", False, 0),
    (64, "mse4", "mse4", 12, 1, [17, 25], [600, 1536], 16, "none", False, 0),
    (128, "mse4", "mse4", 1, 32, [1, 1], [31, 5000], 48, "half", True, 1000),
    (128, "mse4", "mse4", 2, 4, [8, 5, 0, 6], [3, 0, 4, 6], 16, "none", True, 0),   # rows before the first position, no keys
    (128, "mse4", "mse4", 2, 4, [7, 100, 1, 5], [4000, 400, 1, 5], 16, "half", True, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,kf,vf,Hkv,G,news,lens,page,prep,causal,window", EIGHTS)
def test_attention_of_several_eights_of_rows(tq, d, kf, vf, Hkv, G, news, lens, page, prep, causal, window, dtype):
    c = attention_case(tq, d, kf, vf, Hkv, G, news, lens, page, dtype, prep, causal, window)
    check_case(tq, c, 1 / np.sqrt(d), causal, window, H_F16)


def test_eights_of_rows_stay_in_their_workspace(tq):
    """A batch with more tokens than max_q in a sequence: nothing is written behind the workspace or in other sequences' rows."""
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, [2, 6, 1], [700, 900, 30], 16, "bf16")
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    less = tq.PagedBatch(bt.q_start, bt.len, bt.block_table, bt.ntok, 2)
    size = tq.tq_attn_paged_workspace_bytes(fk.handle.ptr, fv.handle.ptr, less.struct, 8, 2, kc.struct)
    guard = torch.full((size + 65536,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    tq.attn_paged(fk.handle, fv.handle, q, kc, vc, less, 0.09, out=out, workspace=guard[:size])
    fk.handle.status()
    assert (guard[size:] == 77).all()
    ref, tol = pu.attention_ref(bt, q, fk, fv, kr, vr, 0.09, True, 0, None, H_F16)
    for rows in (slice(0, 2), slice(8, 9)):
        pu.check_attention(out[rows], ref[rows], tol[rows], q.dtype)


@pytest.mark.parametrize("B", [300, 2100])
def test_attention_many_sequences(tq, B):
    """More sequences than CTAs, than threads, than the single-token kernel takes."""
    lens = [1 + (7 * b) % 40 for b in range(B)]
    news = [1 + (b % 3 == 0) * min(1, lens[b] - 1) for b in range(B)]
    c = attention_case(tq, 64, "mse4", "mse4", 2, 2, news, lens, 16, "fp16")
    check_case(tq, c, 0.12, True, 0, H_F16)


def test_attention_wide_tables(tq):
    """A table far wider than the sequences: the f16 rows of all heads would not fit their space, the heads go in rounds."""
    c = attention_case(tq, 128, "prod3", "prod3", 10, 4, [40, 1], [300, 100], 1024, "bf16", "half", max_pages=300)
    fk, bt, kc = c[0], c[2], c[3]
    size = tq.tq_attn_paged_workspace_bytes(fk.handle.ptr, c[1].handle.ptr, bt.struct, 40, 10, kc.struct)
    assert size < 1.5 * 2 ** 30
    check_case(tq, c, 0.09, True, 0, H_F16)


def test_simt_switch_agrees(tq, monkeypatch):
    """TQ_SIMT=1 sends every call to the general kernels: the same codes and, to f16's roundings, the same attention."""
    c = attention_case(tq, 128, "prod3", "mse4", 2, 4, [140, 1], [400, 900], 32, "bf16", "norm+half")
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    fast = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, prep=pr)
    k, v = heads(2, 600, 4, 128, torch.bfloat16), heads(3, 600, 4, 128, torch.bfloat16)
    ab = pu.make_batch(tq, [600], [600], 32)
    a = run_append(tq, fk, fv, ab, k, v, pr, 4)
    monkeypatch.setenv("TQ_SIMT", "1")
    check_case(tq, c, 0.09, True, 0, H_FP32)
    slow = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, prep=pr)
    assert not torch.equal(fast, slow)
    b = run_append(tq, fk, fv, ab, k, v, pr, 4)
    check_cache(a[0], b[0]), check_cache(a[1], b[1])


@pytest.mark.parametrize("n", [2, 300])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_of_vectors_whose_squares_overflow(tq, n, dtype):
    """Heads of 1e25 (their squares pass fp32) come out of the norm like heads of one: codes, signs and attention."""
    fk, fv = fmt(tq, 128, "prod3", 0), fmt(tq, 128, "mse4", 1)
    bt = pu.make_batch(tq, [n], [n], 16)
    x, v = heads(13, n, 2, 128, DT[dtype]), heads(14, n, 2, 128, DT[dtype])
    x[::2] *= 2.0 ** 83
    pr = make_prep(tq, "norm+half", 128, DT[dtype])
    kc, vc = run_append(tq, fk, fv, bt, x, v, pr, 2)
    check_cache(kc, expected_cache(tq, fk, bt, 2, 1, x, pr))
    fk, fv, bt, kc, vc, kr, vr, q, pr = attention_case(tq, 128, "mse4", "mse4", 2, 4, [n, 1], [400, 90], 16, dtype, "norm+half")
    q[::2] *= 2.0 ** 83
    check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, pr), 0.09, True, 0, H_FP32 if dtype == "fp32" else H_F16)


def test_caches_of_another_format_are_refused(tq):
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, [1], [40], 16, "bf16")
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    for name, norm in (("mse2", "f16"), ("prod3", "f16"), ("mse4", "f32")):
        other = fmt(tq, 128, name, 5, norm).handle
        for hk, hv in ((other, fv.handle), (fk.handle, other)):
            with pytest.raises(tq.TQError, match="another format"):
                tq.attn_paged(hk, hv, q, kc, vc, bt, 0.09)
            with pytest.raises(tq.TQError, match="another format"):
                tq.append_paged(hk, hv, q[:, :2], q[:, 2:4], kc, vc, bt)
    again = fmt(tq, 128, "mse4", 0).handle   # one with the rows' format is taken
    tq.attn_paged(again, fv.handle, q, kc, vc, bt, 0.09)


def test_offsets_past_32_bits(tq):
    """The last pages of caches whose codes and f16 rows' places pass 2^32 bytes: the same bytes and results as in small ones."""
    fk, fv = fmt(tq, 128, "mse4", 0), fmt(tq, 128, "mse4", 1)
    Hkv, page, big = 2, 64, 2 ** 19 + 1024           # 2^19 pages x 2 heads x 64 rows x 64 bytes = 2^32
    news, lens = [150, 1, 5], [700, 900, 40]
    bt = pu.make_batch(tq, news, lens, page)
    full = pu.make_batch(tq, lens, lens, page)
    shift = big - bt.num_pages
    x, v = heads(15, full.ntok, Hkv, 128, torch.bfloat16), heads(16, full.ntok, Hkv, 128, torch.bfloat16)
    q = heads(17, bt.ntok, 4 * Hkv, 128, torch.bfloat16, outliers=False)
    small = [tq.PagedCache(f.handle, bt.num_pages, Hkv, page) for f in (fk, fv)]
    large = [tq.PagedCache(f.handle, big, Hkv, page) for f in (fk, fv)]
    for caches, off in ((small, 0), (large, shift)):
        table = torch.where(full.block_table >= 0, full.block_table + off, full.block_table)
        tq.append_paged(fk.handle, fv.handle, x, v, *caches, tq.PagedBatch(full.q_start, full.len, table, full.ntok))
    assert fk.handle.status() == tq.TQ_OK
    for a, b in zip(small, large):
        assert torch.equal(a.codes, b.codes[shift:]) and torch.equal(a.norms, b.norms[shift:])
        assert not b.codes[:shift].any()
    for dtype in (torch.bfloat16, torch.float32):
        outs = []
        for caches, off in ((small, 0), (large, shift)):
            table = torch.where(full.block_table >= 0, full.block_table + off, full.block_table)
            b = tq.PagedBatch(bt.q_start, bt.len, table, bt.ntok)
            outs.append(tq.attn_paged(fk.handle, fv.handle, q.to(dtype), *caches, b, 0.09))
        assert fk.handle.status() == tq.TQ_OK and torch.equal(*outs) and outs[0].abs().sum() > 0


@pytest.mark.parametrize("d,kf,news,lens,causal", [
    (128, "mse4", [1, 2, 1, 1, 5], [3000, 0, 2500, 0, 1700], False),          # sequences without keys between long ones
    (128, "prod3", [1, 3, 1], [4000, 2, 1999], True),                         # a row before the first position
    (64, "mse4", [1, 1, 1, 1] * 16, [20, 0, 33, 0] * 16, False),              # more items than CTAs
])
def test_sequences_without_keys_among_others(tq, d, kf, news, lens, causal):
    """Empty sequences get zeros, whatever their neighbours' parts and the workspace hold."""
    c = attention_case(tq, d, kf, kf, 6, 2, news, lens, 16, "bf16")
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    size = tq.tq_attn_paged_workspace_bytes(fk.handle.ptr, fv.handle.ptr, bt.struct, 12, 6, kc.struct)
    ws = torch.full((size,), 68, dtype=torch.uint8, device="cuda")   # finite numbers
    got = check_case(tq, c, 0.09, causal, 0, H_F16, workspace=ws)
    for b, L in enumerate(lens):
        if L == 0:
            assert not got[sum(news[:b]):sum(news[:b + 1])].any()


def test_workspaces_serve_smaller_batches(tq):
    """The size for a batch is enough for every batch with no argument larger."""
    g = np.random.default_rng(0)
    one = torch.zeros(2, dtype=torch.int32, device="cuda")
    for d, kf in ((128, "mse4"), (128, "prod3"), (64, "mse4"), (96, "mse3")):
        h = fmt(tq, d, kf, 0).handle
        cache = tq.PagedCache(h, 1, 1, 64)

        def size(B, ntok, pages, max_q, Hq, Hkv):
            s = tq.PagedBatch(one, one[:1], one[:1, None], 1).struct
            s.B, s.ntok, s.max_pages, s.max_q = B, ntok, pages, max_q
            return tq.tq_attn_paged_workspace_bytes(h.ptr, h.ptr, s, Hq, Hkv, cache.struct)

        for _ in range(3000):
            Hkv = int(g.choice([1, 2, 8, 12, 32]))
            Hq = Hkv * int(g.choice([1, 3, 4, 8, 16, 32]))
            B, ntok, pages = (int(2 ** g.uniform(0, top)) for top in (13, 16, 10))
            max_q = int(g.integers(1, ntok + 1))
            B2, n2, p2 = (int(x if g.random() < 0.4 else g.integers(1, x + 1)) for x in (B, ntok, pages))
            q2 = min(n2, int(max_q if g.random() < 0.4 else g.integers(1, max_q + 1)))
            assert 0 < size(B2, n2, p2, q2, Hq, Hkv) <= size(B, ntok, pages, max_q, Hq, Hkv)


def test_two_streams_at_once(tq):
    """Two batches on two streams, each with its own workspace, appended and attended to at the same time."""
    jobs = []
    for i in range(2):
        c = attention_case(tq, 128, "mse4", "mse4", 2, 4, [200, 1, 1], [500, 300, 40], 16, "bf16", "half", seed=i)
        fk, fv, bt, kc, vc, kr, vr, q, pr = c
        size = tq.tq_attn_paged_workspace_bytes(fk.handle.ptr, fv.handle.ptr, bt.struct, 8, 2, kc.struct)
        jobs.append((c, torch.empty(size, dtype=torch.uint8, device="cuda"), torch.cuda.Stream(), torch.zeros_like(q),
                     tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, prep=pr)))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, ws, s, out, want in jobs:
            fk, fv, bt, kc, vc, kr, vr, q, pr = c
            tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, prep=pr, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, ws, s, out, want in jobs:
        assert torch.equal(out, want)


def test_batches_that_are_not_what_they_say(tq):
    """Bounds that leave the batch's rows, or descend: those sequences are not computed, nothing else is touched."""
    for dtype in ("fp32", "bf16"):
        for news in ([1, 1, 1], [40, 1, 30]):
            c = attention_case(tq, 128, "mse4", "mse4", 2, 4, news, [100, 60, 90], 16, dtype)
            fk, fv, bt, kc, vc, kr, vr, q, pr = c
            want = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09)
            n0 = news[0]
            for start in ([0, n0, n0, bt.ntok + 7], [-5, 0, n0 + 1, n0], [0, n0, bt.ntok + 1, 2 ** 31 - 1]):
                bad = tq.PagedBatch(torch.tensor(start, dtype=torch.int32).cuda(), bt.len, bt.block_table, bt.ntok)
                out = torch.full_like(q, 3.0)
                tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bad, 0.09, out=out)
                assert fk.handle.status() in (tq.TQ_OK, tq.TQ_EINVAL)
                if start[:2] == [0, n0]:
                    assert torch.equal(out[:n0], want[:n0]) and (out[n0:] == 3.0).all()


def test_append_then_attend_as_a_server_does(tq):
    """Prompts in chunks, then decode steps, some sequences joining late: append and attend each step, both on a side
    stream, against attention over the package's own rows in 64 bits."""
    d, Hkv, G, page = 128, 2, 4, 16
    fk, fv = fmt(tq, d, "prod3", 0), fmt(tq, d, "mse4", 1)
    pr = make_prep(tq, "norm+half", d, torch.bfloat16)
    num_pages, max_pages = 64, 20
    kc, vc = tq.PagedCache(fk.handle, num_pages, Hkv, page), tq.PagedCache(fv.handle, num_pages, Hkv, page)
    order = torch.randperm(num_pages, generator=torch.Generator().manual_seed(0)).to(torch.int32)
    table = order[:60].reshape(3, 20).contiguous().cuda()
    lens, s = [0, 0, 0], torch.cuda.Stream()
    for step, news in enumerate(([100, 0, 7], [60, 1, 1], [1, 80, 1], [1, 1, 1], [1, 1, 1], [0, 1, 0])):
        lens = [a + b for a, b in zip(lens, news)]
        start = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32).cuda()
        bt = tq.PagedBatch(start, torch.tensor(lens, dtype=torch.int32).cuda(), table, sum(news), max(news))
        bt.news, bt.lens, bt.page = news, list(lens), page
        x = heads(50 + step, sum(news), Hkv * (G + 2), d, torch.bfloat16, outliers=False)
        q, k, v = x[:, :Hkv * G], x[:, Hkv * G:Hkv * (G + 1)], x[:, Hkv * (G + 1):]
        s.wait_stream(torch.cuda.current_stream())
        tq.append_paged(fk.handle, fv.handle, k, v, kc, vc, bt, prep=pr, stream=s)
        out = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, d ** -0.5, prep=pr, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert fk.handle.status() == tq.TQ_OK
        kr, vr = [], []
        for b, L in enumerate(lens):
            pg, sl = pu.slots(bt, b, 0, L)
            for cache, f, rows in ((kc, fk, kr), (vc, fv, vr)):
                codes = cache.codes[pg, :, sl].long()
                idx = ((codes[..., None] >> (torch.arange(8 // f.bits, device="cuda") * f.bits)) & ((1 << f.bits) - 1)).flatten(-2)
                sg = ((cache.signs[pg, :, sl].long()[..., None] >> torch.arange(8, device="cuda")) & 1).flatten(-2) if f.m else None
                rows.append((idx, sg, cache.norms[pg, :, sl].double(), cache.rnorms[pg, :, sl].double() if f.m else None))
        ref, tol = pu.attention_ref(bt, q, fk, fv, kr, vr, d ** -0.5, True, 0, pr, H_F16)
        pu.check_attention(out, ref, tol, torch.bfloat16)


def test_captured_step_replays_with_new_lengths(tq):
    """One decode step (append, attend) captured with padding and replayed with other lengths, tables and batch sizes."""
    d, Hkv, G, page, B = 128, 2, 4, 16, 4
    fk, fv = fmt(tq, d, "mse4", 0), fmt(tq, d, "mse4", 1)
    bt0 = pu.make_batch(tq, [1] * B, [200, 190, 180, 170], page)
    kc, vc = pu.garbage_cache(tq, fk, bt0, Hkv, 1), pu.garbage_cache(tq, fv, bt0, Hkv, 2)
    kr = pu.fill_cache(kc, fk, bt0, [heads(100 + b, L, Hkv, d) for b, L in enumerate(bt0.lens)])
    vr = pu.fill_cache(vc, fv, bt0, [heads(200 + b, L, Hkv, d) for b, L in enumerate(bt0.lens)])
    start, lens, table = bt0.q_start.clone(), bt0.len.clone(), bt0.block_table.clone()
    bt = tq.PagedBatch(start, lens, table, B, 1)
    k, v, q = (heads(i, B, H, d, torch.bfloat16) for i, H in ((1, Hkv), (2, Hkv), (3, Hkv * G)))
    out = torch.zeros_like(q)
    ws = torch.empty(tq.tq_attn_paged_workspace_bytes(fk.handle.ptr, fv.handle.ptr, bt.struct, Hkv * G, Hkv, kc.struct),
                     dtype=torch.uint8, device="cuda")

    def step():
        tq.append_paged(fk.handle, fv.handle, k, v, kc, vc, bt)
        tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, out=out, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for live, ls in ((4, [150, 33, 17, 100]), (2, [16, 160, 0, 0]), (0, [0, 0, 0, 0]), (3, [170, 160, 1, 0])):
        q.copy_(heads(400 + live, B, Hkv * G, d, torch.bfloat16))
        start.copy_(torch.tensor([min(i, live) for i in range(B + 1)], dtype=torch.int32))
        lens.copy_(torch.tensor(ls, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        assert fk.handle.status() == tq.TQ_OK
        got = out.clone()
        assert (got[live:] == 7.0).all()
        step()   # the same step without the graph: the same bits
        assert torch.equal(got, out)
        for b in range(live):   # and right: the newest row is the appended one
            bt1 = tq.PagedBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(), lens[b:b + 1].clone(), table[b:b + 1].contiguous(), 1)
            bt1.news, bt1.lens, bt1.page = [1], [ls[b]], page
            rows = []
            for cache, f in ((kc, fk), (vc, fv)):
                pg, sl = pu.slots(bt1, 0, 0, ls[b])
                codes = cache.codes[pg, :, sl].long()
                rows.append((torch.stack([codes & 15, codes >> 4], -1).flatten(-2), None, cache.norms[pg, :, sl].double(), None))
            ref, tol = pu.attention_ref(bt1, q[b:b + 1], fk, fv, rows[:1], rows[1:], 0.09, True, 0, None, H_F16)
            pu.check_attention(got[b:b + 1], ref, tol, torch.bfloat16)
