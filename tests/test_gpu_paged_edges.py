"""Paged attention at its edges: rows that see nothing, freed pages, lengths past the table, norms far apart, values and keys that
are not finite, queries at the ends of their type's range; against 64 bits."""

import numpy as np
import pytest
import torch

import paged_util as pu
from test_gpu_paged import DT, H_F16, H_FP32, attention_case, check_case, fmt, heads, tq  # noqa: F401  (tq: the fixture)

pytestmark = pytest.mark.gpu


def h_of(dtype):
    return H_FP32 if dtype == "fp32" else H_F16


def cached(tq, fk, fv, news, lens, page, Hkv, k, v, seed=0):
    """A batch whose sequences hold the vectors k[b], v[b]: batch, caches and their stored rows."""
    bt = pu.make_batch(tq, news, lens, page, seed=seed)
    kc, vc = pu.garbage_cache(tq, fk, bt, Hkv, 1), pu.garbage_cache(tq, fv, bt, Hkv, 2)
    return bt, kc, vc, pu.fill_cache(kc, fk, bt, k), pu.fill_cache(vc, fv, bt, v)


# ------------------------------------------------------------------ rows that see nothing
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("size", [100.0, 1000.0])   # value norms of about 1e3 and 1e4
@pytest.mark.parametrize("news,lens", [([40], [10]), ([3, 340, 45], [2, 300, 20])])
def test_rows_before_the_first_position_are_zeros(tq, news, lens, size, dtype):
    """More new tokens than cached ones: the first see nothing, however large the values that the others see."""
    fk, fv = fmt(tq, 128, "mse4", 0), fmt(tq, 128, "mse4", 1)
    k, v = [heads(1 + b, L, 2, 128) for b, L in enumerate(lens)], [size * heads(9 + b, L, 2, 128) for b, L in enumerate(lens)]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, k, v)
    q = heads(3, bt.ntok, 8, 128, DT[dtype], outliers=False)
    got = check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, None), 0.09, True, 0, h_of(dtype))
    for b, (n, L) in enumerate(zip(news, lens)):
        t0 = sum(news[:b])
        assert (got[t0:t0 + max(0, n - L)] == 0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("news", [[1, 2], [60, 1], [340, 50]])
def test_refused_rotation_positions_are_zeros(tq, news, dtype):
    """The same for rows without a rotation, among one and several key tiles of large values."""
    fk, fv = fmt(tq, 128, "mse4", 0), fmt(tq, 128, "prod3", 1)
    lens = [700, 90]
    k, v = [heads(1 + b, L, 1, 128) for b, L in enumerate(lens)], [1000 * heads(9 + b, L, 1, 128) for b, L in enumerate(lens)]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 1, k, v)
    q = heads(3, bt.ntok, 4, 128, DT[dtype], outliers=False)
    pos = torch.randint(0, 4096, (bt.ntok,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    table = pu.rope_table(4096, 128)
    want = check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, tq.HeadPrep(cos_sin=table, pos=pos)), 0.09, False, 0, h_of(dtype))
    bad = torch.arange(bt.ntok, device="cuda") % 3 == 1
    pos = torch.where(bad, torch.full_like(pos, 4096), pos)
    got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, causal=False, prep=tq.HeadPrep(cos_sin=table, pos=pos))
    assert fk.handle.status() == tq.TQ_EINVAL
    assert (got[bad] == 0).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_sequences_whose_pages_are_all_bad_are_zeros(tq, dtype):
    fk, fv = fmt(tq, 128, "mse4", 0), fmt(tq, 128, "mse4", 1)
    news, lens = [50, 60, 1, 2], [300, 200, 400, 90]
    k, v = [heads(1 + b, L, 2, 128) for b, L in enumerate(lens)], [1000 * heads(9 + b, L, 2, 128) for b, L in enumerate(lens)]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, k, v)
    q = heads(3, bt.ntok, 8, 128, DT[dtype], outliers=False)
    want = check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, None), 0.09, True, 0, h_of(dtype))
    t = bt.block_table.clone()
    t[0], t[2] = -1, bt.num_pages
    got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, tq.PagedBatch(bt.q_start, bt.len, t, bt.ntok), 0.09)
    assert fk.handle.status() == tq.TQ_EINVAL
    assert (got[:50] == 0).all() and (got[110] == 0).all()
    assert torch.equal(got[50:110], want[50:110]) and torch.equal(got[111:], want[111:])


# ------------------------------------------------------------------ pages behind the window


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kf,vf", [("mse4", "mse4"), ("prod3", "mse4")])
@pytest.mark.parametrize("news,lens,window", [([1, 60, 3], [700, 500, 333], 100), ([200], [1000], 16), ([64, 1], [640, 2000], 257)])
def test_pages_behind_the_window_may_be_freed(tq, news, lens, window, kf, vf, dtype):
    """Table entries of pages that lie behind the window of a sequence's first new token are not used: -1, or a page that belongs
    to someone else by now."""
    fk, fv = fmt(tq, 128, kf, 0), fmt(tq, 128, vf, 1)
    k, v = [heads(1 + b, L, 2, 128) for b, L in enumerate(lens)], [heads(9 + b, L, 2, 128) for b, L in enumerate(lens)]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, k, v)
    q = heads(3, bt.ntok, 8, 128, DT[dtype], outliers=False)
    want = check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, None), 0.09, True, window, h_of(dtype))
    spare = next(p for p in range(bt.num_pages) if not (bt.block_table == p).any())
    for page in (-1, spare):   # the spare pages' norms are NaN
        for b, (n, L) in enumerate(zip(news, lens)):
            bt.block_table[b, :(L - n - window + 1) // 16] = page
        got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, window=window)
        assert fk.handle.status() == tq.TQ_OK
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("news,lens", [([8, 1], [3, 300]), ([340, 45], [300, 20])])
def test_a_window_as_wide_as_its_type_is_none(tq, news, lens, dtype):
    """Also where the first tokens stand before the first position."""
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, news, lens, 16, dtype)
    want = check_case(tq, c, 0.09, True, 0, h_of(dtype))
    for window in (2 ** 31 - 1, 2 ** 31 - 5, 2 ** 30):
        assert torch.equal(check_case(tq, c, 0.09, True, window, h_of(dtype)), want)


# ------------------------------------------------------------------ lengths and bounds that are not what they say


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("news", [[1, 2, 1], [50, 40, 1], [50, 60, 70]])
@pytest.mark.parametrize("which", [0, 2])
def test_lengths_past_the_table_are_recorded(tq, which, news, dtype):
    """What the table has of the sequence is seen, the call is recorded; the others stay as they are."""
    lens = [160, 130, 158]
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, news, lens, 16, dtype)
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    full = bt.len.clone()
    full[which] = 160                       # all slots of its pages: the reference's rows are those up to its length
    for t in (kc.norms, vc.norms):
        t.nan_to_num_(nan=1.0)
    for causal in (False, True):
        # causal: every token of the long sequence stands behind the table's end, and sees all of it
        want = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, tq.PagedBatch(bt.q_start, full, bt.block_table, bt.ntok), 0.09, causal=False)
        others = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, causal=causal)
        assert fk.handle.status() == tq.TQ_OK
        over = full.clone()
        over[which] = 160 + 200
        got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, tq.PagedBatch(bt.q_start, over, bt.block_table, bt.ntok), 0.09, causal=causal)
        assert fk.handle.status() == tq.TQ_EINVAL and fk.handle.status() == tq.TQ_OK
        mine = torch.zeros(bt.ntok, dtype=torch.bool, device="cuda")
        mine[sum(news[:which]):sum(news[:which + 1])] = True
        assert torch.equal(got[mine], want[mine]) and torch.equal(got[~mine], others[~mine])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("news", [[1, 1, 1], [2, 3, 1], [40, 1, 30], [1, 50, 2]])
def test_bad_bounds_are_recorded_and_their_rows_kept(tq, news, dtype):
    """Sequences whose rows leave the batch's, descend, or are more than max_q: recorded, their rows of out as they were."""
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, news, [100, 60, 90], 16, dtype)
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    n0, N = news[0], bt.ntok

    def run(start, max_q=None):
        out = torch.full_like(q, 3.0)
        b = tq.PagedBatch(torch.tensor(start, dtype=torch.int32).cuda(), bt.len, bt.block_table, N, max_q)
        tq.attn_paged(fk.handle, fv.handle, q, kc, vc, b, 0.09, out=out)
        return out

    for start, good, used in (([0, n0, n0, N + 7], [0, n0, n0, n0], n0), ([0, n0, N + 1, 2 ** 31 - 1], [0, n0, n0, n0], n0),
                              ([-5, 0, n0 + 1, n0], [0, 0, n0 + 1, n0 + 1], n0 + 1), ([-2 ** 31, 0, n0 + 1, n0 - 1], [0, 0, n0 + 1, n0 + 1], n0 + 1)):
        want = run(good)
        assert fk.handle.status() == tq.TQ_OK and (want[used:] == 3.0).all() and not (want[:used] == 3.0).all()
        got = run(start)
        assert fk.handle.status() == tq.TQ_EINVAL and fk.handle.status() == tq.TQ_OK
        assert torch.equal(got, want)
    starts = bt.q_start.tolist()
    want = run(starts)
    for b, n in enumerate(news):
        if n != max(news) or news.count(n) > 1 or n == 1:
            continue
        got = run(starts, n - 1)
        assert fk.handle.status() == tq.TQ_EINVAL
        rows = torch.arange(N, device="cuda")
        mine = (rows >= starts[b]) & (rows < starts[b + 1])
        assert (got[mine] == 3.0).all()
        room = torch.finfo(q.dtype).eps * 4 * want.abs().amax()   # other splits of the keys: the same sums in another order
        assert ((got - want)[~mine].abs() <= room).all()


def test_more_tile_pairs_than_are_counted_are_refused(tq):
    """2^24 tokens of 64 query heads over 2^30 positions: refused before the workspace is looked at."""
    h = fmt(tq, 128, "mse4", 0).handle
    cache = tq._lib.tq_paged_cache(1 << 12, None, 1 << 12, None, 1 << 20, 1024)
    batch = tq._lib.tq_paged_batch(1 << 12, 1 << 12, 1 << 12, 1, 1 << 20, 1 << 24, 1 << 24)
    r = tq._lib.ctypes.byref
    st = tq._lib.lib.tq_attn_paged(h.ptr, h.ptr, 4096, tq.TQ_BF16, 64 * 128, 64, 1, r(batch), None, r(cache), r(cache), 0.1, 1, 0,
                                   4096, 4096, 16, None)
    assert st == tq.TQ_EUNSUPPORTED and "split the batch" in tq.tq_last_error()


# ------------------------------------------------------------------ norms far apart


FAR = [([1], [300]), ([5, 1], [300, 40]), ([40], [41]), ([200, 3], [400, 150])]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("d,kf,vf,norm", [(128, "mse4", "mse4", "f16"), (128, "prod3", "prod3", "f16"), (64, "mse4", "mse4", "f32"), (128, "mse3", "prod3", "f16")])
@pytest.mark.parametrize("news,lens", FAR)
def test_values_that_a_row_does_not_see_cost_it_nothing(tq, news, lens, d, kf, vf, norm, dtype):
    """The newest token's value is 4e6 times (fp32 norms: 1e20 times) its neighbours': rows that come before it are as exact as
    without it, and so is the newest where its own key turns it away."""
    fk, fv = fmt(tq, d, kf, 0), fmt(tq, d, vf, 1, norm)
    small, large = (1e-3, 4e3) if norm == "f16" else (1e-12, 1e8)
    u = heads(77, 1, 1, d)
    k, v = [], []
    for b, L in enumerate(lens):
        kk, vv = heads(1 + b, L, 2, d, outliers=False), small * heads(9 + b, L, 2, d, outliers=False)
        kk[-1] = -6.0 * u[0]          # its score: about -6 * 4 * |u|^2 scale, a weight below e^-100
        vv[-1] *= large / small
        k.append(kk), v.append(vv)
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, k, v)
    q = (heads(3, bt.ntok, 4, d, outliers=False) * 0.3 + 4 * u).to(DT[dtype])
    check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, None), 0.09, True, 0, h_of(dtype))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("kf,norm", [("mse4", "f16"), ("prod3", "f16"), ("mse3", "f32")])
@pytest.mark.parametrize("news,lens", FAR)
def test_keys_that_a_row_does_not_see_cost_it_nothing(tq, news, lens, kf, norm, dtype):
    """The same for the newest token's key."""
    fk, fv = fmt(tq, 128, kf, 0, norm), fmt(tq, 128, "mse4", 1)
    small, large = (1e-3, 4e3) if norm == "f16" else (1e-12, 1e8)
    k = [small * heads(1 + b, L, 2, 128, outliers=False) for b, L in enumerate(lens)]
    for x in k:
        x[-1] *= large / small
    v = [heads(9 + b, L, 2, 128, outliers=False) for b, L in enumerate(lens)]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, k, v)
    q = heads(3, bt.ntok, 4, 128, DT[dtype], outliers=False)
    fk_, fv_, got = fk, fv, tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.15 / small)
    ref, tol = pu.attention_ref(bt, q, fk, fv, kr, vr, 0.15 / small, True, 0, None, h_of(dtype))
    last = torch.zeros(bt.ntok, dtype=torch.bool, device="cuda")
    last[bt.q_start[1:].long() - 1] = True     # these see a score of 1e6: all or nothing, whichever side rounding takes
    pu.check_attention(got[~last], ref[~last], tol[~last], q.dtype)
    assert got.isfinite().all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("norm", ["f16", "f32"])
@pytest.mark.parametrize("news", [[1, 2], [100, 50]])
def test_norms_spread_over_their_type(tq, news, norm, dtype):
    """Keys and values whose norms are spread evenly over 2^26 (fp16 norms) or 2^120 (fp32), in no order; causal and not."""
    fk, fv = fmt(tq, 128, "mse4", 0, norm), fmt(tq, 128, "prod3", 1) if norm == "f16" else fmt(tq, 128, "mse4", 1, norm)
    lens, g = [700, 130], torch.Generator().manual_seed(5)
    span = 26 if norm == "f16" else 120

    def spread(L, lo):
        return torch.exp2(lo + span * torch.rand(L, 2, 1, generator=g).double()).cuda()

    k = [heads(1 + b, L, 2, 128, outliers=False) * spread(L, -span + 2) for b, L in enumerate(lens)]
    v = [heads(9 + b, L, 2, 128, outliers=False) * spread(L, -14 if norm == "f16" else -60) for b, L in enumerate(lens)]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, k, v)
    q = heads(3, bt.ntok, 4, 128, DT[dtype], outliers=False)
    for causal in (True, False):
        got = tq.attn_paged(fk.handle, fv.handle, q.float() if dtype == "fp32" else q, kc, vc, bt, 0.2, causal=causal)
        ref, tol = pu.attention_ref(bt, q, fk, fv, kr, vr, 0.2, causal, 0, None, h_of(dtype))
        fits = ref.abs() < torch.finfo(q.dtype).max / 2   # fp16 has no room for the largest
        assert got[fits].isfinite().all()
        pu.check_attention(got[fits], ref[fits], tol[fits], q.dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 1e-38, -3e-38])
@pytest.mark.parametrize("news", [[1, 2], [100, 50]])
def test_scales_that_make_up_for_the_keys_norms(tq, news, scale, dtype):
    """Keys of norms up to 1e37 under a scale as small, or of zero, which averages."""
    fk, fv = fmt(tq, 128, "mse4", 0, "f32"), fmt(tq, 128, "mse4", 1, "f32")
    lens, g = [700, 130], torch.Generator().manual_seed(6)
    k = [heads(1 + b, L, 2, 128, outliers=False) * torch.exp2(120 * torch.rand(L, 2, 1, generator=g).double()).cuda() for b, L in enumerate(lens)]
    v = [heads(9 + b, L, 2, 128, outliers=False) for b, L in enumerate(lens)]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, k, v)
    q = heads(3, bt.ntok, 4, 128, DT[dtype], outliers=False)
    check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, None), scale, True, 0, h_of(dtype))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("what", [float("inf"), float("nan")])
@pytest.mark.parametrize("kf,vf", [("mse4", "mse4"), ("prod3", "prod3"), ("mse3", "qjl")])
@pytest.mark.parametrize("news,lens,window", [([5], [40], 0), ([3, 1], [200, 17], 20), ([60, 70], [90, 300], 0), ([80], [400], 50)])
def test_rows_that_are_not_finite_and_not_seen(tq, news, lens, window, kf, vf, what, dtype):
    """The newest key and value, and (with a window) one just behind the window of the later tokens, have a norm of infinity or
    NaN: the rows that do not see them are as if they were not there."""
    fk, fv = fmt(tq, 128, kf, 0), fmt(tq, 128, vf, 1)
    k, v = [heads(1 + b, L, 2, 128) for b, L in enumerate(lens)], [heads(9 + b, L, 2, 128) for b, L in enumerate(lens)]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, k, v)
    q = heads(3, bt.ntok, 4, 128, DT[dtype], outliers=False)
    want = check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, None), 0.09, True, window, h_of(dtype))
    ref, tol = pu.attention_ref(bt, q, fk, fv, kr, vr, 0.09, True, window, None, h_of(dtype))
    keep = torch.ones(bt.ntok, dtype=torch.bool, device="cuda")
    for b, (n, L) in enumerate(zip(news, lens)):
        t0 = sum(news[:b])
        for p in [L - 1] + ([L - n - window + 1] if window and L - n - window + 1 >= 0 else []):
            page, slot = pu.slots(bt, b, p, p + 1)
            for c in (kc, vc):
                c.norms[page, :, slot] = what
                if c.rnorms is not None:
                    c.rnorms[page, :, slot] = what
            for i in range(n):
                pos = L - n + i
                if p <= pos and not (window and p <= pos - window):
                    keep[t0 + i] = False
    got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, window=window)
    assert got[keep].isfinite().all()
    pu.check_attention(got[keep], ref[keep], tol[keep], q.dtype)


# ------------------------------------------------------------------ NaN that is seen


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("kf", ["mse4", "prod3", "mse3"])
@pytest.mark.parametrize("side", ["key", "value", "query"])
@pytest.mark.parametrize("news", [[1], [5], [70]])
def test_nan_goes_to_the_rows_that_see_it(tq, news, side, kf, dtype):
    """A NaN key, value or query makes the rows that use it NaN, wherever it stands, and no others."""
    fk, fv = fmt(tq, 128, kf, 0), fmt(tq, 128, kf, 1)
    n, L = news[0], 300
    c = attention_case(tq, 128, kf, kf, 1, 4, news, [L], 16, dtype)
    _, _, bt, kc, vc, kr, vr, q, pr = c
    want = check_case(tq, c, 0.09, True, 0, h_of(dtype))
    if side == "query":
        q[0, 1] = float("nan")
        got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09)
        assert got[0, 1].isnan().all()
        got[0, 1] = want[0, 1]
        assert torch.equal(got, want)
        return
    cache = kc if side == "key" else vc
    for p in [0, 1, 2, 3, 4, 5, 6, 7, 14, 15, 126, 127, 128, 134, L - n] + list(range(L - 9, L)):
        page, slot = pu.slots(bt, 0, p, p + 1)
        old = cache.norms[page, :, slot].clone()
        cache.norms[page, :, slot] = float("nan")
        got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09)
        cache.norms[page, :, slot] = old
        sees = torch.arange(L - n, L, device="cuda") >= p
        assert got[sees].isnan().all(), f"position {p}"
        room = torch.finfo(q.dtype).eps * 4 * want.abs().amax() + 0.02 * (dtype != "fp32")
        assert ((got - want)[~sees].abs() <= room).all(), f"position {p}"


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 70])
def test_rows_of_nan_alone(tq, n, dtype):
    """Every key that a row sees is NaN: NaN, not the zeros of a row without keys."""
    c = attention_case(tq, 128, "mse4", "mse4", 2, 4, [n], [n], 16, dtype)
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    kc.norms.fill_(float("nan"))
    assert tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09).isnan().all()


# ------------------------------------------------------------------ queries at the ends of their range


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kf", ["mse4", "prod3"])
@pytest.mark.parametrize("size", [1e-38, 3e-39, 1e-30, 1e20, 1e37])
@pytest.mark.parametrize("news,prep", [([1, 1], "none"), ([5, 2], "half"), ([70, 1], "none"), ([70, 40], "half"), ([70, 2], "partial")])
def test_queries_of_any_size(tq, news, prep, size, kf, dtype):
    """Tiny queries average the values; large ones with a scale as small give ordinary scores."""
    c = attention_case(tq, 128, kf, kf, 2, 4, news, [300, 90], 16, dtype, prep)
    fk, fv, bt, kc, vc, kr, vr, q, pr = c
    q = (q.double() * size).to(q.dtype)
    if dtype == "fp32" and size < 1e-37:
        q = q.to(torch.bfloat16).float()   # (subnormal inputs lose their own digits)
    scale = 0.09 if size < 1 else 0.09 / size
    check_case(tq, (fk, fv, bt, kc, vc, kr, vr, q, pr), scale, True, 0, h_of(dtype))


# ------------------------------------------------------------------ handles and caches


def test_caches_of_another_shape_with_rows_as_wide_are_refused(tq):
    """64 coordinates of 4 bits and 128 of 2 have rows of one size and are still not the same rows."""
    fa, fb = fmt(tq, 128, "mse2", 0), fmt(tq, 64, "mse4", 0)
    bt = pu.make_batch(tq, [1], [20], 16)
    q = heads(1, 1, 4, 128, torch.bfloat16)
    ca, cb = pu.garbage_cache(tq, fa, bt, 2, 1), pu.garbage_cache(tq, fb, bt, 2, 1)
    assert fa.handle.codes_B == fb.handle.codes_B
    for kc, vc in ((cb, ca), (ca, cb), (cb, cb)):
        with pytest.raises(tq.TQError, match="another format"):
            tq.attn_paged(fa.handle, fa.handle, q, kc, vc, bt, 0.09)
        with pytest.raises(tq.TQError, match="another format"):
            tq.append_paged(fa.handle, fa.handle, q[:, :2], q[:, 2:], kc, vc, bt)
# ------------------------------------------------------------------ precision


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 8])
def test_one_key_gives_its_value_rounded_once(tq, d, G):
    """One key has weight one: the output is its value. The tables hold four centroids to 3.4e-6 of themselves (d = 64; 9e-7 at
    d = 128), which Pi, keeping lengths, makes as much of the value's length at most; sums of d products in fp32 cost at most
    23 * 2^-24 of it; beyond that the output may only be rounded to its type."""
    fk, fv = fmt(tq, d, "mse2", 0), fmt(tq, d, "mse2", 1)
    lens = [1] * 40
    bt, kc, vc, kr, vr = cached(tq, fk, fv, [1] * 40, lens, 16, 2, [heads(b, 1, 2, d) for b in range(40)], [heads(99 + b, 1, 2, d) for b in range(40)])
    q = heads(3, bt.ntok, 2 * G, d, torch.float16, outliers=False)
    got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09)
    assert fk.handle.status() == tq.TQ_OK
    want = torch.stack([fv.rotated(*r)[0][0] @ fv.Pi for r in vr]).repeat_interleave(G, 1)
    room = 2.0 ** -11 * want.abs() + (3.4e-6 + 23 * 2.0 ** -24) * want.norm(dim=-1, keepdim=True) + 2.0 ** -25
    assert ((got.double() - want).abs() <= room).all()


def test_one_key_of_a_chunk_gives_its_value_rounded_once(tq):
    """The same for a chunk's rows, whose values are expanded to f16 first: that is the one rounding (f16 outputs take it over)."""
    fk, fv = fmt(tq, 128, "mse2", 0), fmt(tq, 128, "mse2", 1)
    news, lens = [40, 50], [1, 1]
    bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 16, 2, [heads(b, 1, 2, 128) for b in range(2)], [heads(99 + b, 1, 2, 128) for b in range(2)])
    q = heads(3, bt.ntok, 4, 128, torch.float16, outliers=False)
    got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, 0.09, causal=False)
    assert fk.handle.status() == tq.TQ_OK
    for b, t0 in ((0, 0), (1, 40)):
        want = (fv.rotated(*vr[b])[0][0] @ fv.Pi).repeat_interleave(2, 0)
        room = 2.0 ** -11 * want.abs() + (3.4e-6 + 23 * 2.0 ** -24) * want.norm(dim=-1, keepdim=True) + 2.0 ** -25
        assert ((got[t0:t0 + news[b]].double() - want).abs() <= room).all()


@pytest.mark.parametrize("d,name", [(128, "mse4"), (64, "mse4"), (128, "mse2"), (128, "mse3"), (128, "prod3"), (64, "prod3"), (128, "prod4")])
def test_documented_precision_with_outlier_channels(tq, d, name):
    """Channels of log-normal size and two outliers of ten times that in each head: every head of a chunk within the documented
    1.5e-3 of 64 bits, single tokens (formats with a kernel of their own) within 1e-3 altogether."""
    fk, fv = fmt(tq, d, name, 0), fmt(tq, d, name, 1)
    H = 8

    def data(g, n):
        s = torch.exp(0.5 * torch.randn(H, d, generator=g, dtype=torch.float64))
        at = torch.rand(H, d, generator=g).argsort(1)[:, :2]
        return (torch.randn(n, H, d, generator=g, dtype=torch.float64) * s.scatter(1, at, s.gather(1, at) * 10)).cuda()

    for news, lens in (([300], [1500]), ([1] * 6, [1500] * 6)):
        g = torch.Generator().manual_seed(7)
        k, v = [data(g, L) for L in lens], [data(g, L) for L in lens]
        bt, kc, vc, kr, vr = cached(tq, fk, fv, news, lens, 64, H, k, v)
        q = torch.randn(bt.ntok, H, d, generator=g).half().cuda()
        got = tq.attn_paged(fk.handle, fv.handle, q, kc, vc, bt, d ** -0.5).double()
        ref, _ = pu.attention_ref(bt, q, fk, fv, kr, vr, d ** -0.5, True, 0, None, H_F16)
        off = (got - ref).square().sum((0, 2)).sqrt() / ref.square().sum((0, 2)).sqrt()
        if len(news) == 1:
            assert off.max() <= 1.5e-3
        elif name in ("mse4", "mse2", "prod3"):
            assert (got - ref).norm() <= 1e-3 * ref.norm()
