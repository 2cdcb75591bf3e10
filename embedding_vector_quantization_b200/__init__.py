"""B200-native TurboQuant-style vector quantization (libtq.so + thin binding).

Encode stores each vector's norm, rotates it by a seeded random orthogonal
matrix, maps every rotated coordinate to a Lloyd-Max codebook index and
bit-packs the indices; prod handles add a 1-bit QJL sign sketch of the
residual and its norm ("Google TurboQuant: 6x KV-cache compression",
sections "Stage 1: PolarQuant" and "Stage 2: QJL residual correction").
Scores, GQA decode attention and top-k search read only the packed codes.

The ``tq_*`` functions mirror the C ABI of ``include/tq.h`` one to one;
:class:`Handle` and :class:`Cache` only allocate PyTorch tensors for them.
Everything runs in the library's CUDA kernels; if libtq.so is missing the
import fails.
"""

from . import _lib
from ._lib import (  # noqa: F401  (the C ABI, same names)
    TQ_BF16, TQ_EINVAL, TQ_ECAPACITY, TQ_ECUDA, TQ_ENOMEM, TQ_ETIMEOUT, TQ_EUNSUPPORTED, TQ_F16, TQ_F32, TQ_OK,
    TQError, make_cache, make_head_prep, make_paged_batch, make_paged_cache, tq_append, tq_append_paged, tq_attn_paged,
    tq_attn_paged_workspace_bytes, tq_attn_decode, tq_attn_decode_noalloc, tq_decode_step, tq_attn_workspace_bytes, tq_code_bytes, tq_codebook_host,
    tq_create, tq_create_polar, tq_create_prod, tq_destroy, tq_get_polar_codebook, tq_polar_codebook_host,
    tq_polar_info, tq_encode, tq_get_codebook, tq_get_info, tq_get_rotation,
    tq_last_error, tq_last_status, tq_pack_indices, tq_rotation_host, tq_score, tq_score_workspace_bytes,
    tq_search_topk, tq_search_workspace_bytes, tq_selftest_wait_timeout, tq_set_norm_dtype, tq_timer_enable,
    tq_timer_read,
)


def _torch():
    import torch
    return torch


class Handle:
    """Owns one library handle: Pi, S, S Pi^T and the codebook on the current device.

    ``bits`` is the total bits per coordinate; with ``qjl_m > 0`` it splits into
    ``bits - 1`` MSE bits plus one QJL sign per projection. ``bits = 1`` with
    ``qjl_m > 0`` gives QJL-only rows: the signs and the norm, no codes.
    """

    def __init__(self, d, bits, seed=0, qjl_m=0, norm_dtype=None):
        self._h = tq_create_prod(d, bits, qjl_m, seed) if qjl_m else tq_create(d, bits, seed)
        if norm_dtype is not None:
            tq_set_norm_dtype(self._h, norm_dtype)
        self.d, self.bits_mse, self.m, self.norm_dtype = tq_get_info(self._h)
        self.codes_B, self.signs_B = tq_code_bytes(self._h)
        self.seed = seed
        self.index = _torch().cuda.current_device()   # where its tables are

    @property
    def prod(self):
        return self.m > 0

    @property
    def qjl_only(self):
        return self.m > 0 and self.bits_mse == 0

    @property
    def ptr(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            tq_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def codebook(self):
        return tq_get_codebook(self._h, self.bits_mse)

    def rotation(self):
        return tq_get_rotation(self._h, self.d, self.m)

    def norm_torch_dtype(self):
        torch = _torch()
        return torch.float16 if self.norm_dtype == TQ_F16 else torch.float32

    def alloc_rows(self, shape, device="cuda"):
        """Empty packed storage for vectors of leading shape ``shape``."""
        torch = _torch()
        shape = tuple(shape) if isinstance(shape, (tuple, list)) else (shape,)
        out = {"codes": None, "norms": torch.empty(shape, dtype=self.norm_torch_dtype(), device=device),
               "signs": None, "rnorms": None}
        if self.codes_B:
            out["codes"] = torch.empty(shape + (self.codes_B,), dtype=torch.uint8, device=device)
        if self.prod:
            out["signs"] = torch.empty(shape + (self.signs_B,), dtype=torch.uint8, device=device)
        if self.prod and not self.qjl_only:
            out["rnorms"] = torch.empty(shape, dtype=torch.float16, device=device)
        return out

    def encode(self, x, out=None, stream=None):
        """Encodes x [..., d] (fp32 / fp16 / bf16, contiguous, on the GPU)."""
        x = x.contiguous()
        lead = tuple(x.shape[:-1])
        n = 1
        for s in lead:
            n *= s
        out = out or self.alloc_rows(lead, x.device)
        tq_encode(self._h, x, n, out["codes"], out["signs"], out["norms"], out["rnorms"], stream)
        return out

    def pack_indices(self, idx, stream=None):
        torch = _torch()
        n = idx.shape[0]
        codes = torch.empty((n, self.codes_B), dtype=torch.uint8, device=idx.device)
        tq_pack_indices(self._h, idx.contiguous(), n, codes, stream)
        return codes

    def status(self, stream=None):
        return tq_last_status(self._h, stream)

    def search_topk(self, q, codes, norms, k, workspace=None, stream=None):
        torch = _torch()
        nq, n = q.shape[0], codes.shape[0]
        idx = torch.empty((nq, k), dtype=torch.int64, device=q.device)
        score = torch.empty((nq, k), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = torch.empty(tq_search_workspace_bytes(self._h, nq, n, k), dtype=torch.uint8,
                                    device=q.device)
        tq_search_topk(self._h, q.contiguous(), nq, codes, norms, n, k, idx, score, workspace, stream)
        return idx, score


class PolarHandle(Handle):
    """Recursive polar transform handle ("PolarQuant explainer", sections 1 and 3): log2(d)
    levels of angles, ``bits_level1`` bits at level 1 and ``bits_upper`` at the others."""

    def __init__(self, d, bits_level1, bits_upper, seed=0, norm_dtype=None):
        self._h = tq_create_polar(d, bits_level1, bits_upper, seed)
        if norm_dtype is not None:
            tq_set_norm_dtype(self._h, norm_dtype)
        self.d, self.bits_mse, self.m, self.norm_dtype = tq_get_info(self._h)
        self.codes_B, self.signs_B = tq_code_bytes(self._h)
        self.levels, self.bits_level1, self.bits_upper = tq_polar_info(self._h)
        self.seed = seed
        self.index = _torch().cuda.current_device()

    def level_bits(self):
        return [self.bits_level1] + [self.bits_upper] * (self.levels - 1)

    def codebook(self, level=1):
        return tq_get_polar_codebook(self._h, level, self.level_bits()[level - 1])


class Cache:
    """A quantized K or V cache [B][Hkv][L_cap] for one handle (tensors + ABI struct)."""

    def __init__(self, handle, B, Hkv, L_cap, device="cuda"):
        self.handle, self.B, self.Hkv, self.L_cap = handle, B, Hkv, L_cap
        rows = handle.alloc_rows((B, Hkv, L_cap), device)
        self.codes, self.signs, self.norms, self.rnorms = rows["codes"], rows["signs"], rows["norms"], rows["rnorms"]
        self.struct = make_cache(self.codes, self.signs, self.norms, self.rnorms, L_cap)

    def fill(self, x, stream=None):
        """Encodes x [B, Hkv, L, d] into slots 0 .. L-1 of every (sequence, head)."""
        B, Hkv, L, d = x.shape
        assert (B, Hkv) == (self.B, self.Hkv) and L <= self.L_cap and d == self.handle.d
        if L == self.L_cap:
            tq_encode(self.handle.ptr, x.contiguous(), B * Hkv * L, self.codes, self.signs, self.norms,
                      self.rnorms, stream)
            return
        tmp = self.handle.encode(x.contiguous(), stream=stream)
        for name in ("codes", "norms", "signs", "rnorms"):
            if tmp[name] is not None:
                getattr(self, name)[:, :, :L].copy_(tmp[name])

    def append(self, x_new, len_, advance=True, stream=None):
        tq_append(self.handle.ptr, x_new.contiguous(), self.B, self.Hkv, self.struct, len_, advance, stream)


def score(hk, q, kcache, len_, logits=None, workspace=None, stream=None):
    """Scores q [B, Hq, d] fp32 against a key cache; logits [B, Hq, L_cap] fp32."""
    torch = _torch()
    B, Hq, _ = q.shape
    if logits is None:
        logits = torch.zeros((B, Hq, kcache.L_cap), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(tq_score_workspace_bytes(hk.ptr, B, Hq), dtype=torch.uint8, device=q.device)
    tq_score(hk.ptr, q.contiguous(), B, Hq, kcache.Hkv, kcache.struct, len_, logits, workspace, stream)
    return logits


def attn_decode(hk, hv, q, kcache, vcache, len_, scale, out=None, workspace=None, stream=None):
    """GQA decode attention of q [B, Hq, d] (fp32 or bf16) over quantized K/V caches -> fp32 [B, Hq, d]."""
    torch = _torch()
    B, Hq, d = q.shape
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(tq_attn_workspace_bytes(hk.ptr, hv.ptr, B, Hq, kcache.Hkv, kcache.L_cap),
                                dtype=torch.uint8, device=q.device)
    tq_attn_decode(hk.ptr, hv.ptr, q.contiguous(), B, Hq, kcache.Hkv, kcache.struct, vcache.struct, len_, scale,
                   out, workspace, stream)
    return out


# ------------------------------------------------------------------ paged caches


def _need(ok, what):
    if not ok:
        raise TQError(TQ_EINVAL, "paged", what)


class PagedCache:
    """A quantized K or V cache [num_pages][Hkv][page_size] for one handle (tensors + ABI struct).

    ``tensors`` wraps existing storage: a dict with "codes", "norms" and, for prod handles, "signs" and "rnorms",
    contiguous and of these shapes. New storage starts as zeros.
    """

    def __init__(self, handle, num_pages, Hkv, page_size, device="cuda", tensors=None):
        torch = _torch()
        self.handle, self.num_pages, self.Hkv, self.page_size = handle, num_pages, Hkv, page_size
        shape = (num_pages, Hkv, page_size)
        if tensors is None:
            tensors = {k: None if t is None else t.zero_() for k, t in handle.alloc_rows(shape, device).items()}
        want = {"codes": (handle.codes_B, torch.uint8), "norms": (0, handle.norm_torch_dtype()),
                "signs": (handle.signs_B, torch.uint8),
                "rnorms": (0, torch.float16) if handle.prod and not handle.qjl_only else None}
        for name, w in want.items():
            t = tensors.get(name)
            if w is None or (name in ("codes", "signs") and not w[0]):
                t = None
            else:
                _need(t is not None and t.dtype == w[1] and t.is_contiguous() and t.is_cuda
                      and tuple(t.shape) == shape + ((w[0],) if w[0] else ()),
                      f"{name}: contiguous {w[1]} {list(shape) + ([w[0]] if w[0] else [])} on the GPU wanted")
            setattr(self, name, t)
        self.device = self.norms.device
        _need(all(t is None or t.device == self.device for t in (self.codes, self.signs, self.rnorms)),
              "the cache's tensors must be on one device")
        self.index = self.norms.get_device()
        self.struct = make_paged_cache(self.codes, self.signs, self.norms, self.rnorms, num_pages, page_size)


class PagedBatch:
    """A ragged batch: token rows q_start[b] .. q_start[b+1] - 1 are the newest tokens of sequence b, which has len[b]
    tokens in the cache once they are in it; block_table [B, max_pages] names its pages. int32 tensors on the GPU, read
    when the work runs. ``ntok``: token rows of the call's tensors (rows past q_start[B] are padding); ``max_q``: no
    sequence has more token rows (default: ntok)."""

    def __init__(self, q_start, len_, block_table, ntok, max_q=None):
        torch = _torch()
        for name, t, n in (("q_start", q_start, 1), ("len", len_, 1), ("block_table", block_table, 2)):
            _need(t.dtype == torch.int32 and t.dim() == n and t.is_contiguous() and t.is_cuda and t.device == len_.device,
                  f"{name}: contiguous int32 tensor of {n} dimension(s) on the GPU wanted")
        _need(q_start.shape[0] == len_.shape[0] + 1 and block_table.shape[0] == len_.shape[0],
              "q_start [B + 1], len [B] and block_table [B, max_pages] disagree")
        self.q_start, self.len, self.block_table, self.ntok = q_start, len_, block_table, int(ntok)
        self.device, self.index = len_.device, len_.get_device()
        self.struct = make_paged_batch(q_start, len_, block_table, ntok, ntok if max_q is None else max_q)


class HeadPrep:
    """What each head goes through first: an RMS norm with ``weight`` [d] and ``eps``, then the rotation of its first
    cos_sin.shape[1] coordinates by the token's position (row of ``cos_sin`` [max_pos, rot_dim] fp32: rot_dim / 2 cosines,
    then the sines); pairs (i, i + rot_dim / 2), or (2 i, 2 i + 1) if ``interleaved``. ``pos`` int32 [ntok]: positions to
    rotate by (default: the positions in the cache)."""

    def __init__(self, cos_sin=None, interleaved=False, pos=None, weight=None, eps=1e-6):
        torch = _torch()
        if cos_sin is not None:
            _need(cos_sin.dtype == torch.float32 and cos_sin.dim() == 2 and cos_sin.is_contiguous() and cos_sin.is_cuda,
                  "cos_sin: contiguous float32 [max_pos, rot_dim] on the GPU wanted")
        if pos is not None:
            _need(cos_sin is not None, "pos without cos_sin")
            _need(pos.dtype == torch.int32 and pos.dim() == 1 and pos.is_contiguous() and pos.is_cuda,
                  "pos: contiguous int32 [ntok] on the GPU wanted")
        if weight is not None:
            _need(weight.dtype in (torch.float32, torch.float16, torch.bfloat16) and weight.dim() == 1
                  and weight.is_contiguous() and weight.is_cuda, "weight: contiguous [d] on the GPU wanted")
        self.cos_sin, self.pos, self.weight = cos_sin, pos, weight
        index = {t.get_device() for t in (cos_sin, pos, weight) if t is not None}
        _need(len(index) <= 1, "cos_sin, pos and weight are on different devices")
        self.index = index.pop() if index else None
        self.struct = make_head_prep(cos_sin, pos, weight, interleaved, eps)


def _head_rows(x, name, ntok, d):
    """x [ntok, H, d] with contiguous heads and 16-byte token strides; copied (on the current stream) if it is laid out
    otherwise."""
    if x.dim() != 3 or not x.is_cuda or x.shape[0] != ntok or x.shape[2] != d:
        _need(False, f"{name}: [{ntok}, heads, {d}] on the GPU wanted")
    s0, s1, s2 = x.stride()
    H = x.shape[1]
    if (s2 != 1 or (H > 1 and s1 != d) or s0 < H * d or s0 * x.element_size() % 16 or x.data_ptr() % 16):
        x = x.clone(memory_format=_torch().contiguous_format)
    return x


def _check_paged(hk, hv, kcache, vcache, batch, prep):
    for h, own in ((hk, kcache.handle), (hv, vcache.handle)):
        if h is not own and (h.d, h.bits_mse, h.m, h.norm_dtype) != (own.d, own.bits_mse, own.m, own.norm_dtype):
            _need(False, "a cache was made for rows of another format than its handle's")
    d = hk.d
    if kcache.Hkv != vcache.Hkv:
        _need(False, "the caches differ in Hkv")
    if not hk.index == hv.index == kcache.index == vcache.index == batch.index:
        _need(False, "handles, caches and batch are on different devices")
    if prep is not None:
        if prep.index is not None and prep.index != kcache.index:
            _need(False, "prep is on another device")
        if prep.weight is not None and prep.weight.shape[0] != d:
            _need(False, "weight: one value for each of the head's coordinates wanted")
        if prep.pos is not None and prep.pos.shape[0] < batch.ntok:
            _need(False, "pos: one position for each token row wanted")


def _raw_stream(index):
    """The current stream of a device, as the address the library takes."""
    return _torch().cuda.current_stream(index).cuda_stream


try:   # the same without a Stream object around it: calls for single tokens are bound by the host
    from torch._C import _cuda_getCurrentRawStream as _raw_stream  # noqa: F811
except ImportError:
    pass


def _on(stream, device):
    """The stream a call runs on, made current: what the call allocates or copies belongs to it too."""
    torch = _torch()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    _need(stream.device_index == device.index, "the stream and the caches are on different devices")
    return torch.cuda.stream(stream)


def append_paged(hk, hv, k, v, kcache, vcache, batch, prep=None, stream=None):
    """Quantizes the batch's keys (after ``prep``) and values k, v [ntok, Hkv, d] into their sequences' pages."""
    if stream is not None:
        with _on(stream, kcache.device):
            return append_paged(hk, hv, k, v, kcache, vcache, batch, prep)
    _check_paged(hk, hv, kcache, vcache, batch, prep)
    k, v = _head_rows(k, "k", batch.ntok, hk.d), _head_rows(v, "v", batch.ntok, hk.d)
    if not k.shape[1] == v.shape[1] == kcache.Hkv:
        _need(False, "k and v need one head for each of the caches'")
    if not k.get_device() == v.get_device() == kcache.index:
        _need(False, "k, v and the caches are on different devices")
    tq_append_paged(hk.ptr, hv.ptr, k, v, kcache.Hkv, batch.struct, None if prep is None else prep.struct, kcache.struct,
                    vcache.struct, _raw_stream(kcache.index))


def attn_paged(hk, hv, q, kcache, vcache, batch, scale, causal=True, window=0, prep=None, out=None, workspace=None,
               stream=None):
    """Attention of the batch's queries q [ntok, Hq, d] (after ``prep``) over their sequences' pages -> [ntok, Hq, d] of
    q's dtype. causal: each token over the positions up to its own (the last ``window`` of them if window > 0); not
    causal: over all len[b] cached tokens (cross attention). Rows of padding keep what ``out`` held (new: zeros)."""
    if stream is not None:
        with _on(stream, kcache.device):
            return attn_paged(hk, hv, q, kcache, vcache, batch, scale, causal, window, prep, out, workspace)
    _check_paged(hk, hv, kcache, vcache, batch, prep)
    q = _head_rows(q, "q", batch.ntok, hk.d)
    Hq = q.shape[1]
    if q.get_device() != kcache.index:
        _need(False, "q and the caches are on different devices")
    if out is None:
        out = _torch().zeros(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.get_device() != kcache.index:
        _need(False, "out: contiguous, of q's shape, dtype and device wanted")
    if workspace is None:
        size = tq_attn_paged_workspace_bytes(hk.ptr, hv.ptr, batch.struct, Hq, kcache.Hkv, kcache.struct)
        workspace = _torch().empty(max(16, size), dtype=_torch().uint8, device=q.device)
    elif workspace.get_device() != kcache.index or not workspace.is_contiguous():
        _need(False, "workspace: contiguous and on q's device wanted")
    tq_attn_paged(hk.ptr, hv.ptr, q, Hq, kcache.Hkv, batch.struct, None if prep is None else prep.struct, kcache.struct,
                  vcache.struct, scale, causal, window, out, workspace, _raw_stream(kcache.index))
    return out
