"""ctypes binding of the operators around the attention calls (include/smla.h):
rotary positions, the write and read side of the paged caches, attention over
whole caches and in the expanded form, the 4-bit cache, and the 8-bit projections.

As in ``_lib``: argument marshalling only.  Every function checks its
tensors' types, layouts, sizes and device before the call, runs on the
current CUDA stream unless given one, and raises SmlaError when the library
returns a non-OK status.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import SMLA_BF16, SMLA_E4M3, SMLA_F32, RopeT, Seqs, SeqsT, _check, _stream

ROPE_INTERLEAVED, ROPE_HALF = 0, 1
_SCALINGS = {"plain": 0, "linear": 1, "yarn": 2}
_DTYPES = {torch.bfloat16: SMLA_BF16, torch.uint8: SMLA_E4M3, torch.float32: SMLA_F32}


# These calls take a few microseconds on the GPU, so the checks below keep to
# the cheapest queries of a tensor, and the message is put together only when
# one fails.
_U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _refuse(t, name, dtypes, dev, ndim):
    """The reason a tensor was not accepted, raised."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device (cuda:{dev}), got {t.device}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    raise ValueError(f"{name} must be contiguous")


def _flat(t, name, dtype, dev, ndim):
    """Pointer of a contiguous tensor of this type on the current device (the
    kernels launch there); None for None."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == ndim and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, (dtype,), dev, ndim)


def _rows(t, name, dtypes, dev, ndim):
    """Pointer, shape and leading strides (in elements) of a tensor whose last
    dimension is dense.  A dimension of one element has no stride to speak of:
    its row's width stands in."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.get_device() != dev or t.dim() != ndim:
        _refuse(t, name, dtypes, dev, ndim)
    shape, strides = t.shape, t.stride()
    width = shape[-1]
    if width > 1 and strides[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    if 1 in shape:
        strides = tuple(st if n > 1 else width for st, n in zip(strides, shape))
    return t.data_ptr(), shape, strides


def _seqs(s: Seqs, dev: int, paged: bool = True) -> SeqsT:
    """The C struct of a batch whose arrays hold what the kernels read: B + 1
    entries, B, and (`paged`: where pages are looked up) B rows of max_pages."""
    cu, kv, table, B = s.cu_q, s.kv_len, s.page_table, s.B
    try:  # (all checks at once; which one fails is found out below)
        nc, nk, nt = cu.shape, kv.shape, table.shape
        if (cu.dtype is _I32 and kv.dtype is _I32 and table.dtype is _I32 and cu.get_device() == dev and
                kv.get_device() == dev and table.get_device() == dev and len(nc) == 1 and len(nk) == 1 and len(nt) == 2 and
                nc[0] > B and nk[0] >= B and (not paged or nt[0] >= B and nt[1] == s.max_pages) and cu.is_contiguous() and
                kv.is_contiguous() and table.is_contiguous()):
            return SeqsT(cu.data_ptr(), kv.data_ptr(), table.data_ptr(), B, s.max_pages, s.page_size, s.T)
    except AttributeError:
        pass
    for t, name, ndim in ((cu, "cu_q", 1), (kv, "kv_len", 1), (table, "page_table", 2)):
        _flat(t, name, _I32, dev, ndim)
    raise ValueError(f"seqs: cu_q {tuple(cu.shape)}, kv_len {tuple(kv.shape)} and page_table "
                     f"{tuple(table.shape)} do not hold B={B} sequences of max_pages={s.max_pages}")


def _on(stream, dev: int) -> int:
    return _raw_stream(dev) if stream is None else _stream(stream)


def _pool(pool, dev: int):
    """(pointer, type code, rows, row width) of a cache pool."""
    bf16 = pool.dtype is torch.bfloat16
    ptr = _flat(pool, "pool", torch.bfloat16 if bf16 else torch.uint8, dev, 2)
    rows, width = pool.shape
    return ptr, SMLA_BF16 if bf16 else SMLA_E4M3, rows, width


def _scales(scales, rows: int, D: int, sbs: int, dev: int):
    """Pointer of a pool's scales [rows, ceil(D / sbs)]; None without."""
    if sbs == 0:
        if scales is not None:
            raise ValueError("scales must be None with scale_block_size 0")
        return None
    ptr = _flat(scales, "scales", torch.float32, dev, 2)
    want = (rows, 1 if sbs >= D else D // max(sbs, 1))
    if scales is None or scales.shape != want:
        raise ValueError(f"scales must be {want}, got {None if scales is None else tuple(scales.shape)}")
    return ptr


class Rope:
    """A rotary embedding over columns [offset, offset + 2 * len(inv_freq)) of
    a row: inv_freq f64 [dim/2] on the device (radians per position; see
    rope_frequencies), layout ROPE_INTERLEAVED or ROPE_HALF."""

    def __init__(self, inv_freq: torch.Tensor, offset: int, layout: int = ROPE_INTERLEAVED, amplitude: float = 1.0):
        self.inv_freq, self.offset, self.layout, self.amplitude = inv_freq, int(offset), int(layout), float(amplitude)

    def as_c(self, dev: Optional[int] = None) -> RopeT:
        dev, f = _device() if dev is None else dev, self.inv_freq
        return RopeT(_flat(f, "inv_freq", torch.float64, dev, 1), self.offset, 2 * f.shape[0], self.layout, self.amplitude)


def rope_frequencies(dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(inv_freq f64 [dim/2] on `device`, amplitude) of a rotary embedding:
    scaling "plain", "linear" (position interpolation) or "yarn"."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
    lib = _lib.load()
    out = torch.empty(max(int(dim), 0) // 2, dtype=torch.float64)
    amplitude = ctypes.c_float()
    _check(lib, lib.smla_rope_frequencies(int(dim), float(base), _SCALINGS[scaling], float(factor), int(original_len),
                                          float(beta_fast), float(beta_slow), out.data_ptr(),
                                          ctypes.byref(amplitude)))
    return out.to(device), amplitude.value


def rope(x: torch.Tensor, seqs: Seqs, rope: Rope, out: torch.Tensor, stream=None) -> torch.Tensor:
    """out[t, h] = x[t, h] with its rotary columns turned by token t's
    position.  x bf16 or f32 [T, H, D]; out bf16, f32 or uint8 (e4m3 bytes)
    [T, H, D], x itself for an in-place rotation.  Both may be strided views
    with dense rows."""
    lib, dev = _lib._lib or _lib.load(), _device()
    xp, shape, xs = _rows(x, "x", (torch.bfloat16, torch.float32), dev, 3)
    op, out_shape, os_ = _rows(out, "out", (torch.bfloat16, torch.float32, torch.uint8), dev, 3)
    if shape != out_shape or shape[0] != seqs.T:
        raise ValueError(f"x {tuple(shape)} and out {tuple(out_shape)} must both be [T={seqs.T}, H, D]")
    st = lib.smla_rope(xp, _DTYPES[x.dtype], xs[0], xs[1], _seqs(seqs, dev, False), shape[1], shape[2], rope.as_c(dev), op,
                       _DTYPES[out.dtype], os_[0], os_[1], _on(stream, dev))
    if st:
        _check(lib, st)
    return out


def cache_append(x: torch.Tensor, seqs: Seqs, pool: torch.Tensor, scales: Optional[torch.Tensor],
                 scale_block_size: int, rope: Optional[Rope] = None, norm_weight: Optional[torch.Tensor] = None,
                 norm_eps: float = 1e-6, rows_out: Optional[torch.Tensor] = None, stream=None):
    """Writes the batch's new rows x bf16 [T, D] into the paged pool (uint8
    e4m3 bytes or bf16, [phys_rows, D]) at their tokens' physical rows:
    RMS-normalised over the first norm_weight.shape[0] columns when a weight
    is given, rotated, quantised (scales f32 [phys_rows, nscale] written too);
    rows_out bf16 [T, D] also receives the finished rows."""
    lib, dev = _lib._lib or _lib.load(), _device()
    xp, (T, D), xs = _rows(x, "x", (torch.bfloat16,), dev, 2)
    rp, rs = None, D
    if rows_out is not None:
        rp, rows_shape, rs = _rows(rows_out, "rows_out", (torch.bfloat16,), dev, 2)
        rs = rs[0]
        if rows_shape != x.shape:
            raise ValueError("rows_out must have x's shape")
    pp, pd, phys_rows, width = _pool(pool, dev)
    if T != seqs.T or D != width:
        raise ValueError(f"x {tuple(x.shape)} must be [T={seqs.T}, D={width}]")
    sp = _scales(scales, phys_rows, D, scale_block_size, dev)
    st = lib.smla_cache_append(xp, xs[0], _seqs(seqs, dev), D, _flat(norm_weight, "norm_weight", torch.bfloat16, dev, 1),
                               0 if norm_weight is None else norm_weight.shape[0], norm_eps,
                               rope.as_c(dev) if rope is not None else RopeT(), pp, pd, phys_rows, sp, scale_block_size,
                               rp, rs, _on(stream, dev))
    if st:
        _check(lib, st)


def cache_gather(pool: torch.Tensor, scales: Optional[torch.Tensor], scale_block_size: int, seqs: Seqs,
                 rows: torch.Tensor, stream=None) -> torch.Tensor:
    """rows[t] bf16 = the cached row of seqs' token t, dequantised.  A Seqs
    whose cu_q is the running sum of kv_len reads the whole context."""
    lib, dev = _lib._lib or _lib.load(), _device()
    rp, (T, D), rs = _rows(rows, "rows", (torch.bfloat16,), dev, 2)
    pp, pd, phys_rows, width = _pool(pool, dev)
    if T != seqs.T or D != width:
        raise ValueError(f"rows {tuple(rows.shape)} must be [T={seqs.T}, D={width}]")
    sp = _scales(scales, phys_rows, D, scale_block_size, dev)
    st = lib.smla_cache_gather(pp, pd, phys_rows, sp, scale_block_size, _seqs(seqs, dev), D, rp, rs[0], _on(stream, dev))
    if st:
        _check(lib, st)
    return rows


def expanded_prefill_workspace_size(T: int, S: int, B: int, H: int) -> int:
    """Bytes of device scratch smla_expanded_prefill needs on the current device."""
    return int(_lib.load().smla_expanded_prefill_workspace_size(int(T), int(S), int(B), int(H)))


def expanded_prefill(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                     cu_kv: torch.Tensor, softmax_scale: float, out: torch.Tensor,
                     workspace: Optional[torch.Tensor], attn_sink: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, stream=None, p_terms: int = 0) -> torch.Tensor:
    """out bf16 [T, H, 128] = causal attention of q bf16 [T, H, 192] over keys
    [k_nope [S, H, 128] | k_rope [S, 64]] and values v [S, H, 128] (bf16,
    strided views with dense rows); cu_q, cu_kv int32 [B+1]; workspace a uint8
    CUDA tensor of at least expanded_prefill_workspace_size() bytes (None when
    that is 0); attn_sink f32 [H], lse f32 [T, H] (output).  p_terms: the bf16
    terms that the softmax weights are carried in, 1 or 2 (more exact, slower);
    0 leaves it to the library, which takes 2 in calls of up to 64 rows (T * H)."""
    lib, dev = _lib._lib or _lib.load(), _device()
    bf, f32, i32 = (torch.bfloat16,), torch.float32, torch.int32
    qp, q_shape, qs = _rows(q, "q", bf, dev, 3)
    kp, k_shape, ks = _rows(k_nope, "k_nope", bf, dev, 3)
    rp, r_shape, rs = _rows(k_rope, "k_rope", bf, dev, 2)
    vp, v_shape, vs = _rows(v, "v", bf, dev, 3)
    T, H, S, B = q_shape[0], q_shape[1], v_shape[0], cu_q.shape[0] - 1
    if (q_shape[2] != 192 or k_shape != (S, H, 128) or r_shape != (S, 64) or v_shape != (S, H, 128) or
            out.shape != (T, H, 128) or cu_kv.shape != (B + 1,) or
            (attn_sink is not None and attn_sink.shape != (H,)) or (lse is not None and lse.shape != (T, H))):
        raise ValueError("q [T, H, 192], k_nope [S, H, 128], k_rope [S, 64], v [S, H, 128], out [T, H, 128], cu_q and "
                         "cu_kv [B + 1], attn_sink [H], lse [T, H] do not fit each other")
    st = lib.smla_expanded_prefill_terms(qp, qs[0], qs[1], kp, ks[0], ks[1], rp, rs[0], vp, vs[0], vs[1],
                                         _flat(cu_q, "cu_q", i32, dev, 1), _flat(cu_kv, "cu_kv", i32, dev, 1), B, T, S,
                                         H, softmax_scale, p_terms, _flat(attn_sink, "attn_sink", f32, dev, 1),
                                         _flat(out, "out", torch.bfloat16, dev, 3), _flat(lse, "lse", f32, dev, 2),
                                         _flat(workspace, "workspace", torch.uint8, dev, 1),
                                         0 if workspace is None else workspace.numel(), _on(stream, dev))
    if st:
        _check(lib, st)
    return out


def dense_decode_workspace_size(T: int, H: int, max_kv_len: int) -> int:
    """Bytes of device scratch smla_dense_decode needs on the current device."""
    return int(_lib.load().smla_dense_decode_workspace_size(int(T), int(H), int(max_kv_len)))


def dense_decode(q: torch.Tensor, latent: torch.Tensor, scales: Optional[torch.Tensor], scale_block_size: int,
                 seqs: Seqs, max_kv_len: int, softmax_scale: float, out: torch.Tensor,
                 workspace: Optional[torch.Tensor], attn_sink: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """out bf16 [T, H, 512] = attention of each new token over its sequence's
    whole cache.  q bf16 or uint8 (e4m3 bytes) [T, H, 576]; latent uint8 (e4m3
    bytes) or bf16 [phys_rows, 576] with scales f32 [phys_rows, nscale] or
    None; workspace a uint8 CUDA tensor of at least
    dense_decode_workspace_size() bytes (None when that is 0)."""
    lib, dev = _lib._lib or _lib.load(), _device()
    bf16 = q.dtype is torch.bfloat16
    qp = _flat(q, "q", torch.bfloat16 if bf16 else torch.uint8, dev, 3)
    pp, pd, phys_rows, width = _pool(latent, dev)
    T, H, D = q.shape
    if (T != seqs.T or D != 576 or width != 576 or out.shape[:2] != (T, H) or
            (attn_sink is not None and attn_sink.shape != (H,))):
        raise ValueError(f"q must be [T={seqs.T}, H, 576], latent [phys_rows, 576], out [T, H, 512], attn_sink [H]")
    sp = _scales(scales, phys_rows, D, scale_block_size, dev)
    st = lib.smla_dense_decode(qp, SMLA_BF16 if bf16 else SMLA_E4M3, pp, pd, phys_rows, sp, scale_block_size,
                               _seqs(seqs, dev), max_kv_len, H, out.shape[2], softmax_scale,
                               _flat(attn_sink, "attn_sink", torch.float32, dev, 1),
                               _flat(out, "out", torch.bfloat16, dev, 3),
                               _flat(workspace, "workspace", torch.uint8, dev, 1),
                               0 if workspace is None else workspace.numel(), _on(stream, dev))
    if st:
        _check(lib, st)
    return out


FP4_ROW = 320  # bytes of a 4-bit cache row


# The calls below make all their checks in one condition, with the cheapest queries
# of a tensor; which check failed is found out behind it.  (A 16-row quantisation
# takes 2 us on the GPU, and a helper call for each tensor 4 us on the host.)
def _refuse_fp4_pool(pool, dev: int):
    _flat(pool, "pool", _U8, dev, 2)
    if pool.shape[1] != FP4_ROW:
        raise ValueError(f"a 4-bit pool must be [phys_rows, {FP4_ROW}], got {tuple(pool.shape)}")


def _on_device(t, dtype, dev: int) -> bool:
    """A contiguous tensor of this type on the device."""
    return t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def cache_append_fp4(x: torch.Tensor, seqs: Seqs, pool: torch.Tensor, rope: Optional[Rope] = None,
                     norm_weight: Optional[torch.Tensor] = None, norm_eps: float = 1e-6,
                     rows_out: Optional[torch.Tensor] = None, stream=None):
    """cache_append into a 4-bit latent cache: x bf16 [T, 576], pool uint8
    [phys_rows, 320] (codes, block shifts and the row's scale; include/smla.h)."""
    lib, dev = _lib._lib or _lib.load(), _device()
    T, shape, p_shape, n = seqs.T, x.shape, pool.shape, 0
    if not (shape == (T, 576) and len(p_shape) == 2 and p_shape[1] == FP4_ROW and x.dtype is _BF16 and
            x.get_device() == dev and x.stride(1) == 1 and _on_device(pool, _U8, dev)):
        _rows(x, "x", (_BF16,), dev, 2)
        _refuse_fp4_pool(pool, dev)
        raise ValueError(f"x {tuple(shape)} must be [T={T}, 576]")
    w = r = None
    r_stride = 576
    if norm_weight is not None:
        w, n = _flat(norm_weight, "norm_weight", _BF16, dev, 1), norm_weight.shape[0]
    if rows_out is not None:
        r, r_shape, r_stride = _rows(rows_out, "rows_out", (_BF16,), dev, 2)
        r_stride = r_stride[0]
        if r_shape != shape:
            raise ValueError("rows_out must have x's shape")
    st = lib.smla_cache_append_fp4(x.data_ptr(), x.stride(0) if T > 1 else 576, _seqs(seqs, dev), w, n, norm_eps,
                                   rope.as_c(dev) if rope is not None else RopeT(), pool.data_ptr(), p_shape[0], r,
                                   r_stride, _on(stream, dev))
    if st:
        _check(lib, st)


def cache_gather_fp4(pool: torch.Tensor, seqs: Seqs, rows: torch.Tensor, row_scales: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """rows[t] = the 4-bit cached row of seqs' token t: bf16 [T, 576], or, with
    row_scales f32 [T, 1], uint8 (e4m3 bytes) [T, 576], which hold the same
    values exactly and serve as a pool of the calls over e4m3 caches
    (scale_block_size 576)."""
    lib, dev = _lib._lib or _lib.load(), _device()
    T, shape, p_shape = seqs.T, rows.shape, pool.shape
    bf16 = row_scales is None
    if not (shape == (T, 576) and len(p_shape) == 2 and p_shape[1] == FP4_ROW and rows.dtype is (_BF16 if bf16 else _U8) and
            rows.get_device() == dev and rows.stride(1) == 1 and _on_device(pool, _U8, dev) and
            (bf16 or row_scales.shape == (T, 1) and _on_device(row_scales, _F32, dev))):
        _rows(rows, "rows", (_BF16 if bf16 else _U8,), dev, 2)
        _refuse_fp4_pool(pool, dev)
        _flat(row_scales, "row_scales", _F32, dev, 2)
        raise ValueError(f"rows {tuple(shape)} must be [T={T}, 576], row_scales [T, 1]")
    st = lib.smla_cache_gather_fp4(pool.data_ptr(), p_shape[0], _seqs(seqs, dev), rows.data_ptr(),
                                   SMLA_BF16 if bf16 else SMLA_E4M3, rows.stride(0) if T > 1 else 576,
                                   None if bf16 else row_scales.data_ptr(), _on(stream, dev))
    if st:
        _check(lib, st)
    return rows


def dense_decode_fp4(q: torch.Tensor, pool: torch.Tensor, seqs: Seqs, max_kv_len: int, softmax_scale: float,
                     out: torch.Tensor, workspace: Optional[torch.Tensor], attn_sink: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """dense_decode over a 4-bit latent cache, pool uint8 [phys_rows, 320];
    workspace of dense_decode_workspace_size() bytes."""
    lib, dev = _lib._lib or _lib.load(), _device()
    T, shape, p_shape, o_shape = seqs.T, q.shape, pool.shape, out.shape
    bf16 = q.dtype is _BF16
    if not (len(shape) == 3 and shape[0] == T and shape[2] == 576 and len(p_shape) == 2 and p_shape[1] == FP4_ROW and
            len(o_shape) == 3 and o_shape[:2] == shape[:2] and _on_device(q, _BF16 if bf16 else _U8, dev) and
            _on_device(pool, _U8, dev) and _on_device(out, _BF16, dev)):
        _flat(q, "q", _BF16 if bf16 else _U8, dev, 3)
        _refuse_fp4_pool(pool, dev)
        _flat(out, "out", _BF16, dev, 3)
        raise ValueError(f"q must be [T={T}, H, 576], out [T, H, 512]")
    H = shape[1]
    if attn_sink is not None and attn_sink.shape != (H,):
        raise ValueError(f"attn_sink must be [H={H}]")
    st = lib.smla_dense_decode_fp4(q.data_ptr(), SMLA_BF16 if bf16 else SMLA_E4M3, pool.data_ptr(), p_shape[0],
                                   _seqs(seqs, dev), max_kv_len, H, o_shape[2], softmax_scale,
                                   _flat(attn_sink, "attn_sink", _F32, dev, 1), out.data_ptr(),
                                   _flat(workspace, "workspace", _U8, dev, 1), 0 if workspace is None else workspace.numel(),
                                   _on(stream, dev))
    if st:
        _check(lib, st)
    return out


def quantize_blocks(x: torch.Tensor, out: torch.Tensor, scales: torch.Tensor, norm_weight: Optional[torch.Tensor] = None,
                    norm_eps: float = 1e-6, stream=None):
    """out uint8 (e4m3 bytes) [M, K] and scales f32 [M, ceil(K / 128)] of x bf16
    [M, K] (rows may be strided): a scale for each 128 columns, after an RMS norm
    over the row when its weight bf16 [K] is given."""
    lib, dev = _lib._lib or _lib.load(), _device()
    shape = x.shape
    M, K = shape if len(shape) == 2 else (0, 0)
    if not (len(shape) == 2 and out.shape == shape and scales.shape == (M, (K + 127) >> 7) and x.dtype is _BF16 and
            x.get_device() == dev and (x.stride(1) == 1 or K <= 1) and _on_device(out, _U8, dev) and
            _on_device(scales, _F32, dev) and (norm_weight is None or norm_weight.shape == (K,))):
        _rows(x, "x", (_BF16,), dev, 2)
        _flat(out, "out", _U8, dev, 2)
        _flat(scales, "scales", _F32, dev, 2)
        raise ValueError(f"out must be [M={M}, K={K}], scales [M, {-(-K // 128)}], norm_weight [K]")
    st = lib.smla_quantize_blocks(x.data_ptr(), x.stride(0) if M > 1 else K, M, K,
                                  _flat(norm_weight, "norm_weight", _BF16, dev, 1), norm_eps, out.data_ptr(),
                                  scales.data_ptr(), _on(stream, dev))
    if st:
        _check(lib, st)


def block_matmul(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor, out: torch.Tensor,
                 stream=None) -> torch.Tensor:
    """out[g] bf16 or f32 [M, N] = a[g] b[g]^T of e4m3 operands with a scale for
    each block of 128: a uint8 [G, M, K] with a_scales f32 [G, M, ceil(K / 128)]
    (both may be strided, as heads of a token-major tensor are; out too), b uint8
    [G, N, K] with b_scales f32 [G, ceil(N / 128), ceil(K / 128)] (contiguous).
    Without a batch all five are 2-D."""
    lib, dev = _lib._lib or _lib.load(), _device()
    shape, o_shape = a.shape, out.shape
    n = len(shape)
    if n == 3:
        G, M, K = shape
        lead = (G,)
    elif n == 2:
        (M, K), G, lead = shape, 1, ()
    else:
        raise ValueError(f"a must have 2 or 3 dims, got {n}")
    N, kb = o_shape[-1] if len(o_shape) else 0, (K + 127) >> 7
    a_st, s_st, o_st, out_type = a.stride(), a_scales.stride(), out.stride(), out.dtype
    # (all checks at once; which one fails is found out below)
    if not (o_shape == (*lead, M, N) and a_scales.shape == (*lead, M, kb) and b.shape == (*lead, N, K) and
            b_scales.shape == (*lead, (N + 127) >> 7, kb) and a.dtype is _U8 and b.dtype is _U8 and a_scales.dtype is _F32 and
            b_scales.dtype is _F32 and (out_type is _BF16 or out_type is _F32) and a.get_device() == dev and
            a_scales.get_device() == dev and b.get_device() == dev and b_scales.get_device() == dev and
            out.get_device() == dev and (a_st[-1] == 1 or K <= 1) and (o_st[-1] == 1 or N <= 1) and
            (kb == 1 or s_st[-1] == 1) and b.is_contiguous() and b_scales.is_contiguous()):
        _rows(a, "a", (_U8,), dev, n)
        _rows(a_scales, "a_scales", (_F32,), dev, n)
        _rows(out, "out", (_BF16, _F32), dev, n)
        _flat(b, "b", _U8, dev, n)
        _flat(b_scales, "b_scales", _F32, dev, n)
        raise ValueError("a [G, M, K], a_scales [G, M, ceil(K / 128)], b [G, N, K], b_scales [G, ceil(N / 128), ceil(K / "
                         "128)] and out [G, M, N] do not fit each other")
    st = lib.smla_block_matmul(a.data_ptr(), a_st[0], a_st[-2], a_scales.data_ptr(), s_st[0], s_st[-2], b.data_ptr(),
                               b_scales.data_ptr(), G, M, N, K, out.data_ptr(), SMLA_BF16 if out_type is _BF16 else SMLA_F32,
                               o_st[0], o_st[-2], _on(stream, dev))
    if st:
        _check(lib, st)
    return out
