"""ctypes binding of the operators around the attention calls (include/smla.h):
rotary positions and the write and read side of the paged caches.

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
    i32, table, B = torch.int32, s.page_table, s.B
    c = SeqsT(_flat(s.cu_q, "cu_q", i32, dev, 1), _flat(s.kv_len, "kv_len", i32, dev, 1),
              _flat(table, "page_table", i32, dev, 2), B, s.max_pages, s.page_size, s.T)
    if s.cu_q.shape[0] <= B or s.kv_len.shape[0] < B or paged and (table.shape[0] < B or table.shape[1] != s.max_pages):
        raise ValueError(f"seqs: cu_q {tuple(s.cu_q.shape)}, kv_len {tuple(s.kv_len.shape)} and page_table "
                         f"{tuple(table.shape)} do not hold B={B} sequences of max_pages={s.max_pages}")
    return c


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
        dev = _device() if dev is None else dev
        return RopeT(_flat(self.inv_freq, "inv_freq", torch.float64, dev, 1), self.offset, 2 * self.inv_freq.shape[0],
                     self.layout, self.amplitude)


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
