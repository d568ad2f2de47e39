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
from ._lib import SMLA_BF16, SMLA_E4M3, SMLA_F32, RopeT, Seqs, _check, _ptr, _stream

ROPE_INTERLEAVED, ROPE_HALF = 0, 1
_SCALINGS = {"plain": 0, "linear": 1, "yarn": 2}
_DTYPES = {torch.bfloat16: SMLA_BF16, torch.uint8: SMLA_E4M3, torch.float32: SMLA_F32}


def _here(*tensors: Optional[torch.Tensor]):
    """The kernels launch on the current device: every tensor must be there."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and (not t.is_cuda or t.device.index != dev):
            raise ValueError(f"tensors must be on the current CUDA device (cuda:{dev}), got {t.device}")


def _rows(t: torch.Tensor, name: str, dtypes, ndim: int):
    """Pointer and the leading strides (in elements) of a tensor whose last
    dimension is dense.  A dimension of one element has no stride to speak
    of: its row's width stands in."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    strides = [t.stride(d) if t.shape[d] > 1 else t.shape[-1] for d in range(ndim - 1)]
    return (t.data_ptr() if t.numel() else None), strides


def _pool(pool: torch.Tensor):
    if pool.dtype not in (torch.uint8, torch.bfloat16):
        raise TypeError(f"pool must be torch.uint8 (e4m3 bytes) or torch.bfloat16, got {pool.dtype}")
    return _ptr(pool, pool.dtype, "pool", 2), SMLA_BF16 if pool.dtype == torch.bfloat16 else SMLA_E4M3


def _check_scales(scales: Optional[torch.Tensor], pool: torch.Tensor, sbs: int):
    if sbs == 0:
        if scales is not None:
            raise ValueError("scales must be None with scale_block_size 0")
        return
    D = int(pool.shape[1])
    want = (int(pool.shape[0]), 1 if sbs >= D else D // max(sbs, 1))
    if scales is None or tuple(scales.shape) != want:
        raise ValueError(f"scales must be {want}, got {None if scales is None else tuple(scales.shape)}")


class Rope:
    """A rotary embedding over columns [offset, offset + 2 * len(inv_freq)) of
    a row: inv_freq f64 [dim/2] on the device (radians per position; see
    rope_frequencies), layout ROPE_INTERLEAVED or ROPE_HALF."""

    def __init__(self, inv_freq: torch.Tensor, offset: int, layout: int = ROPE_INTERLEAVED, amplitude: float = 1.0):
        self.inv_freq, self.offset, self.layout, self.amplitude = inv_freq, int(offset), int(layout), float(amplitude)

    def as_c(self) -> RopeT:
        return RopeT(_ptr(self.inv_freq, torch.float64, "inv_freq", 1), self.offset, 2 * self.inv_freq.shape[0],
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
    lib = _lib.load()
    xp, xs = _rows(x, "x", (torch.bfloat16, torch.float32), 3)
    op, os_ = _rows(out, "out", (torch.bfloat16, torch.float32, torch.uint8), 3)
    _here(x, out, rope.inv_freq, seqs.cu_q, seqs.kv_len, seqs.page_table)
    if x.shape != out.shape or int(x.shape[0]) != seqs.T:
        raise ValueError(f"x {tuple(x.shape)} and out {tuple(out.shape)} must both be [T={seqs.T}, H, D]")
    st = lib.smla_rope(xp, _DTYPES[x.dtype], xs[0], xs[1], seqs.as_c(), int(x.shape[1]), int(x.shape[2]),
                       rope.as_c(), op, _DTYPES[out.dtype], os_[0], os_[1], _stream(stream))
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
    lib = _lib.load()
    xp, (xs,) = _rows(x, "x", (torch.bfloat16,), 2)
    rp, (rs,) = _rows(rows_out, "rows_out", (torch.bfloat16,), 2) if rows_out is not None else (None, (x.shape[1],))
    _here(x, pool, scales, rope.inv_freq if rope else None, norm_weight, rows_out, seqs.cu_q, seqs.kv_len,
          seqs.page_table)
    if int(x.shape[0]) != seqs.T or x.shape[1] != pool.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} must be [T={seqs.T}, D={int(pool.shape[1])}]")
    if rows_out is not None and rows_out.shape != x.shape:
        raise ValueError("rows_out must have x's shape")
    _check_scales(scales, pool, scale_block_size)
    pp, pd = _pool(pool)
    st = lib.smla_cache_append(xp, xs, seqs.as_c(), int(x.shape[1]),
                               _ptr(norm_weight, torch.bfloat16, "norm_weight", 1),
                               0 if norm_weight is None else int(norm_weight.shape[0]), float(norm_eps),
                               rope.as_c() if rope else RopeT(), pp, pd, int(pool.shape[0]),
                               _ptr(scales, torch.float32, "scales", 2), int(scale_block_size), rp, rs,
                               _stream(stream))
    _check(lib, st)


def cache_gather(pool: torch.Tensor, scales: Optional[torch.Tensor], scale_block_size: int, seqs: Seqs,
                 rows: torch.Tensor, stream=None) -> torch.Tensor:
    """rows[t] bf16 = the cached row of seqs' token t, dequantised.  A Seqs
    whose cu_q is the running sum of kv_len reads the whole context."""
    lib = _lib.load()
    rp, (rs,) = _rows(rows, "rows", (torch.bfloat16,), 2)
    _here(pool, scales, rows, seqs.cu_q, seqs.kv_len, seqs.page_table)
    if int(rows.shape[0]) != seqs.T or rows.shape[1] != pool.shape[1]:
        raise ValueError(f"rows {tuple(rows.shape)} must be [T={seqs.T}, D={int(pool.shape[1])}]")
    _check_scales(scales, pool, scale_block_size)
    pp, pd = _pool(pool)
    st = lib.smla_cache_gather(pp, pd, int(pool.shape[0]), _ptr(scales, torch.float32, "scales", 2),
                               int(scale_block_size), seqs.as_c(), int(rows.shape[1]), rp, rs, _stream(stream))
    _check(lib, st)
    return rows


def expanded_prefill_workspace_size(T: int, S: int, B: int, H: int) -> int:
    """Bytes of device scratch smla_expanded_prefill needs on the current device."""
    return int(_lib.load().smla_expanded_prefill_workspace_size(int(T), int(S), int(B), int(H)))


def expanded_prefill(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                     cu_kv: torch.Tensor, softmax_scale: float, out: torch.Tensor,
                     workspace: Optional[torch.Tensor], attn_sink: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out bf16 [T, H, 128] = causal attention of q bf16 [T, H, 192] over keys
    [k_nope [S, H, 128] | k_rope [S, 64]] and values v [S, H, 128] (bf16,
    strided views with dense rows); cu_q, cu_kv int32 [B+1]; workspace a uint8
    CUDA tensor of at least expanded_prefill_workspace_size() bytes (None when
    that is 0); attn_sink f32 [H], lse f32 [T, H] (output)."""
    lib = _lib.load()
    bf = (torch.bfloat16,)
    qp, (qt, qh) = _rows(q, "q", bf, 3)
    kp, (kt, kh) = _rows(k_nope, "k_nope", bf, 3)
    rp, (rt,) = _rows(k_rope, "k_rope", bf, 2)
    vp, (vt, vh) = _rows(v, "v", bf, 3)
    _here(q, k_nope, k_rope, v, cu_q, cu_kv, out, workspace, attn_sink, lse)
    T, H, S, B = int(q.shape[0]), int(q.shape[1]), int(v.shape[0]), int(cu_q.shape[0]) - 1
    if (tuple(q.shape) != (T, H, 192) or tuple(k_nope.shape) != (S, H, 128) or tuple(k_rope.shape) != (S, 64) or
            tuple(v.shape) != (S, H, 128) or tuple(out.shape) != (T, H, 128) or tuple(cu_kv.shape) != (B + 1,) or
            (attn_sink is not None and tuple(attn_sink.shape) != (H,)) or
            (lse is not None and tuple(lse.shape) != (T, H))):
        raise ValueError("q [T, H, 192], k_nope [S, H, 128], k_rope [S, 64], v [S, H, 128], out [T, H, 128], cu_q and "
                         "cu_kv [B + 1], attn_sink [H], lse [T, H] do not fit each other")
    st = lib.smla_expanded_prefill(qp, qt, qh, kp, kt, kh, rp, rt, vp, vt, vh, _ptr(cu_q, torch.int32, "cu_q", 1),
                                   _ptr(cu_kv, torch.int32, "cu_kv", 1), B, T, S, H, float(softmax_scale),
                                   _ptr(attn_sink, torch.float32, "attn_sink", 1),
                                   _ptr(out, torch.bfloat16, "out", 3), _ptr(lse, torch.float32, "lse", 2),
                                   _ptr(workspace, torch.uint8, "workspace", 1),
                                   0 if workspace is None else int(workspace.numel()), _stream(stream))
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
    lib = _lib.load()
    qd, qp = _lib._q_arg(q)
    _here(q, latent, scales, out, workspace, attn_sink, seqs.cu_q, seqs.kv_len, seqs.page_table)
    T, H = int(q.shape[0]), int(q.shape[1])
    if (T != seqs.T or tuple(q.shape) != (T, H, 576) or latent.shape[1] != 576 or tuple(out.shape[:2]) != (T, H) or
            (attn_sink is not None and tuple(attn_sink.shape) != (H,))):
        raise ValueError(f"q must be [T={seqs.T}, H, 576], latent [phys_rows, 576], out [T, H, 512], attn_sink [H]")
    _check_scales(scales, latent, scale_block_size)
    pp, pd = _pool(latent)
    st = lib.smla_dense_decode(qp, qd, pp, pd, int(latent.shape[0]), _ptr(scales, torch.float32, "scales", 2),
                               int(scale_block_size), seqs.as_c(), int(max_kv_len), H, int(out.shape[2]),
                               float(softmax_scale), _ptr(attn_sink, torch.float32, "attn_sink", 1),
                               _ptr(out, torch.bfloat16, "out", 3), _ptr(workspace, torch.uint8, "workspace", 1),
                               0 if workspace is None else int(workspace.numel()), _stream(stream))
    _check(lib, st)
    return out
