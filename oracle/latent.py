"""Float64 reference of the operators around the attention calls: rotary
positions, the caches' write and read side, and attention in the expanded
form (test infrastructure only).  Written from the definitions in
include/smla.h."""
from __future__ import annotations

import math

import numpy as np

from .reference import dequant_rows, phys_rows_of, softmax_weights, token_positions

E4M3_MAX = 448.0


def rope_frequencies(dim, base=10000.0, scaling="plain", factor=1.0, original_len=4096, beta_fast=32.0,
                     beta_slow=1.0):
    """(inv_freq f64 [dim/2], amplitude).  YaRN: pair i turns original_len *
    f_i / (2 pi) times over the original length; pairs that turn more than
    beta_fast times keep f_i, fewer than beta_slow times f_i / factor, and the
    share of the latter rises linearly over the pair index between the two
    (rounded outwards to whole pairs)."""
    i = np.arange(dim // 2, dtype=np.float64)
    f = base ** (-2.0 * i / dim)
    if scaling == "plain":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    at = [dim / 2 * math.log(original_len / (2 * math.pi * turns), base) for turns in (beta_fast, beta_slow)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
    ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def rope(x, pos, inv_freq, offset, half, amplitude=1.0):
    """x float64 [T, ..., D] with columns [offset, offset + dim) turned by
    pos[t] * inv_freq[i]; also the sum |p| + |q| of each column's pair (0
    outside), the scale of its rounding errors."""
    y = np.array(x, dtype=np.float64)
    mass = np.zeros_like(y)
    n = len(inv_freq)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    shape = (y.shape[0],) + (1,) * (y.ndim - 2) + (n,)
    c, s = np.cos(ang).reshape(shape) * amplitude, np.sin(ang).reshape(shape) * amplitude
    first = offset + (np.arange(n) if half else 2 * np.arange(n))
    second = first + (n if half else 1)
    p, q = np.array(y[..., first]), np.array(y[..., second])
    y[..., first], y[..., second] = p * c - q * s, q * c + p * s
    mass[..., first] = mass[..., second] = (np.abs(p) + np.abs(q)) * abs(amplitude)
    return y, mass


def append_rows(x, pos, norm_weight=None, norm_eps=0.0, rope_args=None):
    """The finished rows of cache_append before quantisation, and the
    magnitude their rounding errors scale with."""
    r = np.array(x, dtype=np.float64)
    if norm_weight is not None:
        n = len(norm_weight)
        rms = np.sqrt((r[:, :n] ** 2).mean(axis=1, keepdims=True) + norm_eps)
        r[:, :n] = r[:, :n] / rms * norm_weight
    if rope_args is None:
        return r, np.abs(r)
    inv_freq, offset, half, amplitude = rope_args
    y, mass = rope(r, pos, inv_freq, offset, half, amplitude)
    return y, np.maximum(mass, np.abs(y))


def row_scales(rows, sbs):
    """The scales of e4m3 rows: largest finite magnitude / 448, 1 where that
    is 0, at least the smallest normal float32."""
    T, D = rows.shape
    width = D if sbs >= D else sbs
    a = np.abs(rows).reshape(T, D // width, width)
    amax = np.where(np.isfinite(a), a, 0.0).max(axis=2)
    return np.where(amax > 0, np.maximum(amax / E4M3_MAX, 2.0 ** -126), 1.0)


def gather(pool, scales, sbs, cu_q, kv_len, page_table, page_size):
    """Dequantised cached row of every token, float64."""
    pos, seq = token_positions(cu_q, kv_len)
    D = pool.shape[1]
    rows = np.array([phys_rows_of(page_table, page_size, int(b), np.array([p]))[0] for b, p in zip(seq, pos)],
                    dtype=np.int64)
    return dequant_rows(pool, scales, sbs, rows, D)


def expanded_prefill(q, k_nope, k_rope, v, cu_q, cu_kv, softmax_scale, attn_sink=None):
    """out[t, h] = softmax over keys 0..pos(t) of softmax_scale * (q_nope .
    k_nope[j, h] + q_rope . k_rope[j]), times v[j, h]; float64 [T, H, dv], and
    the natural-log sum of exponentials [T, H] (the sink included; -inf where
    nothing is attended).  A token before its sequence's first key attends to
    nothing: zeros."""
    T, H, _ = q.shape
    dn = k_nope.shape[2]
    out = np.zeros((T, H, v.shape[2]))
    lse = np.full((T, H), -np.inf)
    for b in range(len(cu_q) - 1):
        k0, n = int(cu_kv[b]), int(cu_kv[b + 1] - cu_kv[b])
        q0, m = int(cu_q[b]), int(cu_q[b + 1] - cu_q[b])
        for h in range(H):
            s = softmax_scale * (q[q0:q0 + m, h, :dn] @ k_nope[k0:k0 + n, h].T + q[q0:q0 + m, h, dn:] @ k_rope[k0:k0 + n].T)
            for i in range(m):
                keys = n - m + i + 1
                if keys > 0:
                    row = s[i:i + 1, :keys]
                    sink = None if attn_sink is None else attn_sink[h:h + 1]
                    out[q0 + i, h] = softmax_weights(row, sink) @ v[k0:k0 + keys, h]
                    top = row.max() if sink is None else max(row.max(), sink[0])
                    total = np.exp(row - top).sum() + (0.0 if sink is None else np.exp(sink[0] - top))
                    lse[q0 + i, h] = top + np.log(total)
                elif attn_sink is not None:
                    lse[q0 + i, h] = attn_sink[h]
    return out, lse
