"""How exactly dense decode weighs its keys, against float64.

The queries are zero outside the rotary columns, so that a key's logit is set
by its rotary columns and its values by the others, each apart.

Tolerance, from the arithmetic and at its worst (nothing is taken as random).
  weights   each is off by at most 2^-8 of itself: bf16's rounding; three e5m2
            terms are off by 2^-9, and 2^-11 for the f16 that they are taken
            from.  Terms of e5m2 end at half of its smallest step, 2^-17, in
            units that put a row's largest weight at 2^11 or more: 2^-28 of that
            largest (of p_j s_j, s_j the key row's scale; f16's floor is lower).
  logits    64 products, of two terms each where q is bf16, summed in float32:
            off by 128 * 2^-23 of sum |q k| * scale, and a weight by twice the
            largest of that; 2^-18 for the exponential and its argument.
  sums      n keys in float32: n * 2^-24 of sum p |v|.
  output    rounded to bf16, 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

import serving_fp8_indexer_gb300 as smla
import test_gpu_dense_decode as dense
from serving_fp8_indexer_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5
MODES = [("bf16", "unit"), ("bf16", "row"), ("e4m3", "unit"), ("e4m3", "row"), ("e4m3", "block"), ("bf16", "bf16")]


def _e4m3(x):
    return x.to(torch.float8_e4m3fn)


def _pool(values, mode, gen):
    """(pool, scales, scale_block_size, float64 values) of rows near `values`
    [rows, 576]; row and block scales are powers of two, so that nothing but
    the weights is rounded on the way."""
    if mode == "bf16":
        b = values.bfloat16()
        return b, None, 0, b.double()
    if mode == "unit":
        b = _e4m3(values)
        return b.view(torch.uint8), None, 0, b.double()
    rows, blocks = values.shape[0], 1 if mode == "row" else 18
    s = 2.0 ** torch.randint(-3, 3, (rows, blocks), generator=gen, device="cuda").float()
    b = _e4m3((values.view(rows, blocks, -1) / s[:, :, None]).view(rows, 576))
    val = (b.double().view(rows, blocks, -1) * s.double()[:, :, None]).view(rows, 576)
    return b.view(torch.uint8), s.contiguous(), 576 // blocks, val


def _floor(mode):
    return 0.0 if mode == "bf16" else 2.0 ** -28


def _reference(q, val, scales, kv_lens, table, page, mode):
    """(out, tolerance) float64 of one token for each sequence."""
    q64 = q.double() if q.dtype == torch.bfloat16 else q.view(torch.float8_e4m3fn).double()
    out = torch.zeros((q.shape[0], q.shape[1], 512), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for b, n in enumerate(kv_lens):
        key = torch.arange(n, device="cuda")
        rows = table[b].long()[key // page] * page + key % page
        k = val[rows]
        p = torch.softmax(SCALE * q64[b] @ k.T, 1)
        v = k[:, :512]
        out[b] = p @ v
        mass = SCALE * (q64[b].abs() @ k.abs().T).amax(1, keepdim=True)
        rel = 2.0 ** -8 + 2 * 128 * 2.0 ** -23 * mass + 2.0 ** -18 + n * 2.0 ** -24
        sj = torch.ones(n, dtype=torch.float64, device="cuda") if scales is None else scales[rows].double().amax(1)
        floor = _floor(mode) * (p * sj).amax(1, keepdim=True) * (v / sj[:, None]).abs().sum(0)
        tol[b] = rel * (p @ v.abs()) + floor + 2.0 ** -8 * out[b].abs()
    return out, tol


def _decode(q, pool, scales, sbs, seqs, most):
    n = smla.dense_decode_workspace_size(seqs.T, q.shape[1], most)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    out = torch.full((seqs.T, q.shape[1], 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    smla.dense_decode(q, pool, scales, sbs, seqs, most, SCALE, out, ws)
    smla.check_device_errors()
    return out


def _batch(kv_lens, page=64, seed=0):
    s = wl.make_seqs(np.random.default_rng(seed), [1] * len(kv_lens), kv_lens, page)
    return s, smla.Seqs.from_host(s)


def _close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp_min(1e-30)).max()):.3g} x the tolerance"


def _peaked(s, seqs, H, qd, mode, peaks, jitter, seed):
    """Keys `peaks` of every sequence lie 4 to 14 nats (by head) above the
    others, which lie within `jitter` of each other; the peaks' values are 0,
    the others' have mean 0.5."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = max(s.phys_rows, 1)
    x = torch.zeros((rows, 576), device="cuda")
    x[:, :512] = 0.5 + 0.25 * torch.randn((rows, 512), generator=g, device="cuda") if jitter else 0.5
    x[:, 513:] = jitter * torch.randn((rows, 63), generator=g, device="cuda")
    for b in range(s.B):
        at = torch.from_numpy(wl.logical_to_phys(s, b, peaks[peaks < int(s.kv_len[b])])).cuda()
        x[at] = 0.0
        x[at, 512] = 1.0
    pool, scales, sbs, val = _pool(x, mode, g)
    q = torch.zeros((s.T, H, 576), device="cuda")
    q[:, :, 512] = 24.0 * torch.linspace(4.0, 14.0, H, device="cuda")
    if jitter:
        q[:, :, 513:] = torch.randn((s.T, H, 63), generator=g, device="cuda") * 4
    q = q.bfloat16() if qd == "bf16" else _e4m3(q).view(torch.uint8)
    return q, pool, scales, sbs, val


@pytest.mark.parametrize("qd,mode", MODES)
@pytest.mark.parametrize("jitter", [0.0, 0.25])
@pytest.mark.parametrize("n,H", [(700, 16), (4099, 64), (32768, 16), (9001, 32), (20000, 128)])
def test_a_dominant_key_does_not_take_the_others_weight(qd, mode, jitter, n, H):
    """One key far above thousands of others, in the first block or a late one,
    whole (one CTA for everything) and cut over the CTAs."""
    s, seqs = _batch([n])
    for at in (0, n - 130):
        q, pool, scales, sbs, val = _peaked(s, seqs, H, qd, mode, np.array([at]), jitter, seed=n)
        ref, tol = _reference(q, val, scales, [n], seqs.page_table, 64, mode)
        for most in (1, n):
            _close(_decode(q, pool, scales, sbs, seqs, most), ref, tol)


@pytest.mark.parametrize("qd,mode", MODES)
@pytest.mark.parametrize("H", [16, 32, 64])
def test_dominant_keys_in_every_block(qd, mode, H):
    """Each block of 128 keys has one, so that no block's weights are near each
    other; more sequences than CTAs, so that items are whole."""
    lens = [300 + 13 * i for i in range(3)] + [257] * 160
    s, seqs = _batch(lens)
    q, pool, scales, sbs, val = _peaked(s, seqs, H, qd, mode, np.arange(5, 400, 100), 0.25, seed=7)
    ref, tol = _reference(q, val, scales, lens, seqs.page_table, 64, mode)
    _close(_decode(q, pool, scales, sbs, seqs, max(lens)), ref, tol)


@pytest.mark.parametrize("qd,mode", [("bf16", "unit"), ("bf16", "row"), ("bf16", "bf16")])
@pytest.mark.parametrize("H", [16, 64, 128])
def test_infinite_queries_give_nan_whatever_their_logits(qd, mode, H):
    """An infinite query element against keys of one sign: every logit is -inf
    (or +inf), and the row NaN all the same; the other rows do not see it, and a
    token without keys still gets zeros."""
    lens = [1, 900, 0, 40, 129]
    s, seqs = _batch([max(n, 1) for n in lens])
    seqs.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((s.phys_rows, 576), generator=g, device="cuda").abs() + 0.1
    pool, scales, sbs, _ = _pool(x, mode, g)
    q = torch.randn((5, H, 576), generator=g, device="cuda").bfloat16()
    clean = {most: _decode(q, pool, scales, sbs, seqs, most) for most in (1, 900)}
    bad = q.clone()
    rows = torch.zeros((5, H), dtype=torch.bool, device="cuda")
    for b in range(5):
        bad[b, 1, 7] = -float("inf")
        bad[b, H - 1, 575] = float("inf")
        rows[b, 1] = rows[b, H - 1] = lens[b] > 0
    for most in (1, 900):  # whole, and cut
        got = _decode(bad, pool, scales, sbs, seqs, most)
        assert bool(got[rows].isnan().all())
        assert torch.equal(got[~rows], clean[most][~rows]) and bool((got[2] == 0).all())


def _spread_blocks(rows, spread, zeros, gen):
    """A block-scaled pool whose row blocks differ by the powers of two `spread`
    (in turn, by block), with other scales' bits at random; the rotary blocks'
    scales are 1.  `zeros`: the blocks of the largest scale hold nothing."""
    x = torch.randn((rows, 18, 32), generator=gen, device="cuda") * 64
    e = torch.tensor([spread[i % len(spread)] for i in range(16)] + [0, 0], device="cuda").float()
    s = 2.0 ** -e * (1 + torch.rand((rows, 18), generator=gen, device="cuda"))
    s[:, 16:] = 1.0
    if zeros:
        x[:, :16][:, e[:16] == 0] = 0.0
    x[:, 16:] /= 64
    b = _e4m3(x)
    return b.view(rows, 576).view(torch.uint8), s.contiguous(), (b.double() * s.double()[:, :, None]).view(rows, 576)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("spread", [(0, 3), (0, 13, 14, 15), (0, 17, 18, 19), (0, 20, 21, 24), (0, 26)])
@pytest.mark.parametrize("H", [16, 64])
def test_blocks_of_very_different_scales(H, spread, zeros):
    """Every block's columns to the same relative accuracy, whatever the scales
    of the row's other blocks.  The rotary part's products are exact in f16, so
    no logit is off by more than its float32 sum; a value is off by 2^-11 for its
    scale and 2^-11 for its product, or half of f16's smallest step in units of
    2^-5 of the row's largest scale (taken as its power of two, 2^-30 at most); a
    weight by 2^-11."""
    lens = [1, 700, 1100]
    s, seqs = _batch(lens, seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    pool, scales, val = _spread_blocks(s.phys_rows, spread, zeros, g)
    q = torch.zeros((3, H, 576), device="cuda")
    q[:, :, 512:] = torch.randn((3, H, 64), generator=g, device="cuda") * 4
    q8 = _e4m3(q).view(torch.uint8)
    ref, _ = _reference(q8, val, scales, lens, seqs.page_table, 64, "block")
    tol = torch.zeros_like(ref)
    q64 = q8.view(torch.float8_e4m3fn).double()
    for b, n in enumerate(lens):
        key = torch.arange(n, device="cuda")
        rows = seqs.page_table[b].long()[key // 64] * 64 + key % 64
        p = torch.softmax(SCALE * q64[b] @ val[rows].T, 1)
        mass = SCALE * (q64[b].abs() @ val[rows].abs().T).amax(1, keepdim=True)
        rel = 3 * 2.0 ** -11 + 2 * 64 * 2.0 ** -23 * mass + 2.0 ** -18 + n * 2.0 ** -24
        tol[b] = rel * (p @ val[rows, :512].abs()) + 2.0 ** -30 * (p @ scales[rows].double().amax(1))[:, None]
    tol += 2.0 ** -8 * ref.abs()
    for most in (1, 1100):
        _close(_decode(q8, pool, scales, 32, seqs, most), ref, tol)


@pytest.mark.parametrize("qd,mode", MODES)
@pytest.mark.parametrize("q_lens,kv_lens,H", [([1, 2], [3000, 1100], 16), ([2], [5000], 32), ([1, 1], [777, 2500], 128)])
def test_error_beside_the_rounding_of_the_output(qd, mode, q_lens, kv_lens, H):
    """Root mean square, in units of the output's own rounding r (2^-8 / sqrt(3) of
    an element where that is largest, as for every rounding below).  Unit and row
    scales: q and K are exact and a weight is off by half of r (2^-9): sqrt(1 +
    1/4) = 1.12.  Block scales: scale and product off by r / 8 each, in the logits
    and in the values, the weight by r / 8: sqrt(1 + 5 / 64) = 1.04.  bf16: the
    weight by r: 1.42.  A tenth more for the sums in float32 and the sample."""
    s, seqs, q, pool, scales, sbs, val = dense._case(q_lens, kv_lens, H, qd, mode, seed=41)
    ref, _ = dense._reference(s, q, val, **dense._carried(scales, pool))
    most = {"bf16": 1.42, "block": 1.04}.get(mode, 1.12) * 1.1
    rounding = float((ref.bfloat16().double() - ref).norm())
    for bound in (1, max(kv_lens)):
        got = _decode(q, pool, scales, sbs, seqs, bound)
        assert float((got.double() - ref).norm()) <= most * rounding


@pytest.mark.parametrize("mode", ["unit", "row", "bf16"])
@pytest.mark.parametrize("large", [30.0, 3000.0])
@pytest.mark.parametrize("H", [16, 64])
def test_one_large_query_element_leaves_the_others_their_bits(mode, large, H):
    """A query element far above the others, in a column where the keys are 0: the
    logits come from the others alone.  Over an e4m3 cache bf16 elements are exact
    down to 2^-14 of the largest and off by 2^-22 of it below (3000: 0.0007 beside
    elements of size 1), which moves a logit by less than 0.0007 and a weight by
    0.07 %, a fifth of the output's rounding; the rest as in the test above."""
    s, seqs, q, pool, scales, sbs, val = dense._case([1, 2], [2000, 700], H, "bf16", mode, seed=43)
    q[:, :, 300] = large
    q[:, ::2, 300] = -large
    pool[:, 300] = 0
    val[:, 300] = 0
    ref, _ = dense._reference(s, q, val, **dense._carried(scales, pool))
    most = ({"bf16": 1.42}.get(mode, 1.12) + 0.02) * 1.1
    rounding = float((ref.bfloat16().double() - ref).norm())
    for bound in (1, 2000):
        got = _decode(q, pool, scales, sbs, seqs, bound)
        assert float((got.double() - ref).norm()) <= most * rounding
