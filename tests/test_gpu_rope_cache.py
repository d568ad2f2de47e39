"""Rotary positions and the caches' write and read side against the float64
oracle.

Tolerances, from the arithmetic (u = 2^-24, the rounding of one float32
operation):
  * rotation: the reduced angle is off by at most pi * 2^-25 (1.6 u), sin and
    cos by 2 ulp (4 u) and the amplitude's product by 1 u; each of p cos and
    q sin adds a rounding and so does their sum: below 9 u of |p| + |q|,
    times the amplitude.  ROT = 16 u.
  * norm: a sum of 512 squares, at most 32 in a row in one lane and then five
    exchanges, is off by 37 u, its root by half of that, and the division,
    root and two products add 4: below 23 u.  NORM = 32 u, and ROT more where
    the normalised value is rotated.
  * a scale is its block's largest magnitude / 448, off by that magnitude's
    error (twice its relative size where it was rotated: |p| + |q| is at most
    twice the larger of the two results) and one division: 2 (NORM + ROT) + u.
  * outputs round once more: bf16 by 2^-8 of the value, e4m3 by 2^-4, or half
    its smallest step, 2^-10.
"""
import numpy as np
import pytest
import torch

import oracle
import oracle.latent as ol
import serving_fp8_indexer_gb300 as smla
from oracle.reference import decode_bf16, phys_rows_of, token_positions
from serving_fp8_indexer_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROT, NORM = 16 * U, 32 * U
HALF_STEP = {"bf16": (2.0 ** -8, 0.0), "e4m3": (2.0 ** -4, 2.0 ** -10), "f32": (0.0, 0.0)}
OUT = {"bf16": torch.bfloat16, "e4m3": torch.uint8, "f32": torch.float32}


def _bf16(x):
    """float64 values of x rounded to bf16, and the tensor."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def _np(t):
    return t.cpu().view(torch.float8_e4m3fn).double().numpy() if t.dtype == torch.uint8 else t.double().cpu().numpy()


def _batch(rng, q_lens, kv_lens, page=64):
    s = wl.make_seqs(rng, q_lens, kv_lens, page)
    return s, smla.Seqs.from_host(s), token_positions(s.cu_q, s.kv_len)[0]


def _freq(dim, scaling="plain"):
    return ol.rope_frequencies(dim, scaling=scaling, factor=40.0)


def _rope(dim, offset, half, scaling="plain"):
    f, a = smla.rope_frequencies(dim, scaling=scaling, factor=40.0)
    return smla.Rope(f, offset, smla.ROPE_HALF if half else smla.ROPE_INTERLEAVED, a)


@pytest.mark.parametrize("scaling", ["plain", "linear", "yarn"])
@pytest.mark.parametrize("dim", [16, 64, 128])
def test_frequencies(scaling, dim):
    f, a = ol.rope_frequencies(dim, scaling=scaling, factor=16.0, original_len=8192)
    g, b = smla.rope_frequencies(dim, scaling=scaling, factor=16.0, original_len=8192, device="cpu")
    np.testing.assert_allclose(g.numpy(), f, rtol=1e-14)
    assert abs(a - b) <= 2.0 ** -24 * a


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("H,D,offset,dim", [(1, 16, 0, 16), (3, 64, 0, 64), (128, 576, 512, 64), (5, 200, 8, 160),
                                            (2, 1024, 0, 1024), (7, 192, 128, 64)])
@pytest.mark.parametrize("out", ["bf16", "e4m3", "f32"])
def test_rope(half, H, D, offset, dim, out):
    rng = np.random.default_rng(H * D + dim)
    # one token, a batch with an empty sequence, and far positions
    s, seqs, pos = _batch(rng, [1, 0, 5, 3], [1, 9, 5, 260001])
    x64, x = _bf16(rng.standard_normal((s.T, H, D)) * 3)
    y = torch.empty((s.T, H, D), dtype=OUT[out], device="cuda")
    smla.rope(x, seqs, _rope(dim, offset, half, "yarn"), y)
    smla.check_device_errors()
    f, a = _freq(dim, "yarn")
    ref, mass = ol.rope(x64, pos, f, offset, half, a)
    rel, step = HALF_STEP[out]
    tol = ROT * mass * (1 + rel) + rel * np.abs(ref) + step
    assert (np.abs(_np(y) - np.clip(ref, -448, 448) if out == "e4m3" else _np(y) - ref) <= tol).all()


def test_rope_f32_input_and_saturation():
    rng = np.random.default_rng(1)
    s, seqs, pos = _batch(rng, [4], [4])
    x = torch.randn((4, 2, 32), device="cuda") * 400
    y = torch.empty((4, 2, 32), dtype=torch.uint8, device="cuda")
    smla.rope(x, seqs, _rope(16, 16, True), y)
    f, a = _freq(16)
    ref, mass = ol.rope(x.double().cpu().numpy(), pos, f, 16, True, a)
    ref = np.clip(ref, -448, 448)
    assert (np.abs(_np(y) - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 + 2 * ROT * mass).all()
    assert (np.abs(ref) == 448).any()


def test_rope_far_positions_keep_their_angle():
    """At position 2^30 a float32 angle would be off by many turns."""
    s, seqs, pos = _batch(np.random.default_rng(2), [2], [2], 4096)
    seqs.kv_len.fill_(2 ** 30)
    x = torch.randn((2, 1, 64), device="cuda")
    y = torch.empty_like(x)
    smla.rope(x, seqs, _rope(64, 0, False), y)
    smla.check_device_errors()
    # the oracle's angle rounds once, by 2^-24 radians at 2^30; the kernel's
    # step of f / 2 pi turns twice, by 2^-55 turns, 2^-22 radians after 2^30
    # positions: 2^-21 covers both
    f, a = _freq(64)
    ref, mass = ol.rope(x.double().cpu().numpy(), np.array([2 ** 30 - 2, 2 ** 30 - 1]), f, 0, False, a)
    assert (np.abs(_np(y) - ref) <= (ROT + 2.0 ** -21) * mass).all()


@pytest.mark.parametrize("half", [False, True])
def test_rope_in_place_and_strided(half):
    """The rotary part of a projection's output, a strided view, in place and
    into the tail of the absorbed query: nothing else changes."""
    rng = np.random.default_rng(3)
    s, seqs, pos = _batch(rng, [33], [70])
    x64, proj = _bf16(rng.standard_normal((33, 6, 192)))
    q = torch.full((33, 6, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    rope = _rope(64, 0, half)
    smla.rope(proj[:, :, 128:], seqs, rope, q[:, :, 512:])
    before = proj.clone()
    whole = torch.empty_like(proj)
    smla.rope(proj, seqs, _rope(64, 128, half), whole)
    smla.rope(proj[:, :, 128:], seqs, rope, proj[:, :, 128:])
    smla.check_device_errors()
    assert torch.equal(proj[:, :, :128], before[:, :, :128]) and bool((q[:, :, :512] == 7).all())
    assert torch.equal(proj[:, :, 128:], q[:, :, 512:]) and torch.equal(whole, proj)
    ref, mass = ol.rope(x64, pos, _freq(64)[0], 128, half)
    assert (np.abs(_np(whole) - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * ROT * mass).all()


def test_padded_batch_and_short_sequence():
    """Tokens behind the last sequence keep their outputs; a sequence with
    more new tokens than cached ones is reported."""
    rng = np.random.default_rng(4)
    s, seqs, pos = _batch(rng, [3, 2], [10, 5])
    padded = smla.Seqs(seqs.cu_q, seqs.kv_len, seqs.page_table, 64, 9)
    x = torch.randn((9, 4, 64), device="cuda").bfloat16()
    y = torch.full_like(x, 5.0)
    smla.rope(x, padded, _rope(64, 0, False), y)
    pool = torch.full((s.phys_rows, 64), 0xA5, dtype=torch.uint8, device="cuda")
    rows = torch.full((9, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    smla.cache_append(x[:, 0], padded, pool, None, 0, rows_out=rows)
    back = torch.full((9, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    smla.cache_gather(pool, None, 0, padded, back)
    smla.check_device_errors()
    for t in (y, rows, back):
        assert bool((t[5:] == 5).all()) and bool((t[:5] != 5).any())
    assert int((pool != 0xA5).any(1).sum()) == 5
    seqs.kv_len[1] = 1  # two new tokens, one cached
    smla.rope(x, padded, _rope(64, 0, False), y)
    with pytest.raises(smla.SmlaError) as e:
        smla.check_device_errors()
    assert e.value.status == 5


CASES = [  # D, norm_dim, offset, dim, half, sbs
    (576, 512, 512, 64, False, 0), (576, 512, 512, 64, False, 576), (576, 512, 512, 64, True, 32),
    (576, 512, 512, 64, True, None), (128, 0, 64, 64, True, 128), (128, 128, 0, 128, True, 32),
    (128, 0, 0, 64, False, None), (1024, 1024, 0, 1024, True, 1024), (16, 8, 0, 16, False, 0), (40, 0, 0, 0, False, 40),
]


@pytest.mark.parametrize("D,norm,offset,dim,half,sbs", CASES)
@pytest.mark.parametrize("q_lens,kv_lens,page", [([1], [1], 64), ([0, 3, 70, 1], [4, 3, 201, 65], 8)])
def test_append_then_gather(D, norm, offset, dim, half, sbs, q_lens, kv_lens, page):
    rng = np.random.default_rng(D + norm + offset)
    s, seqs, pos = _batch(rng, q_lens, kv_lens, page)
    x64, wide = _bf16(rng.standard_normal((s.T, D + 24)) * np.exp(rng.uniform(-3, 3, (s.T, 1))))
    x64, x = x64[:, 8:D + 8], wide[:, 8:D + 8]  # strided rows
    w64, w = _bf16(1 + 0.2 * rng.standard_normal(norm))
    if not norm:
        w64 = w = None
    rope = _rope(dim, offset, half, "yarn") if dim else None
    bf16 = sbs is None
    mode = 0 if bf16 else sbs
    ns = 0 if mode == 0 else D // min(mode, D)
    pool = torch.full((s.phys_rows, D), 0x25, dtype=torch.uint8, device="cuda")
    if bf16:
        pool = torch.full((s.phys_rows, D), 9.0, dtype=torch.bfloat16, device="cuda")
    scales = torch.full((s.phys_rows, ns), 3.0, device="cuda") if ns else None
    before = pool.clone()
    rows_out = torch.empty((s.T, D), dtype=torch.bfloat16, device="cuda")
    smla.cache_append(x, seqs, pool, scales, mode, rope, norm_weight=w, norm_eps=1e-5, rows_out=rows_out)
    back = torch.empty((s.T, D), dtype=torch.bfloat16, device="cuda")
    smla.cache_gather(pool, scales, mode, seqs, back)
    smla.check_device_errors()

    f, a = _freq(dim, "yarn") if dim else (None, 1.0)
    ref, mass = ol.append_rows(x64, pos, w64, 1e-5, (f, offset, half, a) if dim else None)
    err = (NORM + ROT) * mass
    assert (np.abs(_np(rows_out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * err).all()
    sid = token_positions(s.cu_q, s.kv_len)[1]
    at = np.array([phys_rows_of(s.page_table, page, int(b), np.array([p]))[0] for b, p in zip(sid, pos)], dtype=np.int64)
    sel = torch.from_numpy(at).cuda()
    got = pool[sel]
    if bf16:
        assert torch.equal(got, rows_out)
        assert torch.equal(back, rows_out)
    else:
        sc = np.ones((s.T, 1))
        if ns:
            want = ol.row_scales(ref, mode)
            sc = scales[sel].double().cpu().numpy()
            assert (np.abs(sc - want) <= (2 * (NORM + ROT) + U) * want).all()
        sc = np.repeat(sc, D // sc.shape[1], axis=1)
        ref_c = np.clip(ref, -448 * sc, 448 * sc)
        assert (np.abs(_np(got) * sc - ref_c) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * sc + 2 * err).all()
        # the read side is exact up to its one rounding: a float32 product, then bf16
        values = got.view(torch.float8_e4m3fn).float()
        if ns:
            values = (values.view(s.T, ns, -1) * scales[sel][:, :, None]).view(s.T, D)
        assert torch.equal(back, values.to(torch.bfloat16))
    # every other row of the pool is untouched
    keep = torch.ones(s.phys_rows, dtype=torch.bool, device="cuda")
    keep[sel] = False
    assert torch.equal(pool[keep], before[keep])
    if ns:
        assert bool((scales[keep] == 3).all())


def test_append_special_values():
    """Zero rows get scale 1; infinities saturate and NaN stays, without
    reaching their neighbours; a row of tiny values keeps a finite quotient."""
    s, seqs, pos = _batch(np.random.default_rng(5), [4], [4])
    x = torch.randn((4, 64), device="cuda").bfloat16()
    x[0] = 0
    x[1, 3], x[1, 40] = float("inf"), float("nan")
    x[2] = 1e-39
    for sbs in (0, 64, 32):
        pool = torch.zeros((s.phys_rows, 64), dtype=torch.uint8, device="cuda")
        ns = 0 if sbs == 0 else 64 // sbs
        scales = torch.zeros((s.phys_rows, ns), device="cuda") if ns else None
        smla.cache_append(x, seqs, pool, scales, sbs)
        smla.check_device_errors()
        row0 = int(s.page_table[0, 0]) * 64
        got = pool[row0:row0 + 4].view(torch.float8_e4m3fn).float().cpu()
        assert bool((got[0] == 0).all()) and got[1, 3] == 448 and bool(got[1, 40].isnan())
        assert bool(got[1, torch.arange(64) != 40].isfinite().all()) and bool(got[2:].isfinite().all())
        if ns:
            sc = scales[row0:row0 + 4].cpu()
            assert bool((sc[0] == 1).all()) and bool((sc[2] == 2.0 ** -126).all())
            finite = x[1].float().abs().cpu()
            finite[3] = finite[40] = 0
            # one float32 division of an exact maximum: nothing to tolerate
            assert torch.equal(sc[1], finite.view(ns, -1).amax(1) / 448)


def test_bad_pages_are_reported_and_skipped():
    s, seqs, pos = _batch(np.random.default_rng(6), [3], [130])
    x = torch.ones((3, 64), device="cuda").bfloat16()
    for bad in (-1, 1 << 20):
        pool = torch.zeros((s.phys_rows, 64), dtype=torch.uint8, device="cuda")
        seqs.page_table[0, 2] = bad  # tokens 128, 129; token 127 is on page 1
        smla.cache_append(x, seqs, pool, None, 0)
        with pytest.raises(smla.SmlaError) as e:
            smla.check_device_errors()
        assert e.value.status == 5 and int((pool != 0).any(1).sum()) == 1
        back = torch.full((3, 64), 5.0, device="cuda", dtype=torch.bfloat16)
        smla.cache_gather(pool, None, 0, seqs, back)
        with pytest.raises(smla.SmlaError):
            smla.check_device_errors()
        assert bool((back[0] == 1).all()) and bool((back[1:] == 5).all())


def test_offsets_past_32_bits():
    """Rows of a pool larger than 2^32 bytes."""
    rows = (1 << 32) // 1152 // 64 * 64 + 128
    pool = torch.empty((rows, 576), dtype=torch.bfloat16, device="cuda")
    pool[-192:] = 0
    table = torch.tensor([[rows // 64 - 1, 0]], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    seqs = smla.Seqs(one, torch.tensor([64], dtype=torch.int32, device="cuda"), table, 64, 64)
    x = torch.randn((64, 576), device="cuda").bfloat16()
    smla.cache_append(x, seqs, pool, None, 0)
    back = torch.empty_like(x)
    smla.cache_gather(pool, None, 0, seqs, back)
    smla.check_device_errors()
    assert torch.equal(pool[-64:], x) and torch.equal(back, x) and bool((pool[-192:-64] == 0).all())


def test_captured_and_on_another_stream():
    """A decode step's rotation and write, captured once and replayed for
    later positions: the positions are read from kv_len on the device."""
    rng = np.random.default_rng(7)
    s, seqs, _ = _batch(rng, [2, 2], [130, 70])
    x = torch.randn((4, 2, 64), device="cuda").bfloat16()
    y, pool = torch.empty_like(x), torch.zeros((s.phys_rows, 64), dtype=torch.uint8, device="cuda")
    rope = _rope(64, 0, True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    smla.rope(x, seqs, rope, y, stream=stream)
    smla.cache_append(x[:, 0], seqs, pool, None, 0, rope, stream=stream)
    smla.check_device_errors(stream)
    first, first_pool = y.clone(), pool.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        smla.rope(x, seqs, rope, y)
        smla.cache_append(x[:, 0], seqs, pool, None, 0, rope)
    y.zero_()
    pool.zero_()
    g.replay()
    smla.check_device_errors()
    assert torch.equal(y, first) and torch.equal(pool, first_pool)
    seqs.kv_len.sub_(1)
    g.replay()
    smla.check_device_errors()
    assert not torch.equal(y, first)
    assert int((pool != 0).any(1).sum()) == 6  # positions 127..129 and 67..69
