"""Dense MLA decode against its definition in 64 bits.

Tolerance, from the arithmetic.  The output is rounded to bf16, off by at most
2^-8 of itself.  The weights, and a bf16 query, are carried as two e4m3 terms
(a bf16 cache: as bf16), off by at most 2^-8 of each value and, being rounding
errors of unrelated values, independent of each other with a standard
deviation of at most e = 2^-8 / sqrt(3).  Weight errors move the output by e *
sqrt(sum p_j^2 v_j^2); query errors move each logit by e * scale * sqrt(sum
q_d^2 k_d^2), at most s = e * scale * |q|_4 |k|_4, and the output by s * sqrt(sum
p_j^2 (v_j - out)^2) where the logits' errors are independent and by s * sum
p_j |v_j - out| at most; the square root form is used, times 8 standard
deviations (one element in 10^15).  Float32 sums add 2^-20 of sum p_j |v_j|.

Two e4m3 terms end at half of e4m3's smallest step, 2^-10, whatever the
weight: a weight is carried as P_j = p_j s_j (s_j its row's scale) in units that
put the largest of them at 2^4 or more, so each is off by up to 2^-14 of that
largest, again independently, and moves the output by that much of the row's
unscaled values v_j / s_j.  Block-scaled rows are carried so too, as two terms
of x / s_j: off by up to 2^-8 of each value and 2^-10 of s_j, which enters as the
weights' and the query's errors do.
"""
import math

import numpy as np
import pytest
import torch

import serving_fp8_indexer_gb300 as smla
from serving_fp8_indexer_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5
E = 2.0 ** -8 / math.sqrt(3)


def _cache(rows, mode, gen):
    """(pool, scales, scale_block_size, values f64 [rows, 576])"""
    x = torch.randn((rows, 576), generator=gen, device="cuda")
    if mode == "bf16":
        return x.bfloat16(), None, 0, x.bfloat16().double()
    if mode == "unit":
        b = x.to(torch.float8_e4m3fn)
        return b.view(torch.uint8), None, 0, b.double()
    w = 576 if mode == "row" else 32
    blk = x.view(rows, -1, w) * torch.exp(torch.randn((rows, 576 // w, 1), generator=gen, device="cuda") * 0.3)
    s = blk.abs().amax(2) / 448
    b = (blk / s[:, :, None]).to(torch.float8_e4m3fn)
    return b.view(rows, 576).view(torch.uint8), s.contiguous(), w, (b.double() * s.double()[:, :, None]).view(rows, 576)


def _carried(scales, pool):
    """(row scale, block-scaled?) of _reference: the one scale a row's values are carried with (its largest), None for a bf16 cache."""
    if pool.dtype == torch.bfloat16:
        return dict(srow=None)
    if scales is None:
        return dict(srow=torch.ones(pool.shape[0], dtype=torch.float64, device="cuda"))
    return dict(srow=scales.double().amax(1), block=scales.shape[1] > 1)


def _case(q_lens, kv_lens, H, qd, mode, page=64, seed=0):
    rng = np.random.default_rng(seed)
    s = wl.make_seqs(rng, q_lens, kv_lens, page)
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool, scales, sbs, val = _cache(max(s.phys_rows, 1), mode, g)
    x = torch.randn((s.T, H, 576), generator=g, device="cuda")
    q = x.bfloat16() if qd == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)
    return s, smla.Seqs.from_host(s), q, pool, scales, sbs, val


def _reference(s, q, val, srow, sink=None, block=False):
    """(out, tolerance) in float64."""
    q64 = q.double() if q.dtype == torch.bfloat16 else q.view(torch.float8_e4m3fn).double()
    out = torch.zeros((s.T, q.shape[1], 512), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for b in range(s.B):
        rows = torch.from_numpy(wl.logical_to_phys(s, b, np.arange(int(s.kv_len[b])))).cuda()
        k = val[rows]
        for t in range(int(s.cu_q[b]), int(s.cu_q[b + 1])):
            n = int(s.kv_len[b]) - int(s.cu_q[b + 1]) + t + 1
            if n <= 0:  # nothing to attend to: zeros
                continue
            z = SCALE * q64[t] @ k[:n].T
            if sink is not None:
                z = torch.cat([z, sink.double()[:, None]], 1)
            p = torch.softmax(z, 1)[:, :n]
            v = k[:n, :512]
            o = p @ v
            out[t] = o
            p2 = p * p
            var_p = p2 @ (v * v)
            about = (var_p - 2 * o * (p2 @ v) + o * o * p2.sum(1, keepdim=True)).clamp_min(0)  # sum p^2 (v - out)^2
            s2 = (SCALE * SCALE) * (q64[t].pow(4).sum(1).sqrt() * k[:n].pow(4).sum(1).max().sqrt())[:, None]
            if srow is not None:
                sj = srow[rows[:n]]
                largest = (p * sj).amax(1, keepdim=True)
                if block:
                    var_p = 2 * var_p + p2 @ (sj * sj)[:, None] / 16  # 2^-10 = 2^-8 / 4
                    s2 = 2 * s2 + (SCALE * sj.max() / 4) ** 2 * q64[t].pow(2).sum(1)[:, None]
                var_p = var_p + (2.0 ** -6 * largest) ** 2 * ((v / sj[:, None]) ** 2).sum(0)  # 2^-14 = 2^-6 * 2^-8
            var_q = s2 * about
            tol[t] = 8 * E * (var_p + var_q).sqrt() + 2.0 ** -8 * o.abs() + 2.0 ** -20 * (p @ v.abs())
    return out, tol


def _run(seqs, q, pool, scales, sbs, most, sink=None, out=None, stream=None):
    n = smla.dense_decode_workspace_size(seqs.T, q.shape[1], most)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None  # NaN in every float
    out = torch.full((seqs.T, q.shape[1], 512), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    smla.dense_decode(q, pool, scales, sbs, seqs, most, SCALE, out, ws, attn_sink=sink, stream=stream)
    smla.check_device_errors(stream)
    return out


def _close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp_min(1e-30)).max()):.3g} x the tolerance"


MODES = [("bf16", "unit"), ("bf16", "row"), ("e4m3", "unit"), ("e4m3", "row"), ("e4m3", "block"), ("bf16", "bf16")]
SHAPES = [([1], [1], 16, 64), ([1, 1, 1], [127, 128, 129], 64, 64), ([2, 0, 3, 1], [700, 5, 3, 2049], 128, 16),
          ([4, 4], [4100, 77], 16, 8), ([1], [20011], 32, 256), ([3, 2], [300, 1000], 48, 64),
          ([2, 1, 4, 1], [30001, 5, 9000, 12345], 64, 64), ([1, 1], [60000, 777], 16, 128)]


@pytest.mark.parametrize("qd,mode", MODES)
@pytest.mark.parametrize("q_lens,kv_lens,H,page", SHAPES)
def test_matches_the_definition(qd, mode, q_lens, kv_lens, H, page):
    s, seqs, q, pool, scales, sbs, val = _case(q_lens, kv_lens, H, qd, mode, page, seed=len(q_lens) * 100 + H)
    out = _run(seqs, q, pool, scales, sbs, max(kv_lens))
    _close(out, *_reference(s, q, val, **_carried(scales, pool)))


@pytest.mark.parametrize("qd,mode", MODES)
def test_many_tokens_and_a_sink(qd, mode):
    """Enough tokens that nothing is split, and a sink with either form."""
    for q_lens, kv_lens, H in (([4] * 45, [200 + 7 * i for i in range(45)], 64), ([1, 2], [900, 1500], 128)):
        s, seqs, q, pool, scales, sbs, val = _case(q_lens, kv_lens, H, qd, mode, seed=5)
        sink = torch.randn(H, device="cuda") * 2
        out = _run(seqs, q, pool, scales, sbs, max(kv_lens), sink)
        _close(out, *_reference(s, q, val, sink=sink, **_carried(scales, pool)))


@pytest.mark.parametrize("qd,mode", MODES)
def test_bound_on_the_lengths_only_chooses_the_split(qd, mode):
    s, seqs, q, pool, scales, sbs, val = _case([1, 2], [1500, 700], 16, qd, mode, seed=6)
    ref, tol = _reference(s, q, val, **_carried(scales, pool))
    for most in (1, 100, 1500, 100000):
        _close(_run(seqs, q, pool, scales, sbs, most), ref, tol)


@pytest.mark.parametrize("qd,mode", MODES)
def test_unused_rows_and_padded_batches(qd, mode):
    """Whatever the pool holds outside the sequences' keys (NaN here) never
    reaches an output, and tokens behind the last sequence keep theirs."""
    s, seqs, q, pool, scales, sbs, val = _case([2, 1], [70, 333], 64, qd, mode, page=128, seed=7)
    clean = _run(seqs, q, pool, scales, sbs, 333)
    used = torch.zeros(s.phys_rows, dtype=torch.bool, device="cuda")
    for b in range(2):
        used[torch.from_numpy(wl.logical_to_phys(s, b, np.arange(int(s.kv_len[b])))).cuda()] = True
    pool = pool.clone()
    pool[~used] = float("nan") if mode == "bf16" else 0x7F
    if scales is not None:
        scales = scales.clone()
        scales[~used] = float("nan")
    pad = smla.Seqs(seqs.cu_q, seqs.kv_len, seqs.page_table, 128, 8)
    q8 = torch.cat([q, q[:1].expand(5, -1, -1)]).contiguous()
    for most in (333, 1):  # split and not
        out = torch.full((8, 64, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        _run(pad, q8, pool, scales, sbs, most, out=out)
        assert bool((out[3:] == 5).all())
        _close(out[:3], *_reference(s, q, val, **_carried(scales, pool)))
    _close(clean, *_reference(s, q, val, **_carried(scales, pool)))


def test_rows_without_keys():
    s, seqs, q, pool, scales, sbs, val = _case([1, 1], [1, 900], 16, "bf16", "unit", seed=8)
    seqs.kv_len[0] = 0
    for most in (900, 1):
        out = _run(seqs, q, pool, scales, sbs, most)
        assert bool((out[0] == 0).all()) and bool((out[1] != 0).any())


def test_peaked_and_growing_logits():
    """A key that takes almost all the weight in a late block, and logits that
    grow along the keys (the running reference is raised many times)."""
    s, seqs, q, pool, scales, sbs, val = _case([1], [1200], 16, "bf16", "unit", seed=9)
    rows = torch.from_numpy(wl.logical_to_phys(s, 0, np.arange(1200))).cuda()
    base = torch.randn(576, device="cuda").sign()
    ramp = torch.linspace(-2, 2, 1200, device="cuda")[:, None] * base + 0.2 * torch.randn((1200, 576), device="cuda")
    pool[rows] = ramp.to(torch.float8_e4m3fn).view(torch.uint8)
    val[rows] = pool[rows].view(torch.float8_e4m3fn).double()
    q = (base * torch.linspace(0.1, 1.5, 16, device="cuda")[None, :, None]).bfloat16()
    for most in (1200, 1):
        _close(_run(seqs, q, pool, scales, sbs, most), *_reference(s, q, val, **_carried(scales, pool)))


def test_captured_replay_and_another_stream():
    s, seqs, q, pool, scales, sbs, val = _case([1, 1], [600, 420], 128, "bf16", "row", seed=10)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        _close(_run(seqs, q, pool, scales, sbs, 600, stream=stream), *_reference(s, q, val, **_carried(scales, pool)))
    torch.cuda.current_stream().wait_stream(stream)
    n = smla.dense_decode_workspace_size(2, 128, 600)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    out = torch.zeros((2, 128, 512), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        smla.dense_decode(q, pool, scales, sbs, seqs, 600, SCALE, out, ws)
    for shorter in (0, 131):
        seqs.kv_len.copy_(torch.tensor([600 - shorter, 420 - shorter], dtype=torch.int32))
        s.kv_len = seqs.kv_len.cpu().numpy()
        g.replay()
        smla.check_device_errors()
        _close(out, *_reference(s, q, val, **_carried(scales, pool)))


def test_bad_pages_are_reported():
    s, seqs, q, pool, scales, sbs, val = _case([1], [200], 64, "bf16", "unit", seed=11)
    for bad in (-1, 1 << 24):
        seqs.page_table[0, 1] = bad
        with pytest.raises(smla.SmlaError) as e:
            _run(seqs, q, pool, scales, sbs, 200)
        assert e.value.status == 5


def test_rows_past_32_bits():
    """Pages at the far end of a cache larger than 2^32 bytes."""
    rows = (1 << 32) // 576 // 64 * 64 + 256
    pool = torch.empty((rows, 576), dtype=torch.uint8, device="cuda")
    s, seqs, q, small, scales, sbs, val = _case([2], [100], 16, "bf16", "unit", seed=12)
    far = torch.tensor([[rows // 64 - 1, rows // 64 - 2]], dtype=torch.int32, device="cuda")
    for i in range(2):
        a = int(s.page_table[0, i]) * 64
        b = int(far[0, i]) * 64
        pool[b:b + 64] = small[a:a + 64]
    seqs = smla.Seqs(seqs.cu_q, seqs.kv_len, far, 64, 2)
    _close(_run(seqs, q, pool, None, 0, 100), *_reference(s, q, val, **_carried(scales, pool)))


def test_zero_and_tiny_row_scales_keep_their_weight():
    """A row of scale 0 (or almost) has value 0, logit 0 and still its share of
    the softmax."""
    s, seqs, q, pool, scales, sbs, val = _case([1], [300], 16, "bf16", "row", seed=13)
    rows = torch.from_numpy(wl.logical_to_phys(s, 0, np.arange(300))).cuda()
    scales[rows[10:200]] = 0.0
    scales[rows[200:220]] = 1e-36
    val[rows[10:220]] *= 0.0
    pool[rows[10:200]] = 0x38
    got = _run(seqs, q, pool, scales, sbs, 300)
    srow = scales.double()[:, 0].clamp_min(1e-30)
    _close(got, *_reference(s, q, val, srow=srow))


@pytest.mark.parametrize("qd,mode", [("bf16", "unit"), ("bf16", "row"), ("e4m3", "row")])
def test_the_same_call_gives_the_same_bits(qd, mode):
    for q_lens, kv_lens, H in (([1, 2], [3000, 1100], 128), ([2] * 3, [500, 900, 1300], 16)):
        s, seqs, q, pool, scales, sbs, val = _case(q_lens, kv_lens, H, qd, mode, seed=14)
        first = _run(seqs, q, pool, scales, sbs, 3000)
        for _ in range(4):
            assert torch.equal(_run(seqs, q, pool, scales, sbs, 3000), first)


def test_a_page_that_hangs_over_the_pool_is_reported():
    """A pool that ends inside a page: keys before its end are read, later ones
    reported."""
    s, seqs, q, pool, scales, sbs, val = _case([1], [60], 16, "bf16", "unit", seed=15)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    one = smla.Seqs(seqs.cu_q, seqs.kv_len, table, 64, 1)
    _run(one, q, pool[:60].contiguous(), None, 0, 60)
    with pytest.raises(smla.SmlaError) as e:
        _run(one, q, pool[:59].contiguous(), None, 0, 60)
    assert e.value.status == 5


def test_many_sequences_and_odd_groups():
    """More sequences than a warp holds at once, empty ones among them, and
    token groups that end inside a sequence's tokens."""
    q_lens = [(3 * i) % 4 for i in range(70)]
    kv_lens = [max(q, (37 * i) % 300) for i, q in enumerate(q_lens)]
    for H in (16, 32):
        s, seqs, q, pool, scales, sbs, val = _case(q_lens, kv_lens, H, "bf16", "row", page=16, seed=16)
        for most in (300, 1):
            _close(_run(seqs, q, pool, scales, sbs, most), *_reference(s, q, val, **_carried(scales, pool)))


@pytest.mark.parametrize("mode", ["unit", "row"])
@pytest.mark.parametrize("H", [16, 64, 128])
def test_infinite_and_nan_queries_stay_in_their_row(mode, H):
    """Every logit of such a row is infinite or NaN, and so its softmax NaN;
    the other rows do not see it."""
    s, seqs, q, pool, scales, sbs, val = _case([2, 1], [400, 90], H, "bf16", mode, seed=17)
    clean = _run(seqs, q, pool, scales, sbs, 400)
    bad = q.clone()
    bad[0, 3, 100] = float("inf")
    bad[1, H - 1, 575] = float("-inf")
    bad[2, 0, 0] = float("nan")
    got = _run(seqs, bad, pool, scales, sbs, 400)
    rows = torch.zeros((3, H), dtype=torch.bool, device="cuda")
    rows[0, 3] = rows[1, H - 1] = rows[2, 0] = True
    assert bool(got[rows].isnan().all())
    assert torch.equal(got[~rows], clean[~rows])


@pytest.mark.parametrize("qd,mode", [("bf16", "row"), ("e4m3", "row"), ("e4m3", "block")])
@pytest.mark.parametrize("tiny", [0.0, 1e-36])
def test_rows_of_tiny_scale_ahead_of_the_others(qd, mode, tiny):
    """The first blocks' rows have scale 0 (or almost), the later ones' ordinary
    scales: the first ones' logits and values are 0, their share is not."""
    s, seqs, q, pool, scales, sbs, val = _case([1], [700], 16, qd, mode, seed=18)
    rows = torch.from_numpy(wl.logical_to_phys(s, 0, np.arange(700))).cuda()
    scales[rows[:400]] = tiny
    val[rows[:400]] *= 0.0
    carried = _carried(scales.clamp_min(1e-30), pool)
    for most in (700, 1):
        _close(_run(seqs, q, pool, scales, sbs, most), *_reference(s, q, val, **carried))
    scales[rows] = tiny
    got = _run(seqs, q, pool, scales, sbs, 700)
    assert bool((got.float().abs() <= 1e-33).all())


@pytest.mark.parametrize("qd,mode", [("e4m3", "block"), ("bf16", "bf16"), ("bf16", "row"), ("e4m3", "unit")])
@pytest.mark.parametrize("q_lens,kv_lens,H,page", [SHAPES[4], SHAPES[6], SHAPES[7], ([1] * 5, [4000 + i for i in range(5)], 128, 32)])
def test_forty_calls_give_the_same_bits(qd, mode, q_lens, kv_lens, H, page):
    """Ring slots that are handed back too early, or seen a phase early, show
    as results that differ from call to call."""
    s, seqs, q, pool, scales, sbs, val = _case(q_lens, kv_lens, H, qd, mode, page, seed=19)
    first = _run(seqs, q, pool, scales, sbs, max(kv_lens))
    for _ in range(40):
        assert torch.equal(_run(seqs, q, pool, scales, sbs, max(kv_lens)), first)


@pytest.mark.parametrize("qd,mode", MODES)
@pytest.mark.parametrize("H,page", [(192, 4096), (256, 8), (48, 32)])
def test_more_heads_and_extreme_pages(qd, mode, H, page):
    s, seqs, q, pool, scales, sbs, val = _case([1, 3], [777, 1500], H, qd, mode, page, seed=20)
    ref, tol = _reference(s, q, val, **_carried(scales, pool))
    for most in (1500, 1):
        _close(_run(seqs, q, pool, scales, sbs, most), ref, tol)


@pytest.mark.parametrize("qd,mode", MODES)
def test_one_captured_call_serves_growing_lengths(qd, mode):
    """The grid is chosen from max_kv_len at the capture; lengths beyond it and
    empty sequences are served by the same graph."""
    s, seqs, q, pool, scales, sbs, val = _case([1, 2, 1], [2000, 1200, 300], 32, qd, mode, seed=22)
    n = smla.dense_decode_workspace_size(4, 32, 500)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.zeros((4, 32, 512), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        smla.dense_decode(q, pool, scales, sbs, seqs, 500, SCALE, out, ws)
    for lens in ([5, 130, 0], [2000, 1200, 300], [1, 2, 257]):
        seqs.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        s.kv_len = seqs.kv_len.cpu().numpy()
        g.replay()
        smla.check_device_errors()
        _close(out, *_reference(s, q, val, **_carried(scales, pool)))
