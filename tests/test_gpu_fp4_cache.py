"""The latent cache in 4 bits: writing, reading back and dense decode over it.

Without norm and rotation a written row is compared bit by bit with the host's:
scale, shifts and codes are single roundings of exact quantities.  With them a
finished row is off by NORM + ROT = 48 u of its pair's magnitudes (the float32
arithmetic of the same kernel over e4m3 caches, derived there; u = 2^-24), its
scale by twice that and a division, so that a value in units of its block's code is
within 2^-17 of the exact one (at most 8 units) when it is rounded to the nearest code:
off by half a step, 0.25 up to 2 units, else at most a quarter of the value.

Attention over the cache reads e2m1 * 2^(6 - shift) as e4m3 bytes with the scale by
the row, so its result is, bit by bit, that of the dense decode over the e4m3 rows
that the gather returns, and holds its derived tolerance against 64 bits."""
import math

import numpy as np
import pytest
import torch

import oracle.latent as ol
import serving_fp8_indexer_gb300 as smla
from oracle.reference import token_positions
from serving_fp8_indexer_gb300 import workloads as wl
from test_gpu_dense_decode import SCALE, _close, _reference

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
CODES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _fields(pool):
    """(codes [n, 576], shifts [n, 36], scales f32 [n]) of rows, on the host."""
    p = pool.cpu()
    codes = torch.stack((p[:, :288] & 15, p[:, :288] >> 4), 2).view(-1, 576)
    shifts = torch.stack((p[:, 288:306] & 15, p[:, 288:306] >> 4), 2).view(-1, 36)
    return codes, shifts, p[:, 308:312].contiguous().view(torch.float32)[:, 0]


def _values(pool):
    """(values in units of the row's scale, scales), float64 on the host."""
    codes, shifts, scales = _fields(pool)
    v = CODES[(codes & 7).long()] * torch.where(codes > 7, -1.0, 1.0)
    unit = torch.where(shifts == 15, 0.0, torch.exp2(6 - shifts.double()))
    return (v.view(-1, 36, 16) * unit[:, :, None]).view(-1, 576), scales.double()


def _expected(x):
    """The row's bytes for finished float32 rows, on the host."""
    v = x.float().cpu().view(-1, 36, 16)
    a = torch.where(v.isfinite(), v.abs(), torch.zeros(()))
    top = a.amax(2)
    most = top.amax(1)
    scale = torch.where(most > 0, (most / torch.full_like(most, 384.0)).clamp_min(2.0 ** -126), torch.ones(()))
    shift = sum((top.double() * 2.0 ** k <= most.double()[:, None]).int() for k in range(1, 15))
    # the f32 quotient, then an exact power of two, then the nearest code (ties to the even one)
    y = (v / scale[:, None, None]).double() * torch.exp2(shift.double() - 6)[:, :, None]
    m = y.abs()
    code = sum((m > b if even else m >= b).int() for b, even in
               ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)))
    code = torch.where(v.isnan(), torch.zeros((), dtype=code.dtype), code) | torch.signbit(v).int() << 3
    code, shift = code.view(-1, 576), shift
    rows = torch.zeros((v.shape[0], 320), dtype=torch.uint8)
    rows[:, :288] = (code[:, 0::2] | code[:, 1::2] << 4).byte()
    rows[:, 288:306] = (shift[:, 0::2] | shift[:, 1::2] << 4).byte()
    scale = torch.where(v.isnan().view(-1, 576).any(1), torch.full_like(scale, math.nan), scale)
    rows[:, 308:312] = scale.view(-1, 1).view(torch.uint8)
    return rows


def _flat_batch(T, page=64):
    pages = -(-T // page)
    i32 = dict(dtype=torch.int32, device="cuda")
    return smla.Seqs(torch.tensor([0, T], **i32), torch.tensor([T], **i32), torch.arange(pages, **i32)[None], page, T), pages * page


def _written(x):
    seqs, n = _flat_batch(x.shape[0])
    pool = torch.full((n, 320), 0xEE, dtype=torch.uint8, device="cuda")
    smla.cache_append_fp4(x, seqs, pool)
    smla.check_device_errors()
    assert bool((pool[x.shape[0]:] == 0xEE).all())
    return pool[:x.shape[0]], seqs, pool


@pytest.mark.parametrize("size", [1.0, 2.0 ** -90, 2.0 ** 119])
def test_rows_are_written_bit_by_bit(size):
    g = _gen(1)
    # blocks over 22 binary places, and values on the borders between codes
    x = torch.randn((1500, 576), generator=g, device="cuda")
    x *= torch.exp2(-torch.randint(0, 22, (1500, 36, 1), generator=g, device="cuda")).expand(1500, 36, 16).reshape(1500, 576)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.24, 4.99], device="cuda")
    x[:600] = borders[torch.randint(0, 10, (600, 576), generator=g, device="cuda")] * x[:600].sign()
    x[:600, ::16] = 6.0
    x[300:600] *= torch.exp2(-torch.randint(0, 16, (300, 36, 1), generator=g, device="cuda")).expand(300, 36, 16).reshape(300, 576)
    x = (x * size).bfloat16()
    assert bool(x.isfinite().all())
    rows, _, _ = _written(x)
    assert torch.equal(rows.cpu(), _expected(x))


def test_zeros_infinities_nan_and_subnormals():
    x = torch.randn((8, 576), generator=_gen(2), device="cuda").bfloat16()
    x[0] = 0
    x[1, 16:560] = 0
    x[2, 5], x[2, 40] = math.inf, -math.inf
    x[3, 100] = math.nan
    x[4] = 2.0 ** -133
    x[4, 0] = 2.0 ** -128
    x[5] *= 2.0 ** -126
    x[6] = math.inf
    x[7, 32:48] = 2.0 ** -130
    rows, seqs, pool = _written(x)
    want = _expected(x)
    # (the codes of a NaN are not told: the scale says NaN)
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(rows.cpu()[keep], want[keep])
    assert torch.equal(rows.cpu()[3, 288:], want[3, 288:])
    back = torch.empty((8, 576), dtype=torch.bfloat16, device="cuda")
    smla.cache_gather_fp4(pool, seqs, back)
    assert bool((back[0] == 0).all()) and bool(back[3].isnan().all()) and bool(back[keep].isfinite().all())


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("norm", [0, 512, 576])
def test_finished_rows(half, norm):
    rng = np.random.default_rng(3)
    s = wl.make_seqs(rng, [3, 0, 130, 1, 17], [3, 5, 700, 64, 129], 16)
    seqs = smla.Seqs.from_host(s)
    pos, _ = token_positions(s.cu_q, s.kv_len)
    wide = torch.randn((s.T, 640), generator=_gen(norm), device="cuda").bfloat16()
    x = wide[:, :576]
    f, amp = smla.rope_frequencies(64, scaling="yarn", factor=40.0)
    w = (1 + 0.1 * torch.randn(norm, generator=_gen(5), device="cuda")).bfloat16() if norm else None
    pool = torch.zeros((s.phys_rows, 320), dtype=torch.uint8, device="cuda")
    kept = torch.empty((s.T, 584), dtype=torch.bfloat16, device="cuda")[:, :576]
    smla.cache_append_fp4(x, seqs, pool, smla.Rope(f, 512, smla.ROPE_HALF if half else smla.ROPE_INTERLEAVED, amp), w, 1e-5, kept)
    smla.check_device_errors()
    of, oa = ol.rope_frequencies(64, scaling="yarn", factor=40.0)
    want, mass = ol.append_rows(x.double().cpu().numpy(), pos, None if w is None else w.double().cpu().numpy(), 1e-5, (of, 512, half, oa))
    want, mass = torch.from_numpy(want), torch.from_numpy(mass)
    err = (kept.double().cpu() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + 50 * U * mass).all())
    rows = torch.from_numpy(np.concatenate([wl.logical_to_phys(s, b, np.arange(int(s.kv_len[b]) - int(s.cu_q[b + 1] - s.cu_q[b]),
                                                                               int(s.kv_len[b]))) for b in range(s.B)]))
    value, scale = _values(pool[rows.cuda()])
    _, shifts, _ = _fields(pool[rows.cuda()])
    most = want.abs().amax(1)
    assert bool(((scale - most / 384).abs() <= 200 * U * most / 384).all())
    top = want.abs().view(-1, 36, 16).amax(2)
    # a shift may be one off only where the maxima's ratio is a power of two, within their error
    ratio = torch.log2(most[:, None] / top)
    near = (ratio - ratio.round()).abs() < 2.0 ** -15
    assert bool((near | (shifts.double() == ratio.floor().clamp(0, 14))).all())
    unit = torch.exp2(6 - shifts.double()).repeat_interleave(16, 1)
    y, got = want / (most[:, None] / 384) / unit, value / unit
    assert bool(((got - y).abs() <= torch.clamp_min(y.abs() / 4, 0.25) + 2.0 ** -17).all())
    untouched = torch.ones(s.phys_rows, dtype=torch.bool)
    untouched[rows] = False
    assert bool((pool.cpu()[untouched] == 0).all())


def test_rows_behind_the_last_sequence_and_bad_pages():
    x = torch.randn((6, 576), generator=_gen(6), device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = torch.full((16, 320), 0xEE, dtype=torch.uint8, device="cuda")
    seqs = smla.Seqs(torch.tensor([0, 2, 4], **i32), torch.tensor([2, 10], **i32), torch.tensor([[0, -1], [5, 1]], **i32), 8, 6)
    smla.cache_append_fp4(x, seqs, pool)  # sequence 1: positions 8, 9 on its second page
    smla.check_device_errors()
    want = _expected(x)
    assert torch.equal(pool.cpu()[[0, 1, 8, 9]], want[:4]) and bool((pool[[2, 7, 10, 15]] == 0xEE).all())
    rows, sc = torch.full((6, 576), 0x55, dtype=torch.uint8, device="cuda"), torch.full((6, 1), 9.0, device="cuda")
    smla.cache_gather_fp4(pool, seqs, rows, sc)
    smla.check_device_errors()
    v, s = _values(pool[[0, 1, 8, 9]])
    assert torch.equal(rows[:4].view(torch.float8_e4m3fn).double().cpu(), v) and torch.equal(sc[:4, 0].double().cpu(), s)
    assert bool((rows[4:] == 0x55).all()) and bool((sc[4:] == 9.0).all())
    # a page outside the pool is reported, its tokens skipped, the others done
    before = pool.clone()
    bad = smla.Seqs(seqs.cu_q, seqs.kv_len, torch.tensor([[0, -1], [5, 2]], **i32), 8, 6)
    smla.cache_append_fp4(x.flip(0), bad, pool)
    with pytest.raises(smla.SmlaError) as e:
        smla.check_device_errors()
    assert e.value.status == 5 and torch.equal(pool[8:], before[8:])
    bf = torch.full((6, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    smla.cache_gather_fp4(pool, bad, bf)
    with pytest.raises(smla.SmlaError):
        smla.check_device_errors()
    assert bool((bf[2:] == 3.0).all()) and not bool((bf[:2] == 3.0).all())


def _random_pool(n, g):
    """Rows of every code and shift (15 among them), scales over ten binary places."""
    pool = torch.randint(0, 256, (n, 320), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.exp2(10 * torch.rand((n, 1), generator=g, device="cuda") - 12)
    pool[:, 308:312] = scale.view(torch.uint8)
    return pool


@pytest.mark.parametrize("page", [8, 64, 1024])
def test_gather_is_exact(page):
    rng = np.random.default_rng(page)
    kv = [1, 777, 64, 2100]
    s = wl.make_seqs(rng, kv, kv, page)
    seqs = smla.Seqs.from_host(s)
    pool = _random_pool(s.phys_rows, _gen(page))
    phys = torch.from_numpy(np.concatenate([wl.logical_to_phys(s, b, np.arange(n)) for b, n in enumerate(kv)])).cuda()
    v, sc = _values(pool[phys])
    rows = torch.empty((s.T, 592), dtype=torch.uint8, device="cuda")[:, :576]
    scales = torch.empty((s.T, 1), device="cuda")
    smla.cache_gather_fp4(pool, seqs, rows, scales)
    bf = torch.empty((s.T, 584), dtype=torch.bfloat16, device="cuda")[:, :576]
    smla.cache_gather_fp4(pool, seqs, bf)
    smla.check_device_errors()
    assert torch.equal(rows.contiguous().view(torch.float8_e4m3fn).double().cpu(), v)
    assert torch.equal(scales[:, 0].double().cpu(), sc)
    # (a product of 4 and 24 significant bits, rounded to f32 and then to bf16)
    want = (v * sc[:, None]).float().bfloat16()
    assert torch.equal(bf.cpu(), want)


def _decode(seqs, q, pool, most, sink=None, out=None, stream=None):
    n = smla.dense_decode_workspace_size(seqs.T, q.shape[1], most)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None  # NaN in every float
    out = torch.full((seqs.T, q.shape[1], 512), math.nan, dtype=torch.bfloat16, device="cuda") if out is None else out
    smla.dense_decode_fp4(q, pool, seqs, most, SCALE, out, ws, attn_sink=sink, stream=stream)
    smla.check_device_errors(stream)
    return out


def _cache(n, g):
    """A pool written by the append, and its values."""
    x = torch.randn((n, 36, 16), generator=g, device="cuda") * torch.exp2(-6 * torch.rand((n, 36, 1), generator=g, device="cuda"))
    x = (x.view(n, 576) * torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda"))).bfloat16()
    seqs, rows = _flat_batch(n, 8)
    pool = torch.zeros((rows, 320), dtype=torch.uint8, device="cuda")
    smla.cache_append_fp4(x, seqs, pool)
    return pool[:n].contiguous()


def _as_e4m3(pool):
    seqs, _ = _flat_batch(pool.shape[0], 8)
    rows, scales = torch.empty((pool.shape[0], 576), dtype=torch.uint8, device="cuda"), torch.empty((pool.shape[0], 1), device="cuda")
    smla.cache_gather_fp4(pool, seqs, rows, scales)
    return rows, scales


SHAPES = [([1], [1], 16, 64), ([1, 1, 1], [127, 128, 129], 64, 64), ([2, 0, 3, 1], [700, 5, 3, 2049], 128, 16),
          ([1, 1], [63, 65], 32, 8), ([4, 1, 2], [1500, 1, 2], 16, 256), ([1], [40000], 16, 64), ([2, 2], [1000, 333], 48, 1024),
          ([1, 1, 1, 1, 1], [5000, 1, 900, 3000, 64], 32, 32)]


@pytest.mark.parametrize("qd", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,kv_lens,H,page", SHAPES)
def test_decode(q_lens, kv_lens, H, page, qd):
    rng = np.random.default_rng(sum(kv_lens))
    s = wl.make_seqs(rng, q_lens, kv_lens, page)
    seqs, g = smla.Seqs.from_host(s), _gen(sum(kv_lens) + H)
    pool = _cache(max(s.phys_rows, 8), g)
    x = torch.randn((s.T, H, 576), generator=g, device="cuda")
    q = x.bfloat16() if qd == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)
    sink = torch.randn(H, generator=g, device="cuda") if len(kv_lens) > 2 else None
    most = max(kv_lens)
    out = _decode(seqs, q, pool, most, sink)
    v, sc = (t.cuda() for t in _values(pool))
    ref, tol = _reference(s, q, v * sc[:, None], sc, sink)
    _close(out, ref, tol)
    rows, scales = _as_e4m3(pool)
    n = smla.dense_decode_workspace_size(s.T, H, most)
    other = torch.empty_like(out)
    smla.dense_decode(q, rows, scales, 576, seqs, most, SCALE, other, torch.empty(n, dtype=torch.uint8, device="cuda") if n else None,
                      attn_sink=sink)
    assert torch.equal(out, other)


def test_every_code_and_shift_enters():
    """Random bytes: -0 codes, the highest shifts and blocks marked as zeros."""
    rng = np.random.default_rng(8)
    s = wl.make_seqs(rng, [2], [500], 64)
    g = _gen(8)
    pool = _random_pool(s.phys_rows, g)
    q = torch.randn((2, 64, 576), generator=g, device="cuda").bfloat16() * 0.05
    out = _decode(smla.Seqs.from_host(s), q, pool, 500)
    v, sc = (t.cuda() for t in _values(pool))
    ref, tol = _reference(s, q, v * sc[:, None], sc)
    _close(out, ref, tol)


def test_decode_without_keys_past_the_last_sequence_and_foreign_rows():
    """Zeros for a sequence without keys; tokens behind the last sequence keep their
    outputs; what lies in rows that are nobody's (NaN everywhere) does not matter."""
    i32 = dict(dtype=torch.int32, device="cuda")
    g = _gen(9)
    pool = _cache(64, g)
    foreign = torch.ones(64, dtype=torch.bool)
    foreign[24:32] = foreign[40:43] = False  # pages 3 and the head of 5
    pool[foreign.cuda()] = 0xFF
    seqs = smla.Seqs(torch.tensor([0, 1, 2, 3], **i32), torch.tensor([0, 11, 11], **i32),
                     torch.tensor([[-1, -1], [3, 5], [3, 5]], **i32), 8, 5)
    for H in (16, 64):
        q = torch.randn((5, H, 576), generator=g, device="cuda").bfloat16()
        out = torch.full((5, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        _decode(seqs, q, pool, 11, out=out)
        assert bool((out[0] == 0).all()) and bool((out[3:] == 5.0).all()) and bool(out[1:3].isfinite().all())
        v, sc = (t.cuda() for t in _values(pool[[*range(24, 32), 40, 41, 42]]))
        k = v * sc[:, None]
        p = torch.softmax(SCALE * q[1:3].double() @ k.T, 2)
        want = p @ k[:, :512]
        assert float((out[1:3].double() - want).norm() / want.norm()) < 2.0 ** -7


def test_decode_reports_bad_pages():
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = _cache(64, _gen(10))
    q = torch.randn((1, 16, 576), generator=_gen(11), device="cuda").bfloat16()
    for pages in ([3, -1], [3, 8], [3, 1 << 27]):
        seqs = smla.Seqs(torch.tensor([0, 1], **i32), torch.tensor([12], **i32), torch.tensor([pages], **i32), 8, 1)
        with pytest.raises(smla.SmlaError) as e:
            _decode(seqs, q, pool, 12)
        assert e.value.status == 5
    # a page that hangs over the pool's end
    seqs = smla.Seqs(torch.tensor([0, 1], **i32), torch.tensor([64], **i32), torch.tensor([[0]], **i32), 64, 1)
    with pytest.raises(smla.SmlaError):
        _decode(seqs, q, pool[:60].contiguous(), 64)
    _decode(smla.Seqs(seqs.cu_q, torch.tensor([60], **i32), seqs.page_table, 64, 1), q, pool[:60].contiguous(), 60)


def test_nan_rows_and_queries():
    g = _gen(12)
    rng = np.random.default_rng(12)
    s = wl.make_seqs(rng, [1, 1], [200, 200], 64)
    seqs = smla.Seqs.from_host(s)
    pool = _cache(s.phys_rows, g)
    q = torch.randn((2, 16, 576), generator=g, device="cuda").bfloat16()
    ref = _decode(seqs, q, pool, 200)
    row = int(wl.logical_to_phys(s, 1, np.array([150]))[0])
    pool[row, 308:312] = torch.tensor([math.nan], device="cuda").view(torch.uint8)
    out = _decode(seqs, q, pool, 200)
    assert torch.equal(out[0], ref[0]) and bool(out[1].isnan().all())
    q[0, 3, 7] = math.inf
    out = _decode(seqs, q, pool, 200)
    keep = torch.arange(16, device="cuda") != 3
    assert bool(out[0, 3].isnan().all()) and torch.equal(out[0, keep], ref[0, keep])


@pytest.mark.parametrize("H", [16, 128])
def test_same_bits_each_time_and_captured(H):
    rng = np.random.default_rng(13)
    s = wl.make_seqs(rng, [1, 2, 1], [6000, 350, 2222], 64)
    seqs, g = smla.Seqs.from_host(s), _gen(13)
    pool = _cache(s.phys_rows, g)
    q = torch.randn((4, H, 576), generator=g, device="cuda").bfloat16()
    ref = _decode(seqs, q, pool, 6000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(ref, _decode(seqs, q, pool, 6000, stream=side))
    for _ in range(10):
        assert torch.equal(ref, _decode(seqs, q, pool, 6000))
    # one captured step: the new tokens written, then attended to, over growing lengths
    x = torch.randn((4, 576), generator=g, device="cuda").bfloat16()
    kv = seqs.kv_len.clone()
    live = smla.Seqs(seqs.cu_q, kv, seqs.page_table, 64, 4)
    ws = torch.empty(smla.dense_decode_workspace_size(4, H, 6000), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smla.cache_append_fp4(x, live, pool)
        smla.dense_decode_fp4(q, pool, live, 6000, SCALE, out, ws)
    for cut in (3, 1, 0):
        kv.copy_(seqs.kv_len - cut)
        x.copy_(torch.randn((4, 576), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        smla.check_device_errors()
        assert torch.equal(out, _decode(live, q, pool, 6000))


def test_rows_taken_back_serve_the_sparse_calls():
    """The gathered e4m3 rows with their scales as the pool of sparse attention."""
    g = _gen(14)
    n, H, k = 300, 64, 64
    pool = _cache(304, g)
    rows, scales = _as_e4m3(pool)
    q = torch.randn((5, H, 576), generator=g, device="cuda").bfloat16()
    idx = torch.stack([torch.randperm(n, generator=g, device="cuda")[:k] for _ in range(5)])
    lens = torch.full((5,), k, dtype=torch.int32, device="cuda").view(torch.uint32)
    out = torch.empty((5, H, 512), dtype=torch.bfloat16, device="cuda")
    smla.sparse_prefill(q, rows, scales, 576, idx.int().view(torch.uint32), lens, SCALE, out)
    smla.check_device_errors()
    v, sc = (t.cuda() for t in _values(pool))
    for t in range(5):
        c = (v * sc[:, None])[idx[t]]
        want = torch.softmax(SCALE * q[t].double() @ c.T, 1) @ c[:, :512]
        assert float((out[t].double() - want).norm() / want.norm()) < 1e-2
