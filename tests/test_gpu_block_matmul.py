"""The block-scaled 8-bit matrix product and the quantisation of its left operand
against their definitions in 64 bits.

Tolerance of the product, from the arithmetic (u = 2^-24).  A product of two e4m3
values has 8 significant bits, exact in f32.  A block's 128 products and the sums
over the blocks are added in f32; in whatever order, and with the sum cut off
instead of rounded at each step, the 128 are off by at most 128 * 2u of the sum of
their magnitudes.  Each scale's product, its product with the block's sum and the
addition to the blocks before round once, the addition relative to the sum so far:
with kb blocks, 256 u + 2 u + kb u of the whole sum of magnitudes.  (A cluster's
partial sums are added the same way.)  The output rounds once more: bf16 by 2^-8 of
the value.

Quantised without a norm, scale and byte are single roundings of exact quantities
and compared bit by bit.  With it: a row's sum of squares is added by up to 256
threads with up to 64 each, then in five exchanges and at most 8 additions, off by
77 u of itself, its root by half of that; the division, the root and the two
products add 4 u: below 48 u.  Scales are off by that and one division; a value
relative to its scale by twice that, and then by half an e4m3 step: 2^-4 of it, or
2^-10.
"""
import pytest
import torch

import serving_fp8_indexer_gb300 as smla

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
E4 = torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _operand(g, G, R, K, by_rows):
    """(bytes, scales, values f64) of a [G, R, K] operand: a scale for each 128
    columns of a row, or of 128 rows."""
    kb, nb = -(-K // 128), R if by_rows else -(-R // 128)
    x = (torch.randn((G, R, K), generator=g, device="cuda") * 60).to(E4)
    s = torch.exp(torch.randn((G, nb, kb), generator=g, device="cuda"))
    full = s if by_rows else s.repeat_interleave(128, 1)[:, :R]
    return x.view(torch.uint8), s, x.double() * full.repeat_interleave(128, 2)[:, :, :K].double()


def _close(out, av, bv):
    ref = torch.bmm(av, bv.transpose(1, 2))
    mass = torch.bmm(av.abs(), bv.abs().transpose(1, 2))
    kb = -(-av.shape[2] // 128)
    tol = (258 + kb) * U * mass + (2.0 ** -8 * ref.abs() if out.dtype == torch.bfloat16 else U * ref.abs())
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp_min(1e-300)).max()):.3g} x the tolerance"


SHAPES = [(1, 1, 8, 16), (1, 1, 128, 128), (1, 15, 136, 112), (1, 16, 576, 144), (1, 17, 120, 1040), (1, 33, 264, 512),
          (1, 64, 2048, 4096), (1, 65, 384, 256), (1, 128, 128, 16384), (1, 129, 8, 2048), (1, 300, 1000, 784),
          (1, 1000, 5000, 400), (1, 2049, 1160, 128), (3, 5, 72, 208), (16, 16, 512, 128), (128, 16, 128, 512),
          (8, 130, 512, 128), (4, 700, 1032, 272), (2, 1, 8, 16), (1, 4101, 2056, 512)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N,K", SHAPES)
def test_product(G, M, N, K, dtype):
    g = _gen(G + M + N + K)
    a, sa, av = _operand(g, G, M, K, True)
    b, sb, bv = _operand(g, G, N, K, False)
    out = torch.full((G, M, N), float("nan"), dtype=dtype, device="cuda")
    if G == 1:
        smla.block_matmul(a[0], sa[0], b[0], sb[0], out[0])
    else:
        smla.block_matmul(a, sa, b, sb, out)
    smla.check_device_errors()
    _close(out, av, bv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N,K", [(1, 2050, 2056, 16), (1, 2600, 1800, 272), (1, 2100, 2296, 1296), (3, 700, 2200, 640),
                                     (1, 4000, 3904, 400), (1, 512, 4104, 2064), (2, 300, 1168, 8192), (1, 257, 8200, 144)])
def test_whole_and_half_tiles(G, M, N, K, dtype):
    """Tiles beyond whole waves of the GPU's pairs of CTAs, few of them: the last
    ones are divided, behind whole ones of one block of columns and of many, and with
    their second half past N; or all of a call's are."""
    test_product(G, M, N, K, dtype)


@pytest.mark.parametrize("G,M,N,K", [(16, 3, 64, 256), (8, 130, 136, 384), (128, 300, 128, 144)])
def test_heads_of_a_token_major_tensor(G, M, N, K):
    """Every operand strided as the heads of a [T, H, wider] tensor are; what lies
    between the rows is neither read (NaN) nor written."""
    g = _gen(G)
    a, sa, av = _operand(g, G, M, K, True)
    b, sb, bv = _operand(g, G, N, K, False)
    kb = sa.shape[2]
    wide = torch.full((M, G, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :, :K] = a.transpose(0, 1)
    scales = torch.full((M + 1, G + 1, kb + 3), float("nan"), device="cuda")
    scales[:M, :G, :kb] = sa.transpose(0, 1)
    out = torch.full((M, G, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    smla.block_matmul(wide[:, :, :K].transpose(0, 1), scales[:M, :G, :kb].transpose(0, 1), b, sb,
                      out[:, :, :N].transpose(0, 1))
    smla.check_device_errors()
    _close(out[:, :, :N].transpose(0, 1), av, bv)
    assert bool((out[:, :, N:] == 7.0).all())


def test_broadcast_scales_and_one_element_dimensions():
    """a_scales may have strides of 0, and strides of dimensions of one element do not matter."""
    g = _gen(3)
    a, _, _ = _operand(g, 4, 20, 256, True)
    b, sb, bv = _operand(g, 4, 40, 256, False)
    one = torch.full((1, 1, 1), 0.5, device="cuda")
    out = torch.empty((4, 20, 40), device="cuda")
    smla.block_matmul(a, one.expand(4, 20, 1).repeat(1, 1, 2), b, sb, out)
    _close(out, 0.5 * a.view(E4).double(), bv)
    two = torch.full((1, 1, 2), 0.5, device="cuda").expand(4, 20, 2)
    again = torch.empty_like(out)
    smla.block_matmul(a, two, b, sb, again)
    smla.check_device_errors()
    assert torch.equal(out, again)


@pytest.mark.parametrize("G,M", [(1, 1), (1, 300), (5, 1)])
def test_strides_of_one_element_do_not_matter(G, M):
    """As the C interface says: whatever stands there, 0 and negative numbers too."""
    from serving_fp8_indexer_gb300 import _lib

    lib, N, K = _lib.load(), 20000, 256
    g = _gen(6)
    a, sa, av = _operand(g, G, M, K, True)
    b, sb, bv = _operand(g, G, N, K, False)
    for odd in (0, -32, 1 << 40):
        out = torch.full((G, M, N), float("nan"), device="cuda")
        st = lib.smla_block_matmul(a.data_ptr(), odd if G == 1 else M * K, odd if M == 1 else K, sa.data_ptr(),
                                   odd if G == 1 else M * 2, odd if M == 1 else 2, b.data_ptr(), sb.data_ptr(), G, M, N, K,
                                   out.data_ptr(), 2, odd if G == 1 else M * N, odd if M == 1 else N, None)
        assert st == 0, _lib.last_error(lib)
        smla.check_device_errors()
        _close(out, av, bv)


@pytest.mark.parametrize("N", [8, 40, 264, 2088])
def test_many_tiles_with_few_columns(N):
    """Tiles whose last columns lie past N, one after the other on each SM: a
    place on the way out is not taken again before it has been read."""
    g = _gen(N)
    M, K = 60000, 128
    a, sa, av = _operand(g, 1, M, K, True)
    b, sb, bv = _operand(g, 1, N, K, False)
    for dtype in (torch.bfloat16, torch.float32):
        first = None
        for _ in range(4):
            out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
            smla.block_matmul(a[0], sa[0], b[0], sb[0], out)
            if first is None:
                first = out
                _close(out[None], av, bv)
            assert torch.equal(first, out)
    smla.check_device_errors()


@pytest.mark.parametrize("M", [4, 200])
def test_special_values_stay_in_their_rows_and_columns(M):
    g = _gen(4)
    N, K = 20000 if M > 64 else 264, 384
    a, sa, av = _operand(g, 1, M, K, True)
    b, sb, bv = _operand(g, 1, N, K, False)
    ref = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    smla.block_matmul(a[0], sa[0], b[0], sb[0], ref)
    a[0, 1, 200] = 0x7F              # NaN
    sa[0, 2, 1] = float("inf")
    sa[0, 3] = 0.0
    b[0, 5, 0] = 0xFF                # NaN
    out = torch.empty_like(ref)
    smla.block_matmul(a[0], sa[0], b[0], sb[0], out)
    smla.check_device_errors()
    assert bool(out[1].isnan().all()) and bool(out[:, 5].isnan().all())
    assert not bool(out[2].isfinite().any())
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[1:4] = False
    cols = torch.arange(N, device="cuda") != 5
    assert bool((out[3][cols] == 0).all())
    assert torch.equal(out[keep][:, cols], ref[keep][:, cols])


@pytest.mark.parametrize("M,N,K", [(16, 1024, 8192), (1030, 4104, 528)])
def test_same_bits_each_time_other_streams_and_graphs(M, N, K):
    g = _gen(5)
    a, sa, av = _operand(g, 1, M, K, True)
    b, sb, _ = _operand(g, 1, N, K, False)
    ref = torch.empty((M, N), device="cuda")
    smla.block_matmul(a[0], sa[0], b[0], sb[0], ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [torch.full_like(ref, float("nan")) for _ in range(6)]
    with torch.cuda.stream(side):  # two calls at once on two streams
        for o in outs[:3]:
            smla.block_matmul(a[0], sa[0], b[0], sb[0], o)
    for o in outs[3:5]:
        smla.block_matmul(a[0], sa[0], b[0], sb[0], o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smla.block_matmul(a[0], sa[0], b[0], sb[0], outs[5])
    graph.replay()
    torch.cuda.synchronize()
    smla.check_device_errors()
    assert all(torch.equal(ref, o) for o in outs)
    outs[5].fill_(float("nan"))
    sa *= 2  # the graph reads its inputs anew
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(2 * ref, outs[5])


# ------------------------------------------------------------------ quantisation
def _expected(x):
    """(bytes, scales) of float rows on the host: IEEE quotients, one rounding."""
    v = x.float().cpu()
    M, K = v.shape
    kb = -(-K // 128)
    v = torch.nn.functional.pad(v, (0, kb * 128 - K)).view(M, kb, 128)
    top = torch.where(v.isfinite(), v.abs(), torch.zeros(()))
    most = top.amax(2)
    s = torch.where(most > 0, (most / torch.full_like(most, 448.0)).clamp_min(2.0 ** -126), torch.ones(()))
    q = (v / s[:, :, None]).clamp(-448, 448)  # (NaN stays)
    return q.to(E4).view(torch.uint8).view(M, kb * 128)[:, :K], s


def _quantized(x, weight=None, eps=1e-6):
    M, K = x.shape
    out = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((M, -(-K // 128)), float("nan"), device="cuda")
    smla.quantize_blocks(x, out, s, norm_weight=weight, norm_eps=eps)
    smla.check_device_errors()
    return out, s


@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (16, 2048), (257, 1552), (1000, 576), (4100, 1168), (2, 16384),
                                 (1, 128), (2047, 128), (70001, 128), (3001, 256), (11003, 384), (9001, 512), (4097, 1024),
                                 (3000, 4112), (2500, 2048)])
def test_bytes_and_scales_are_the_quotients(M, K):
    g = _gen(M + K)
    wide = torch.randn((M, K + 64), generator=g, device="cuda").bfloat16() * torch.exp(2 * torch.randn((M, 1), generator=g, device="cuda")).bfloat16()
    x = wide[:, :K]
    out, s = _quantized(x)
    want, ws = _expected(x)
    assert torch.equal(s.cpu(), ws) and torch.equal(out.cpu(), want)


def test_zeros_infinities_nan_and_tiny_blocks():
    x = torch.randn((6, 400), generator=_gen(9), device="cuda").bfloat16()
    x[0] = 0
    x[1, 128:256] = 0
    x[2, 3] = float("inf")
    x[2, 130] = -float("inf")
    x[3, 5] = float("nan")
    x[4, 256:] = 2.0 ** -130
    x[5, :128] = float("inf")
    out, s = _quantized(x)
    want, ws = _expected(x)
    assert torch.equal(s.cpu(), ws)
    nan = want & 0x7F == 0x7F
    assert torch.equal(out.cpu() & 0x7F == 0x7F, nan) and torch.equal(out.cpu()[~nan], want[~nan])
    assert int(nan.sum()) == 1 and float(s[0, 0]) == 1.0 and int(out[2, 3]) == 0x7E and int(out[2, 130]) == 0xFE


@pytest.mark.parametrize("M,K", [(1, 16), (7, 128), (9, 1024), (16, 2048), (3, 4096), (130, 1040), (5, 16384), (2, 4112),
                                 (1, 48), (33, 96), (1001, 208), (17, 256), (1003, 512), (2001, 640), (1301, 1552), (1300, 2048),
                                 (1501, 4096), (1219, 4112), (1217, 8192), (1218, 16384)])
def test_normalised_rows(M, K):
    g = _gen(M * K)
    wide = (torch.randn((M, K + 8), generator=g, device="cuda") * torch.exp(3 * torch.randn((M, 1), generator=g, device="cuda"))).bfloat16()
    x, w = wide[:, :K], (1 + 0.2 * torch.randn(K, generator=g, device="cuda")).bfloat16()
    out, s = _quantized(x, w, 1e-3)
    v = x.double()
    v = v / (v.square().mean(1, keepdim=True) + 1e-3).sqrt() * w.double()
    kb = s.shape[1]
    blocks = torch.nn.functional.pad(v, (0, kb * 128 - K)).view(M, kb, 128)
    want = blocks.abs().amax(2) / 448
    assert bool(((s.double() - want).abs() <= 50 * U * want).all())
    q = (blocks / want[:, :, None]).view(M, kb * 128)[:, :K]
    err = (out.view(E4).double() - q).abs()
    assert bool((err <= 100 * U * q.abs() + (2.0 ** -4 * q.abs()).clamp_min(2.0 ** -10) * (1 + 100 * U)).all())


def test_rows_that_share_memory_are_read():
    x = torch.randn((1, 256), generator=_gen(2), device="cuda").bfloat16()
    out, s = _quantized(x.expand(5, 256))
    one, so = _quantized(x)
    assert torch.equal(out, one.expand(5, 256)) and torch.equal(s, so.expand(5, 2))
