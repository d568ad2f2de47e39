"""The block-scaled product where its two forms end, meet and take strided operands.

Which form a call takes is the launcher's rule on costs, repeated here so that a
shape that is meant for one of them says so.  Tolerances: those of the product
itself."""
import pytest
import torch

import serving_fp8_indexer_gb300 as smla
from test_gpu_block_matmul import _close, _gen, _operand

pytestmark = pytest.mark.gpu


def _sms():
    return torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count


def _tiles(G, M, N, rows, cols):
    return G * -(-M // rows) * -(-N // cols)


def _halves(G, M, N):
    """Tiles of the wide form that go as halves."""
    pairs = _sms() // 2
    last = _tiles(G, M, N, 256, 256) % pairs
    return last if 2 * last <= pairs else 0


def _wide(G, M, N, K):
    kb, pairs, last = -(-K // 128), _sms() // 2, _halves(G, M, N)
    waves = -(-(_tiles(G, M, N, 256, 256) - last) // pairs)
    cost = (waves * (72 + 20 * kb) + ((72 + 13 * kb) if last else 0)) * _sms()
    return M > 32 and cost < _tiles(G, M, N, 64, 128) * (72 + 13 * kb)


@pytest.mark.parametrize("G,M,N,K", [(1, 2048, 2560, 16), (1, 2048, 2560, 144), (1, 3000, 7000, 128), (4, 700, 1032, 272)])
def test_calls_on_end_of_pairs_that_end_early(G, M, N, K):
    """One to three blocks a tile: a pair of CTAs is over as its last products are.
    What comes next on the same SMs (the same product, a quantisation) is not touched
    by what the pair before was still told."""
    assert _wide(G, M, N, K)
    g = _gen(K)
    a, sa, av = _operand(g, G, M, K, True)
    b, sb, bv = _operand(g, G, N, K, False)
    x = torch.randn((400, 1552), generator=g, device="cuda").bfloat16()
    w = torch.ones(1552, dtype=torch.bfloat16, device="cuda")
    outs = [torch.full((G, M, N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(12)]
    xb = [torch.empty((400, 1552), dtype=torch.uint8, device="cuda") for _ in outs]
    xs = [torch.empty((400, 13), device="cuda") for _ in outs]
    for o, q, s in zip(outs, xb, xs):
        smla.block_matmul(a, sa, b, sb, o)
        smla.quantize_blocks(x, q, s, norm_weight=w)
    smla.check_device_errors()
    _close(outs[0], av, bv)
    assert all(torch.equal(outs[0], o) for o in outs)
    assert all(torch.equal(xb[0], q) for q in xb) and all(torch.equal(xs[0], s) for s in xs)


@pytest.mark.parametrize("M,N,K", [(2300, 4096, 1040), (600, 2600, 2064)])
def test_new_operands_in_the_same_stages(M, N, K):
    """Products of new operands call after call: bytes that the second CTA of a pair has
    loaded are the ones that the first one's MMAs read, not those of the block or
    call before."""
    assert _wide(1, M, N, K)
    g = _gen(M)
    b, sb, bv = _operand(g, 1, N, K, False)
    calls = [_operand(g, 1, M, K, True) for _ in range(6)]
    outs = [torch.full((M, N), float("nan"), device="cuda") for _ in calls]
    for (a, sa, _), o in zip(calls, outs):
        smla.block_matmul(a[0], sa[0], b[0], sb[0], o)
    smla.check_device_errors()
    for (_, _, av), o in zip(calls, outs):
        _close(o[None], av, bv)


def _token_major(G, M, N, K, dtype, pad=24):
    """Operands strided as the heads of a [T, H, wider] tensor are, and what lies between
    their rows: NaN that is not read, 7.0 that is not written."""
    g = _gen(G + M)
    a, sa, av = _operand(g, G, M, K, True)
    b, sb, bv = _operand(g, G, N, K, False)
    kb = sa.shape[2]
    wide = torch.full((M, G, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :, :K] = a.transpose(0, 1)
    scales = torch.full((M + 1, G + 1, kb + 3), float("nan"), device="cuda")
    scales[:M, :G, :kb] = sa.transpose(0, 1)
    out = torch.full((M + 3, G, N + pad), 7.0, dtype=dtype, device="cuda")
    smla.block_matmul(wide[:, :, :K].transpose(0, 1), scales[:M, :G, :kb].transpose(0, 1), b, sb,
                      out[:M, :, :N].transpose(0, 1))
    smla.check_device_errors()
    _close(out[:M, :, :N].transpose(0, 1), av, bv)
    assert bool((out[:, :, N:] == 7.0).all()) and bool((out[M:] == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N,K,halves", [(8, 512, 1024, 272, 0), (3, 700, 2200, 640, 5), (16, 600, 384, 528, 20),
                                            (9, 250, 2056, 400, 5), (2, 257, 2056, 2064, 36)])
def test_heads_of_a_token_major_tensor_in_the_wide_form(G, M, N, K, halves, dtype):
    """The batch before the rows in a's and out's memory, with ends of tiles inside rows
    and columns, in whole tiles and halves."""
    assert _wide(G, M, N, K) and (_sms() != 152 or _halves(G, M, N) == halves)
    _token_major(G, M, N, K, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(700, 2200, 640), (300, 8200, 272)])
def test_padded_rows_in_the_wide_form(M, N, K, dtype):
    """One matrix with gaps between the rows of a, of its scales and of out."""
    assert _wide(1, M, N, K)
    _token_major(1, M, N, K, dtype)
    g = _gen(N)
    a, sa, av = _operand(g, 1, M, K, True)
    b, sb, bv = _operand(g, 1, N, K, False)
    wide = torch.full((M, K + 16), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :K] = a[0]
    out = torch.full((M, N + 8), 7.0, dtype=dtype, device="cuda")
    smla.block_matmul(wide[:, :K], sa[0], b[0], sb[0], out[:, :N])
    smla.check_device_errors()
    _close(out[None, :, :N], av, bv)
    assert bool((out[:, N:] == 7.0).all())


@pytest.mark.parametrize("G,M,N,K,halves", [(1, 2300, 4096, 8208, 0), (1, 2300, 5000, 4240, 28), (1, 700, 4104, 8208, 0)])
def test_long_columns_in_the_wide_form(G, M, N, K, halves):
    """More blocks than the scales' groups of eight many times over, the last group of
    one block or two, in whole tiles and halves."""
    assert _wide(G, M, N, K) and (_sms() != 152 or _halves(G, M, N) == halves)
    g = _gen(K)
    a, sa, av = _operand(g, G, M, K, True)
    b, sb, bv = _operand(g, G, N, K, False)
    out = torch.full((G, M, N), float("nan"), device="cuda")
    smla.block_matmul(a[0], sa[0], b[0], sb[0], out[0])
    smla.check_device_errors()
    _close(out, av, bv)


def _narrow_blocks(G, M, N, K):
    """Blocks of K that a CTA of the narrow form takes."""
    kb, cs = -(-K // 128), 1
    n = _tiles(G, M, N, 16 if M <= 16 else 32 if M <= 32 else 64, 128)
    while cs < 8 and 2 * n * cs <= 2 * _sms() - _sms() // 4 and kb >= 4 * cs:
        cs *= 2
    return -(-kb // cs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N,K", [(1, 16, 24576, 8208), (1, 30, 17160, 8336), (1, 50, 17200, 6160), (1, 64, 24576, 8208),
                                     (2, 10, 9000, 4240), (1, 300, 2304, 8208), (1, 5, 24568, 16400), (1, 17, 9000, 16400)])
def test_chunks_of_scales_in_the_narrow_form(G, M, N, K, dtype):
    """More than 32 blocks a CTA, whose scales come a chunk of 32 at a time: two chunks
    to five, the last of one block or more, with and without a cluster."""
    assert not _wide(G, M, N, K) and (_sms() != 152 or _narrow_blocks(G, M, N, K) > 32)
    g = _gen(M + K)
    a, sa, av = _operand(g, G, M, K, True)
    b, sb, bv = _operand(g, G, N, K, False)
    out = torch.full((G, M, N), float("nan"), dtype=dtype, device="cuda")
    smla.block_matmul(a, sa, b, sb, out)
    smla.check_device_errors()
    _close(out, av, bv)
