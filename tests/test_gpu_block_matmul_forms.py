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
