"""Offsets past 2^31 and 2^32: a 4-bit pool of 4.5 GB, quantisations of 4.4 G elements, products
with 2.3 G outputs, rows of operands 4.6 GB apart and weights of 2.1 GB.  What lies far
is compared with the same data near by, or with the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import serving_fp8_indexer_gb300 as smla
from test_gpu_block_matmul import E4, U, _gen, _quantized
from test_gpu_dense_decode import SCALE

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def test_a_4_bit_pool_past_32_bits():
    """Pages at the pool's start, around 2^31 and 2^32 bytes and at its end: written, read
    back in both types and attended to as in a small pool."""
    page, n = 64, 14_000_000 // 64
    far = [0, (1 << 31) // (64 * 320), (1 << 31) // (64 * 320) + 1, (1 << 32) // (64 * 320), (1 << 32) // (64 * 320) + 1, n - 2, n - 1]
    i32 = dict(dtype=torch.int32, device="cuda")
    kv = 7 * page - 5
    x = torch.randn((kv, 576), generator=_gen(1), device="cuda").bfloat16()
    q = torch.randn((2, 64, 576), generator=_gen(2), device="cuda").bfloat16()
    got = []
    for pages, phys in ((far, n * page), (range(7), 7 * page)):
        pool = torch.full((phys, 320), 0xFF, dtype=torch.uint8, device="cuda")
        table = torch.tensor([list(pages)], **i32)
        fill = smla.Seqs(torch.tensor([0, kv], **i32), torch.tensor([kv], **i32), table, page, kv)
        smla.cache_append_fp4(x, fill, pool)
        rows, scales = torch.empty((kv, 576), dtype=torch.uint8, device="cuda"), torch.empty((kv, 1), device="cuda")
        smla.cache_gather_fp4(pool, fill, rows, scales)
        bf = torch.empty((kv, 576), dtype=torch.bfloat16, device="cuda")
        smla.cache_gather_fp4(pool, fill, bf)
        outs = []
        for H in (16, 64):
            step = smla.Seqs(torch.tensor([0, 2], **i32), torch.tensor([kv], **i32), table, page, 2)
            out = torch.full((2, H, 512), math.nan, dtype=torch.bfloat16, device="cuda")
            ws = torch.empty(smla.dense_decode_workspace_size(2, H, kv), dtype=torch.uint8, device="cuda")
            smla.dense_decode_fp4(q[:, :H].contiguous(), pool, step, kv, SCALE, out, ws)
            outs.append(out)
        smla.check_device_errors()
        written = torch.cat([pool[p * page:(p + 1) * page] for p in pages])[:kv]
        assert bool((pool.view(-1, page, 320)[pages[-1], page - 5:] == 0xFF).all())
        got.append((written, rows, scales, bf, *outs))
        del pool
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got))
    assert bool(got[0][-1].isfinite().all()) and bool(got[0][3].isfinite().all())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("K", [128, 1552, 4096, 16384])
def test_quantisations_past_32_bits(K, norm):
    M = (1 << 32) // K + 1003
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    piece = torch.randn(1 << 22, generator=_gen(K), device="cuda").bfloat16()
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 22):
        part = flat[i:i + (1 << 22)]
        part.copy_(piece[:part.numel()])
    w = (1 + 0.2 * torch.randn(K, generator=_gen(3), device="cuda")).bfloat16() if norm else None
    out = torch.full((M, K), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full((M, -(-K // 128)), math.nan, device="cuda")
    smla.quantize_blocks(x, out, s, norm_weight=w)
    smla.check_device_errors()
    # the form that a few rows take sums them in another order where there is a norm: a
    # scale is off by 50 u on each side, and a byte by one step
    for row in (0, (1 << 31) // K - 20, (1 << 32) // K - 20, M - 40):
        few, fs = _quantized(x[row:row + 40].contiguous(), w)
        part, ps = out[row:row + 40], s[row:row + 40]
        if norm:
            assert bool(((ps - fs).abs() <= 100 * U * fs).all())
            a, b = part.view(E4).float(), few.view(E4).float()
            assert bool(((a - b).abs() <= (2.0 ** -3 * torch.maximum(a.abs(), b.abs())).clamp_min(2.0 ** -9)).all())
            assert float((part != few).float().mean()) < 1e-3
        else:
            assert torch.equal(ps, fs) and torch.equal(part, few)


def _rows_close(out, a, sa, b, sb):
    """Some rows and columns of a product of one block of columns against 64 bits."""
    av, bv = a.view(E4).double() * sa.double(), b.view(E4).double() * sb.double()
    ref, mass = av @ bv.T, av.abs() @ bv.abs().T
    tol = 259 * U * mass + (2.0 ** -8 * ref.abs() if out.dtype == torch.bfloat16 else U * ref.abs())
    assert bool(((out.double() - ref).abs() <= tol).all())


def test_products_past_32_bits_many_rows():
    """Rows of a and of its scales far apart, 2.3 G outputs."""
    M, N, K, far = 70_000, 32_776, 128, 65_536
    g = _gen(7)
    room = torch.empty((M, far), dtype=torch.uint8, device="cuda")
    a = room[:, far - K:]
    a.copy_((torch.randn((M, K), generator=g, device="cuda") * 60).to(E4).view(torch.uint8))
    scales = torch.empty((M, 31_000), device="cuda")[:, 30_999:]
    scales.copy_(torch.exp(torch.randn((M, 1), generator=g, device="cuda")))
    b = (torch.randn((N, K), generator=g, device="cuda") * 60).to(E4).view(torch.uint8)
    sb = torch.exp(torch.randn((-(-N // 128), 1), generator=g, device="cuda"))
    out = torch.full((M, N), math.nan, dtype=torch.bfloat16, device="cuda")
    smla.block_matmul(a, scales, b, sb, out)
    smla.check_device_errors()
    full = sb.repeat_interleave(128, 0)[:N]
    for row in (0, (1 << 31) // far - 128, (1 << 32) // far - 128, (1 << 31) // N - 128, M - 256):
        _rows_close(out[row:row + 256], a[row:row + 256], scales[row:row + 256], b, full)
    assert not bool(torch.stack([o.isnan().any() for o in out.split(5000)]).any())


@pytest.mark.parametrize("M,dtype", [(16, torch.float32), (30, torch.bfloat16)])
def test_products_past_32_bits_many_columns(M, dtype):
    """Weights of 2.1 GB, rows of 134 M outputs."""
    N, K = (1 << 27) + 2056, 16
    g = _gen(8)
    a = (torch.randn((M, K), generator=g, device="cuda") * 60).to(E4).view(torch.uint8)
    sa = torch.exp(torch.randn((M, 1), generator=g, device="cuda"))
    b = torch.randint(0, 0x7F, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    sb = torch.rand((-(-N // 128), 1), generator=g, device="cuda") + 0.5
    out = torch.full((M, N), math.nan, dtype=dtype, device="cuda")
    smla.block_matmul(a, sa, b, sb, out)
    smla.check_device_errors()
    for c in (0, (1 << 26) - 512, (1 << 27) - 512, N - 1024):
        cols = slice(c, c + 1024)
        _rows_close(out[:, cols], a, sa, b[cols], sb[torch.arange(c, c + 1024, device="cuda") // 128])
    assert not bool(torch.stack([o.isnan().any() for o in out.split(1 << 24, 1)]).any())


def test_heads_past_32_bits():
    """A batch whose heads' outputs lie 4.4 GB apart, between rows that are not written."""
    G, M, N, K = 3, 300, 1032, 272
    g = _gen(9)
    a = (torch.randn((G, M, K), generator=g, device="cuda") * 60).to(E4).view(torch.uint8)
    b = (torch.randn((G, N, K), generator=g, device="cuda") * 60).to(E4).view(torch.uint8)
    sa, sb = torch.ones((G, M, 3), device="cuda"), torch.ones((G, 9, 3), device="cuda")
    near = torch.empty((G, M, N), dtype=torch.bfloat16, device="cuda")
    smla.block_matmul(a, sa, b, sb, near)
    apart = 2_200_000_000 // 8 * 8
    room = torch.zeros(2 * apart + M * N, dtype=torch.bfloat16, device="cuda")
    out = room.as_strided((G, M, N), (apart, N, 1))
    smla.block_matmul(a, sa, b, sb, out)
    smla.check_device_errors()
    assert torch.equal(out, near)
    assert np.isclose(float(sum(p.float().abs().sum(dtype=torch.float64) for p in room.split(1 << 28))),
                      float(near.float().abs().sum(dtype=torch.float64)), rtol=1e-9)
