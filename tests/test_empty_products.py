"""A product without batches, rows or columns does nothing, whatever strides its empty
tensors have (torch gives those of a [M, 0] tensor as 1)."""
import pytest
import torch

from serving_fp8_indexer_gb300 import _latent, _lib
from serving_fp8_indexer_gb300 import build as smla_build


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N", [(2, 4, 0), (2, 0, 64), (0, 4, 64), (None, 4, 0), (None, 0, 64), (None, 0, 0), (2, 1, 0)])
def test_empty_products(monkeypatch, G, M, N, dtype):
    monkeypatch.setattr(_latent, "_device", lambda: -1)  # (host tensors count as device -1)
    smla_build.build()
    lead = () if G is None else (G,)
    u8 = lambda *n: torch.zeros((*lead, *n), dtype=torch.uint8)  # noqa: E731
    f = lambda *n: torch.zeros((*lead, *n))  # noqa: E731
    out = torch.zeros((*lead, M, N), dtype=dtype)
    assert _latent.block_matmul(u8(M, 272), f(M, 3), u8(N, 272), f(-(-N // 128), 3), out, stream=0) is out


def test_empty_products_of_any_strides():
    smla_build.build()
    lib, P = _lib.load(), 0x10000
    for G, M, N in ((0, 4, 64), (3, 0, 64), (3, 4, 0)):
        for odd in (0, 1, 7, -16, 1 << 50):
            assert lib.smla_block_matmul(P, odd, odd, P, odd, odd, P, P, G, M, N, 128, P, 0, odd, odd, None) == 0
    assert lib.smla_block_matmul(P, 0, 0, P, 0, 0, P, P, 3, 4, 0, 120, P, 0, 0, 0, None) != 0  # K is still checked
