"""The bytes that cache_append writes are e4m3 of the float32 quotient value /
scale, to the last bit: rows without norm and rotation, so that nothing else is
rounded.  Every bf16 largest magnitude of a binade is paired with every bf16
value of eleven binades below it; many quotients lie next to a border between two
bytes, where the product with a rounded reciprocal falls on the other side."""
import pytest
import torch

import serving_fp8_indexer_gb300 as smla

pytestmark = pytest.mark.gpu


def _rows(width):
    """bf16 rows [n, width]: column 0 the largest of the row (and of each
    32-column block: its first), the others values of it at random order."""
    m = torch.arange(128, 256, device="cuda").float()
    small = torch.cat([m * 2.0 ** -e for e in range(1, 12)])
    g = torch.Generator(device="cuda").manual_seed(1)
    per = -(-small.numel() // (width - width // 32))
    rows = []
    for a in m:
        v = torch.zeros(per * (width - width // 32), device="cuda")
        v[:small.numel()] = small[torch.randperm(small.numel(), generator=g, device="cuda")]
        v *= torch.randint(0, 2, v.shape, generator=g, device="cuda") * 2.0 - 1
        v = v.view(per, width // 32, 31)
        rows.append(torch.cat([a.expand(per, width // 32, 1), v], 2).reshape(per, width))
    return torch.cat(rows).bfloat16()


@pytest.mark.parametrize("size", [1.0, 2.0 ** -112, 2.0 ** 119])
@pytest.mark.parametrize("width,sbs", [(576, 576), (576, 32), (128, 128), (1024, 32)])
def test_bytes_are_the_quotients(width, sbs, size):
    x = _rows(width) * size
    T = x.shape[0]
    pages = -(-T // 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    seqs = smla.Seqs(torch.tensor([0, T], **i32), torch.tensor([T], **i32), torch.arange(pages, **i32)[None], 64, T)
    pool = torch.zeros((pages * 64, width), dtype=torch.uint8, device="cuda")
    blocks = width // min(sbs, width)
    scales = torch.zeros((pages * 64, blocks), device="cuda")
    smla.cache_append(x, seqs, pool, scales, sbs)
    smla.check_device_errors()
    # on the host: tensors by tensors there, IEEE quotients (a division by a number
    # is a product with its reciprocal on the GPU)
    v = x.float().cpu().view(T, blocks, -1)
    want = v.abs().amax(2) / torch.full((T, blocks), 448.0)
    assert torch.equal(scales[:T].cpu(), want)
    # a float32 quotient, and one rounding to e4m3 (nothing exceeds 448 by a whole step)
    byte = (v / want[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(T, width)
    assert torch.equal(pool[:T].cpu(), byte)
