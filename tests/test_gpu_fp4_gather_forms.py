"""Every form of the 4-bit gather against the rows' values, bit by bit: bf16 rows on
32-byte boundaries (one store a block) and on 16-byte ones, e4m3 rows, and calls of so
many tokens that a CTA takes 32 of them in several passes, with a ragged end.

A value is a product of 4 and 24 significant bits, rounded to f32 and then to bf16."""
import numpy as np
import pytest
import torch

import serving_fp8_indexer_gb300 as smla
from serving_fp8_indexer_gb300 import workloads as wl
from test_gpu_fp4_cache import _gen, _random_pool, _values

pytestmark = pytest.mark.gpu


def _rows(T, stride, offset, dtype):
    """[T, 576] rows `stride` elements apart, `offset` elements into their memory, which
    is marked."""
    room = torch.full((T * stride + offset + 64,), 0x55 if dtype is torch.uint8 else 7.0, dtype=dtype, device="cuda")
    return room, room[offset:offset + T * stride].view(T, stride)[:, :576]


def _check(s, seqs, pool, kv, stride, offset, dtype):
    phys = torch.from_numpy(np.concatenate([wl.logical_to_phys(s, b, np.arange(n)) for b, n in enumerate(kv)])).cuda()
    v, sc = _values(pool[phys])
    T = int(sum(kv))
    room, rows = _rows(T, stride, offset, dtype)
    before = room.clone()
    scales = torch.full((T, 1), float("nan"), device="cuda") if dtype is torch.uint8 else None
    smla.cache_gather_fp4(pool, seqs, rows, scales)
    smla.check_device_errors()
    if scales is None:
        assert torch.equal(rows.cpu(), (v * sc[:, None]).float().bfloat16())
    else:
        assert torch.equal(rows.contiguous().view(torch.float8_e4m3fn).double().cpu(), v)
        assert torch.equal(scales[:, 0].double().cpu(), sc)
    rows.copy_(before[offset:offset + T * stride].view(T, stride)[:, :576])
    assert torch.equal(room.view(torch.uint8), before.view(torch.uint8))  # nothing else was written


FORMS = [(576, 0, torch.bfloat16), (592, 16, torch.bfloat16), (584, 0, torch.bfloat16), (576, 8, torch.bfloat16),
         (576, 0, torch.uint8), (592, 16, torch.uint8)]


@pytest.mark.parametrize("stride,offset,dtype", FORMS)
@pytest.mark.parametrize("kv", [[1], [1, 777, 64, 2100]])
def test_few_rows(kv, stride, offset, dtype):
    s = wl.make_seqs(np.random.default_rng(len(kv)), kv, kv, 64)
    _check(s, smla.Seqs.from_host(s), _random_pool(s.phys_rows, _gen(3)), kv, stride, offset, dtype)


@pytest.mark.parametrize("stride,offset,dtype", FORMS)
def test_many_rows(stride, offset, dtype):
    """32 tokens a CTA: the last CTA has 11 of them, sequences end inside CTAs, and one has
    no tokens."""
    least = 64 * torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    kv = [1, least // 2 + 5, 0, 31, 33]
    kv.append(-(-least // 32) * 32 + 32 + 11 - sum(kv))
    assert sum(kv) >= least and sum(kv) % 32 == 11
    s = wl.make_seqs(np.random.default_rng(4), kv, kv, 16)
    _check(s, smla.Seqs.from_host(s), _random_pool(s.phys_rows, _gen(4)), kv, stride, offset, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8])
def test_many_rows_of_a_padded_batch(dtype):
    """Tokens behind the last sequence, whole CTAs of them, keep their rows."""
    least = 64 * torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    kv = [3000, 45]
    s = wl.make_seqs(np.random.default_rng(5), kv, kv, 64)
    seqs = smla.Seqs.from_host(s)
    T = least + 7
    padded = smla.Seqs(seqs.cu_q, seqs.kv_len, seqs.page_table, seqs.page_size, T)
    pool = _random_pool(s.phys_rows, _gen(5))
    mark = 0x55 if dtype is torch.uint8 else 7.0
    rows = torch.full((T, 576), mark, dtype=dtype, device="cuda")
    scales = torch.full((T, 1), 9.0, device="cuda") if dtype is torch.uint8 else None
    smla.cache_gather_fp4(pool, padded, rows, scales)
    few = torch.empty((3045, 576), dtype=dtype, device="cuda")
    few_scales = torch.empty((3045, 1), device="cuda") if dtype is torch.uint8 else None
    smla.cache_gather_fp4(pool, seqs, few, few_scales)
    smla.check_device_errors()
    assert torch.equal(rows[:3045].view(torch.uint8), few.view(torch.uint8)) and bool((rows[3045:] == mark).all())
    if scales is not None:
        assert torch.equal(scales[:3045], few_scales) and bool((scales[3045:] == 9.0).all())
