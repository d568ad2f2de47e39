"""The softmax weights of the expanded prefill in one bf16 term or two, as the
caller asks: the accuracy of a row is the same whatever else its call holds."""
import pytest
import torch

import serving_fp8_indexer_gb300 as smla
from test_gpu_expanded import SCALE, _close, _inputs, _reference

pytestmark = pytest.mark.gpu


def _run(q, kv, kr, cu_q, cu_kv, p_terms):
    T, H = q.shape[:2]
    n = smla.expanded_prefill_workspace_size(T, kv.shape[0], cu_q.shape[0] - 1, H)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    out = torch.full((T, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    smla.expanded_prefill(q, kv[..., :128], kr, kv[..., 128:], cu_q, cu_kv, SCALE, out, ws, p_terms=p_terms)
    smla.check_device_errors()
    return out


@pytest.mark.parametrize("q_lens,kv_lens,H", [([1], [300], 1), ([64], [64], 1), ([65], [65], 1), ([300], [700], 8),
                                              ([64, 65, 1], [64, 3000, 513], 4), ([1000], [1000], 3), ([2], [9000], 64)])
def test_two_terms_round_only_the_output_at_every_size(q_lens, kv_lens, H):
    """Two terms are off by 2^-16 of a weight, a hundredth of the output's rounding
    (2^-8 / sqrt(3) of an element, root mean square), on either side of the size
    up to which they are taken unasked."""
    q, kv, kr, cu_q, cu_kv = _inputs(q_lens, kv_lens, H, seed=31)
    ref, _, tol = _reference(q, kv, kr, q_lens, kv_lens)
    got = _run(q, kv, kr, cu_q, cu_kv, 2)
    _close(got, ref, tol)
    assert float((got.double() - ref).norm()) <= 1.1 * float((ref.bfloat16().double() - ref).norm())
    _close(_run(q, kv, kr, cu_q, cu_kv, 1), ref, tol)


def test_a_row_is_as_exact_among_many_as_alone():
    q, kv, kr, cu_q, cu_kv = _inputs([1, 200], [150, 200], 8, seed=32)
    ref, _, _ = _reference(q, kv, kr, [1, 200], [150, 200])
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for many, alone in ((_run(q, kv, kr, cu_q, cu_kv, 2)[:1], _run(q[:1], kv, kr, one, cu_kv[:2].contiguous(), 2)),):
        rounding = float((ref[:1].bfloat16().double() - ref[:1]).norm())
        assert float((many.double() - ref[:1]).norm()) <= 1.1 * rounding
        assert float((alone.double() - ref[:1]).norm()) <= 1.1 * rounding


@pytest.mark.parametrize("q_len,terms", [(64, 2), (65, 1)])
def test_unasked_the_size_of_the_call_decides(q_len, terms):
    q, kv, kr, cu_q, cu_kv = _inputs([q_len], [200], 1, seed=33)
    assert torch.equal(_run(q, kv, kr, cu_q, cu_kv, 0), _run(q, kv, kr, cu_q, cu_kv, terms))
    assert not torch.equal(_run(q, kv, kr, cu_q, cu_kv, 0), _run(q, kv, kr, cu_q, cu_kv, 3 - terms))
