"""Rotary angles far below one turn, in f32: pairs (0, 1), whose first element
becomes -amplitude * sin(angle), to its last digits.

Tolerance (u = 2^-24): the reduced angle is rounded to a float, 1 u of itself, and
a sine below a quarter turn by no more of itself; sincospif is off by 2 ulp, 4 u;
the products with the amplitude and with 1 add a rounding each: 7 u."""
import numpy as np
import pytest
import torch

import serving_fp8_indexer_gb300 as smla

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("scaling,base", [("plain", 10000.0), ("yarn", 10000.0), ("linear", 5e6)])
@pytest.mark.parametrize("first", [0, 1, 100, 9000])
def test_small_angles_keep_their_relative_accuracy(half, scaling, base, first):
    T, dim = 70, 64
    freq, amp = smla.rope_frequencies(dim, base=base, scaling=scaling, factor=40.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    seqs = smla.Seqs(torch.tensor([0, T], **i32), torch.tensor([first + T], **i32), torch.zeros((1, 1), **i32), 64, T)
    x = torch.zeros((T, 1, dim), device="cuda")
    one, zero = (slice(dim // 2, dim), slice(0, dim // 2)) if half else (slice(1, dim, 2), slice(0, dim, 2))
    x[..., one] = 1.0
    out = torch.empty_like(x)
    smla.rope(x, seqs, smla.Rope(freq, 0, smla.ROPE_HALF if half else smla.ROPE_INTERLEAVED, amp), out)
    smla.check_device_errors()
    angle = np.outer(np.arange(first, first + T), freq.cpu().numpy())
    small = angle < 1.5
    assert small.any()
    sine = -out[:, 0, zero].double().cpu().numpy()
    want = np.sin(angle) * np.float64(np.float32(amp))
    assert (np.abs(sine - want) <= 7 * U * np.abs(want))[small].all()
