"""Latent attention in the expanded form against its definition in 64 bits.

Tolerance, from the arithmetic.  A logit is a sum of 192 products in float32
on the tensor cores: off by at most 192 * 2^-23 of its mass, which is at most
|q| |k| * scale (2^-23 a step, since the tensor cores may truncate), so a
weight is off by twice that relative to the row's largest, and by 2^-20 for
the exponential and its argument's rounding.  A weight is rounded to bf16
(2^-8).  The weighted sum over n keys adds n * 2^-23.  All of it scales with
sum_j p_j |v_j|; the output's own rounding is 2^-8 of the output.
"""
import numpy as np
import pytest
import torch

import oracle.latent as ol
import serving_fp8_indexer_gb300 as smla

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def _inputs(q_lens, kv_lens, H, seed=0, spare=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, S = sum(q_lens), sum(kv_lens) + spare
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return n(T, H, 192), n(S, H, 256), n(S, 64), _cu(q_lens), _cu(kv_lens)


def _reference(q, kv, kr, q_lens, kv_lens, sink=None):
    """(out, lse, error scale) in float64: the definition, one sequence and
    head at a time."""
    T, H = q.shape[:2]
    out = torch.zeros((T, H, 128), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -float("inf"), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    q0 = k0 = 0
    for m, n in zip(q_lens, kv_lens):
        for h in range(H):
            if m == 0:
                continue
            qq = q[q0:q0 + m, h].double()
            kk = torch.cat([kv[k0:k0 + n, h, :128], kr[k0:k0 + n]], 1).double()
            v = kv[k0:k0 + n, h, 128:].double()
            z = SCALE * qq @ kk.T
            i, j = torch.arange(m, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
            z = z.masked_fill(j > n - m + i, -float("inf"))
            if sink is not None:
                z = torch.cat([z, sink[h].double().expand(m, 1)], 1)
            if z.shape[1] == 0:
                continue
            L = torch.logsumexp(z, 1)
            p = torch.exp(z - L[:, None])[:, :n].nan_to_num(0.0)  # rows without keys: nothing
            out[q0:q0 + m, h] = p @ v
            lse[q0:q0 + m, h] = L
            if n:
                mass = SCALE * qq.norm(dim=1) * kk.norm(dim=1).max()
                rel = 2.0 ** -8 + 2 * 192 * 2.0 ** -23 * mass + n * 2.0 ** -23 + 2.0 ** -20
                tol[q0:q0 + m, h] = rel[:, None] * (p @ v.abs()) + 2.0 ** -8 * out[q0:q0 + m, h].abs()
        q0, k0 = q0 + m, k0 + n
    return out, lse, tol


def _run(q, kv, kr, cu_q, cu_kv, sink=None, lse=False, out=None, stream=None):
    T, H = q.shape[:2]
    n = smla.expanded_prefill_workspace_size(T, kv.shape[0], cu_q.shape[0] - 1, H)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    out = torch.full((T, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    ls = torch.full((T, H), float("nan"), device="cuda") if lse else None
    smla.expanded_prefill(q, kv[..., :128], kr, kv[..., 128:], cu_q, cu_kv, SCALE, out, ws, attn_sink=sink, lse=ls,
                          stream=stream)
    smla.check_device_errors(stream)
    return (out, ls) if lse else out


def _close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert bool((err <= tol + 1e-30).all()), f"worst {float((err / (tol + 1e-30)).max()):.3g} x the tolerance"


SHAPES = [([1], [1], 1), ([1], [2], 3), ([3], [3], 2), ([127], [127], 3), ([128], [128], 2), ([129], [129], 2),
          ([255, 256, 257], [255, 256, 257], 2), ([0, 1, 5, 0, 300], [4, 700, 5, 0, 1025], 4), ([512], [640], 16),
          ([64, 64], [129, 128], 5), ([384], [2000], 1), ([700, 1], [701, 1], 130)]


@pytest.mark.parametrize("q_lens,kv_lens,H", SHAPES)
@pytest.mark.parametrize("sink", [False, True])
def test_matches_the_definition(q_lens, kv_lens, H, sink):
    q, kv, kr, cu_q, cu_kv = _inputs(q_lens, kv_lens, H)
    sk = torch.randn(H, device="cuda") if sink else None
    out, lse = _run(q, kv, kr, cu_q, cu_kv, sk, lse=True)
    ref, ref_lse, tol = _reference(q, kv, kr, q_lens, kv_lens, sk)
    _close(out, ref, tol)
    mass = float(SCALE * q.float().norm(dim=2).max() * torch.cat([kv[..., :128].float().norm(dim=2).max()[None],
                                                                  kr.float().norm(dim=1).max()[None]]).norm())
    assert bool(((lse.double() - ref_lse).abs() <= 192 * 2.0 ** -23 * mass + max(kv_lens) * 2.0 ** -24 + 1e-5).all())


@pytest.mark.parametrize("q_lens,kv_lens,H", [([1], [5000], 1), ([130], [9001], 2), ([2, 1, 3], [3000, 100, 7000], 4),
                                              ([16], [1024], 8)])
@pytest.mark.parametrize("sink", [False, True])
def test_few_queries_split_the_keys(q_lens, kv_lens, H, sink):
    q, kv, kr, cu_q, cu_kv = _inputs(q_lens, kv_lens, H, seed=1)
    assert smla.expanded_prefill_workspace_size(q.shape[0], kv.shape[0], len(q_lens), H) > 0
    sk = torch.randn(H, device="cuda") + 3 if sink else None
    out, lse = _run(q, kv, kr, cu_q, cu_kv, sk, lse=True)
    ref, ref_lse, tol = _reference(q, kv, kr, q_lens, kv_lens, sk)
    _close(out, ref, tol)
    assert bool(((lse.double() - ref_lse).abs() <= 1e-2).all())


def test_rows_that_attend_to_nothing():
    """More new tokens than keys, no keys, and no key rows at all: zeros, and
    with a sink still zeros."""
    for q_lens, kv_lens in (([5, 3], [3, 0]), ([200], [10]), ([4], [0])):
        for sink in (None, torch.tensor([0.5, -2.0], device="cuda")):
            q, kv, kr, cu_q, cu_kv = _inputs(q_lens, kv_lens, 2, seed=2)
            out, lse = _run(q, kv, kr, cu_q, cu_kv, sink, lse=True)
            ref, ref_lse, tol = _reference(q, kv, kr, q_lens, kv_lens, sink)
            _close(out, ref, tol)
            empty = torch.isneginf(ref_lse)
            assert torch.equal(torch.isneginf(lse), empty)
            assert bool(((lse.double() - ref_lse)[~empty].abs() <= 1e-4).all())


def test_growing_logits_rescale():
    """Logits that grow along the keys raise every row's reference in many
    blocks; a sink far above and far below them."""
    q, kv, kr, cu_q, cu_kv = _inputs([300], [900], 2, seed=3)
    kv[..., :128] = (q[:1, :, :128].float().sign() * torch.linspace(0, 1, 900, device="cuda")[:, None, None] * 8).bfloat16()
    q[..., :128] = q[:1, :, :128].abs().bfloat16() * q[:1, :, :128].sign()
    for sink in (None, torch.tensor([90.0, -90.0], device="cuda"), torch.tensor([300.0, float("-inf")], device="cuda")):
        out, lse = _run(q, kv, kr, cu_q, cu_kv, sink, lse=True)
        ref, ref_lse, tol = _reference(q, kv, kr, [300], [900], sink)
        _close(out, ref, tol)
        assert bool(((lse.double() - ref_lse).abs() <= 1e-3 * (1 + ref_lse.abs())).all())


def test_what_lies_outside_a_sequence_never_reaches_it():
    """NaN and infinities in the key rows of other sequences, between and
    behind them, and in the queries behind the last one."""
    q_lens, kv_lens = [70, 3, 140], [70, 33, 200]
    q, kv, kr, cu_q, cu_kv = _inputs(q_lens, kv_lens, 3, seed=4, spare=57)
    clean = _run(q, kv, kr, cu_q, cu_kv)
    for bad in (float("nan"), float("inf"), -3.3e38):
        kv2, kr2 = kv.clone(), kr.clone()
        kv2[70:103], kr2[70:103] = bad, bad  # the middle sequence
        kv2[303:], kr2[303:] = bad, bad
        out = _run(q, kv2, kr2, cu_q, cu_kv)
        keep = torch.cat([torch.arange(70), torch.arange(73, 213)]).cuda()
        assert torch.equal(out[keep], clean[keep])


def test_non_finite_inside_a_sequence_is_seen():
    q, kv, kr, cu_q, cu_kv = _inputs([1], [300], 1, seed=5)
    kv[100, 0, 130] = float("nan")
    out = _run(q, kv, kr, cu_q, cu_kv)
    assert bool(out[0, 0, 2].isnan()) and bool(out[0, 0, 3].isfinite())
    q[0, 0, 0] = float("nan")
    assert bool(_run(q, kv, kr, cu_q, cu_kv).isnan().all())


def test_padded_batch_strides_and_repeat():
    """Tokens behind the last sequence keep their outputs; separate, strided
    and transposed operands give the same result, twice the same bits."""
    q_lens, kv_lens, H = [100, 29], [100, 400], 4
    q, kv, kr, cu_q, cu_kv = _inputs(q_lens, kv_lens, H, seed=6)
    base = _run(q, kv, kr, cu_q, cu_kv)
    pad = torch.cat([q, torch.full((40, H, 192), float("nan"), device="cuda", dtype=torch.bfloat16)])
    out = torch.full((169, H, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    _run(pad, kv, kr, cu_q, cu_kv, out=out)
    assert bool((out[129:] == 5).all())
    ref, _, tol = _reference(q, kv, kr, q_lens, kv_lens)
    _close(out[:129], ref, tol)
    # heads outermost, and a wider rotary row
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    kt = kv.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros((kr.shape[0], 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 64:] = kr
    assert torch.equal(_run(qt, kt, wide[:, 64:], cu_q, cu_kv), base)
    assert torch.equal(_run(q, kv, kr, cu_q, cu_kv), base)


def test_captured_and_on_another_stream():
    """One capture serves later batches of the same bound: lengths are read on
    the device."""
    q, kv, kr, cu_q, cu_kv = _inputs([64, 64], [500, 500], 2, seed=7)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        first = _run(q, kv, kr, cu_q, cu_kv, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    out = torch.zeros((128, 2, 128), dtype=torch.bfloat16, device="cuda")
    n = smla.expanded_prefill_workspace_size(128, 1000, 2, 2)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        smla.expanded_prefill(q, kv[..., :128], kr, kv[..., 128:], cu_q, cu_kv, SCALE, out, ws)
    g.replay()
    smla.check_device_errors()
    assert torch.equal(out, first)
    cu_q.copy_(_cu([100, 28]))
    cu_kv.copy_(_cu([300, 700]))
    g.replay()
    smla.check_device_errors()
    ref, _, tol = _reference(q, kv, kr, [100, 28], [300, 700])
    _close(out, ref, tol)


def test_oracle_agrees_with_the_reference_above():
    """The numpy oracle and this file's reference are two readings of the
    same definition."""
    q, kv, kr, cu_q, cu_kv = _inputs([3, 0, 6], [5, 2, 4], 2, seed=8)
    sink = torch.tensor([0.3, -1.0], device="cuda")
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    for sk in (None, sink):
        ref, lse, _ = _reference(q, kv, kr, [3, 0, 6], [5, 2, 4], sk)
        o, l = ol.expanded_prefill(d(q), d(kv[..., :128]), d(kr), d(kv[..., 128:]), d(cu_q).astype(int),
                                   d(cu_kv).astype(int), SCALE, None if sk is None else d(sk))
        np.testing.assert_allclose(d(ref), o, atol=1e-12)
        np.testing.assert_allclose(d(lse), l, atol=1e-12)


def test_bad_key_offsets_are_reported():
    q, kv, kr, cu_q, cu_kv = _inputs([4], [8], 1, seed=9)
    cu_kv[1] = 9  # one past the key rows
    out = torch.empty((4, 1, 128), dtype=torch.bfloat16, device="cuda")
    smla.expanded_prefill(q, kv[..., :128], kr, kv[..., 128:], cu_q, cu_kv, SCALE, out, None)
    with pytest.raises(smla.SmlaError) as e:
        smla.check_device_errors()
    assert e.value.status == 5


@pytest.mark.parametrize("q_lens,kv_lens,H", [([1], [5000], 1), ([3, 2], [900, 40], 8), ([64], [64], 1),
                                              ([16], [300], 4), ([2, 2, 1], [212, 130, 180], 1)])
def test_calls_of_few_rows_round_only_the_output(q_lens, kv_lens, H):
    """P in two terms is off by 2^-16 of a weight, a hundredth of the output's
    rounding (2^-8 / sqrt(3) of an element, root mean square): beside the exact
    result rounded to bf16 the error may grow by a tenth at most."""
    q, kv, kr, cu_q, cu_kv = _inputs(q_lens, kv_lens, H, seed=21)
    ref, _, tol = _reference(q, kv, kr, q_lens, kv_lens)
    got = _run(q, kv, kr, cu_q, cu_kv)
    _close(got, ref, tol)
    assert float((got.double() - ref).norm()) <= 1.1 * float((ref.bfloat16().double() - ref).norm())
