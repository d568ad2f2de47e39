"""The operators as a serving loop runs them together: a chunk's projections
are normalised, rotated and written to the paged caches; its context is read
back, expanded per head and attended to; later tokens are decoded over the
same cache in the absorbed form, and through the indexer, top-k and sparse
attention.  Expanded and absorbed attention compute the same thing,
  q_nope . (W_uk c) = (W_uk^T q_nope) . c   and   W_uv sum p c = sum p (W_uv c),
so the two agree up to their roundings.

Tolerance.  Both forms read the same cache bytes and the same weights; what
differs is what is rounded to bf16 on the way: the gathered rows, the expanded
keys and values, the absorbed query, the weights P and the outputs, twelve
roundings in all of which each moves the result by at most 2^-8 / sqrt(3) of
its size in the root mean square (rounding errors of unrelated values), the
logits being of unit variance: sqrt(12) * 2^-8 / sqrt(3) = 2^-7 relative.
"""
import numpy as np
import pytest
import torch

import serving_fp8_indexer_gb300 as smla
from serving_fp8_indexer_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
REL = 2.0 ** -7
H, PAGE, SCALE = 16, 64, 192 ** -0.5


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


class Model:
    """One attention layer's weights and caches for sequences of up to `most` tokens."""

    def __init__(self, B, most, sbs, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.g, self.B, self.sbs = g, B, sbs
        self.w_uk = (n(H, 512, 128) / 512 ** 0.5).bfloat16()
        self.w_uv = (n(H, 512, 128) / 512 ** 0.5).bfloat16()
        self.norm = (1 + 0.1 * n(512)).bfloat16()
        self.s = wl.make_seqs(np.random.default_rng(seed), [1] * B, [most] * B, PAGE)
        self.table = torch.from_numpy(self.s.page_table).cuda()
        ns = 0 if sbs == 0 else 576 // min(sbs, 576)
        self.pool = torch.zeros((self.s.phys_rows, 576), dtype=torch.uint8, device="cuda")
        self.scales = torch.ones((self.s.phys_rows, ns), device="cuda") if ns else None
        self.k_pool = torch.zeros((self.s.phys_rows, 128), dtype=torch.uint8, device="cuda")
        self.k_scale = torch.ones((self.s.phys_rows, 1), device="cuda")
        f, a = smla.rope_frequencies(64, scaling="yarn", factor=4.0, original_len=1024)
        self.tail, self.head = smla.Rope(f, 512, smla.ROPE_INTERLEAVED, a), smla.Rope(f, 0, smla.ROPE_INTERLEAVED, a)
        self.key_rope = smla.Rope(f, 0, smla.ROPE_HALF, a)

    def seqs(self, q_lens, kv_lens):
        cu = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32, device="cuda")
        return smla.Seqs(cu, torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), self.table, PAGE, int(sum(q_lens)))

    def draw(self, T):
        n = lambda *s: torch.randn(s, generator=self.g, device="cuda").bfloat16()  # noqa: E731
        return n(T, 576), n(T, H, 192), n(T, 128)

    def write(self, seqs, latent, keys):
        rows = torch.empty_like(latent)
        smla.cache_append(latent, seqs, self.pool, self.scales, self.sbs, self.tail, norm_weight=self.norm, rows_out=rows)
        smla.cache_append(keys, seqs, self.k_pool, self.k_scale, 128, self.key_rope)
        return rows

    def expanded(self, seqs, q, kv_lens):
        whole = self.seqs(kv_lens, kv_lens)
        c = torch.empty((whole.T, 576), dtype=torch.bfloat16, device="cuda")
        smla.cache_gather(self.pool, self.scales, self.sbs, whole, c)
        kv = torch.einsum("sc,hcd->shd", c[:, :512], torch.cat([self.w_uk, self.w_uv], 2))  # [S, H, 256]
        q = q.clone()
        smla.rope(q[..., 128:], seqs, self.head, q[..., 128:])
        out = torch.empty((seqs.T, H, 128), dtype=torch.bfloat16, device="cuda")
        n = smla.expanded_prefill_workspace_size(seqs.T, whole.T, self.B, H)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        return smla.expanded_prefill(q, kv[..., :128], c[:, 512:], kv[..., 128:], seqs.cu_q, whole.cu_q, SCALE, out, ws)

    def absorbed_q(self, seqs, q):
        lat = torch.empty((seqs.T, H, 576), dtype=torch.bfloat16, device="cuda")
        lat[..., :512] = torch.einsum("thd,hcd->thc", q[..., :128], self.w_uk)
        smla.rope(q[..., 128:], seqs, self.head, lat[..., 512:])
        return lat

    def decode(self, seqs, lat, most, out, ws):
        return smla.dense_decode(lat, self.pool, self.scales, self.sbs, seqs, most, SCALE, out, ws)

    def up(self, out):
        return torch.einsum("thc,hcd->thd", out, self.w_uv)


@pytest.mark.parametrize("sbs", [0, 576])
def test_chunks_then_decode_both_forms(sbs):
    m = Model(3, 700, sbs)
    kv = [0, 0, 0]
    for q_lens in ([300, 64, 129], [200, 1, 300], [2, 2, 2], [1, 1, 1]):
        kv = [a + b for a, b in zip(kv, q_lens)]
        seqs = m.seqs(q_lens, kv)
        latent, q, keys = m.draw(seqs.T)
        m.write(seqs, latent, keys)
        a = m.expanded(seqs, q, kv)
        lat = m.absorbed_q(seqs, q)
        out = torch.empty((seqs.T, H, 512), dtype=torch.bfloat16, device="cuda")
        n = smla.dense_decode_workspace_size(seqs.T, H, max(kv))
        b = m.up(m.decode(seqs, lat, max(kv), out, torch.empty(n, dtype=torch.uint8, device="cuda") if n else None))
        smla.check_device_errors()
        assert _rel(b, a) <= REL
        # the dense prefill of the same cache and queries
        dense = torch.empty_like(out)
        smla.dense_prefill(lat, m.pool, m.scales, sbs, seqs, SCALE, dense)
        smla.check_device_errors()
        assert _rel(dense, out) <= REL


def test_written_caches_feed_the_indexer_and_sparse_attention():
    """With k at least the context's length the selection is every key, and
    sparse attention over it is the dense decode."""
    m = Model(2, 500, 576, seed=1)
    seqs = m.seqs([400, 333], [400, 333])
    latent, _, keys = m.draw(seqs.T)
    m.write(seqs, latent, keys)
    seqs = m.seqs([2, 2], [402, 335])
    latent, q, keys = m.draw(4)
    m.write(seqs, latent, keys)
    q_idx = torch.randn((4, 8, 128), generator=m.g, device="cuda").bfloat16()
    q8 = torch.empty((4, 8, 128), dtype=torch.uint8, device="cuda")
    smla.rope(q_idx, seqs, m.key_rope, q8)
    scores = torch.empty((4, 404), device="cuda")
    smla.indexer_scores(q8, torch.ones((4, 8), device="cuda"), m.k_pool, m.k_scale.view(-1), seqs, scores)
    idx = torch.empty((4, 512), dtype=torch.uint32, device="cuda")
    lens = torch.empty((4,), dtype=torch.uint32, device="cuda")
    smla.topk(scores, seqs, 512, idx, lens)
    lat = m.absorbed_q(seqs, q)
    sparse = torch.empty((4, H, 512), dtype=torch.bfloat16, device="cuda")
    smla.sparse_prefill(lat, m.pool, m.scales, 576, idx, lens, SCALE, sparse)
    dense = torch.empty_like(sparse)
    n = smla.dense_decode_workspace_size(4, H, 402)
    m.decode(seqs, lat, 402, dense, torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    smla.check_device_errors()
    assert lens.view(torch.int32).tolist() == [401, 402, 334, 335]
    assert _rel(sparse, dense) <= REL
    # the scores are those of the keys the cache holds: relu, summed over heads
    pos = [401 - 1, 402 - 1, 334 - 1, 335 - 1]
    for t in range(4):
        rows = torch.from_numpy(wl.logical_to_phys(m.s, t // 2, np.arange(pos[t] + 1))).cuda()
        k = m.k_pool[rows].view(torch.float8_e4m3fn).double() * m.k_scale[rows].double()
        ref = (q8[t].view(torch.float8_e4m3fn).double() @ k.T).clamp_min(0).sum(0)
        assert bool(((scores[t, :pos[t] + 1].double() - ref).abs() <= 1e-4 * ref.abs().max()).all())


def test_a_decode_step_captured_once_serves_the_next_tokens():
    """Rotation, cache write and attention of one step in a graph: lengths and
    inputs change between replays, the graph does not.  A padded slot keeps its
    output."""
    m = Model(2, 400, 576, seed=2)
    kv = [130, 64]
    first = m.seqs(kv, kv)
    latent, _, keys = m.draw(first.T)
    m.write(first, latent, keys)
    seqs = m.seqs([1, 1], [131, 65])
    step = smla.Seqs(seqs.cu_q, seqs.kv_len, m.table, PAGE, 3)  # one slot more than sequences
    latent, q, keys = m.draw(3)
    q_lat = torch.zeros((3, H, 576), dtype=torch.bfloat16, device="cuda")
    out = torch.full((3, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    n = smla.dense_decode_workspace_size(3, H, 400)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def run():
        smla.cache_append(latent, step, m.pool, m.scales, 576, m.tail, norm_weight=m.norm)
        q_lat[..., :512] = torch.einsum("thd,hcd->thc", q[..., :128], m.w_uk)
        smla.rope(q[..., 128:], step, m.head, q_lat[..., 512:])
        smla.dense_decode(q_lat, m.pool, m.scales, 576, step, 400, SCALE, out, ws)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for k in range(70):  # across a page's end
        nl, nq, _ = m.draw(3)
        latent.copy_(nl)
        q.copy_(nq)
        g.replay()
        if k % 23 == 0 or k == 69:
            got = out.clone()
            smla.check_device_errors()
            want = m.expanded(seqs, q[:2], seqs.kv_len.tolist())
            assert _rel(m.up(got[:2]), want) <= REL, k
            assert bool((got[2] == 5).all())
        seqs.kv_len.add_(1)
