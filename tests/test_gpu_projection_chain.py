"""An attention layer with 8-bit projections and a 4-bit latent cache, as a serving
loop runs it: hidden states are quantised and projected, the latents normalised,
rotated and written in 4 bits; a chunk attends in the expanded form over keys and
values up-projected from the cached rows, later tokens in the absorbed form over
the cache itself, and the outputs are projected back.

Expanded and absorbed attention compute the same thing from the same cached rows
and the same weights (an absorbed weight is the transpose of the up-projection's
128 x 128 blocks, byte for byte).  What differs are the operands rounded to e4m3 on
the way, each off by at most 2^-4 / sqrt(3) of its size in the root mean square:
the absorbed form's q_nope (in the logits, which have unit variance) and latent
outputs, the expanded form's rows (in the logits and in the values); sqrt(4) of
them together, and the bf16 roundings between, 2^-7 as for the same chain with 16-bit
projections: 2 * 2^-4 / sqrt(3) + 2^-7 = 0.08 of the result.
"""
import math

import numpy as np
import pytest
import torch

import serving_fp8_indexer_gb300 as smla
from serving_fp8_indexer_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
REL = 2 * 2.0 ** -4 / math.sqrt(3) + 2.0 ** -7
H, D, Q, PAGE, SCALE = 16, 1024, 256, 64, 192 ** -0.5


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _weight(g, *shape):
    """8-bit weights of unit gain with their block scales, [..., N, K]."""
    w = torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5
    *lead, N, K = shape
    pad = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128))
    tiles = pad.view(*lead, pad.shape[-2] // 128, 128, pad.shape[-1] // 128, 128)
    scale = tiles.abs().amax((-3, -1)) / 448
    full = scale.repeat_interleave(128, -2).repeat_interleave(128, -1)[..., :N, :K]
    return (w / full).to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), scale.contiguous()


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def _project(x, weight, norm=None):
    """bf16 [T, N] of x bf16 [T, K] through 8-bit weights."""
    T, K = x.shape
    b, s = _empty(T, K, dtype=torch.uint8), _empty(T, -(-K // 128), dtype=torch.float32)
    smla.quantize_blocks(x, b, s, norm_weight=norm)
    return smla.block_matmul(b, s, weight[0], weight[1], _empty(T, weight[0].shape[0]))


def _project_heads(x, weight, out):
    """out [T, H, N] (strided) of x bf16 [T, H, K] (strided rows) through weights [H, N, K]."""
    T, _, K = x.shape
    rows = x.reshape(T * H, K)
    b, s = _empty(T * H, K, dtype=torch.uint8), _empty(T * H, -(-K // 128), dtype=torch.float32)
    smla.quantize_blocks(rows, b, s)
    smla.block_matmul(b.view(T, H, K).transpose(0, 1), s.view(T, H, -1).transpose(0, 1), weight[0], weight[1],
                      out.transpose(0, 1))
    return out


class Layer:
    def __init__(self, B, most, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.B = g, B
        self.down = _weight(g, Q + 576, D)           # hidden -> compressed queries and latents
        self.q_up = _weight(g, H * 192, Q)
        up = _weight(g, H, 256, 512)                 # latents -> keys and values of each head
        self.kv_up = (up[0].view(H * 256, 512), up[1].view(H * 2, 4))
        self.k_t = (up[0][:, :128].transpose(1, 2).contiguous(), up[1][:, :1].transpose(1, 2).contiguous())
        self.v = (up[0][:, 128:].contiguous(), up[1][:, 1:].contiguous())
        self.out = _weight(g, D, H * 128)
        n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.q_norm, self.c_norm = (1 + 0.1 * n(Q)).bfloat16(), (1 + 0.1 * n(512)).bfloat16()
        s = wl.make_seqs(np.random.default_rng(seed), [1] * B, [most] * B, PAGE)
        self.table = torch.from_numpy(s.page_table).cuda()
        self.pool = torch.zeros((s.phys_rows, 320), dtype=torch.uint8, device="cuda")
        f, a = smla.rope_frequencies(64, scaling="yarn", factor=4.0, original_len=1024)
        self.tail, self.head = smla.Rope(f, 512, amplitude=a), smla.Rope(f, 0, amplitude=a)

    def seqs(self, q_lens, kv_lens):
        i32 = dict(dtype=torch.int32, device="cuda")
        return smla.Seqs(torch.tensor([0] + list(np.cumsum(q_lens)), **i32), torch.tensor(kv_lens, **i32), self.table, PAGE,
                         int(sum(q_lens)))

    def write(self, x, seqs):
        """Queries [T, H, 192]; the latents go into the cache."""
        y = _project(x, self.down)
        smla.cache_append_fp4(y[:, Q:], seqs, self.pool, self.tail, norm_weight=self.c_norm)
        return _project(y[:, :Q], self.q_up, self.q_norm).view(seqs.T, H, 192)

    def expanded(self, q, seqs, kv_lens):
        whole = self.seqs(kv_lens, kv_lens)
        c = smla.cache_gather_fp4(self.pool, whole, _empty(whole.T, 576))
        kv = _project(c[:, :512], self.kv_up).view(whole.T, H, 256)
        q = q.clone()
        smla.rope(q[..., 128:], seqs, self.head, q[..., 128:])
        n = smla.expanded_prefill_workspace_size(seqs.T, whole.T, self.B, H)
        return smla.expanded_prefill(q, kv[..., :128], c[:, 512:], kv[..., 128:], seqs.cu_q, whole.cu_q, SCALE,
                                     _empty(seqs.T, H, 128), _empty(n, dtype=torch.uint8) if n else None)

    def absorbed(self, q, seqs, most, ws):
        lat = _empty(seqs.T, H, 576)
        _project_heads(q[..., :128], self.k_t, lat[..., :512])
        smla.rope(q[..., 128:], seqs, self.head, lat[..., 512:])
        o = smla.dense_decode_fp4(lat, self.pool, seqs, most, SCALE, _empty(seqs.T, H, 512), ws)
        return _project_heads(o, self.v, _empty(seqs.T, H, 128))

    def finish(self, o):
        return _project(o.reshape(o.shape[0], H * 128), self.out)


def test_chunks_then_decode_both_forms():
    m = Layer(3, 700)
    kv = [0, 0, 0]
    for q_lens in ([300, 64, 129], [200, 1, 300], [2, 2, 2], [1, 1, 1]):
        kv = [a + b for a, b in zip(kv, q_lens)]
        seqs = m.seqs(q_lens, kv)
        q = m.write(torch.randn((seqs.T, D), generator=m.g, device="cuda").bfloat16(), seqs)
        a = m.expanded(q, seqs, kv)
        n = smla.dense_decode_workspace_size(seqs.T, H, max(kv))
        b = m.absorbed(q, seqs, max(kv), _empty(n, dtype=torch.uint8) if n else None)
        smla.check_device_errors()
        assert _rel(b, a) <= REL
        # the output projections of the two differ as their inputs do, and by their own roundings
        assert _rel(m.finish(b), m.finish(a)) <= REL + 2 * 2.0 ** -4 / math.sqrt(3)


def test_each_projection_of_the_chain_is_its_product():
    """Quantised and multiplied as the chain does, against 64 bits: activations
    rounded to e4m3 (2^-4 / sqrt(3) in the root mean square), outputs to bf16."""
    m = Layer(1, 64)
    x = torch.randn((37, D), generator=m.g, device="cuda").bfloat16()
    w = m.down[0].view(torch.float8_e4m3fn).double()
    full = m.down[1].double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:w.shape[0], :w.shape[1]]
    assert _rel(_project(x, m.down), x.double() @ (w * full).t()) <= 2.0 ** -4 / math.sqrt(3) + 2.0 ** -8
    q = torch.randn((9, H, 192), generator=m.g, device="cuda").bfloat16()
    w = m.k_t[0].view(torch.float8_e4m3fn).double() * m.k_t[1].double().repeat_interleave(128, 1)
    got = _project_heads(q[..., :128], m.k_t, _empty(9, H, 576)[..., :512])
    assert _rel(got, torch.einsum("thk,hnk->thn", q[..., :128].double(), w)) <= 2.0 ** -4 / math.sqrt(3) + 2.0 ** -8


def test_captured_decode_step():
    """The whole step in one graph, replayed over growing lengths, gives the eager step's bits."""
    m, most = Layer(3, 600), 600
    kv = [400, 90, 257]
    first = m.seqs(kv, kv)
    m.write(torch.randn((first.T, D), generator=m.g, device="cuda").bfloat16(), first)
    seqs = m.seqs([1, 1, 1], [k + 1 for k in kv])
    ws = _empty(smla.dense_decode_workspace_size(3, H, most), dtype=torch.uint8)
    x = torch.randn((3, D), generator=m.g, device="cuda").bfloat16()

    def step():
        return m.finish(m.absorbed(m.write(x, seqs), seqs, most, ws))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(torch.randn((3, D), generator=m.g, device="cuda"))
        seqs.kv_len.copy_(torch.tensor([k + 1 + i for k in kv], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())
        smla.check_device_errors()
