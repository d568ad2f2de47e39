"""Refusals of the 8-bit projections and of the 4-bit cache's operators, on the
host: the library and the binding reject what the documentation does not allow
before anything reaches a device."""
import math

import pytest
import torch

from serving_fp8_indexer_gb300 import _latent, _lib
from serving_fp8_indexer_gb300 import build as smla_build

INVALID, UNSUPPORTED = 1, 2
P = 0x10000  # an aligned fake device pointer: validation runs before any launch


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return _lib.load()


def _seqs(T=4, B=1, page_size=64):
    return _lib.SeqsT(P, P, P, B, 1, page_size, T)


def _rope(inv=P, offset=0, dim=16, layout=0, amplitude=1.0):
    return _lib.RopeT(inv, offset, dim, layout, amplitude)


def test_quantize_refusals(lib):
    def call(x=P, xs=128, M=4, K=128, w=None, eps=1e-6, out=P, sc=P):
        return lib.smla_quantize_blocks(x, xs, M, K, w, eps, out, sc, None)

    for kw, st in ((dict(M=-1), INVALID), (dict(K=0), UNSUPPORTED), (dict(K=8), UNSUPPORTED), (dict(K=24), UNSUPPORTED),
                   (dict(K=(1 << 20) + 16), UNSUPPORTED), (dict(K=16400, w=P), UNSUPPORTED), (dict(w=P, eps=-1.0), INVALID),
                   (dict(w=P, eps=math.nan), INVALID), (dict(w=P + 8), INVALID), (dict(xs=-8), INVALID),
                   (dict(xs=130), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(sc=None), INVALID),
                   (dict(x=P + 8), INVALID), (dict(out=P + 8), INVALID), (dict(sc=P + 2), INVALID),
                   (dict(M=1 << 30, K=1 << 20), UNSUPPORTED)):
        assert call(**kw) == st, kw
    assert call(M=0, x=None, out=None, sc=None) == 0


def test_matmul_refusals(lib):
    def call(a=P, ag=512, am=128, s=P, sg=4, sm=1, b=P, bs=P, G=2, M=4, N=64, K=128, out=P, od=0, og=256, om=64):
        return lib.smla_block_matmul(a, ag, am, s, sg, sm, b, bs, G, M, N, K, out, od, og, om, None)

    for kw, st in ((dict(G=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-8), INVALID), (dict(K=0), UNSUPPORTED),
                   (dict(K=40), UNSUPPORTED), (dict(K=1 << 21), UNSUPPORTED), (dict(N=60), UNSUPPORTED),
                   (dict(od=1), INVALID), (dict(am=112), INVALID), (dict(ag=112), INVALID), (dict(am=136), INVALID),
                   (dict(ag=1 << 38), INVALID), (dict(am=0), INVALID), (dict(sg=-1), INVALID), (dict(sm=-1), INVALID),
                   (dict(om=56), INVALID), (dict(om=68), INVALID), (dict(og=0), INVALID), (dict(og=64, om=64), INVALID),
                   (dict(og=248, om=64), INVALID), (dict(og=64, om=120), INVALID), (dict(a=None), INVALID),
                   (dict(s=None), INVALID), (dict(b=None), INVALID), (dict(bs=None), INVALID), (dict(out=None), INVALID),
                   (dict(a=P + 8), INVALID), (dict(b=P + 8), INVALID), (dict(out=P + 8), INVALID), (dict(s=P + 2), INVALID),
                   (dict(bs=P + 1), INVALID), (dict(M=1 << 30, N=256, ag=1 << 37, og=256, om=512), UNSUPPORTED),
                   (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(N=(1 << 28) + 8), UNSUPPORTED), (dict(N=1 << 28, K=1 << 10, am=1024, ag=4096, om=1 << 28, og=1 << 30), UNSUPPORTED)):
        assert call(**kw) == st, (kw, _lib.last_error(lib))
    for kw in (dict(G=0), dict(M=0), dict(N=0)):
        assert call(a=None, s=None, b=None, bs=None, out=None, **kw) == 0, kw


BAD_ROPES = [(dict(layout=2), INVALID), (dict(offset=568), INVALID), (dict(dim=24), UNSUPPORTED), (dict(offset=4), UNSUPPORTED),
             (dict(inv=None), INVALID), (dict(amplitude=math.nan), INVALID)]


def test_fp4_append_and_gather_refusals(lib):
    def append(x=P, xs=576, s=None, w=None, nd=0, eps=1e-6, r=None, pool=P, rows=64, ro=None, rs=576):
        return lib.smla_cache_append_fp4(x, xs, s or _seqs(), w, nd, eps, r or _rope(), pool, rows, ro, rs, None)

    def gather(pool=P, rows=64, s=None, out=P, od=0, rs=576, sc=None):
        return lib.smla_cache_gather_fp4(pool, rows, s or _seqs(), out, od, rs, sc, None)

    for kw, st in ((dict(pool=None), INVALID), (dict(pool=P + 8), INVALID), (dict(rows=0), INVALID), (dict(rows=1 << 31), INVALID),
                   (dict(s=_seqs(page_size=4)), UNSUPPORTED), (dict(s=_seqs(B=0)), INVALID)):
        assert append(**kw) == st and gather(**kw) == st, kw
    for kw, st in ((dict(x=None), INVALID), (dict(x=P + 2), INVALID), (dict(xs=568), INVALID), (dict(xs=580), INVALID),
                   (dict(ro=P + 16, rs=575), INVALID), (dict(ro=P + 8), INVALID), (dict(ro=P), INVALID), (dict(w=P, nd=12), UNSUPPORTED),
                   (dict(w=P, nd=584), UNSUPPORTED), (dict(w=P, nd=0), UNSUPPORTED), (dict(w=P, nd=64, eps=-1.0), INVALID),
                   (dict(w=P + 8, nd=64), INVALID)):
        assert append(**kw) == st, kw
    for kw, st in BAD_ROPES:
        assert append(r=_rope(**kw)) == st, kw
    for kw, st in ((dict(od=2), INVALID), (dict(out=None), INVALID), (dict(out=P + 8), INVALID), (dict(rs=568), INVALID),
                   (dict(rs=580), INVALID), (dict(od=1, sc=P, rs=584), INVALID), (dict(od=1), INVALID), (dict(sc=P), INVALID),
                   (dict(od=1, sc=P + 2), INVALID)):
        assert gather(**kw) == st, kw
    assert append(s=_seqs(T=0), x=None, pool=None, rows=0) == 0
    assert gather(s=_seqs(T=0), pool=None, out=None, rows=0) == 0


def test_fp4_decode_refusals(lib):
    def call(q=P, qd=0, pool=P, rows=64, s=None, most=64, H=64, vd=512, scale=0.04, sink=None, out=P, ws=P, wsb=1 << 30):
        return lib.smla_dense_decode_fp4(q, qd, pool, rows, s or _seqs(), most, H, vd, scale, sink, out, ws, wsb, None)

    for kw, st in ((dict(qd=2), INVALID), (dict(most=0), INVALID), (dict(H=24), UNSUPPORTED), (dict(vd=256), UNSUPPORTED),
                   (dict(scale=math.nan), INVALID), (dict(q=None), INVALID), (dict(pool=None), INVALID), (dict(out=None), INVALID),
                   (dict(q=P + 8), INVALID), (dict(pool=P + 8), INVALID), (dict(sink=P + 2), INVALID), (dict(rows=0), INVALID),
                   (dict(s=_seqs(B=0)), INVALID)):
        assert call(**kw) == st, kw
    need = lib.smla_dense_decode_workspace_size(4, 64, 8192)
    assert call(most=8192, wsb=need - 1) == INVALID and "workspace" in _lib.last_error(lib)
    assert call(most=8192, ws=P + 8) == INVALID
    assert call(s=_seqs(T=0), q=None, pool=None, rows=0, out=None) == 0


def test_binding_refusals(monkeypatch):
    """Shapes that do not fit each other (host tensors count as device -1)."""
    monkeypatch.setattr(_latent, "_device", lambda: -1)
    smla_build.build()
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    f = lambda *n: torch.zeros(n)  # noqa: E731
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16)  # noqa: E731
    ok = dict(a=u8(2, 4, 128), a_scales=f(2, 4, 1), b=u8(2, 64, 128), b_scales=f(2, 1, 1), out=bf(2, 4, 64))
    for kw in (dict(a_scales=f(2, 4, 2)), dict(b=u8(2, 64, 112)), dict(b=u8(3, 64, 128)), dict(b_scales=f(2, 2, 1)),
               dict(out=bf(2, 4, 72)), dict(out=bf(2, 5, 64)), dict(out=bf(1, 4, 64)),
               dict(out=bf(2, 64, 4).transpose(1, 2)), dict(a=u8(2, 128, 4).transpose(1, 2))):
        with pytest.raises(ValueError):
            _latent.block_matmul(**{**ok, **kw}, stream=0)
    for kw in (dict(a=bf(2, 4, 128)), dict(out=u8(2, 4, 64)), dict(a_scales=bf(2, 4, 1)), dict(b=f(2, 64, 128))):
        with pytest.raises(TypeError):
            _latent.block_matmul(**{**ok, **kw}, stream=0)
    for a, rest in ((u8(4, 128), (f(4, 1), u8(1, 64, 128), f(1, 1, 1), bf(4, 64))),
                    (u8(4, 128), (f(1, 4, 1), u8(64, 128), f(1, 1), bf(4, 64))),
                    (u8(1, 1, 4, 128), (f(4, 1), u8(64, 128), f(1, 1), bf(4, 64))),
                    (u8(128), (f(4, 1), u8(64, 128), f(1, 1), bf(4, 64)))):
        with pytest.raises(ValueError):
            _latent.block_matmul(a, *rest, stream=0)
    for out, sc, w in ((u8(4, 64), f(4, 1), None), (u8(4, 128), f(4, 2), None), (u8(4, 128), f(4, 1), bf(64))):
        with pytest.raises(ValueError):
            _latent.quantize_blocks(bf(4, 128), out, sc, w, stream=0)
    z = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    seqs = _lib.Seqs(z(2), z(1), z(1, 1), 64, 4)
    with pytest.raises(ValueError, match="320"):
        _latent.cache_append_fp4(bf(4, 576), seqs, u8(64, 288), stream=0)
    with pytest.raises(ValueError):
        _latent.cache_append_fp4(bf(4, 512), seqs, u8(64, 320), stream=0)
    with pytest.raises(ValueError):
        _latent.cache_append_fp4(bf(4, 576), seqs, u8(64, 320), rows_out=bf(3, 576), stream=0)
    with pytest.raises(ValueError):
        _latent.cache_gather_fp4(u8(64, 320), seqs, u8(4, 576), f(4, 2), stream=0)
    with pytest.raises(TypeError):
        _latent.cache_gather_fp4(u8(64, 320), seqs, u8(4, 576), stream=0)  # e4m3 rows need their scales
    with pytest.raises(TypeError):
        _latent.cache_gather_fp4(u8(64, 320), seqs, bf(4, 576), f(4, 1), stream=0)
    with pytest.raises(ValueError):
        _latent.dense_decode_fp4(bf(3, 16, 576), u8(64, 320), seqs, 64, 0.1, bf(3, 16, 512), None, stream=0)
