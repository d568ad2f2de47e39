"""Refusals of the operators around the attention calls, on the host: the
library and the binding reject what the documentation does not allow before
anything reaches a device."""
import ctypes
import math

import pytest
import torch

from serving_fp8_indexer_gb300 import _lib, _latent
from serving_fp8_indexer_gb300 import build as smla_build

INVALID, UNSUPPORTED = 1, 2
P = 0x10000  # an aligned fake device pointer: validation runs before any launch


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return _lib.load()


def _seqs(T=4, B=1, page_size=64):
    return _lib.SeqsT(P, P, P, B, 1, page_size, T)


def _msg(lib):
    return _lib.last_error(lib)


def _rope(inv=P, offset=0, dim=16, layout=0, amplitude=1.0):
    return _lib.RopeT(inv, offset, dim, layout, amplitude)


BAD_ROPES = [(dict(layout=2), INVALID), (dict(offset=-8), INVALID), (dict(dim=-16), INVALID), (dict(offset=56), INVALID),
             (dict(offset=2147483640), INVALID), (dict(dim=24), UNSUPPORTED), (dict(offset=4), UNSUPPORTED),
             (dict(inv=None), INVALID), (dict(inv=P + 4), INVALID), (dict(amplitude=math.nan), INVALID)]


def test_frequencies_refusals(lib):
    out, amp = (ctypes.c_double * 32)(), ctypes.c_float()

    def call(dim=64, base=1e4, scaling=0, factor=2.0, length=4096, fast=32.0, slow=1.0, o=out, a=ctypes.byref(amp)):
        return lib.smla_rope_frequencies(dim, base, scaling, factor, length, fast, slow, o, a)

    assert call() == 0 and out[0] == 1.0 and amp.value == 1.0
    for kw in (dict(dim=63), dict(dim=0), dict(dim=2000), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
               dict(scaling=3), dict(o=None), dict(a=None), dict(scaling=1, factor=0.5), dict(scaling=2, factor=math.nan),
               dict(scaling=2, length=0), dict(scaling=2, fast=1.0, slow=2.0), dict(scaling=2, slow=0.0)):
        assert call(**kw) == INVALID, kw
    with pytest.raises(ValueError):
        _latent.rope_frequencies(64, scaling="other")


def test_rope_refusals(lib):
    def call(x=P, xd=0, xts=128, xhs=64, s=None, H=2, D=64, r=None, out=P + 0x10000, od=0, ots=128, ohs=64):
        return lib.smla_rope(x, xd, xts, xhs, s or _seqs(), H, D, r or _rope(), out, od, ots, ohs, None)

    for kw, st in ((dict(xd=1), INVALID), (dict(od=3), INVALID), (dict(D=12), UNSUPPORTED), (dict(D=8), UNSUPPORTED),
                   (dict(D=2048), UNSUPPORTED), (dict(H=0), UNSUPPORTED), (dict(H=65536), UNSUPPORTED),
                   (dict(xts=130), INVALID), (dict(ohs=4), INVALID), (dict(ots=0), INVALID), (dict(ohs=0), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
                   (dict(x=P + 8), INVALID), (dict(out=P + 8), INVALID), (dict(out=P + 4, od=1), INVALID),
                   (dict(out=P, od=2), INVALID), (dict(out=P, ots=64), INVALID), (dict(s=_seqs(page_size=48)), UNSUPPORTED),
                   (dict(s=_seqs(B=0)), INVALID)):
        assert call(**kw) == st, kw
    for kw, st in BAD_ROPES:
        assert call(r=_rope(**kw)) == st and "rope" in _msg(lib), kw
    assert call(s=_seqs(T=0), x=None, out=None) == 0


def test_append_and_gather_refusals(lib):
    def append(x=P, xs=64, s=None, D=64, w=None, nd=0, eps=1e-6, r=None, pool=P, pd=1, rows=64, sc=None, sbs=0, ro=None,
               rs=64):
        return lib.smla_cache_append(x, xs, s or _seqs(), D, w, nd, eps, r or _rope(), pool, pd, rows, sc, sbs, ro, rs,
                                     None)

    def gather(pool=P, pd=1, rows=64, sc=None, sbs=0, s=None, D=64, out=P, rs=64):
        return lib.smla_cache_gather(pool, pd, rows, sc, sbs, s or _seqs(), D, out, rs, None)

    both = ((dict(pd=2), INVALID), (dict(D=1032), UNSUPPORTED), (dict(D=20), UNSUPPORTED), (dict(sbs=16), UNSUPPORTED),
            (dict(sbs=-1), UNSUPPORTED), (dict(sbs=32), INVALID), (dict(sbs=64, pd=0, sc=P), INVALID),
            (dict(sbs=32, D=40, sc=P), UNSUPPORTED), (dict(pool=None), INVALID), (dict(pool=P + 8), INVALID),
            (dict(sbs=64, sc=P + 2), INVALID), (dict(rows=0), INVALID), (dict(rows=1 << 31), INVALID),
            (dict(s=_seqs(page_size=4)), UNSUPPORTED))
    for kw, st in both:
        assert append(**kw) == st and gather(**kw) == st, kw
    for kw, st in ((dict(x=None), INVALID), (dict(x=P + 2), INVALID), (dict(xs=56), INVALID), (dict(xs=68), INVALID),
                   (dict(ro=P + 16, rs=63), INVALID), (dict(ro=P + 8), INVALID), (dict(ro=P), INVALID), (dict(w=P, nd=12), UNSUPPORTED),
                   (dict(w=P, nd=72), UNSUPPORTED), (dict(w=P, nd=0), UNSUPPORTED), (dict(w=P, nd=64, eps=-1.0), INVALID),
                   (dict(w=P, nd=64, eps=math.nan), INVALID), (dict(w=P + 8, nd=64), INVALID)):
        assert append(**kw) == st, kw
    for kw, st in BAD_ROPES:
        assert append(r=_rope(**kw)) == st, kw
    for kw, st in ((dict(out=None), INVALID), (dict(out=P + 8), INVALID), (dict(rs=56), INVALID), (dict(rs=65), INVALID)):
        assert gather(**kw) == st, kw
    assert append(s=_seqs(T=0), x=None, pool=None, rows=0) == 0
    assert gather(s=_seqs(T=0), pool=None, out=None, rows=0) == 0


def test_binding_refuses_host_tensors_and_wrong_layouts():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    bf = (torch.bfloat16,)
    with pytest.raises(TypeError):
        _latent._rows(x.half(), "x", bf, -1, 3)
    with pytest.raises(TypeError):
        _latent._rows([1.0], "x", bf, -1, 3)
    with pytest.raises(ValueError, match="device"):
        _latent._rows(x, "x", bf, 0, 3)  # on the host
    with pytest.raises(ValueError):
        _latent._rows(x, "x", bf, -1, 2)
    with pytest.raises(ValueError, match="dense"):
        _latent._rows(x.transpose(1, 2), "x", bf, -1, 3)
    with pytest.raises(ValueError, match="device"):
        _latent._flat(x, "x", torch.bfloat16, 0, 3)
    with pytest.raises(TypeError):
        _latent._flat(x, "x", torch.float32, -1, 3)
    # a dimension of one element has no stride of its own (host tensors count
    # as device -1 in these helpers)
    assert _latent._rows(x[:1, :1], "x", bf, -1, 3)[2] == (64, 64, 1)
    assert _latent._rows(x[..., :8], "x", bf, -1, 3)[2] == (128, 64, 1)
    with pytest.raises(ValueError):
        _latent._scales(torch.ones((64, 1)), 64, 64, 0, -1)
    with pytest.raises(ValueError):
        _latent._scales(torch.ones((64, 1)), 64, 64, 32, -1)
    with pytest.raises(ValueError):
        _latent._scales(None, 64, 64, 64, -1)
    assert _latent._scales(torch.ones((64, 2)), 64, 64, 32, -1) is not None
    assert _latent._scales(None, 64, 64, 0, -1) is None


def test_expanded_refusals(lib):
    def call(q=P, qt=384, qh=192, k=P, kt=512, kh=256, r=P, rt=64, v=P, vt=512, vh=256, cq=P, ck=P, B=1, T=4, S=8, H=2,
             sc=0.1, sink=None, out=P, lse=None, ws=P, wsb=1 << 30):
        return lib.smla_expanded_prefill(q, qt, qh, k, kt, kh, r, rt, v, vt, vh, cq, ck, B, T, S, H, sc, sink, out, lse,
                                         ws, wsb, None)

    for kw, st in ((dict(T=-1), INVALID), (dict(S=-1), INVALID), (dict(B=-1), INVALID), (dict(B=0), INVALID),
                   (dict(H=0), UNSUPPORTED), (dict(H=65536), UNSUPPORTED), (dict(sc=0.0), INVALID),
                   (dict(sc=-0.1), INVALID), (dict(sc=math.nan), INVALID), (dict(sc=math.inf), INVALID),
                   (dict(qh=191), INVALID), (dict(qt=184), INVALID), (dict(kh=120), INVALID), (dict(kt=516), INVALID),
                   (dict(rt=0), INVALID), (dict(vt=0), INVALID), (dict(vh=0), INVALID), (dict(vh=1 << 38), INVALID),
                   (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(r=None), INVALID), (dict(v=None), INVALID),
                   (dict(cq=None), INVALID), (dict(ck=None), INVALID), (dict(out=None), INVALID),
                   (dict(q=P + 8), INVALID), (dict(v=P + 8), INVALID), (dict(out=P + 8), INVALID),
                   (dict(sink=P + 2), INVALID), (dict(lse=P + 1), INVALID), (dict(cq=P + 2), INVALID),
                   (dict(T=1 << 25, H=64), UNSUPPORTED)):
        assert call(**kw) == st, kw
    need = lib.smla_expanded_prefill_workspace_size(1, 8192, 1, 1)
    assert need > 0
    assert call(T=1, S=8192, H=1, wsb=need - 1) == INVALID and "workspace" in _msg(lib)
    assert call(T=1, S=8192, H=1, ws=None, wsb=0) == INVALID
    assert call(T=1, S=8192, H=1, ws=P + 8) == INVALID and "aligned" in _msg(lib)
    assert call(T=0, B=0, q=None, k=None, r=None, v=None, cq=None, ck=None, out=None) == 0
    assert lib.smla_expanded_prefill_workspace_size(0, 1, 1, 1) == 0


def test_dense_decode_refusals(lib):
    def call(q=P, qd=0, pool=P, pd=1, rows=64, sc=None, sbs=0, s=None, most=64, H=64, vd=512, scale=0.04, sink=None,
             out=P, ws=P, wsb=1 << 30):
        return lib.smla_dense_decode(q, qd, pool, pd, rows, sc, sbs, s or _seqs(), most, H, vd, scale, sink, out, ws, wsb,
                                     None)

    for kw, st in ((dict(qd=2), INVALID), (dict(pd=2), INVALID), (dict(pd=0, qd=1), UNSUPPORTED),
                   (dict(pd=0, sbs=576, sc=P), UNSUPPORTED), (dict(sbs=32, sc=P), UNSUPPORTED), (dict(most=0), INVALID),
                   (dict(H=24), UNSUPPORTED), (dict(vd=256), UNSUPPORTED), (dict(sbs=576), INVALID),
                   (dict(scale=math.nan), INVALID), (dict(q=None), INVALID), (dict(pool=None), INVALID),
                   (dict(out=None), INVALID), (dict(q=P + 8), INVALID), (dict(pool=P + 8), INVALID),
                   (dict(sink=P + 2), INVALID), (dict(rows=0), INVALID), (dict(s=_seqs(B=0)), INVALID)):
        assert call(**kw) == st, kw
    need = lib.smla_dense_decode_workspace_size(4, 64, 8192)
    assert need > 0 and lib.smla_dense_decode_workspace_size(0, 64, 8192) == 0
    assert call(most=8192, wsb=need - 1) == INVALID and "workspace" in _msg(lib)
    assert call(most=8192, ws=None, wsb=0) == INVALID
    assert call(most=8192, ws=P + 8) == INVALID and "aligned" in _msg(lib)
    assert call(s=_seqs(T=0), q=None, pool=None, rows=0, out=None) == 0
