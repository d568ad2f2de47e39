"""Further refusals of the operators around the attention calls, on the host."""
import pytest
import torch

from serving_fp8_indexer_gb300 import _latent, _lib
from serving_fp8_indexer_gb300 import build as smla_build

P = 0x10000  # an aligned fake device pointer: validation runs before any launch


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return _lib.load()


def test_expanded_terms_are_one_or_two_or_unsaid(lib):
    def call(terms, T=0):
        return lib.smla_expanded_prefill_terms(P, 384, 192, P, 512, 256, P, 64, P, 512, 256, P, P, 1, T, 8, 2, 0.1, terms,
                                               None, P, None, P, 1 << 30, None)

    for terms in (0, 1, 2):
        assert call(terms) == 0  # no tokens: nothing is launched
    for terms in (-1, 3):
        for T in (0, 4):
            assert call(terms, T) == 1 and "p_terms" in _lib.last_error(lib)


def test_batches_whose_arrays_are_too_short():
    """The kernels read cu_q[B], kv_len[B - 1] and B rows of the page table (host
    tensors count as device -1 in this helper)."""
    def seqs(cu=4, kv=3, rows=3, pages=5):
        z = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
        return _lib.Seqs(z(cu), z(kv), z(rows, pages), 64, 2)

    assert _latent._seqs(seqs(), -1).B == 3
    assert _latent._seqs(seqs(cu=9, rows=7), -1).B == 3  # longer ones are the head of a larger buffer
    for kw in (dict(cu=3), dict(rows=2), dict(kv=4)):
        with pytest.raises(ValueError, match="seqs"):
            _latent._seqs(seqs(**kw), -1)
    s = seqs()
    s.page_table = torch.zeros((3, 4), dtype=torch.int32)  # narrower than max_pages
    with pytest.raises(ValueError, match="max_pages"):
        _latent._seqs(s, -1)
    s = seqs()
    s.kv_len = s.kv_len[:2]
    with pytest.raises(ValueError, match="seqs"):
        _latent._seqs(s, -1)
    with pytest.raises(TypeError):
        _latent._seqs(_lib.Seqs([0, 1], seqs().kv_len, seqs().page_table, 64, 2), -1)
    # a rotation looks no page up
    assert _latent._seqs(seqs(rows=1, pages=1), -1, False).B == 3
    with pytest.raises(ValueError, match="seqs"):
        _latent._seqs(seqs(cu=3, rows=1), -1, False)
