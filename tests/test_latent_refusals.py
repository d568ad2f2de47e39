"""Further refusals of the operators around the attention calls, on the host."""
import pytest

from serving_fp8_indexer_gb300 import _lib
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
