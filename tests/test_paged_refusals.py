"""Refusals of the paged calls, without a GPU (device pointers are fake aligned
addresses)."""
import pytest

import indexed_sparse_attention_gb300 as qsa
from indexed_sparse_attention_gb300 import build as qsa_build
from indexed_sparse_attention_gb300 import paged

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    qsa_build.build()
    return qsa.lib()


def test_extend_step_checks(L):
    pool = paged.PagePoolDesc(FAKE, 8, FAKE, FAKE, 4, 10, 16)
    call = lambda p=pool, seqs=FAKE, new=FAKE, n=1, to=FAKE: L.qsa_pages_extend_step(p, seqs, new, n, to, None)
    assert call(to=None) == 1 and call(to=None, n=0) == 1
    assert call(seqs=None) == 1 and call(new=None) == 1 and call(n=-1) == 1 and call(n=1025) == 2
    assert call(p=None) == 1 and call(p=paged.PagePoolDesc(FAKE, 8, FAKE, FAKE, 4, 10, 20)) == 2
    assert "qsa_pages_extend_step" in L.qsa_last_error().decode()
