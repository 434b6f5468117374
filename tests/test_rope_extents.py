"""Refusals of rotations whose rows and strides do not fit 64 bits together (fake aligned addresses, no GPU)."""
import pytest

import indexed_sparse_attention_gb300 as qsa

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    from indexed_sparse_attention_gb300 import build
    build.build()
    return qsa.lib()


def test_overlap_is_seen_whatever_the_products(L):
    # (n_rows - 1) * row stride passes 2^63 (and wraps below zero, to zero, or to a small number): y's rows lie over
    # its heads all the same.
    r = qsa.Rope(64)
    call = lambda rows, heads, xr, yr, yh: L.qsa_rotate(r.byref, FAKE, rows, heads, 128, 1, FAKE, xr, 128, FAKE * 2, yr, yh, None)
    for rows, yr in ((2 ** 31 - 1, 2 ** 33), (2 ** 30 + 1, 2 ** 34), (2 ** 31 - 1, 2 ** 40), (2 ** 24 + 1, 2 ** 40)):
        assert call(rows, 4, 512, yr, yr) == 1, (rows, yr)
    # Rows of x that no address reaches are refused as well.
    assert call(2 ** 31 - 1, 1, 2 ** 40, 128, 128) == 1 and "64 bits" in L.qsa_last_error().decode()
    assert call(2 ** 31 - 1, 1, 128, 2 ** 40, 128) == 1 and "64 bits" in L.qsa_last_error().decode()
