"""Sizes beyond 32-bit coordinates: what is refused before any launch (no GPU)."""

import ctypes

import pytest

from virtual_noise_perturbed_gb300 import _lib, build

P = ctypes.c_void_p
F = 1 << 44          # never dereferenced: every call below returns from the host's checks
FAR = 1 << 42


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_features_beyond_32_bits(lib):
    most = 2 ** 31 - 512

    def call(rows, k, n):
        return lib.vn_linear(P(F), P(F + FAR), 1, P(0), 0, P(0), rows, k, n, 0, P(F + 2), P(0), P(F + 5 * FAR), 1 << 60, P(0))
    for k, n in ((most + 1, 1), (1, most + 1), (1 << 33, 1)):
        assert call(9, k, n) == 6                                     # VN_ERR_OVERFLOW
        assert lib.vn_linear_workspace(9, k, n, 1, 1) == -1
        assert lib.vn_linear_backward_workspace(9, k, n, 1, 0, 1) == -1
        assert call(8, k, n) == 4                                     # allowed: refused for y over x
    assert lib.vn_linear_workspace(8, 1 << 33, 1, 1, 1) == 0
    assert call(9, most, 1) == 4 and call(9, 1, most) == 4


def test_sums_over_rows_beyond_32_bits(lib):
    """One kernel would add 2^31 rows one after the other, for minutes and without precision."""
    def call(rows, k, n, gx, gw, gb):
        return lib.vn_linear_backward(P(F), P(F + FAR), P(F + 2 * FAR), P(0), 1, rows, k, n, 0, P(gx), P(gw), P(gb), 1,
                                      P(F + 5 * FAR), 1 << 60, P(0))
    rows = 2 ** 31 - 511
    assert call(rows, 1, 1, F + 3 * FAR, F + 4 * FAR, 0) == 6
    assert call(rows, 1, 1, F + 3 * FAR, 0, F + 4 * FAR) == 6
    assert call(rows, 1, 1, F + 2, 0, 0) == 4                         # grad_x alone is taken: refused for its place
    assert call(rows, 0, 1, 0, 0, F + 4 * FAR) == 6
    assert lib.vn_linear_backward_workspace(rows, 1, 1, 1, 0, 1) > 0
    assert lib.vn_linear_workspace(1 << 33, 64, 64, 0, 1) == lib.vn_linear_workspace(1 << 30, 64, 64, 0, 1)
