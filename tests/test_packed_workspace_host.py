"""The workspace of the layer on weights in 4 bits, without a GPU."""

import pytest

from virtual_noise_perturbed_gb300 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_many_rows_in_bf16(lib):
    w = lib.vn_linear_packed_workspace
    assert w(33, 512, 256, 1, 1) == 4 * 512 * 256 + -(-4 * 512 * 33 // 256) * 256     # two terms of a weight, two copies of x
    assert w(33, 511, 256, 1, 0) == w(33, 512, 256, 1, 1)                             # rows are padded to 16 bytes
    assert w(16384, 512, 256, 1, 1) == w(10 ** 9, 512, 256, 1, 1)                     # x is laid out some rows at a time
    assert w(33, 2 ** 30 - 256, 3, 1, 1) > 0 and w(33, 2 ** 30 - 255, 3, 1, 1) == 0   # longer rows need none
    assert w(33, 2 ** 26, 2 ** 31 - 512, 1, 1) > 2 ** 58                              # the largest weights that sizes allow
