"""Weights in 4 bits without a GPU: refusals before any launch, sizes, and the oracle against hand-worked groups."""

import ctypes

import numpy as np
import pytest

from oracle import acting as ora
from virtual_noise_perturbed_gb300 import _lib, build

P = ctypes.c_void_p
F = 0x100000          # never dereferenced: every call below returns from the host's checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_row_bytes(lib):
    assert [lib.vn_packed_row_bytes(k) for k in (-1, 0, 1, 128, 129, 4096, (1 << 40) + 1)] == [-1, 0, 64, 64, 128, 2048, -1]


def test_pack_refusals(lib):
    for name, swap in (("vn_pack_weight", False), ("vn_unpack_weight", True)):
        def call(w=F, dt=0, out=4, k=64, group=64, codes=F + 0x10000, scales=F + 0x20000):
            f = getattr(lib, name)
            return f(P(codes), P(scales), dt, out, k, group, P(w), P(0)) if swap else f(P(w), dt, out, k, group, P(codes), P(scales), P(0))
        assert call(dt=4) == 3
        assert call(group=48) == 4 and call(group=0) == 4 and call(group=256) == 4
        assert call(out=-1) == 2 and call(k=-1) == 2
        assert call(out=1 << 40, k=1 << 39) == 6 and call(k=(1 << 40) + 1) == 6
        assert call(w=0) == 1 and call(codes=0) == 1 and call(scales=0) == 1
        assert call(w=F + 2) == 5 and call(codes=F + 0x10008) == 5 and call(scales=F + 0x20001) == 5
        assert call(codes=F + 1008) == 4 and call(w=F + 0x20000) == 4
        assert call(out=0, w=0, codes=0, scales=0) == 0 and call(k=0, w=0, codes=0, scales=0) == 0
    assert lib.vn_pack_weight(P(F), 0, 4, 64, 64, P(F + 0x10000), P(F + 0x10000), P(0)) == 4


def test_linear_refusals(lib):
    def call(x=F, codes=F + 0x10000, scales=F + 0x20000, dt=0, group=64, b=0, bdt=0, r=0, rows=4, k=64, n=8, act=0, y=F + 0x30000,
             ws=0, wb=0):
        return lib.vn_linear_packed(P(x), P(codes), P(scales), dt, group, P(b), bdt, P(r), rows, k, n, act, P(y), P(ws), wb, P(0))
    assert call(dt=5) == 3 and call(b=F, bdt=5) == 3
    assert call(group=31) == 4 and call(act=7) == 4
    assert call(rows=-1) == 2 and call(n=-1) == 2
    assert call(rows=1 << 40, n=1 << 40) == 6
    assert call(x=0) == 1 and call(codes=0) == 1 and call(scales=0) == 1 and call(y=0) == 1
    assert call(x=F + 2) == 5 and call(codes=F + 0x10004) == 5 and call(r=F + 0x40001) == 5 and call(ws=F + 0x50001) == 5
    for at in (F + 32, F + 0x10000, F + 0x20000):
        assert call(y=at) == 4
    assert call(r=F + 0x30000) == 4 and call(b=F + 0x30000) == 4
    assert call(rows=100) == 11 and call(rows=100, ws=F + 0x50000, wb=16) == 11
    assert call(rows=0, x=0, y=0) == 0 and call(n=0, y=0) == 0
    w = lib.vn_linear_packed_workspace
    assert w(32, 512, 256, 1, 1) == 0 and w(10, 512, 256, 0, 1) == 0
    assert w(33, 512, 256, 1, 1) >= 2 * 512 * 256 and w(11, 512, 256, 0, 1) >= 4 * 512 * 256
    assert w(-1, 4, 4, 0, 1) == -1 and w(4, 4, 4, 9, 1) == -1


def test_oracle_by_hand():
    w = np.array([[7.0, -3.4, 3.5, 0.5, 1.5, -0.5, 0.0, 14.0]])
    codes, scales = ora.pack4(w, 4, lambda v: v)
    assert scales.tolist() == [[1.0, 2.0]] and codes.tolist() == [[7, -3, 4, 0, 1, 0, 0, 7]]
    assert ora.values4(codes, scales, 4).tolist() == [[7, -3, 4, 0, 2, 0, 0, 14]]
    codes, scales = ora.pack4(np.zeros((2, 3)), 32, lambda v: v)
    assert not codes.any() and not scales.any() and scales.shape == (2, 1)
