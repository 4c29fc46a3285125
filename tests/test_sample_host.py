"""Drawing an index without a GPU: refusals before any launch, and the oracle against hand-worked rows."""

import ctypes
import math

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


def test_refusals(lib):
    def call(x=F, dt=0, rows=4, n=8, u=F + 0x1000, t=1.0, ts=0, k=0, ks=0, p=1.0, ps=0, m=0.0, ms=0, i=F + 0x2000, lp=F + 0x3000):
        return lib.vn_sample(P(x), dt, rows, n, P(u), t, P(ts), k, P(ks), p, P(ps), m, P(ms), P(i), P(lp), P(0))
    assert call(dt=3) == 3
    assert call(rows=-1) == 2 and call(n=0) == 2 and call(n=524289) == 2
    assert call(rows=1 << 60, n=1 << 10) == 6
    assert call(t=math.nan) == 4 and call(t=math.inf) == 4 and call(p=math.nan) == 4 and call(m=-math.inf) == 4
    assert call(x=0) == 1 and call(u=0) == 1 and call(i=0) == 1
    assert call(x=F + 2) == 5 and call(u=F + 0x1002) == 5 and call(i=F + 0x2004) == 5 and call(lp=F + 0x3001) == 5
    assert call(ts=F + 0x4002) == 5 and call(ks=F + 0x4004) == 5 and call(ps=F + 1) == 5 and call(ms=F + 2) == 5
    assert call(i=F) == 4 and call(i=F + 0x1008) == 4 and call(lp=F + 0x2010) == 4 and call(lp=F + 124) == 4
    assert call(ts=F + 0x2000) == 4 and call(ks=F + 0x2000) == 4 and call(ps=F + 0x3000) == 4 and call(ms=F + 0x3008) == 4
    assert call(rows=0, x=0, u=0, i=0) == 0


def test_oracle_filters_by_hand():
    x = np.log([1.0, 4.0, 2.0, 4.0, 1.0])  # sorted: 4 (1), 4 (3), 2 (2), 1 (0), 1 (4); shares of 12
    kept = lambda **f: np.flatnonzero(ora.keep(x, **f)).tolist()  # noqa: E731
    assert kept() == [0, 1, 2, 3, 4]
    assert kept(top_k=1) == [1] and kept(top_k=2) == [1, 3] and kept(top_k=4) == [0, 1, 2, 3] and kept(top_k=9) == [0, 1, 2, 3, 4]
    assert kept(top_p=0.3) == [1] and kept(top_p=0.34) == [1, 3] and kept(top_p=0.8) == [1, 2, 3] and kept(top_p=0.0) == [1]
    assert kept(top_p=0.9) == [0, 1, 2, 3]
    assert kept(top_k=3, top_p=0.41) == [1, 3]       # of ten, not of twelve
    assert kept(min_p=0.4) == [1, 2, 3] and kept(min_p=1.0) == [1, 3]
    assert kept(temperature=0.0) == [1]
    assert kept(temperature=0.5, min_p=0.2) == [1, 2, 3]   # squares: 16, 4, 1


def test_oracle_draws_by_hand():
    x = np.log([1.0, 4.0, 2.0, 1.0])
    draw = lambda u, **f: ora.sample(x, u, **f)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.124, 0.126, 0.6, 0.63, 0.87, 0.88, 0.999, 1.0)] == [0, 0, 1, 1, 2, 2, 3, 3, 3]
    assert draw(0.0, top_k=2) == 1 and draw(0.67, top_k=2) == 2
    assert math.isclose(ora.sample(x, 0.3)[1], math.log(0.5))
    assert ora.sample(np.array([-math.inf, -math.inf]), 0.5)[0] == -1 and ora.sample(np.array([0.0, math.nan]), 0.5)[0] == -1
    assert ora.sample(np.array([0.0, math.inf, math.inf]), 0.6)[0] == 2
    assert ora.sample(np.array([0.0, -math.inf]), 1.0)[0] == 0
