"""The gradient norm's and clipping's entry points without a GPU: refusals before any launch."""

import ctypes

import numpy as np
import pytest

from oracle import network as ora
from virtual_noise_perturbed_gb300 import _lib, build

P = ctypes.c_void_p
F = 0x100000          # never dereferenced: every call below returns from the host's checks
WS = F + 0x80000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


class Gradient(ctypes.Structure):
    _fields_ = [("g", P), ("out", P), ("n", ctypes.c_int64)]


def table(*rows):
    return (Gradient * len(rows))(*[Gradient(*r) for r in rows])


def test_workspace(lib):
    w = lib.vn_gradient_norm_workspace
    assert w(-1) == -1 and w((1 << 32) + 1) == -1
    assert w(0) >= 8 and w(1) >= 8 + 8 * 152 and w(5000) > w(1)


def test_norm_and_clip_refusals(lib):
    need = lib.vn_gradient_norm_workspace(2)

    def norm(rows=((F, 0, 8), (F + 0x1000, 0, 8)), dt=0, norm=F + 0x4000, ws=WS, wb=need, count=None):
        return lib.vn_gradient_norm(ctypes.cast(table(*rows), P), len(rows) if count is None else count, dt, P(norm), P(ws), wb, P(0))

    assert norm(dt=2) == 3
    assert norm(count=-1) == 2 and norm(rows=((F, 0, -1),)) == 2
    assert norm(count=(1 << 32) + 1) == 6 and norm(rows=((F, 0, 1 << 60),)) == 6
    assert norm(norm=0) == 1 and norm(rows=((0, 0, 8),)) == 1
    assert norm(norm=F + 0x4002) == 5 and norm(rows=((F + 2, 0, 8),)) == 5 and norm(ws=WS + 8) == 5
    assert norm(ws=0) == 11 and norm(wb=need - 1) == 11
    assert norm(norm=F + 28) == 4                                     # over a gradient
    assert norm(rows=((WS + 64, 0, 8),)) == 4 and norm(norm=WS) == 4  # in the workspace
    assert lib.vn_gradient_norm(P(0), 2, 0, P(F), P(WS), need, P(0)) == 1

    def clip(rows=((F, F, 8), (F + 0x1000, F + 0x2000, 8)), dt=0, bound=1.0, norm=F + 0x4000, wb=need):
        return lib.vn_clip_gradients(ctypes.cast(table(*rows), P), len(rows), dt, bound, P(norm), P(WS), wb, P(0))

    assert clip(bound=-1.0) == 4 and clip(bound=float("nan")) == 4
    assert clip(rows=((F, 0, 8),)) == 1
    assert clip(rows=((F, F + 0x2002, 8),)) == 5
    assert clip(rows=((F, F + 4, 8),)) == 4                                   # out over its own grad, shifted
    assert clip(rows=((F, F, 8), (F, F, 8))) == 4                             # one tensor twice in place
    assert clip(rows=((F, F + 0x1000, 8), (F + 0x1000, F, 8))) == 4           # exchanged
    assert clip(rows=((F, F + 0x2000, 8), (F + 0x100, F + 0x201c, 8))) == 4   # two outs
    assert clip(norm=F + 0x2000) == 4


class Tensor(ctypes.Structure):
    _fields_ = [("p", P), ("g", P), ("m", P), ("v", P), ("ms", P), ("vs", P), ("n", ctypes.c_int64), ("wd", ctypes.c_double)]


def test_clipped_step_refusals(lib):
    need = lib.vn_gradient_norm_workspace(1)

    def call(bits=32, pdt=0, bound=1.0, norm=F + 0x8000, ws=WS, wb=need, step=1, **k):
        t = dict(p=F, g=F + 0x1000, m=F + 0x2000, v=F + 0x3000, ms=F + 0x4000, vs=F + 0x5000, n=8)
        t.update(k)
        arr = (Tensor * 1)(Tensor(t["p"], t["g"], t["m"], t["v"], t["ms"], t["vs"], t["n"], 0.0))
        return lib.vn_adamw_clipped(ctypes.cast(arr, P), 1, pdt, 0, bits, 0.1, 0.9, 0.99, 1e-8, step, 0, bound, P(norm), P(ws), wb, P(0))

    assert call(pdt=4) == 3 and call(bits=16) == 4 and call(step=0) == 4 and call(n=-1) == 2 and call(g=0) == 1
    assert call(bound=-0.5) == 4 and call(bound=float("nan")) == 4
    assert call(norm=0) == 1 and call(norm=F + 0x8001) == 5 and call(ws=0) == 11 and call(wb=8) == 11 and call(ws=WS + 1) == 5
    for at in (F, F + 0x1000, F + 0x2000, F + 0x301c, WS + 8):
        assert call(norm=at) == 4
    assert call(bits=8, norm=F + 0x4000) == 4
    assert call(p=WS) == 4


def test_oracle_norm():
    assert ora.gradient_norm([np.array([3.0]), np.array([[4.0]]), np.zeros(0)]) == 5.0
    assert ora.clip_factor(5.0, 5.0) == 1.0 and ora.clip_factor(5.0, 2.0) == 0.4
    assert ora.clip_factor(np.inf, 1.0) == 0.0 and np.isnan(ora.clip_factor(np.nan, 1.0)) and ora.clip_factor(0.0, 0.0) == 1.0
