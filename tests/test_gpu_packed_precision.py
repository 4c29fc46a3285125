"""The layer on weights in 4 bits is as exact with many rows as with few, over the whole range of x, and may be empty.

With A = sum |x| |v| of an output. A product on the tensor cores is exact, and each step of 16 k cut below 2^-23 of what it adds up;
the sums of groups, of splits of k and of warps are fp32. Few rows: as in test_gpu_packed.py. Many rows in bf16: a value is the sum of two
bf16 terms, exactly, so k counts twice: 2 k / 16 + 1 steps, and up to 8 splits joined (8 2^-24 A). Results by half a step, 2^-8."""

import numpy as np
import pytest
import torch

from oracle import acting as ora
from oracle import network
import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16}
FEW = {"fp32": 10, "bf16": 32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def randn(*shape, kind="fp32", seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(KINDS[kind])


def packed(w, group, kind):
    codes, scales = ora.pack4(f64(w), group, lambda v: torch.from_numpy(np.asarray(v)).to(KINDS[kind]).double().numpy())
    return vn.pack4(w.to(DEV), group=group), ora.values4(codes, scales, group)


def check(p, values, x, kind, bias=None, act=None, residual=None):
    y = vn.linear4(x.to(DEV), p, None if bias is None else bias.to(DEV), activation=act,
                   residual=None if residual is None else residual.to(DEV), check_status=True)
    xs = f64(x)
    rows, k = xs.shape
    r = None if residual is None else f64(residual)
    want, z = network.linear(xs, values, None if bias is None else f64(bias), act or "none", r)
    a = np.abs(xs) @ np.abs(values).T + (0 if bias is None else np.abs(f64(bias)))
    if rows <= FEW[kind]:
        steps = 2.0 ** -20 + (k / p.group / 8 + 16) * 2.0 ** -24
    elif kind == "bf16":
        steps = (2 * (k + 15) // 16 + 1) * 2.0 ** -23 + 8 * 2.0 ** -24
    else:
        steps = 2.0 ** -18  # linear's own
    tol = steps * a * 1.2 + (2.0 ** -20 * (1 + np.abs(z)) if act else 0)        # no slope is above 1.2
    tol = tol + (2.0 ** -8 if kind == "bf16" else 2.0 ** -23) * (np.abs(want) + (0 if r is None else np.abs(r)))
    err = np.abs(f64(y) - want)
    assert np.all(err <= tol + 1e-30), (err.max(), (err / (tol + 1e-30)).max())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [32, 33, 40, 64, 129, 300])
@pytest.mark.parametrize("out,k", [(1, 1), (7, 31), (100, 333), (256, 256), (129, 1003), (64, 2048)])
def test_values_are_not_rounded_with_many_rows(out, k, rows, group):
    w = randn(out, k, kind="bf16", seed=1, scale=k ** -0.5)
    p, v = packed(w, group, "bf16")
    x = randn(rows, k, kind="bf16", seed=2)
    check(p, v, x, "bf16")
    check(p, v, x, "bf16", randn(out, seed=3), "gelu", randn(rows, out, kind="bf16", seed=4))


def test_a_large_layer_with_many_rows():
    w = randn(4096, 4096, kind="bf16", seed=5, scale=1 / 64)
    p, v = packed(w, 64, "bf16")
    for rows in (33, 500):
        check(p, v, randn(rows, 4096, kind="bf16", seed=6), "bf16", randn(4096, kind="bf16", seed=7), "silu")


def test_one_hot_rows_read_the_values_with_many_rows():
    w = randn(50, 300, kind="bf16", seed=8)
    p, v = packed(w, 64, "bf16")
    eye = torch.eye(300, dtype=torch.bfloat16, device=DEV)
    for n in (33, 300):
        assert torch.equal(vn.linear4(eye[:n], p), p.dequantize()[:, :n].t())


def test_views_at_odd_offsets_with_many_rows():
    """x and y that start anywhere; what lies around y stays as it is."""
    w = randn(37, 91, kind="bf16", seed=9)
    p, v = packed(w, 32, "bf16")
    x = randn(70, 91, kind="bf16", seed=10)
    want = vn.linear4(x.to(DEV), p)
    for shift in (1, 2, 3, 5):
        flat = torch.full((70 * 91 + 16,), float("nan"), dtype=torch.bfloat16, device=DEV)
        there = flat[shift:shift + 70 * 91].view(70, 91)
        there.copy_(x)
        buf = torch.full((70 * 37 + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
        out = buf[shift:shift + 70 * 37].view(70, 37)
        assert vn.linear4(there, p, out=out) is out and torch.equal(out, want)
        assert bool((buf[:shift] == 7).all()) and bool((buf[shift + 70 * 37:] == 7).all())


@pytest.mark.parametrize("rows", [4, 40])
def test_infinities_in_x_are_the_products_in_bf16(rows):
    """An infinity times a value is an infinity or, where the value is 0, a NaN; other rows are as without it."""
    w = randn(20, 300, kind="bf16", seed=11)
    w[7, 100] = 0.0
    w[9] = 0.0
    p, v = packed(w, 64, "bf16")
    x = randn(rows, 300, kind="bf16", seed=12)
    clean = vn.linear4(x.to(DEV), p)
    x[1, 100] = float("inf")
    x[2, 299] = -float("inf")
    x[3, 5] = float("nan")
    got = vn.linear4(x.to(DEV), p).cpu()
    for r, at in ((1, 100), (2, 299)):
        with np.errstate(invalid="ignore"):
            want = f64(x)[r, at] * v[:, at]
        assert np.array_equal(f64(got)[r], want, equal_nan=True), r
    assert bool(torch.isnan(got[3]).all())
    assert torch.equal(got[0], clean[0].cpu()) and torch.equal(got[4:], clean[4:].cpu())


def test_infinite_and_nan_groups_with_many_rows():
    w = randn(20, 300, kind="bf16", seed=13)
    w[3, 40], w[5, 299] = float("inf"), float("nan")
    p = vn.pack4(w.to(DEV))
    y = vn.linear4(randn(50, 300, kind="bf16", seed=14).to(DEV), p)
    bad = torch.zeros(20, dtype=torch.bool)
    bad[[3, 5]] = True
    assert torch.equal(torch.isnan(y).cpu(), bad.expand(50, 20))


def test_rows_too_long_for_twice_their_length():
    """Rows of 2^30, twice whose length no coordinate of the plain layer holds: taken a few at a time from the packed weights."""
    k, rows = 2 ** 30, 33
    if torch.cuda.mem_get_info(DEV)[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GB")
    g = torch.Generator().manual_seed(16)
    at = torch.cat([torch.tensor([0, 1, 2 ** 29 - 1, 2 ** 29, k - 2, k - 1]), torch.randint(0, k, (200,), generator=g)]).unique()
    w = torch.zeros(3, k, dtype=torch.bfloat16, device=DEV)
    w[:, at] = randn(3, len(at), kind="bf16", seed=17).to(DEV)
    p = vn.pack4(w, group=128)
    p.dequantize(out=w)
    few = w[:, at].clone()
    # Unrounded: the scale times the code next to the rounded value over it.
    scale = p.scales[:, at // 128].double()
    values = torch.where(scale > 0, torch.round(few.double() / scale.clamp(min=1e-30)), 0.0) * scale
    del w
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device=DEV)
    xs = randn(rows, len(at), kind="bf16", seed=18).to(DEV)
    x[:, at] = xs
    y = vn.linear4(x, p, check_status=True).double()
    want = xs.double() @ values.t()
    a = xs.double().abs() @ values.abs().t()
    # Some 200 groups are not zero: as many sums in fp32.
    assert bool(((y - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * a).all())


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 10, 11, 32, 33, 100])
def test_an_empty_layer_for_any_number_of_rows(rows, kind):
    empty = vn.pack4(torch.empty(4, 0, dtype=KINDS[kind], device=DEV))
    b = torch.arange(4.0, device=DEV)
    r = torch.ones(rows, 4, dtype=KINDS[kind], device=DEV)
    x = torch.empty(rows, 0, dtype=KINDS[kind], device=DEV)
    assert torch.equal(vn.linear4(x, empty, b).float(), b.expand(rows, 4))
    assert torch.equal(vn.linear4(x, empty, b, activation="relu", residual=r).float(), b.expand(rows, 4) + 1)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 5, 20, 40])
def test_the_whole_range_of_x(rows, kind):
    """Results that fp32 holds are finite, whatever the size of x: a group's sum of x times codes, up to 7 * 128 |x|, would not be."""
    k = 256
    for size, scale in ((3e38, 1e-4), (1e36, 1e-3), (4e36, 0.05), (1e-3, 1e37), (1e-25, 1.0), (1e-25, 1e20)):
        g = torch.Generator().manual_seed(15)
        w = (torch.rand(12, k, generator=g) * scale).to(KINDS[kind])
        w[1] *= -1
        w[2, ::2] *= -1
        p, v = packed(w, 128, kind)
        x = ((torch.rand(rows, k, generator=g) * 0.5 + 0.5) * size).to(KINDS[kind])
        if size > 1e38:
            x[:, 3:] *= 0.005
        check(p, v, x, kind)


@pytest.mark.parametrize("rows", [16384, 16385, 50001])
def test_more_rows_than_are_laid_out_at_once(rows):
    w = randn(24, 70, kind="bf16", seed=19, scale=0.1)
    p, v = packed(w, 32, "bf16")
    x = randn(rows, 70, kind="bf16", seed=20)
    check(p, v, x, "bf16", randn(24, seed=21), "tanh", randn(rows, 24, kind="bf16", seed=22))
