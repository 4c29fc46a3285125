"""fp32 sums of one sign over a long k: their error as a whole does not grow with k.

The tensor cores' accumulators round every step's sum towards zero, so terms of one sign shrink together.
Limit of the mean relative error, whatever k (u = 2^-23, the spacing of fp32 at 1):
  - products of the operands' bf16 terms that are left out: below 2^-7 2^-15 twice, 4 u (2^-21);
  - the leading products: at most 32 steps in an accumulator, each of which loses less than u of what
    it holds by then, so less than (32 + 1) / 2 u of their sum;
  - the smaller products, below 2^-6 of the sum: at most 512 steps, (512 + 1) / 2 / 64 u.
Together 24.6 u, 2.9e-6. Adding the accumulators up rounds to nearest, with no sign: a mean over many
results sees nothing of it, one result about sqrt(k / 512) u / 2 of it (512 of k an accumulator)."""

import pytest
import torch

import virtual_noise_perturbed_gb300 as vn
from tests.network_routes import plan
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STEP = 2.0 ** -23
LIMIT = (4 + 33 / 2 + 513 / 128) * STEP


def check(got, want, k, what):
    error = (got.double() - want) / want
    assert abs(float(error.mean())) <= LIMIT, (what, float(error.mean()))
    spread = float((error * error).mean().sqrt())
    assert spread <= LIMIT + (1 + (k / 512) ** 0.5) * STEP, (what, spread)


def positive(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEV) + 0.5


def check_forward(rows, k, n):
    g = torch.Generator(device=DEV).manual_seed(k)
    x, w, r = positive(g, rows, k), positive(g, n, k), positive(g, rows, n)
    want = x.double() @ w.double().t()
    check(vn.linear(x, w, check_status=True), want, k, "y")
    check(vn.linear(x, w, residual=r, check_status=True), want + r.double(), k, "y with a residual")


def check_backward(rows, k, n):
    g = torch.Generator(device=DEV).manual_seed(rows)
    d, x, w = positive(g, rows, n), positive(g, rows, k), positive(g, n, k)
    gx, gw, gb = vn.linear_backward(d, x, w, check_status=True)
    check(gw, d.double().t() @ x.double(), rows, "grad_w")
    check(gx, d.double() @ w.double(), n, "grad_x")
    check(gb, d.double().sum(0), rows, "grad_b")


@pytest.mark.parametrize("rows,k,n", [(1031, 4095, 1031), (3000, 8192, 3000), (1100, 16390, 2047), (4096, 16384, 2048)])
def test_pairs_of_ctas(rows, k, n):
    build()
    p = plan(rows, k, n, "fp32", False)
    assert p[0] == 3 and p[4] == 1
    check_forward(rows, k, n)


@pytest.mark.parametrize("rows,k,n", [(128, 16390, 130), (130, 16390, 1000), (147, 44719, 211), (64, 36970, 64), (270, 4957, 704)])
def test_single_ctas(rows, k, n):
    build()
    p = plan(rows, k, n, "fp32", False)
    assert p[0] == 3 and p[4] == 0
    check_forward(rows, k, n)


@pytest.mark.parametrize("rows,k,n", [(16384, 1024, 1024), (65536, 256, 256), (65536, 1024, 1021), (100000, 130, 130)])
def test_gradients_over_many_rows_on_tiles(rows, k, n):
    build()
    assert plan(rows, k, n, "fp32", True)[0] == 3
    check_backward(rows, k, n)


@pytest.mark.parametrize("rows,k,n,columns", [(2048, 16384, 1024, 128), (640, 16390, 130, 128), (130, 16390, 600, 64),
                                              (9, 65536, 520, 16), (1021, 4099, 256, 64)])
def test_gathered(rows, k, n, columns):
    build()
    assert plan(rows, k, n, "fp32", False)[:2] == [2, columns]
    check_forward(rows, k, n)


@pytest.mark.parametrize("rows,k,n,columns", [(262144, 64, 64, 64), (1000003, 16, 8, 64), (20000, 300, 100, 128),
                                              (40000, 200, 128, 64), (1021, 256, 256, 64)])
def test_gradients_over_many_rows_gathered(rows, k, n, columns):
    build()
    assert plan(rows, k, n, "fp32", True)[:2] == [2, columns]
    check_backward(rows, k, n)
