"""The centre network's linear layer and layer norm on the GPU, forward and backward, against the
float64 oracle element by element.

Tolerances. u = 2^-24 is fp32's unit roundoff. A sum of k products held in fp32 is off by at most
about k u S, S the sum of the products' magnitudes (the order is free); twice that is allowed, plus
16 u S for the splitting of fp32 operands into bf16 terms. An activation of slope <= 1.13 passes the
error on and adds a few u (tanhf, normcdff, expf and a quotient: 16 u (1 + |z|) allowed); results in
bf16 add their rounding, 2^-8 (8 significant bits), and may take activations good to 2^-14. d = g act'(z) is rounded once to
bf16 (2^-8 of each |d|) before the bf16 products. Layer norm adds a handful of roundings to the
error of its two sums."""

import numpy as np
import pytest
import torch

from oracle import network as ora
import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
ACTS = ["none", "tanh", "relu", "gelu", "silu"]
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def normal(gen, shape, kind, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=gen) * scale + shift).to(KINDS[kind]).to(DEV)


def within(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), f"{what}: NaN/Inf pattern differs"
    worst = np.max((np.abs(got - want) - bound)) if got.size else -1.0
    assert worst <= 0, f"{what}: {worst:.3e} beyond the bound, largest error {np.max(np.abs(got - want)):.3e}"


def rounding(kind, y):
    return (2.0 ** -8 if kind == "bf16" else U) * np.abs(y) * 1.01 + 1e-37


def act_slack(kind, z):
    return (2.0 ** -14 if kind == "bf16" else 16 * U) * (1 + np.abs(z))


# rows, in, out: single elements, odd sizes, below and across the tiles of every kernel, long sums
SHAPES = [(1, 1, 1), (1, 256, 256), (1, 4096, 72), (3, 64, 7), (5, 17, 33), (8, 1024, 40), (9, 8, 16), (16, 512, 130),
          (17, 72, 264), (33, 100, 256), (64, 64, 64), (129, 136, 257), (255, 24, 128), (256, 1000, 96), (1021, 256, 256),
          (300, 520, 1032), (2, 2048, 1000), (31, 4104, 128), (700, 65, 700)]


def check_linear(rows, k, n, kind, act, bias, residual, preact, seed=0):
    g = torch.Generator().manual_seed(rows * 7919 + k * 31 + n + seed)
    x, w = normal(g, (rows, k), kind), normal(g, (n, k), kind, k ** -0.5)
    b = normal(g, (n,), bias) if bias else None
    r = normal(g, (rows, n), kind) if residual else None
    got = vn.linear(x, w, b, activation=act, residual=r, preact=preact)
    y, z = got if preact else (got, None)
    wy, wz = ora.linear(f64(x), f64(w), None if b is None else f64(b), act, None if r is None else f64(r))
    s = np.abs(f64(x)) @ np.abs(f64(w)).T + (0 if b is None else np.abs(f64(b)))
    err = (2 * k + 18) * U * s
    if preact:
        within(z, wz, err + rounding(kind, wz), "preact")
    rr = 0 if r is None else np.abs(f64(r))
    within(y, wy, 1.13 * err + (act_slack(kind, wz) if act != "none" else 0) + 2 * U * rr + rounding(kind, wy), "y")


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_linear_shapes(rows, k, n, kind):
    check_linear(rows, k, n, kind, "gelu", kind, True, True)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 6, 150])
def test_linear_activations(rows, act, kind):
    check_linear(rows, 192, 200, kind, act, None, False, False)
    check_linear(rows, 192, 200, kind, act, "fp32" if kind == "bf16" else "bf16", True, False, seed=1)


def test_linear_large_bf16_on_the_gpu_in_fp64():
    """A size of many tiles, against torch's float64 product on the device."""
    g = torch.Generator().manual_seed(3)
    rows, k, n = 2000, 2056, 3000
    x, w, b = normal(g, (rows, k), "bf16"), normal(g, (n, k), "bf16", k ** -0.5), normal(g, (n,), "bf16")
    y = vn.linear(x, w, b, check_status=True)
    want = x.double() @ w.double().t() + b.double()
    s = x.double().abs() @ w.double().abs().t() + b.double().abs()
    bound = (2 * k + 18) * U * s + 2.0 ** -8 * want.abs() * 1.01
    assert bool(((y.double() - want).abs() <= bound).all())


def test_linear_large_fp32_on_the_gpu_in_fp64():
    g = torch.Generator().manual_seed(4)
    rows, k, n = 1500, 1031, 1100
    x, w = normal(g, (rows, k), "fp32"), normal(g, (n, k), "fp32", k ** -0.5)
    y = vn.linear(x, w, check_status=True)
    want = x.double() @ w.double().t()
    s = x.double().abs() @ w.double().abs().t()
    assert bool(((y.double() - want).abs() <= (2 * k + 18) * U * s).all())
    # The error as a whole is that of fp32 sums, far below the bound on one element.
    rel = float((y.double() - want).norm() / want.norm())
    assert rel <= 2e-6, rel


def test_linear_leading_shape_strides_and_out():
    g = torch.Generator().manual_seed(5)
    x = normal(g, (40, 6, 5), "fp32").permute(2, 1, 0)          # (5, 6, 40), not contiguous
    w = normal(g, (40, 24), "fp32").t()                          # (24, 40), not contiguous
    out = torch.full((5, 6, 24), float("nan"), device=DEV)
    y = vn.linear(x, w, out=out)
    assert y is out
    want = f64(x) @ f64(w).T
    within(y, want, (2 * 40 + 18) * U * (np.abs(f64(x)) @ np.abs(f64(w)).T), "y")


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_linear_unaligned_base(kind):
    """Inputs that start inside a buffer, off the 16-byte boundaries of vector loads."""
    g = torch.Generator().manual_seed(6)
    flat = normal(g, (1 + 200 * 128,), kind)
    x = flat[1:1 + 200 * 128].view(200, 128)
    wflat = normal(g, (1 + 64 * 128,), kind, 0.1)
    w = wflat[1:].view(64, 128)
    y = vn.linear(x, w)
    want = f64(x) @ f64(w).T
    within(y, want, (2 * 128 + 18) * U * (np.abs(f64(x)) @ np.abs(f64(w)).T) + rounding(kind, want), "y")
    d = normal(g, (1 + 200 * 64,), kind)[1:].view(200, 64)
    gx, gw, gb = vn.linear_backward(d, x, w)
    wx, ww, wb, _ = ora.linear_backward(f64(d), f64(x), f64(w))
    within(gx, wx, (2 * 64 + 18) * U * (np.abs(f64(d)) @ np.abs(f64(w))) + rounding(kind, wx), "grad_x")
    within(gw, ww, (2 * 200 + 18) * U * (np.abs(f64(d)).T @ np.abs(f64(x))) + rounding(kind, ww), "grad_w")
    within(gb, wb, 2 * 200 * U * np.abs(f64(d)).sum(0) + rounding(kind, wb), "grad_b")


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_linear_empty_sizes(kind):
    k = KINDS[kind]
    assert vn.linear(torch.empty(0, 8, dtype=k, device=DEV), torch.ones(4, 8, dtype=k, device=DEV)).shape == (0, 4)
    assert vn.linear(torch.ones(3, 8, dtype=k, device=DEV), torch.empty(0, 8, dtype=k, device=DEV)).shape == (3, 0)
    b = torch.arange(4, dtype=k, device=DEV)
    y = vn.linear(torch.empty(3, 0, dtype=k, device=DEV), torch.empty(4, 0, dtype=k, device=DEV), b)
    assert torch.equal(y, b.expand(3, 4))
    gx, gw, gb = vn.linear_backward(torch.empty(0, 4, dtype=k, device=DEV), torch.empty(0, 8, dtype=k, device=DEV),
                                    torch.ones(4, 8, dtype=k, device=DEV))
    assert gx.shape == (0, 8) and not gw.any() and not gb.any()
    gx, gw, gb = vn.linear_backward(torch.empty(3, 0, dtype=k, device=DEV), torch.ones(3, 8, dtype=k, device=DEV),
                                    torch.empty(0, 8, dtype=k, device=DEV))
    assert not gx.any() and gw.shape == (0, 8) and gb.shape == (0,)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,k,n", [(4, 64, 40), (300, 264, 200)])
def test_linear_not_finite(rows, k, n, kind):
    """A NaN of x reaches its row of y and nothing else; an infinity leaves its row not finite."""
    g = torch.Generator().manual_seed(7)
    x, w = normal(g, (rows, k), kind), normal(g, (n, k), kind)
    x[1, 5], x[2, 3] = float("nan"), float("inf")
    y = f64(vn.linear(x, w))
    assert np.isnan(y[1]).all() and not np.isfinite(y[2]).any()
    assert np.isfinite(np.delete(y, (1, 2), axis=0)).all()


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [1e-18, 1e15])
def test_linear_scales(scale, kind):
    """Far from 1, the splitting into bf16 terms keeps fp32's precision."""
    g = torch.Generator().manual_seed(8)
    x, w = normal(g, (600, 520), kind, scale), normal(g, (300, 520), kind, 1 / 20)
    y = vn.linear(x, w)
    want = f64(x) @ f64(w).T
    within(y, want, (2 * 520 + 18) * U * (np.abs(f64(x)) @ np.abs(f64(w)).T) + rounding(kind, want), "y")


def check_backward(rows, k, n, kind, act, bias=True):
    g = torch.Generator().manual_seed(rows * 7919 + k * 31 + n + 1)
    x, w, d = normal(g, (rows, k), kind), normal(g, (n, k), kind, k ** -0.5), normal(g, (rows, n), kind)
    z = normal(g, (rows, n), kind) if act != "none" else None
    gx, gw, gb = vn.linear_backward(d, x, w, z, activation=act, bias=bias)
    wx, ww, wb, wd = ora.linear_backward(f64(d), f64(x), f64(w), None if z is None else f64(z), act)
    ad = np.abs(wd) + np.abs(f64(d)) * (act_slack(kind, f64(z)) if act != "none" else 0)
    e = np.abs(f64(d)) * (act_slack(kind, f64(z)) if act != "none" else 0)   # of d itself
    er = e + (2.0 ** -8 * ad if kind == "bf16" and act != "none" else 0)      # of d as the products take it
    aw, ax = np.abs(f64(w)), np.abs(f64(x))
    within(gx, wx, (2 * n + 18) * U * (ad @ aw) + er @ aw + rounding(kind, wx), "grad_x")
    within(gw, ww, (2 * rows + 18) * U * (ad.T @ ax) + er.T @ ax + rounding(kind, ww), "grad_w")
    if bias:
        within(gb, wb, (2 * rows + 2) * U * ad.sum(0) + e.sum(0) + rounding(kind, wb), "grad_b")
    else:
        assert gb is None


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_linear_backward_shapes(rows, k, n, kind):
    check_backward(rows, k, n, kind, "none")
    check_backward(rows, k, n, kind, "gelu", bias=False)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_activations(act, kind):
    check_backward(150, 192, 200, kind, act)


@pytest.mark.parametrize("rows,k,n,kind", [(4100, 260, 136, "bf16"), (2500, 264, 520, "bf16"), (2100, 300, 264, "fp32")])
def test_linear_backward_long_sums(rows, k, n, kind):
    check_backward(rows, k, n, kind, "silu")


@pytest.mark.parametrize("act", ACTS)
def test_linear_gradient_against_differences(act):
    """<c, y> along directions of x, w and b, by central differences of the float64 forward."""
    rng = np.random.default_rng(11)
    rows, k, n = 37, 24, 19
    x, w, b, c = (rng.standard_normal(s).astype(np.float32) for s in ((rows, k), (n, k), (n,), (rows, n)))
    w /= np.float32(5)
    dev = [torch.from_numpy(a).to(DEV) for a in (x, w, b, c)]
    y, z = vn.linear(dev[0], dev[1], dev[2], activation=act, preact=True)
    gx, gw, gb = vn.linear_backward(dev[3], dev[0], dev[1], z, activation=act)
    args = [a.astype(np.float64) for a in (x, w, b)]
    h = 1e-6
    for i, grad in enumerate((gx, gw, gb)):
        u = rng.standard_normal(args[i].shape)
        u /= np.linalg.norm(u)

        def loss(s):
            a = list(args)
            a[i] = a[i] + s * h * u
            return float((ora.linear(a[0], a[1], a[2], act)[0] * c).sum())
        diff = (loss(1) - loss(-1)) / (2 * h)
        got = float((f64(grad) * u).sum())
        # differences: h^2 of the third derivative and 2^-52 |loss| / h; fp32 gradient: 1e-5 of its norm
        tol = 1e-5 * float(np.linalg.norm(f64(grad))) + 1e-6 * (1 + abs(diff))
        if act == "relu":     # a kink within h of z = 0 contributes at most its |c| |dz|
            tol += 1e-3
        assert abs(got - diff) <= tol, (i, got, diff)


# ---------------------------------------------------------------- layer norm
NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (5, 32), (2, 255), (9, 256), (4, 257), (33, 512), (7, 1000), (6, 1021), (3, 1024),
               (5, 2048), (3, 2056), (2, 3001), (7, 4096), (2, 4104), (3, 8192), (2, 8200), (2, 9001), (2, 16384), (1, 20000),
               (3, 33000), (2, 40001), (700, 64), (1500, 96), (5000, 40)]


def norm_inputs(rows, n, kind, wkind):
    g = torch.Generator().manual_seed(rows * 131 + n)
    x = (torch.randn((rows, n), generator=g) * (0.1 + 2 * torch.rand((rows, 1), generator=g))
         + 3 * torch.randn((rows, 1), generator=g)).to(KINDS[kind]).to(DEV)
    return g, x, normal(g, (n,), wkind, 0.3, 1.0), normal(g, (n,), wkind, 0.3)


@pytest.mark.parametrize("kind,wkind", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,n", NORM_SHAPES)
def test_layer_norm(rows, n, kind, wkind):
    g, x, w, b = norm_inputs(rows, n, kind, wkind)
    y, mean, rstd = vn.layer_norm(x, w, b, eps=1e-5)
    wy, wm, wr = ora.layer_norm(f64(x), f64(w), f64(b), 1e-5)
    ax = np.abs(f64(x))
    # a thread adds at most 2 + n/32 values before the tree of 10 additions
    steps = min(n, 2 + n // 32) + 12
    em = steps * U * ax.mean(1) + U * np.abs(wm)
    within(mean, wm, em, "mean")
    # the centred squares' sum: its own additions, and each c off by em + 2u|c|
    er = wr * (steps * U + 8 * U + 0.5 * (em * wr) ** 2 + 4 * U * ax.max(1) * wr)
    within(rstd, wr, er, "rstd")
    h = np.abs((f64(x) - wm[:, None]) * wr[:, None])
    ey = np.abs(f64(w)) * (h * (er / wr + 4 * U)[:, None] + (em + U * ax.max(1))[:, None] * wr[:, None])
    within(y, wy, ey + 4 * U * (h * np.abs(f64(w)) + np.abs(f64(b))) + rounding(kind, wy), "y")


def test_layer_norm_without_parameters_and_large_offset():
    g = torch.Generator().manual_seed(2)
    x = normal(g, (64, 300), "fp32", 1.0, 1000.0)       # the mean is 1000 times the deviation
    y, mean, rstd = vn.layer_norm(x)
    wy, wm, wr = ora.layer_norm(f64(x))
    within(y, wy, 300 * U * 1000 * np.ones_like(wy), "y")  # one sum's error over the deviation
    flat = torch.full((5, 128), 7.25, device=DEV)
    y, mean, rstd = vn.layer_norm(flat, eps=1e-5)
    assert not y.any() and bool((mean == 7.25).all())
    within(rstd, np.full(5, 1e-5 ** -0.5), 4 * U * 1e-5 ** -0.5, "rstd of a constant row")


def test_layer_norm_not_finite_stays_in_its_row():
    g = torch.Generator().manual_seed(3)
    for n in (96, 1021, 4096, 20001):
        x = normal(g, (6, n), "fp32")
        x[2, n // 2], x[4, 1] = float("nan"), float("inf")
        y, mean, rstd = vn.layer_norm(x)
        bad = ~torch.isfinite(y).all(1)
        assert bad.tolist() == [False, False, True, False, True, False]


def check_norm_backward(rows, n, kind, wkind):
    g, x, w, _ = norm_inputs(rows, n, kind, wkind)
    d = normal(g, (rows, n), kind)
    _, wm, wr = ora.layer_norm(f64(x))
    mean, rstd = (torch.from_numpy(a.astype(np.float32)).to(DEV) for a in (wm, wr))
    gx, gw, gb = vn.layer_norm_backward(d, x, mean, rstd, w)
    wm, wr = f64(mean), f64(rstd)
    wx, ww, wb = ora.layer_norm_backward(f64(d), f64(x), wm, wr, f64(w))
    h = (f64(x) - wm[:, None]) * wr[:, None]
    t = np.abs(f64(d) * f64(w))
    eh = 3 * U * np.abs(h) + U * np.abs(wm * wr)[:, None]         # of h: a difference and a product
    steps = min(n, 2 + n // 32) + 14
    m1 = (steps * U * t).mean(1, keepdims=True)
    m2 = (steps * U * t * np.abs(h) + t * eh).mean(1, keepdims=True)
    am2 = (t * np.abs(h)).mean(1, keepdims=True)
    bound = wr[:, None] * (m1 + np.abs(h) * m2 + eh * am2 + 6 * U * (t + t.mean(1, keepdims=True) + np.abs(h) * am2))
    within(gx, wx, bound + rounding(kind, wx), "grad_x")
    ad = np.abs(f64(d))
    within(gw, ww, ((rows + 12) * U * ad * np.abs(h) + ad * eh).sum(0) + rounding(wkind, ww), "grad_w")
    within(gb, wb, (rows + 12) * U * ad.sum(0) + rounding(wkind, wb), "grad_b")


@pytest.mark.parametrize("kind,wkind", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,n", NORM_SHAPES)
def test_layer_norm_backward(rows, n, kind, wkind):
    check_norm_backward(rows, n, kind, wkind)


def test_layer_norm_backward_without_weight_and_without_rows():
    g, x, w, _ = norm_inputs(11, 96, "fp32", "fp32")
    d = normal(g, (11, 96), "fp32")
    _, mean, rstd = vn.layer_norm(x)
    gx, gw, gb = vn.layer_norm_backward(d, x, mean, rstd)
    assert gw is None and gb is None
    one, _, _ = vn.layer_norm_backward(d, x, mean, rstd, torch.ones(96, device=DEV))
    assert torch.equal(gx, one)
    e = torch.empty(0, 96, device=DEV)
    gx, gw, gb = vn.layer_norm_backward(e, e, e[:, 0], e[:, 0], w)
    assert gx.shape == (0, 96) and not gw.any() and not gb.any()


def test_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(13)
    x, w, b, c = (rng.standard_normal(s).astype(np.float32) for s in ((29, 45), (45,), (45,), (29, 45)))
    dev = [torch.from_numpy(a).to(DEV) for a in (x, w, b, c)]
    _, mean, rstd = vn.layer_norm(dev[0], dev[1], dev[2])
    grads = vn.layer_norm_backward(dev[3], dev[0], mean, rstd, dev[1])
    args = [a.astype(np.float64) for a in (x, w, b)]
    for i, grad in enumerate(grads):
        u = rng.standard_normal(args[i].shape)
        u /= np.linalg.norm(u)

        def loss(s):
            a = list(args)
            a[i] = a[i] + s * 1e-6 * u
            return float((ora.layer_norm(a[0], a[1], a[2])[0] * c).sum())
        diff = (loss(1) - loss(-1)) / 2e-6
        got = float((f64(grad) * u).sum())
        assert abs(got - diff) <= 1e-5 * float(np.linalg.norm(f64(grad))) + 1e-6 * (1 + abs(diff)), i


def test_repeatable_and_on_another_stream():
    """The same call gives the same bits, also on a stream of its own."""
    g = torch.Generator().manual_seed(21)
    x, w, d = normal(g, (777, 264), "bf16"), normal(g, (200, 264), "bf16", 0.1), normal(g, (777, 200), "bf16")
    z = normal(g, (777, 200), "bf16")
    gamma = normal(g, (264,), "fp32")

    def every():
        y = vn.linear(x, w, activation="gelu")
        n, mean, rstd = vn.layer_norm(x, gamma, gamma)
        return [y, n, mean, rstd, *vn.linear_backward(d, x, w, z, activation="gelu"),
                *vn.layer_norm_backward(x, x, mean, rstd, gamma)]
    first = every()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = every()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    vn.device_status()


def test_capture_in_a_graph():
    """The operators launch without synchronising or allocating: a graph of them replays."""
    g = torch.Generator().manual_seed(22)
    x, w, b = normal(g, (256, 256), "bf16"), normal(g, (256, 256), "bf16", 1 / 16), normal(g, (256,), "bf16")
    y0 = vn.linear(x, w, b, activation="tanh")
    n0, _, _ = vn.layer_norm(y0, b, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = vn.linear(x, w, b, activation="tanh")
        n, _, _ = vn.layer_norm(y, b, b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(n, n0)


def test_refusals():
    x, w = torch.ones(3, 8, device=DEV), torch.ones(4, 8, device=DEV)
    with pytest.raises(ValueError):
        vn.linear(x.cpu(), w)
    with pytest.raises(ValueError):
        vn.linear(x, w[:, :7])
    with pytest.raises(TypeError):
        vn.linear(x, w.bfloat16())
    with pytest.raises(TypeError):
        vn.linear(x.double(), w.double())
    with pytest.raises(ValueError):
        vn.linear(x, w, torch.ones(5, device=DEV))
    with pytest.raises(ValueError):
        vn.linear(x, w, activation="softmax")
    with pytest.raises(ValueError):
        vn.linear(x, w, residual=torch.ones(3, 5, device=DEV))
    with pytest.raises(TypeError):
        vn.linear(x, w, residual=torch.ones(3, 4, device=DEV).bfloat16())
    with pytest.raises(ValueError):
        vn.linear(x, w, out=torch.ones(4, 3, device=DEV))
    buf = torch.ones(64, device=DEV)
    with pytest.raises(vn.VNError) as e:       # y over x
        vn.linear(buf[:24].view(3, 8), w, out=buf[20:32].view(3, 4))
    assert e.value.status == 4
    with pytest.raises(ValueError):
        vn.linear_backward(torch.ones(3, 4, device=DEV), x, w, activation="tanh")
    with pytest.raises(ValueError):
        vn.linear_backward(torch.ones(4, 4, device=DEV), x, w)
    with pytest.raises(ValueError):
        vn.layer_norm(x, torch.ones(7, device=DEV))
    with pytest.raises(TypeError):
        vn.layer_norm(x, torch.ones(8, device=DEV), torch.ones(8, device=DEV).bfloat16())
    with pytest.raises(TypeError):
        vn.layer_norm(x.half())
    with pytest.raises(vn.VNError):
        vn.layer_norm(x, eps=-1.0)
    with pytest.raises(vn.VNError):
        vn.layer_norm(x, eps=float("nan"))
    with pytest.raises(ValueError):
        vn.layer_norm(torch.ones(3, 0, device=DEV))
    with pytest.raises(ValueError):
        vn.layer_norm_backward(x, x, torch.ones(4, device=DEV), torch.ones(3, device=DEV))
    with pytest.raises(TypeError):
        vn.layer_norm_backward(x, x, torch.ones(3, device=DEV).double(), torch.ones(3, device=DEV))


# Rows that start anywhere: lengths beside every boundary of the kernels' choices, and tensors that start
# on any element between others' memory.
ANY_N = (3, 9, 17, 31, 65, 127, 129, 250, 257, 301, 511, 513, 1023, 1025, 2047, 2049, 4095, 4097, 8191, 8193, 16383)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", ANY_N)
def test_layer_norm_of_any_length(n, kind):
    for rows in (1, 5, 1300):
        if rows * n > 4_000_000:
            continue
        test_layer_norm(rows, n, kind, "fp32")
        check_norm_backward(rows, n, kind, "fp32")


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", (7, 61, 255, 517, 1021, 3001))
def test_layer_norm_does_not_depend_on_the_place(n, kind):
    """NaN around the inputs reaches nothing, and what lies around the outputs stays. (Odd lengths: where
    16-byte loads divide a row, aligned tensors have a kernel, and an order of sums, of their own.)"""
    g, x, w, b = norm_inputs(19, n, kind, "fp32")
    d = normal(g, (19, n), kind)
    y, mean, rstd = vn.layer_norm(x, w, b)
    grads = None
    for o in range(1, 9):
        def placed(t):
            big = torch.full((t.numel() + 32,), float("nan"), dtype=t.dtype, device=DEV)
            view = big[o:o + t.numel()].view(t.shape)
            view.copy_(t)
            return view

        big = torch.full((x.numel() + 32,), 7.0, dtype=x.dtype, device=DEV)
        out = big[o + 3:o + 3 + x.numel()].view(x.shape)
        y2, mean2, rstd2 = vn.layer_norm(placed(x), w, b, out=out)
        assert torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
        assert bool((big[:o + 3] == 7).all()) and bool((big[o + 3 + x.numel():] == 7).all())
        again = vn.layer_norm_backward(placed(d), placed(x), mean, rstd, w)
        if grads is None:
            grads = again
        for p, q in zip(again, grads):
            assert torch.equal(p, q)
    ref = vn.layer_norm_backward(d, x, mean, rstd, w)
    for p, q in zip(grads, ref):
        assert torch.equal(p, q)


@pytest.mark.parametrize("rows,n_in,n_out", [(9, 7, 5), (33, 65, 63), (130, 127, 129), (257, 191, 70), (64, 250, 38)])
def test_linear_bf16_does_not_depend_on_the_place(rows, n_in, n_out):
    """As above, for operands that are gathered."""
    g = torch.Generator().manual_seed(31)
    x, w = normal(g, (rows, n_in), "bf16"), normal(g, (n_out, n_in), "bf16", 0.2)
    d, z = normal(g, (rows, n_out), "bf16"), normal(g, (rows, n_out), "bf16")
    first = None
    for o in range(1, 9):
        def placed(t):
            big = torch.full((t.numel() + 32,), float("nan"), dtype=t.dtype, device=DEV)
            view = big[o:o + t.numel()].view(t.shape)
            view.copy_(t)
            return view

        got = (vn.linear(placed(x), placed(w)),) + tuple(
            vn.linear_backward(placed(d), placed(x), placed(w), placed(z), activation="silu"))
        assert all(bool(torch.isfinite(t).all()) for t in got)
        if first is None:
            first = got
        for p, q in zip(got, first):
            assert torch.equal(p, q)


def _chain(x, w, gain, n):
    """n residual steps; each call's input is what the call before it wrote."""
    for _ in range(n):
        h, _, _ = vn.layer_norm(x, gain, gain)
        x = vn.linear(h, w, activation="tanh", residual=x)
    return x


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,n", [(3, 64), (130, 96), (1000, 264), (700, 129)])
def test_calls_that_follow_one_another_see_each_other(rows, n, kind):
    """Launches overlap the end of the one before: the same bits with a wait after every call, without,
    over two streams joined by events, and replayed from a graph."""
    g = torch.Generator().manual_seed(41)
    x, w, gain = normal(g, (rows, n), kind), normal(g, (n, n), kind, 0.1), normal(g, (n,), "fp32", 0.1, 1.0)
    want = x
    for _ in range(30):
        want = _chain(want, w, gain, 1)
        torch.cuda.synchronize()
    for _ in range(5):
        assert torch.equal(_chain(x, w, gain, 30), want)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    y, kept = x, []
    for i in range(30):
        here, there = streams[i % 2], streams[(i + 1) % 2]
        with torch.cuda.stream(here):
            y = _chain(y, w, gain, 1)
            kept.append(y)
        there.wait_stream(here)
    torch.cuda.synchronize()
    assert torch.equal(y, want)

    graph, out = torch.cuda.CUDAGraph(), None
    with torch.cuda.graph(graph):
        out = _chain(x, w, gain, 30)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,n_in,n_out", [(4096, 64, 64), (4500, 33, 70), (8192, 130, 60), (30001, 16, 8)])
def test_linear_backward_over_many_rows(rows, n_in, n_out, kind):
    """Sums over rows that are long enough to be split over the largest clusters."""
    check_backward(rows, n_in, n_out, kind, "silu")
