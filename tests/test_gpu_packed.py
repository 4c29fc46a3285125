"""Weights in 4 bits and the linear layer on them on the GPU against float64.

Packing is exact: codes and scales have to be the oracle's, values its values rounded once. The layer, with A = sum |x| |v|
of an output: a group's products are exact and its sum on the tensor cores off by at most 2^-20 A (8 steps, each cut below
2^-23 of what it adds up), the groups' sums and joins in fp32 by (groups / 8 + 16) 2^-24 A, and an activation by 2^-20 (1 + |z|); bf16
results by half a step, 2^-8. With many rows in bf16 the values are rounded first (2^-8 A), and fp32's products are those
of ``linear`` (2^-18 A)."""

import numpy as np
import pytest
import torch

from oracle import acting as ora
from oracle import network
import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300 import VNError
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rounder(kind):
    return lambda v: torch.from_numpy(np.asarray(v)).to(KINDS[kind]).double().numpy()


def randn(*shape, kind="fp32", seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(KINDS[kind])


def check_packed(w, group, kind):
    p = vn.pack4(w.to(DEV), group=group)
    codes, scales = ora.pack4(f64(w), group, rounder(kind))
    assert p.shape == w.shape and p.group == group and p.scales.dtype == w.dtype
    got = f64(p.scales)
    assert np.array_equal(got, scales, equal_nan=True)
    want = rounder(kind)(ora.values4(codes, scales, group))
    assert np.array_equal(f64(p.dequantize()), want, equal_nan=True)
    return p, ora.values4(codes, scales, group)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("out,k", [(1, 1), (3, 31), (5, 32), (16, 33), (17, 127), (40, 128), (7, 129), (9, 1003), (130, 256), (33, 4100)])
def test_packing(out, k, kind, group):
    w = randn(out, k, kind=kind, seed=out + k, scale=0.1)
    w[0, : k // 2] = 0
    check_packed(w, group, kind)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_packing_on_borders_and_at_the_ends_of_the_range(kind):
    """Halves between two codes, their neighbours, groups of zeros, subnormal scales, infinities and NaN."""
    w = torch.zeros(12, 256)
    w[0] = torch.arange(256) % 15 - 7.0
    w[1] = (torch.arange(256) % 29 - 14) * 0.5
    w[1, ::32] = 7.0
    w[2] = torch.nextafter(w[1], torch.full((256,), 9.0))
    w[3] = torch.nextafter(w[1], torch.full((256,), -9.0))
    w[2, ::32] = w[3, ::32] = 7.0
    w[4] = w[1] * 3
    w[5, 40] = 1e-44
    w[6] = torch.arange(256) * 1.4e-45
    w[7] = w[0] * 4e37
    w[8, 33] = float("inf")
    w[9, 200] = float("nan")
    w[9, 100] = -float("inf")
    w[10] = 1e-38 * (torch.arange(256) % 13 - 6)
    w[11, ::32] = 0.7
    w[11, 1::2] = 0.05
    for group in (32, 64, 128):
        check_packed(w.to(KINDS[kind]), group, kind)


def test_packing_many_borders():
    """Random fp32 weights next to every half: the quotient's own rounding decides nothing."""
    g = torch.Generator().manual_seed(5)
    s = torch.rand(512, 1, generator=g) + 0.5
    w = (torch.randint(-7, 7, (512, 256), generator=g) + 0.5) * s
    w += torch.randint(-2, 3, (512, 256), generator=g) * 2.0 ** -24 * w
    w[:, ::32] = 7 * s
    check_packed(w, 32, "fp32")


def check_linear(p, values, x, kind, bias=None, act=None, residual=None, y=None):
    if y is None:
        y = vn.linear4(x.to(DEV), p, None if bias is None else bias.to(DEV), activation=act,
                       residual=None if residual is None else residual.to(DEV), check_status=True)
    assert y.shape == x.shape[:-1] + (values.shape[0],) and y.dtype == x.dtype
    xs = f64(x).reshape(-1, x.shape[-1])
    rows = xs.shape[0]
    r = None if residual is None else f64(residual).reshape(rows, -1)
    want, z = network.linear(xs, values, None if bias is None else f64(bias), act or "none", r)
    a = np.abs(xs) @ np.abs(values).T + (0 if bias is None else np.abs(f64(bias)))
    many = rows > (32 if kind == "bf16" else 10)
    tol = (2.0 ** -20 + (x.shape[-1] / p.group / 8 + 16) * 2.0 ** -24) * a
    if many:
        tol = tol + (2.0 ** -8 if kind == "bf16" else 2.0 ** -18) * a
    tol = tol * 1.2 + (2.0 ** -20 * (1 + np.abs(z)) if act else 0)       # no slope is above 1.2
    tol = tol + (2.0 ** -8 if kind == "bf16" else 2.0 ** -23) * (np.abs(want) + (0 if r is None else np.abs(r)))
    err = np.abs(f64(y).reshape(rows, -1) - want)
    assert np.all(err <= tol + 1e-30), (err.max(), (err / (tol + 1e-30)).max())


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8, 9, 10, 11, 16, 17, 21, 32, 33, 64, 200])
def test_rows(rows, kind):
    w = randn(100, 333, kind=kind, seed=1, scale=0.06)
    p, v = check_packed(w, 64, kind)
    x, b, r = randn(rows, 333, kind=kind, seed=2), randn(100, kind="fp32", seed=3), randn(rows, 100, kind=kind, seed=4)
    check_linear(p, v, x, kind, b, "gelu", r)
    check_linear(p, v, x, kind)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("out,k", [(1, 1), (8, 64), (15, 127), (16, 128), (17, 129), (256, 256), (31, 1003), (64, 4096), (40, 9000)])
def test_sizes(out, k, kind, group):
    w = randn(out, k, kind=kind, seed=6, scale=k ** -0.5)
    p, v = check_packed(w, group, kind)
    for rows in (1, 7):
        check_linear(p, v, randn(rows, k, kind=kind, seed=7), kind, randn(out, kind=kind, seed=8), "tanh")


@pytest.mark.parametrize("act", [None, "tanh", "relu", "gelu", "silu"])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_activations(kind, act):
    w = randn(70, 200, kind=kind, seed=9, scale=0.2)
    p, v = check_packed(w, 32, kind)
    check_linear(p, v, randn(4, 200, kind=kind, seed=10), kind, None, act, randn(4, 70, kind=kind, seed=11))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_one_hot_rows_read_the_values(kind):
    """Exactly: the code times the scale, rounded once."""
    w = randn(50, 300, kind=kind, seed=12)
    p, v = check_packed(w, 64, kind)
    eye = torch.eye(300, dtype=KINDS[kind], device=DEV)
    for a in range(0, 300, 20):
        assert torch.equal(vn.linear4(eye[a:a + 20], p), p.dequantize()[:, a:a + 20].t())


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_a_large_layer(kind):
    w = randn(4096, 4096, kind=kind, seed=13, scale=1 / 64)
    p, v = check_packed(w, 128, kind)
    check_linear(p, v, randn(1, 4096, kind=kind, seed=14), kind, randn(4096, kind=kind, seed=15), "gelu", randn(1, 4096, kind=kind, seed=16))
    check_linear(p, v, randn(8, 4096, kind=kind, seed=17), kind)


def test_shapes_strides_buffers_and_neighbours():
    w = randn(37, 90, seed=18)
    p, v = check_packed(w, 32, "fp32")
    x = randn(2, 3, 90, seed=19)
    want = vn.linear4(x.to(DEV), p)
    check_linear(p, v, x, "fp32", y=want)
    one = vn.linear4(x[0, 0].to(DEV), p)
    assert one.shape == (37,) and torch.equal(one, vn.linear4(x[0, :1].to(DEV), p)[0])
    wide = torch.zeros(2, 3, 181, device=DEV)
    wide[..., 1::2] = x.to(DEV)
    assert torch.equal(vn.linear4(wide[..., 1::2], p), want)
    flat = torch.full((2 * 3 * 90 + 5,), float("nan"), device=DEV)
    there = flat[3:3 + 540].view(2, 3, 90)
    there.copy_(x)
    assert torch.equal(vn.linear4(there, p), want)
    buf = torch.full((2 * 3 * 37 + 6,), 7.0, device=DEV)
    out = buf[3:3 + 222].view(2, 3, 37)
    assert vn.linear4(there, p, out=out) is out and torch.equal(out, want)
    assert bool((buf[:3] == 7).all()) and bool((buf[225:] == 7).all())
    assert vn.linear4(torch.empty(0, 90, device=DEV), p).shape == (0, 37)
    again = vn.Weight4(p.codes.clone(), p.scales.clone(), 90, 32)
    assert torch.equal(vn.linear4(x.to(DEV), again), want)
    values = torch.empty(37, 90, device=DEV)
    assert p.dequantize(out=values) is values and torch.equal(values, p.dequantize())
    empty = vn.pack4(torch.empty(4, 0, device=DEV))
    b = torch.arange(4.0, device=DEV)
    assert torch.equal(vn.linear4(torch.empty(2, 0, device=DEV), empty, b), b.expand(2, 4))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_infinities_and_nan(kind):
    w = randn(20, 300, kind=kind, seed=20)
    w[3, 40], w[5, 299] = float("inf"), float("nan")
    p = vn.pack4(w.to(DEV))
    y = vn.linear4(randn(2, 300, kind=kind, seed=21).to(DEV), p)
    bad = torch.zeros(20, dtype=torch.bool)
    bad[[3, 5]] = True
    assert torch.equal(torch.isnan(y).cpu(), bad.expand(2, 20))
    x = randn(2, 300, kind=kind, seed=22)
    x[1, 7] = float("nan")
    y = vn.linear4(x.to(DEV), vn.pack4(randn(20, 300, kind=kind, seed=23).to(DEV)))
    assert bool(torch.isfinite(y[0]).all()) and bool(torch.isnan(y[1]).all())


@pytest.mark.parametrize("rows", [3, 100])
def test_streams_and_graphs(rows):
    w = randn(200, 500, kind="bf16", seed=24)
    p, v = check_packed(w, 64, "bf16")
    x = randn(rows, 500, kind="bf16", seed=25).to(DEV)
    want = vn.linear4(x, p, activation="silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = vn.linear4(x, p, activation="silu")
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = vn.linear4(x, p, activation="silu")
    for scale in (1.0, 0.5):
        x.mul_(scale)
        graph.replay()
        assert torch.equal(y, vn.linear4(x, p, activation="silu"))


def test_trained_packed_and_acting():
    """The operators as a program uses them: clipped steps on a policy, its layers packed, actions drawn from the packed
    policy's logits; the drawn indices are the oracle's on those logits."""
    g = torch.Generator().manual_seed(26)
    w1, w2 = (torch.randn(64, 40, generator=g) * 0.2).to(DEV), (torch.randn(12, 64, generator=g) * 0.2).to(DEV)
    b1, b2 = torch.zeros(64, device=DEV), torch.zeros(12, device=DEV)
    opt = vn.AdamW([w1, b1, w2, b2], lr=1e-2, weight_decay=0.0)
    x, target = torch.randn(128, 40, generator=g).to(DEV), torch.randn(128, 12, generator=g).to(DEV)
    for _ in range(3):
        h, z = vn.linear(x, w1, b1, activation="tanh", preact=True)
        off = vn.linear(h, w2, b2, residual=-target)
        gh, gw2, gb2 = vn.linear_backward(off, h, w2)
        _, gw1, gb1 = vn.linear_backward(gh, x, w1, z, activation="tanh")
        grads = [gw1, gb1, gw2, gb2]
        norm = opt.step(grads, max_norm=1.0)
        want = network.gradient_norm([f64(t) for t in grads])
        assert abs(float(norm) - want) <= 2.0 ** -23 * want
    p1, p2 = vn.pack4(w1), vn.pack4(w2)
    h = vn.linear4(x[:6], p1, b1, activation="tanh")
    logits = vn.linear4(h, p2, b2)
    u = torch.rand(6, generator=g)
    index = vn.sample(logits, u.to(DEV), temperature=0.7, top_p=0.9)
    for r in range(6):
        assert int(index[r]) == ora.sample(f64(logits[r]), float(u[r]), temperature=0.7, top_p=0.9)[0]


def test_refusals():
    w = torch.ones(6, 40, device=DEV)
    p = vn.pack4(w)
    x = torch.ones(2, 40, device=DEV)
    for call in (lambda: vn.pack4(w.double()), lambda: vn.linear4(x.bfloat16(), p)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: vn.pack4(w.cpu()), lambda: vn.pack4(w, group=16), lambda: vn.pack4(w[0]), lambda: vn.linear4(x[:, :39], p),
                 lambda: vn.linear4(x.cpu(), p), lambda: vn.linear4(x, p, torch.ones(5, device=DEV)),
                 lambda: vn.linear4(x, p, residual=x), lambda: vn.linear4(x, p, out=x), lambda: vn.linear4(x, p, activation="elu"),
                 lambda: vn.Weight4(p.codes, p.scales, 40, 48), lambda: vn.linear4(x, vn.Weight4(p.codes[:, :32], p.scales, 40, 64)),
                 lambda: vn.linear4(x, vn.Weight4(p.codes, p.scales, 40, 32)), lambda: p.dequantize(out=torch.empty(6, 41, device=DEV))):
        with pytest.raises(ValueError):
            call()
    square = vn.pack4(torch.ones(40, 40, device=DEV))
    with pytest.raises(VNError, match="VN_ERR_VALUE"):
        vn.linear4(x, square, out=x)
    odd = torch.zeros(6 * 64 + 1, dtype=torch.uint8, device=DEV)[1:].view(6, 64)
    with pytest.raises(VNError, match="VN_ERR_ALIGN"):
        vn.linear4(x, vn.Weight4(odd, p.scales, 40, 64))
