"""The gradient norm, clipping, and AdamW's clipped step on the GPU against float64.

Tolerances: the norm is the exact one rounded once (half a step, u = 2^-24 of it) but for sums kept to about
2^-36, and the factor likewise; an element then takes the factor's rounding, its product's and, in bf16, half a
step of 2^-8."""

import numpy as np
import pytest
import torch

from oracle import network as ora
import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300 import VNError
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {"fp32": U, "bf16": 2.0 ** -8}
SHAPES = [(1,), (255,), (0,), (17, 19), (64, 64), (4095,), (4096,), (4097,), (3, 5, 7000), (8191,), (8192,), (8193,), ()]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make(shapes, kind, seed=0, scale=0.01):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale * float(torch.exp(torch.randn((), generator=g)))).to(KINDS[kind]).to(DEV)
            for s in shapes]


def norm_close(got, want):
    assert got.shape == () and got.dtype == torch.float32
    assert abs(float(got) - want) <= U * (1 + 2.0 ** -10) * want, (float(got), want)


def check_clipped(out, grads, max_norm, kind):
    norm = ora.gradient_norm([f64(g) for g in grads])
    f = ora.clip_factor(norm, max_norm)
    for o, g in zip(out, grads):
        want = f64(g) * f
        assert np.all(np.abs(f64(o) - want) <= (HALF[kind] + 2.1 * U) * np.abs(want) + 1e-44)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_norm_and_clipping(kind):
    grads = make(SHAPES, kind)
    want = ora.gradient_norm([f64(g) for g in grads])
    norm_close(vn.gradient_norm(grads), want)
    norm_close(vn.gradient_norm(tuple(grads)), want)
    norm_close(vn.gradient_norm(grads[8]), ora.gradient_norm([f64(grads[8])]))
    buf = torch.empty((), device=DEV)
    assert vn.gradient_norm(grads, out=buf) is not None and float(buf) == float(vn.gradient_norm(grads))
    before = [g.clone() for g in grads]
    out = [torch.full_like(g, float("nan")) for g in grads]
    norm_close(vn.clip_gradients(grads, 0.3 * want, out=out), want)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    check_clipped(out, before, 0.3 * want, kind)
    norm_close(vn.clip_gradients(grads, 0.3 * want), want)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_gradients_within_the_bound_keep_their_bits(kind):
    grads = make(SHAPES, kind, seed=1)
    grads[3][0, 0] = -0.0
    before = [g.clone() for g in grads]
    want = ora.gradient_norm([f64(g) for g in grads])
    out = [torch.empty_like(g) for g in grads]
    for bound in (want * 1.001, float("inf")):
        norm_close(vn.clip_gradients(grads, bound), want)
        norm_close(vn.clip_gradients(grads, bound, out=out), want)
        for g, o, b in zip(grads, out, before):
            assert torch.equal(g.view(torch.uint8) if g.dim() else g, b.view(torch.uint8) if b.dim() else b)
            assert torch.equal(o.view(torch.uint8) if o.dim() else o, b.view(torch.uint8) if b.dim() else b)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("size", [1e-41, 1e-30, 1e-19, 1e-13, 1e10, 1e16, 1e19, 1e30, 3e37])
def test_the_whole_range(kind, size):
    """Squares that fp32 cannot hold, and elements of very different sizes side by side."""
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(20001, generator=g, dtype=torch.float64) * size).float().to(KINDS[kind]).to(DEV)
    mixed = x.clone()
    mixed[::3] *= 1e-3
    mixed[1::3] *= 1e-7
    for t in (x, mixed):
        want = ora.gradient_norm([f64(t)])
        if want < 3.4e38:
            assert abs(float(vn.gradient_norm(t)) - want) <= max(U * (1 + 2.0 ** -10) * want, 2.0 ** -150)
        else:
            assert float(vn.gradient_norm(t)) == float("inf")
        if want > 1e-30:
            out = torch.empty_like(t)
            vn.clip_gradients(t, want * 0.25, out=out)
            scaled = f64(t) * 0.25
            assert np.all(np.abs(f64(out) - scaled) <= (HALF[kind] + 2.1 * U) * np.abs(scaled) + 2.0 ** -134)


def test_long_sums_and_many_tensors():
    """A hundred million equal elements, whose sum of squares fp32 could not count; and more tensors than a
    launch takes."""
    x = torch.full((100_000_003,), 0.1, device=DEV)
    norm_close(vn.gradient_norm(x), float(np.float32(0.1)) * np.sqrt(100_000_003.0))
    many = make([(1 + i % 7, 3) for i in range(2001)], "fp32", seed=4)
    want = ora.gradient_norm([f64(g) for g in many])
    norm_close(vn.gradient_norm(many), want)
    before = [g.clone() for g in many]
    norm_close(vn.clip_gradients(many, 0.5 * want), want)
    check_clipped(many, before, 0.5 * want, "fp32")


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_views_at_odd_offsets_and_their_neighbours(kind):
    """Tensors that start anywhere; what lies before and behind them stays as it is."""
    flat = make([(40000,)], kind, seed=5)[0]
    keep = flat.clone()
    at = [(3, 9001), (9010, 17), (9031, 16384), (26001, 13001)]
    views = [flat[o:o + n] for o, n in at]
    want = ora.gradient_norm([f64(v) for v in views])
    before = [v.clone() for v in views]
    norm_close(vn.clip_gradients(views, 0.4 * want), want)
    check_clipped(views, before, 0.4 * want, kind)
    outside = torch.ones(40000, dtype=torch.bool, device=DEV)
    for o, n in at:
        outside[o:o + n] = False
    assert torch.equal(flat[outside], keep[outside])


def test_not_contiguous_gradients_are_read():
    g = make([(33, 65), (65,)], "fp32", seed=6)
    want = ora.gradient_norm([f64(t) for t in g])
    norm_close(vn.gradient_norm([g[0].t(), g[1].expand(1, 65)]), want)
    out = [torch.empty(65, 33, device=DEV), torch.empty(65, device=DEV)]
    norm_close(vn.clip_gradients([g[0].t(), g[1]], 0.5 * want, out=out), want)
    check_clipped([out[0].t(), out[1]], g, 0.5 * want, "fp32")


def test_infinities_and_nan():
    g = [torch.ones(5000, device=DEV), torch.ones(3, device=DEV)]
    g[0][17] = float("inf")
    out = [torch.empty_like(t) for t in g]
    assert float(vn.clip_gradients(g, 1.0, out=out)) == float("inf")
    assert torch.isnan(out[0][17]) and int((out[0] != 0).sum()) == 1 and bool((out[1] == 0).all())
    g[1][0] = float("nan")
    assert np.isnan(float(vn.clip_gradients(g, 1.0, out=out)))
    assert all(bool(torch.isnan(o).all()) for o in out)
    z = [torch.zeros(100, device=DEV), torch.zeros(0, device=DEV)]
    assert float(vn.clip_gradients(z, 0.0)) == 0.0 and bool((z[0] == 0).all())
    assert float(vn.gradient_norm(torch.zeros(0, device=DEV))) == 0.0
    w = torch.ones(100, device=DEV)
    assert float(vn.clip_gradients(w, 0.0)) == 10.0 and bool((w == 0).all())


def test_repeats_streams_and_graphs():
    grads = make([(300, 1000), (1000,), (77, 91)], "bf16", seed=7)
    out = [torch.empty_like(g) for g in grads]
    first = vn.clip_gradients(grads, 0.1, out=out)
    want = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for o in out:
            o.fill_(float("nan"))
        again = vn.clip_gradients(grads, 0.1, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert float(again) == float(first) and all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = vn.clip_gradients(grads, 0.1, out=out)
    for scale in (1.0, 2.0, 1.0):
        for g in grads:
            g.mul_(scale)
        graph.replay()
        assert float(norm) == float(vn.gradient_norm(grads))
        check_clipped(out, grads, 0.1, "bf16")


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kind,gkind", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_a_clipped_step_is_the_step_of_clipped_gradients(kind, gkind, bits):
    shapes = [(1,), (257,), (0,), (64, 64), (3, 5, 700), (2048,)]
    for bound in (0.5, 1e6):
        a, b = make(shapes, kind, seed=8), make(shapes, kind, seed=8)
        grads = make(shapes, gkind, seed=9, scale=1.0)
        o1 = vn.AdamW(a, lr=1e-2, weight_decay=0.1, state_bits=bits)
        o2 = vn.AdamW(b, lr=1e-2, weight_decay=0.1, state_bits=bits)
        for _ in range(2):
            keep = [g.clone() for g in grads]
            n1 = o1.step(grads, max_norm=bound)
            assert all(torch.equal(g, k) for g, k in zip(grads, keep))
            wide = [g.float().clone() for g in grads]  # the factor's product is rounded to fp32 only
            n2 = vn.clip_gradients(wide, bound)
            assert o2.step(wide) is None
            assert float(n1) == float(n2) == float(vn.gradient_norm(grads))
        assert o1.steps == 2
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert all(torch.equal(p, q) for p, q in zip(o1.moments(), o2.moments()))


def test_a_clipped_step_takes_a_flat_gradient_and_many_tensors():
    shapes = [(1 + i % 5, 7) for i in range(1001)]
    a, b = make(shapes, "fp32", seed=10), make(shapes, "fp32", seed=10)
    grads = make(shapes, "fp32", seed=11)
    n1 = vn.AdamW(a).step(torch.cat([g.reshape(-1) for g in grads]), max_norm=0.2)
    n2 = vn.AdamW(b).step(grads, max_norm=0.2)
    want = ora.gradient_norm([f64(g) for g in grads])
    norm_close(n1, want)
    norm_close(n2, want)
    moved = [torch.equal(p, q) or float((p - q).abs().max()) < 1e-6 for p, q in zip(a, b)]
    assert all(moved)


def test_refusals():
    g = [torch.ones(8, device=DEV), torch.ones(4, device=DEV)]
    for call in (lambda: vn.gradient_norm([]), lambda: vn.gradient_norm(None), lambda: vn.clip_gradients(g, None),
                 lambda: vn.gradient_norm([g[0], g[1].bfloat16()]), lambda: vn.gradient_norm(g[0].double())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: vn.gradient_norm([torch.ones(3)]), lambda: vn.gradient_norm(g, out=torch.empty(1, device=DEV)),
                 lambda: vn.clip_gradients(torch.ones(4, 4, device=DEV).t(), 1.0), lambda: vn.clip_gradients(g, 1.0, out=g[:1]),
                 lambda: vn.clip_gradients(g, 1.0, out=[g[1], g[0]])):
        with pytest.raises(ValueError):
            call()
    wide = torch.ones(16, device=DEV)
    for call in (lambda: vn.clip_gradients(g, -1.0), lambda: vn.clip_gradients(g, float("nan")),
                 lambda: vn.clip_gradients([g[0], g[0]], 1.0), lambda: vn.clip_gradients([wide[:8], wide[4:12]], 1.0),
                 lambda: vn.clip_gradients([wide[:8], wide[8:]], 1.0, out=[wide[8:], wide[:8]]),
                 lambda: vn.AdamW([g[0]]).step([torch.ones(8, device=DEV)], max_norm=-1.0)):
        with pytest.raises(VNError, match="VN_ERR_VALUE"):
            call()
    norm_close(vn.gradient_norm([g[0], g[0]]), 4.0)  # read twice, counted twice
    assert float(vn.clip_gradients([wide[:8], wide[8:]], 2.0, out=[wide[:8], wide[8:]])) == 4.0
    assert bool((wide == 0.5).all())


def test_what_is_written_counts_as_changed():
    g = torch.ones(8, device=DEV)
    v = g._version
    vn.gradient_norm(g)
    assert g._version == v
    vn.clip_gradients(g, 1.0)
    assert g._version == v + 1
