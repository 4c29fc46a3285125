"""AdamW over many tensors on the GPU against the float64 oracle.

Tolerances: with 32-bit moments every element takes a handful of fp32 roundings (u = 2^-24): 8u of
each term of the sums. An 8-bit code may fall on the other side of a rounding boundary in float64: then
it is its neighbour, at most 2^-3 of the value (or 2^-9 of the block's unit) away. That happens in few
places, since fp32 is 2^20 times finer than a code -- but bf16 gradients can fall on exact ties: a block
whose largest has a mantissa that is a multiple of 7 (448 = 7 * 64) puts others halfway between two codes,
where each side's last bit decides."""

import numpy as np
import pytest
import torch

from oracle import network as ora
import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16}
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make(shapes, kind, gkind, seed=0):
    g = torch.Generator().manual_seed(seed)
    params = [torch.randn(s, generator=g).to(KINDS[kind]).to(DEV) for s in shapes]
    grads = [(torch.randn(s, generator=g) * 0.01).to(KINDS[gkind]).to(DEV) for s in shapes]
    return params, grads


def step64(opt, i, p, g, m, v, decay):
    return ora.adamw(p, g, m, v, lr=opt.lr, beta1=opt.betas[0], beta2=opt.betas[1], eps=opt.eps, weight_decay=decay,
                     step=opt.steps, maximize=opt.maximize)


SHAPES = [(1,), (255,), (256,), (257,), (0,), (17, 19), (64, 64), (2048,), (3, 5, 700), (8,)]


@pytest.mark.parametrize("maximize", [False, True])
@pytest.mark.parametrize("kind,gkind", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_32_bit_moments(kind, gkind, maximize):
    params, grads = make(SHAPES, kind, gkind)
    decay = [0.1 * (i % 3) for i in range(len(SHAPES))]
    opt = vn.AdamW(params, **HYPER, weight_decay=decay, maximize=maximize)
    m = [np.zeros(p.numel()) for p in params]
    v = [np.zeros(p.numel()) for p in params]
    for k in range(3):
        before = [f64(p).reshape(-1) for p in params]
        gs = [g * (1.0 + 0.5 * k) for g in grads]
        opt.step(gs)
        fm, fv = (f64(t) for t in opt.moments())
        for i, p in enumerate(params):
            g = f64(gs[i]).reshape(-1)
            wp, m[i], v[i] = step64(opt, i, before[i], g, m[i], v[i], decay[i])
            at = slice(opt.offsets[i], opt.offsets[i] + p.numel())
            assert np.all(np.abs(fm[at] - m[i]) <= 8 * U * (k + 1) * (np.abs(g).max(initial=0)) + 1e-37)
            assert np.all(np.abs(fv[at] - v[i]) <= 8 * U * (k + 1) * v[i] + 1e-37)
            move = np.abs(wp - before[i]) + opt.lr * 4
            tol = 2 * U * np.abs(wp) + 32 * U * (k + 1) * move + (2.0 ** -8 * np.abs(wp) if kind == "bf16" else 0)
            assert np.all(np.abs(f64(p).reshape(-1) - wp) <= tol), (k, i)


@pytest.mark.parametrize("maximize", [False, True])
@pytest.mark.parametrize("kind,gkind", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_8_bit_moments(kind, gkind, maximize):
    params, grads = make(SHAPES, kind, gkind, seed=1)
    # magnitudes over many orders within a block, and a block of zeros
    for g in grads[1:]:
        flat = g.view(-1)
        flat.mul_(torch.exp(torch.linspace(-25, 0, flat.numel(), device=DEV)).to(g.dtype))
    grads[7].zero_()
    opt = vn.AdamW(params, **HYPER, weight_decay=0.05, state_bits=8, maximize=maximize)
    for k in range(3):
        before = [f64(p).reshape(-1) for p in params]
        bm, bv = (f64(t) for t in opt.moments())
        opt.step(grads)
        fm, fv = (f64(t) for t in opt.moments())
        off = total = 0
        for i, p in enumerate(params):
            at = slice(opt.offsets[i], opt.offsets[i] + p.numel())
            g = f64(grads[i]).reshape(-1)
            wp, wm, wv = step64(opt, i, before[i], g, bm[at], bv[at], 0.05)
            # the step itself uses the unrounded moments: fp32's tolerance
            move = np.abs(wp - before[i]) + opt.lr * 4
            tol = 2 * U * np.abs(wp) + 64 * U * move + (2.0 ** -8 * np.abs(wp) if kind == "bf16" else 0)
            assert np.all(np.abs(f64(p).reshape(-1) - wp) <= tol), (k, i)
            if not p.numel():
                continue
            for got, want, root in ((fm[at], wm, False), (np.sqrt(fv[at]), np.sqrt(wv), True)):
                q, scale = ora.pack(want, root)
                q, unit = ora.unpack(q, scale), np.repeat(scale, 256)[:p.numel()]
                near = np.abs(got - q) <= 8 * U * np.abs(q)
                neighbour = np.abs(got - q) <= (2.0 ** -3 + 1e-6) * np.abs(q) + 2.0 ** -9 * unit * (1 + 1e-6)
                assert np.all(near | neighbour), (k, i, root)
                off += int((~near).sum())
                total += near.size
                if root:
                    assert np.all(got[(want > 0) & (unit > 0)] > 0)
        # a few u on either side of a boundary, 8 boundaries an octave: about 6e-6 of the elements; ties of
        # bf16 gradients: at most 1 element in 16 of such blocks
        assert off <= (2 + 4e-5 * total if gkind == "fp32" else total / 16), off


def test_8_bit_first_step_has_the_sign_of_the_gradient():
    """After one step every element has moved by about lr against its gradient, however small it is
    beside its block's largest: m and the root are used unrounded, and a stored root is never 0."""
    g = (torch.exp(torch.linspace(-30, 0, 1024, device=DEV)) * torch.tensor([1.0, -1.0], device=DEV).repeat(512))
    p = torch.zeros(1024, device=DEV)
    opt = vn.AdamW([p], lr=0.01, betas=(0.9, 0.999), eps=0.0, weight_decay=0.0, state_bits=8)
    opt.step([g])
    assert torch.allclose(p, -0.01 * torch.sign(g), rtol=1e-5)
    opt.step([g])
    _, v = opt.moments()
    assert bool((v > 0).all()) and bool(torch.isfinite(p).all())


def test_flat_gradient_equals_the_list():
    a, grads = make([(40, 64), (40,), (7, 40), (7,)], "fp32", "fp32", seed=2)
    b = [p.clone() for p in a]
    o1, o2 = vn.AdamW(a, **HYPER), vn.AdamW(b, **HYPER)
    o1.step(grads)
    o2.step(torch.cat([g.reshape(-1) for g in grads]))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert all(torch.equal(p, q) for p, q in zip(o1.moments(), o2.moments()))


@pytest.mark.parametrize("bits", [8, 32])
def test_views_of_one_vector_at_odd_offsets(bits):
    """Parameters that are views of a flat vector, off the vector loads' boundaries: the same bits."""
    shapes = [(3, 7), (3,), (301, 3), (301,)]
    p1, grads = make(shapes, "fp32", "fp32", seed=3)
    flat = torch.cat([p.reshape(-1) for p in p1])
    p2, at = [], 0
    for s in shapes:
        n = int(np.prod(s))
        p2.append(flat[at:at + n].view(s))
        at += n
    o1, o2 = vn.AdamW(p1, **HYPER, state_bits=bits), vn.AdamW(p2, **HYPER, state_bits=bits)
    for _ in range(2):
        o1.step(grads)
        o2.step(torch.cat([g.reshape(-1) for g in grads]))
    assert all(torch.equal(a, b) for a, b in zip(p1, p2))
    assert all(torch.equal(a, b) for a, b in zip(o1.moments(), o2.moments()))


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("count", [1, 16, 17, 448, 449, 1000])
def test_many_tensors(count, bits):
    """Across the kernels' table sizes and several launches: each tensor as if it were alone."""
    g = torch.Generator().manual_seed(count)
    sizes = [int(s) for s in torch.randint(1, 700, (count,), generator=g)]
    params = [torch.randn(s, generator=g).to(DEV) for s in sizes]
    grads = [torch.randn(s, generator=g).to(DEV) for s in sizes]
    alone = {i: params[i].clone() for i in {0, count // 2, count - 1}}
    vn.AdamW(params, **HYPER, state_bits=bits).step(grads)
    for i, p in alone.items():
        vn.AdamW([p], **HYPER, state_bits=bits).step([grads[i]])
        assert torch.equal(p, params[i]), i


@pytest.mark.parametrize("bits", [8, 32])
def test_resume_from_state(bits):
    a, grads = make([(50, 30), (50,)], "fp32", "fp32", seed=4)
    b = [p.clone() for p in a]
    o1 = vn.AdamW(a, **HYPER, state_bits=bits)
    for _ in range(4):
        o1.step(grads)
    o2 = vn.AdamW(b, **HYPER, state_bits=bits)
    o2.step(grads)
    o2.step(grads)
    state = {k: t.view(torch.uint8).clone().view(t.dtype) for k, t in o2.state.items()}
    o3 = vn.AdamW(b, **HYPER, state_bits=bits, state=state, step=o2.steps)
    o3.step(grads)
    o3.step(grads)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_not_finite_gradients():
    """32 bits: the element alone. 8 bits: its block's moments, and no other block."""
    for bits in (32, 8):
        p = torch.ones(1024, device=DEV)
        g = torch.ones(1024, device=DEV)
        g[300] = float("nan")
        g[800] = float("inf")
        opt = vn.AdamW([p], **HYPER, state_bits=bits)
        opt.step([g])
        m, v = opt.moments()
        bad = ~torch.isfinite(m)
        want = torch.zeros(1024, dtype=torch.bool, device=DEV)
        if bits == 32:
            want[[300, 800]] = True
        else:
            want[256:512] = True
            want[768:] = True
        assert torch.equal(bad, want)
        assert torch.isfinite(p).sum() == 1022


def test_hyperparameters_of_one_step():
    p, q = torch.ones(10, device=DEV), torch.ones(10, device=DEV)
    g = torch.full((10,), 0.5, device=DEV)
    vn.AdamW([p], lr=0.1, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0).step([g])
    assert torch.allclose(p, torch.full_like(p, 0.9), rtol=1e-6)
    opt = vn.AdamW([q], lr=0.1, betas=(0.9, 0.999), eps=0.0, weight_decay=0.5)
    opt.step([g], lr=0.2)
    assert torch.allclose(q, torch.full_like(q, 0.9 - 0.2), rtol=1e-5)
    z = torch.ones(10, device=DEV)
    vn.AdamW([z], lr=0.1, eps=1e-8, weight_decay=0.0).step([torch.zeros(10, device=DEV)])
    assert torch.equal(z, torch.ones(10, device=DEV))


def test_refusals():
    p = torch.ones(8, device=DEV)
    with pytest.raises(ValueError):
        vn.AdamW([])
    with pytest.raises(ValueError):
        vn.AdamW([torch.ones(8)])
    with pytest.raises(ValueError):
        vn.AdamW([torch.ones(8, 8, device=DEV).t()[1:]])
    with pytest.raises(TypeError):
        vn.AdamW([p, p.bfloat16()])
    with pytest.raises(TypeError):
        vn.AdamW([p.double()])
    with pytest.raises(ValueError):
        vn.AdamW([p], state_bits=16)
    with pytest.raises(ValueError):
        vn.AdamW([p], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError):
        vn.AdamW([p], state={"m": torch.zeros(8, device=DEV)})
    opt = vn.AdamW([p])
    with pytest.raises(ValueError):
        opt.step([])
    with pytest.raises(ValueError):
        opt.step([torch.ones(9, device=DEV)])
    with pytest.raises(ValueError):
        opt.step(torch.ones(9, device=DEV))
    with pytest.raises(TypeError):
        opt.step([torch.ones(8, device=DEV).double()])
    with pytest.raises(vn.VNError):
        opt.step([p])                      # the gradient over the parameters
    with pytest.raises(vn.VNError):
        vn.AdamW([p], betas=(1.0, 0.9)).step([torch.ones(8, device=DEV)])
    with pytest.raises(vn.VNError):
        vn.AdamW([p], eps=-1.0).step([torch.ones(8, device=DEV)])
    with pytest.raises(vn.VNError):
        opt.step([torch.ones(8, device=DEV)], lr=float("nan"))
    assert opt.steps == 0 and torch.equal(p, torch.ones(8, device=DEV))


def _codes(x, root):
    """The stored form of a flat moment in torch's fp32 operations, one rounding each."""
    x = torch.nn.functional.pad(x, (0, -x.numel() % 256)).view(-1, 256)
    top = x.abs().amax(1, keepdim=True)
    scale = torch.where(top < 1e-30, torch.zeros_like(top), top * (1.0 / 448.0))
    q = torch.where(scale == 0, torch.zeros_like(x), x * (torch.ones_like(scale) / scale))
    q = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    if root:
        q = torch.where((q == 0) & (x > 0) & (scale > 0), torch.full_like(x, 2.0 ** -9), q)
    return q, scale


@pytest.mark.parametrize("maximize", [False, True])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [256 * 700, 256 * 700 + 19])
def test_8_bit_codes_are_those_of_single_roundings(n, kind, maximize):
    """Every operation on the way to a code is one fp32 rounding, so that the codes follow from the
    formulas alone: bit for bit what torch's separate operations give, on aligned and ragged tensors."""
    g = torch.Generator(device=DEV).manual_seed(n)
    p = torch.randn(n, generator=g, device=DEV).to(KINDS[kind])
    opt = vn.AdamW([p], lr=1e-3, betas=(0.9, 0.999), state_bits=8, maximize=maximize)
    for _ in range(3):
        s = opt.state
        scale = lambda k: s[k].repeat_interleave(256)
        m = s["m"].float() * scale("m_scale")
        r = s["v"].float() * scale("v_scale")
        gr = (torch.randn(n, generator=g, device=DEV) * torch.exp(3 * torch.randn(n, generator=g, device=DEV))).to(KINDS[kind])
        opt.step([gr])
        f = gr.float() * (-1.0 if maximize else 1.0)
        m = m[:n] * 0.9 + f * (1 - 0.9)
        v = (r * r)[:n] * 0.999 + (f * f) * (1 - 0.999)
        for key, x, root in (("m", m, False), ("v", torch.sqrt(v), True)):
            q, unit = _codes(x, root)
            assert torch.equal(opt.state[key].float()[:n], q.view(-1)[:n]), key
            assert torch.equal(opt.state[key + "_scale"], unit.view(-1)), key
        em, ev = opt.moments()
        assert torch.equal(em, opt.state["m"].float() * opt.state["m_scale"].repeat_interleave(256))
        er = opt.state["v"].float() * opt.state["v_scale"].repeat_interleave(256)
        assert torch.equal(ev, er * er)
