"""AdamW's handle: what it holds, and what happens to it beside its steps."""

import copy
import io
import pickle

import pytest
import torch

import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def make(bits, seed=0):
    g = torch.Generator().manual_seed(seed)
    params = [torch.randn(s, generator=g).to(DEV) for s in ((70, 30), (70,), (5, 70))]
    grads = [torch.randn(p.shape, generator=g).to(DEV) for p in params]
    return vn.AdamW(params, lr=1e-2, weight_decay=[0.1, 0.0, 0.2], state_bits=bits, maximize=True), grads


def bits_of(opt):
    return [t.clone() for t in opt.params] + [t.view(torch.uint8).clone() for _, t in sorted(opt.state.items())]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def saved(opt):
    f = io.BytesIO()
    torch.save(opt, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("twin", [copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o)), saved])
def test_a_copy_steps_on_its_own_tensors(twin, bits):
    opt, grads = make(bits)
    opt.step(grads)
    before = bits_of(opt)
    other = twin(opt)
    assert other.steps == 1 and same(bits_of(other), before)
    other.step(grads)
    assert same(bits_of(opt), before)                       # nothing of the first has moved
    after = bits_of(other)
    assert not any(torch.equal(p, q) for p, q in zip(after[:3], before[:3])) and not same(after[3:], before[3:])
    assert same([t.reshape(-1) for t in other.moments()], [t.reshape(-1) for t in saved(other).moments()])
    opt.step(grads)
    assert same(bits_of(opt), after) and opt.steps == other.steps == 2
    del opt
    other.step(grads)                                       # the first is gone
    third, _ = make(bits)
    for _ in range(3):
        third.step(grads)
    assert same(bits_of(other), bits_of(third))


def test_a_copy_of_a_policy_and_its_handle_keep_their_views():
    """Parameters that are views of one vector stay views of one vector in a deep copy of both."""
    flat = torch.arange(600, dtype=torch.float32, device=DEV)
    opt = vn.AdamW([flat[:256].view(16, 16), flat[300:]], lr=0.1)
    flat2, opt2 = copy.deepcopy((flat, opt))
    opt2.step([torch.ones(16, 16, device=DEV), torch.ones(300, device=DEV)])
    assert torch.equal(flat, torch.arange(600, dtype=torch.float32, device=DEV))
    assert bool((flat2[:256] != flat[:256]).all()) and torch.equal(flat2[256:300], flat[256:300])


def test_a_handle_loaded_off_the_gpu_is_refused():
    f = io.BytesIO()
    torch.save(make(32)[0], f)
    f.seek(0)
    with pytest.raises(ValueError, match="CUDA"):
        torch.load(f, weights_only=False, map_location="cpu")


@pytest.mark.parametrize("bits", [8, 32])
def test_a_step_is_not_captured(bits):
    """Replays would repeat the capture's step number: refused, and neither counted nor launched."""
    opt, grads = make(bits)
    opt.step(grads)
    before = bits_of(opt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            opt.step(grads)
        kept = grads[0] + 1                                 # the capture itself goes on
    graph.replay()
    torch.cuda.synchronize()
    assert opt.steps == 1 and same(bits_of(opt), before) and torch.equal(kept, grads[0] + 1)
    opt.step(grads)
    assert opt.steps == 2


def test_autograd_notices_a_step_between_forward_and_backward():
    w = torch.ones(4, 4, device=DEV, requires_grad=True)
    x = torch.ones(4, 4, device=DEV, requires_grad=True)
    loss = (x @ w).sum()
    vn.AdamW([w]).step([torch.ones(4, 4, device=DEV)])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        frozen = torch.ones(4, device=DEV)
    vn.AdamW([frozen]).step([torch.ones(4, device=DEV)])
    assert bool((frozen < 1).all())


def test_autograd_notices_an_output_buffer_written_over():
    a, b = torch.ones(3, 8, device=DEV), torch.ones(4, 8, device=DEV)
    for write in (lambda out: vn.linear(a, b, out=out), lambda out: vn.layer_norm(torch.ones(3, 4, device=DEV), out=out)):
        out = torch.ones(3, 4, device=DEV)
        scale = torch.ones(3, 4, device=DEV, requires_grad=True)
        loss = (scale * out).sum()
        write(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_tensors_that_share_memory_are_refused():
    flat = torch.ones(2048, device=DEV)
    m, v = torch.zeros(1024, device=DEV), torch.zeros(1024, device=DEV)
    for params in ([flat[:10], flat[:10]], [flat[5:20], flat[:6]], [flat[:100], flat[50:60], flat[200:]]):
        with pytest.raises(ValueError, match="share memory"):
            vn.AdamW(params)
    for state in ({"m": m, "v": m}, {"m": flat[:1024], "v": v}, {"m": flat[1023:2047], "v": v}):
        with pytest.raises(ValueError, match="share memory"):
            vn.AdamW([flat[:1024]], state=state)
    vn.AdamW([flat[:10], flat[10:20], flat[20:20], flat[15:15], flat[20:]])
    vn.AdamW([flat[:1024]], state={"m": flat[1024:], "v": v})
