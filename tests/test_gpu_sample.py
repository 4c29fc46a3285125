"""Drawing an index from logits on the GPU against the float64 oracle.

Indices have to be equal: weights good to 2^-35 and sums that are exact leave a chance below 1e-6 that one of a test's
random numbers lies between the two sides' borders. Log-probabilities: a distance of logits over the temperature and a
logarithm, each a few fp32 roundings (u = 2^-24): 8u of the sum of their sizes."""

import math

import numpy as np
import pytest
import torch

from oracle import acting as ora
import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300 import VNError
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16}
FILTERS = [
    {},
    dict(temperature=0.7),
    dict(temperature=1.3, top_k=1),
    dict(top_k=5),
    dict(temperature=0.9, top_p=0.9),
    dict(min_p=0.05),
    dict(temperature=1.5, top_k=40, top_p=0.8, min_p=0.02),
    dict(temperature=0.0),
    dict(temperature=2.5, top_p=0.999),
    dict(top_p=0.0),
    dict(min_p=1.0),
    dict(top_k=3, top_p=0.5),
]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def logits(rows, n, kind, seed=0, scale=2.5, masked=0.1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g) * scale
    x[torch.rand(rows, n, generator=g) < masked] = -math.inf
    x[:, n // 2] = torch.randn(rows, generator=g)
    return x.to(KINDS[kind]), torch.rand(rows, generator=g)


def row_filters(filters, i):
    return {k: (v[i].item() if isinstance(v, torch.Tensor) else v) for k, v in filters.items() if v is not None}


def check(x, u, filters, got=None):
    """x and u on the CPU, of any leading shape."""
    there = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in filters.items()}
    index, logp = got or vn.sample(x.to(DEV), u.to(DEV), logprobs=True, **there)
    assert index.shape == u.shape and index.dtype == torch.int64 and logp.shape == u.shape and logp.dtype == torch.float32
    xs, us = x.double().reshape(-1, x.shape[-1]).numpy(), u.double().reshape(-1).numpy()
    index, logp = index.reshape(-1).cpu().numpy(), logp.reshape(-1).double().cpu().numpy()
    for r in range(us.size):
        f = row_filters(filters, r)
        want, want_logp = ora.sample(xs[r], us[r], **f)
        assert index[r] == want, (r, index[r], want, f)
        if want < 0:
            assert math.isnan(logp[r])
            continue
        t = f.get("temperature", 1.0)
        far = (xs[r].max() - xs[r][want]) / t if t > 0 and math.isfinite(xs[r].max()) else 0.0
        assert abs(logp[r] - want_logp) <= 8 * U * (far + abs(want_logp + far)) + 1e-12, (r, logp[r], want_logp)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 200, 256, 257, 300, 1000, 1021, 2048, 4096, 4097])
def test_sizes(n, kind):
    for i, f in enumerate(FILTERS):
        x, u = logits(9, n, kind, seed=i)
        check(x, u, f)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [8192, 20011, 65536, 131071])
def test_long_rows(n, kind):
    for i, f in enumerate(FILTERS):
        if i % 2 == 0 or n < 50000:
            x, u = logits(2, n, kind, seed=10 + i)
            check(x, u, f)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_the_longest_row(kind):
    x, u = logits(1, 524288, kind, seed=30)
    check(x, u, dict(temperature=1.1))
    check(x, u, dict(temperature=0.8, top_k=1000, top_p=0.9))
    check(x[:, 1:], u, dict(top_p=0.95))  # no row on a vector load's boundary: a word more


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,n", [(5001, 3), (4099, 8), (2049, 13), (3000, 100), (700, 256), (600, 513), (310, 1021), (160, 4096), (80, 9001), (150, 40000)])
def test_many_rows(rows, n, kind):
    x, u = logits(rows, n, kind, seed=40)
    check(x, u, dict(temperature=0.8, top_p=0.95))
    check(x, u, dict(temperature=1.2, top_k=n // 3 + 1, min_p=0.01))


def check_repeated(x, u, filters, times):
    """As many rows as run with one or two warps each: `times` copies of x, of which one is compared and the others have to be like
    it. Copies start at other places within 16 bytes, so their fp32 sums are of other groups: each log-probability is within
    check()'s bound of the oracle's, and two of them within twice that."""
    rows = u.numel()
    there = {k: v.repeat(times).to(DEV) if isinstance(v, torch.Tensor) else v for k, v in filters.items()}
    index, logp = vn.sample(x.repeat(times, 1).to(DEV), u.repeat(times).to(DEV), logprobs=True, **there)
    check(x, u, filters, (index[:rows], logp[:rows]))
    index, logp = index.view(times, rows).cpu(), logp.double().view(times, rows).cpu()
    assert torch.equal(index, index[:1].expand(times, rows))
    t = torch.as_tensor(filters.get("temperature", 1.0), dtype=torch.float64).expand(rows)
    top = x.double().max(-1).values
    far = (top - x.double().gather(1, index[0].clamp(min=0)[:, None])[:, 0]) / t
    far = torch.where((t > 0) & top.isfinite() & (index[0] >= 0), far, 0.0)
    assert torch.equal(logp.isnan(), (index < 0))
    off = (logp - logp[:1]).nan_to_num(0.0).abs()
    assert (off <= 16 * U * (far + (logp[:1].nan_to_num(0.0) + far).abs()) + 2e-12).all()


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [257, 600, 640, 1021, 1284, 2048, 2051, 3001, 4096])
def test_rows_side_by_side(n, kind):
    for i, f in enumerate(FILTERS):
        x, u = logits(12, n, kind, seed=200 + i)
        check_repeated(x, u, f, 320)
    x, u = logits(12, n, kind, seed=220)
    g = torch.Generator().manual_seed(221)
    check_repeated(x, u, dict(temperature=torch.rand(12, generator=g) * 2, top_k=torch.randint(0, n + 2, (12,), generator=g),
                              top_p=torch.rand(12, generator=g) * 1.2, min_p=torch.rand(12, generator=g) * 0.2), 320)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [300, 1021, 2051])
def test_rows_side_by_side_with_ties_and_extreme_values(n, kind):
    for seed in range(3):
        x, u = logits(12, n, kind, seed=230 + seed)
        x = (x * 2).round() / 2
        x[0] = 1.0
        x[1, 5] = math.nan
        x[2] = -math.inf
        x[3, 7::11] = math.inf
        x[4, 1:] = -math.inf
        x[5] *= 1e30
        for f in ({}, dict(top_k=max(1, n // 5)), dict(top_p=0.37), dict(temperature=0.5, top_k=n // 2 + 1, top_p=0.61),
                  dict(top_k=3, top_p=0.4, min_p=0.2), dict(temperature=0.0), dict(min_p=0.3)):
            check_repeated(x, u, f, 320)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [4, 7, 16, 40, 256, 300, 5000])
def test_ties(n, kind):
    """Logits of few values: the borders of the filters fall among equal ones, the lower indices of which are kept."""
    for seed in range(6):
        x, u = logits(8, n, kind, seed=50 + seed)
        x = (x * 2).round() / 2
        x[0] = 1.0
        for f in (dict(top_k=max(1, n // 5)), dict(top_p=0.37), dict(temperature=0.5, top_k=n // 2 + 1, top_p=0.61),
                  dict(top_k=3, top_p=0.4, min_p=0.2), dict(temperature=0.0), dict(min_p=0.3)):
            check(x, u, f)


def test_more_kept_than_there_are_finite_logits():
    """The border of top-k among the logits of -infinity, far below the finite ones in the order of their bits."""
    for n in (300, 1021, 5000):
        x, u = logits(6, n, "fp32", seed=55, masked=0.6)
        for f in (dict(temperature=0.07, top_k=n * 3 // 4), dict(temperature=1.0, top_k=n - 1, top_p=0.9)):
            check(x, u, f)


@pytest.mark.parametrize("n", [10, 1000])
def test_zeros_of_both_signs_are_equal(n):
    x = torch.full((2, n), -3.0)
    x[:, 3::2] = -0.0
    x[:, 6::4] = 0.0
    u = torch.tensor([0.1, 0.9])
    for f in (dict(temperature=0.0), dict(top_k=2), dict(top_p=0.3), dict(min_p=1.0)):
        check(x, u, f)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [4, 5, 16, 300, 4096])
def test_rows_without_an_answer_and_extreme_values(n, kind):
    low = torch.finfo(KINDS[kind]).min
    x, u = logits(12, n, kind, seed=60)
    x[0] = -math.inf
    x[1, n - 1] = math.nan
    x[2, 0], x[2, n - 1] = math.inf, math.inf
    x[3] = low
    x[4] = low
    x[4, n - 2] = 0.0
    x[5] = -math.inf
    x[5, 1] = -7.0
    x[6, 0] = torch.finfo(KINDS[kind]).max
    x[7] = 0.0
    x[8] = torch.finfo(KINDS[kind]).tiny
    x[8, 2] = 0.0
    x[9, ::2] = low
    x[10] = math.inf
    x[11] = -x[11].abs() - 50
    for f in FILTERS:
        check(x, u, f)


@pytest.mark.parametrize("n", [6, 70, 300, 6000])
def test_random_numbers_at_the_ends(n):
    x, _ = logits(6, n, "fp32", seed=70, masked=0.4)
    x = x[:1].expand(6, n).clone()
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 3.0, -1.0, 1e-30])
    for f in ({}, dict(top_p=0.8), dict(top_k=2, temperature=0.3)):
        check(x, u, f)
    u[2] = math.nan
    assert vn.sample(x.to(DEV), u.to(DEV)).tolist()[2] == -1


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [3, 8, 13, 20, 256, 1021, 4096])
def test_parameters_of_each_row(n, kind):
    rows = 60
    x, u = logits(rows, n, kind, seed=80)
    g = torch.Generator().manual_seed(81)
    f = dict(temperature=torch.rand(rows, generator=g) * 2, top_k=torch.randint(0, n + 2, (rows,), generator=g),
             top_p=torch.rand(rows, generator=g) * 1.2, min_p=torch.rand(rows, generator=g) * 0.2)
    f["temperature"][:3] = torch.tensor([0.0, -1.0, 1e30])
    f["min_p"][::4] = 0.0
    f["min_p"][5] = 1.0
    f["top_p"][6] = 0.0
    check(x, u, f)
    for name in ("temperature", "top_p", "min_p"):
        bad = dict(f)
        bad[name] = f[name].clone()
        bad[name][7] = math.nan
        check(x, u, bad)


def test_temperatures_at_the_ends_of_their_range():
    x, u = logits(4, 400, "fp32", seed=90, masked=0.0)
    for t in (1e-30, 1e-3, 1e3, 1e30):
        check(x, u, dict(temperature=t))
    index = vn.sample(x.to(DEV), u.to(DEV), temperature=torch.full((4,), math.inf, device=DEV))
    assert index.tolist() == [int(v * 400) for v in u.double().tolist()]


@pytest.mark.parametrize("n", [8, 200, 700])
def test_shares(n):
    """Random numbers spread evenly draw each index in proportion to its weight, to within one."""
    x, _ = logits(1, n, "fp32", seed=100)
    count = 20000
    u = (torch.arange(count, dtype=torch.float64) + 0.5) / count
    f = dict(temperature=0.9, top_k=n // 2, top_p=0.97)
    index = vn.sample(x.to(DEV).expand(count, n), u.float().to(DEV), **f).cpu()
    w = ora.keep(x[0].double().numpy(), **f)
    counts = np.bincount(index.numpy(), minlength=n)
    assert np.all(np.abs(counts - w / w.sum() * count) <= 1.01)


def test_shapes_strides_and_buffers():
    x, u = logits(24, 50, "fp32", seed=110)
    want = vn.sample(x.to(DEV), u.to(DEV), top_p=0.9)
    assert torch.equal(vn.sample(x.to(DEV).view(4, 6, 50), u.to(DEV).view(4, 6), top_p=0.9), want.view(4, 6))
    wide = torch.zeros(24, 101, device=DEV)
    wide[:, 1::2] = x.to(DEV)
    assert torch.equal(vn.sample(wide[:, 1::2], u.to(DEV), top_p=0.9), want)
    out = torch.full((24,), -5, dtype=torch.int64, device=DEV)
    assert vn.sample(x.to(DEV), u.to(DEV), top_p=0.9, out=out) is out and torch.equal(out, want)
    one = vn.sample(x[3].to(DEV), u[3].to(DEV), top_p=0.9)
    assert one.shape == () and one == want[3]
    assert vn.sample(torch.empty(0, 7, device=DEV), torch.empty(0, device=DEV)).shape == (0,)
    flat = torch.zeros(24 * 4001 + 3, device=DEV)
    for kind in ("fp32", "bf16"):
        for n in (100, 4001):
            x, u = logits(24, n, kind, seed=111)
            for shift in (1, 3):
                there = flat.to(KINDS[kind])[shift:shift + 24 * n].view(24, n)
                there.copy_(x)
                check(x, u, dict(top_k=30, top_p=0.9), vn.sample(there, u.to(DEV), top_k=30, top_p=0.9, logprobs=True))


def test_streams_and_graphs():
    x, u = logits(300, 1000, "bf16", seed=120)
    x, u = x.to(DEV), u.to(DEV)
    want = vn.sample(x, u, top_k=50, top_p=0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = vn.sample(x, u, top_k=50, top_p=0.9)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    t = torch.full((300,), 0.8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        index, logp = vn.sample(x, u, temperature=t, top_p=0.9, logprobs=True)
    for temperature in (0.8, 0.0, 1.4):
        t.fill_(temperature)
        u.uniform_()
        graph.replay()
        check(x.cpu(), u.cpu(), dict(temperature=t.cpu(), top_p=0.9), (index, logp))


def test_a_population_acts():
    """A policy's logits, as the population's forward gives them, become an action for each individual."""
    g = torch.Generator().manual_seed(130)
    ws = [torch.randn(32, 12, generator=g).to(DEV), torch.randn(8, 32, generator=g).to(DEV) * 0.3]
    x = torch.randn(5, 12, generator=g).to(DEV)
    seeds = torch.arange(64, device=DEV)
    out = vn.virtual_perturbed_mlp(x, ws, None, seeds, 0.1)
    u = torch.rand(64, 5, generator=g)
    check(out.cpu(), u, dict(temperature=0.5, top_k=4))


def test_refusals():
    x, u = torch.zeros(4, 9, device=DEV), torch.zeros(4, device=DEV)
    for call in (lambda: vn.sample(x.double(), u), lambda: vn.sample(x, u.double()), lambda: vn.sample(x, u, top_k=2.5),
                 lambda: vn.sample(x, u, temperature=u.double()), lambda: vn.sample(x, u, top_k=u)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: vn.sample(x.cpu(), u), lambda: vn.sample(x, u.cpu()), lambda: vn.sample(x, u[:3]),
                 lambda: vn.sample(x[:, :0], u), lambda: vn.sample(x, u, top_p=u[:2]),
                 lambda: vn.sample(x, u, out=torch.empty(4, device=DEV)),
                 lambda: vn.sample(x, u, out=torch.empty(4, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: vn.sample(x, u, temperature=math.nan), lambda: vn.sample(x, u, temperature=math.inf),
                 lambda: vn.sample(x, u, top_p=math.nan), lambda: vn.sample(x, u, min_p=math.inf)):
        with pytest.raises(VNError, match="VN_ERR_VALUE"):
            call()
    with pytest.raises(VNError, match="VN_ERR_SHAPE"):
        vn.sample(torch.zeros(1, 524289, device=DEV), u[:1])
    both = torch.zeros(16, device=DEV)
    with pytest.raises(VNError, match="VN_ERR_VALUE"):
        vn.sample(x, both[:4], out=both.view(torch.int64)[:4])
