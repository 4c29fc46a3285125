"""What is measured of the operators between training the centre network and acting with it: the norm
of a gradient over many tensors with clipping, weights packed to 4 bits with group scales and the linear
layer on them, and sampling from logits with temperature, top-k, top-p and min-p.

A gradient, of the centre network or the population's estimate, is clipped on its way into AdamW; the
trained layers are packed and answer single observations; the policy's logits become actions. Sizes
are those of the package's workloads (widths 8, 64, 256, 1024 and 4096, populations of 1,024 to 16,384),
odd neighbours of them, and vocabularies.

``run`` computes each operator in elementary torch operations where ``own`` is false, and through the
package's entry points where it is true.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ACTS = ("none", "tanh", "relu", "gelu", "silu")
_BLOCK = 256                 # a tensor's moments start on a multiple of this many elements
_BETA1, _BETA2, _EPS, _LR, _DECAY, _STEPS = 0.9, 0.999, 1e-8, 1e-3, 0.01, 37


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # One observation's action among 4,096, with every filter: latency counts.
        {"name": "sample one observation", "op": "sample", "rows": 1, "n": 4096, "type": "bf16", "temperature": 0.8,
         "top_k": 50, "top_p": 0.95, "min_p": 0.02, "per_row": False, "logprobs": False},
        # An action among eight for each of 1,024 environments, with its probability for the learner.
        {"name": "sample environments", "op": "sample", "rows": 1024, "n": 8, "type": "fp32", "temperature": 1.0,
         "top_k": 0, "top_p": 1.0, "min_p": 0.0, "per_row": False, "logprobs": True},
        # A whole population over 4,096 actions, each individual with a temperature and a nucleus of its own.
        {"name": "sample population", "op": "sample", "rows": 16384, "n": 4096, "type": "bf16", "temperature": 0.9,
         "top_k": 0, "top_p": 0.9, "min_p": 0.0, "per_row": True, "logprobs": True},
        # A few rows over a vocabulary whose odd size leaves no row on a vector load's boundary.
        {"name": "sample vocabulary", "op": "sample", "rows": 32, "n": 131071, "type": "fp32", "temperature": 0.7,
         "top_k": 100, "top_p": 0.95, "min_p": 0.0, "per_row": False, "logprobs": False},
        # The policy's six gradients clipped into buffers of their own: launches count.
        {"name": "clip policy", "op": "clip", "layers": 3, "in": 64, "width": 256, "out": 8, "type": "fp32", "limit": 0.5},
        # The large network's gradients, with an odd last layer.
        {"name": "clip large", "op": "clip", "layers": 4, "in": 4096, "width": 4096, "out": 1021, "type": "bf16",
         "limit": 0.25},
        # A clipped step of the policy's parameters, and of the large network's.
        {"name": "clipped step policy", "op": "step", "layers": 3, "in": 64, "width": 256, "out": 8, "type": "fp32",
         "grad": "fp32", "maximize": True, "limit": 0.5},
        {"name": "clipped step large", "op": "step", "layers": 4, "in": 4096, "width": 4096, "out": 4096, "type": "bf16",
         "grad": "bf16", "maximize": False, "limit": 0.25},
        # Packing an odd layer, and a large one, with the values that come out of it again.
        {"name": "pack odd", "op": "pack", "out": 1021, "in": 1003, "type": "fp32", "group": 32},
        {"name": "pack large", "op": "pack", "out": 16384, "in": 4096, "type": "bf16", "group": 128},
        # Acting on one observation with the large network's packed layer: its codes are read once.
        {"name": "linear4 one observation", "op": "linear4", "rows": 1, "in": 4096, "out": 4096, "type": "bf16",
         "group": 64, "act": "gelu", "bias": True, "residual": True},
        # A handful of observations, odd sizes, in fp32.
        {"name": "linear4 handful", "op": "linear4", "rows": 5, "in": 4093, "out": 4099, "type": "fp32", "group": 32,
         "act": "tanh", "bias": True, "residual": False},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm; odd ones, multiples of 8 and of 64 all occur."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.random()
    if kind < 0.3 and v >= 64:
        v -= v % 64
    elif kind < 0.6 and v >= 8:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("sample", "sample", "sample", "clip", "step", "pack", "linear4", "linear4"))
    kind = rng.choice(("bf16", "fp32"))
    if op == "sample":
        n = _spread(rng, 2, 131072)
        return {"op": op, "rows": _spread(rng, 1, max(1, min(65536, 2 ** 25 // n))), "n": n, "type": kind,
                "temperature": rng.choice((0.0, 1.0, round(rng.uniform(0.3, 1.7), 3), round(rng.uniform(0.3, 1.7), 3))),
                "top_k": rng.choice((0, 0, 1, _spread(rng, 2, 200), _spread(rng, 1, n))),
                "top_p": rng.choice((1.0, 1.0, 0.95, round(rng.uniform(0.05, 0.99), 3))),
                "min_p": rng.choice((0.0, 0.0, round(rng.uniform(0.001, 0.3), 4))),
                "per_row": rng.random() < 0.3, "logprobs": rng.random() < 0.5}
    if op == "linear4":
        return {"op": op, "rows": _spread(rng, 1, 256), "in": _spread(rng, 8, 4096), "out": _spread(rng, 8, 4096),
                "type": kind, "group": rng.choice((32, 64, 128)), "act": rng.choice(_ACTS),
                "bias": rng.random() < 0.75, "residual": rng.random() < 0.5}
    if op == "pack":
        return {"op": op, "out": _spread(rng, 1, 8192), "in": _spread(rng, 1, 8192), "type": kind,
                "group": rng.choice((32, 64, 128))}
    width = _spread(rng, 16, 4096)
    case = {"op": op, "layers": rng.randint(2, 3 if width > 2048 else 12), "in": _spread(rng, 8, 4096), "width": width,
            "out": _spread(rng, 1, 4096), "type": kind, "limit": rng.choice((0.1, 0.5, 1.5))}
    if op == "step":
        case.update(grad=rng.choice(("fp32", kind)), maximize=rng.random() < 0.5)
    return case


def _shapes(case):
    """Weight and bias of each layer, as the package lays a policy out."""
    sizes = [case["in"]] + [case["width"]] * (case["layers"] - 1) + [case["out"]]
    return [s for a, b in zip(sizes[:-1], sizes[1:]) for s in ((b, a), (b,))]


def _groups(case):
    return -(-case["in"] // case["group"])


def work(case):
    op = case["op"]
    size = _TYPES[case["type"]].itemsize
    if op == "sample":
        m, n = case["rows"], case["n"]
        return {"bytes": m * n * size + m * (4 + 8 + 4 * case["logprobs"] + 16 * case["per_row"]), "flops": 4 * m * n}
    if op == "linear4":
        m, k, n = case["rows"], case["in"], case["out"]
        packed = n * k / 2 + n * _groups(case) * size
        return {"bytes": int(packed + size * (m * k + n * case["bias"] + m * n * (1 + case["residual"]))),
                "flops": 2 * m * n * k}
    if op == "pack":
        n, k = case["out"], case["in"]
        return {"bytes": int(2 * n * k * size + 2 * n * k / 2 + 2 * n * _groups(case) * size), "flops": 4 * n * k}
    count = sum(math.prod(s) for s in _shapes(case))
    if op == "clip":
        return {"bytes": 2 * count * size, "flops": 3 * count}
    return {"bytes": (2 * size + _TYPES[case["grad"]].itemsize + 16) * count, "flops": 19 * count}


# ---------------------------------------------------------------- the inputs
def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, kind=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(kind)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    op, kind = case["op"], _TYPES[case["type"]]
    s = {"case": case}
    if op == "sample":
        m, n = case["rows"], case["n"]
        # Logits of differing sharpness, one action in twenty not allowed.
        x = normal(m, n) * (1 + 2 * uniform(m, 1))
        x = torch.where(uniform(m, n) < 0.05, torch.full_like(x, -math.inf), x)
        x[:, n // 2] = normal(m)
        s["x"], s["u"] = x.to(kind), uniform(m)
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = (case[k] for k in ("temperature", "top_k", "top_p", "min_p"))
        if case["per_row"]:
            s["temperature"] = (0.5 + uniform(m)) * case["temperature"]
            s["top_k"] = torch.randint(0, 2 * case["top_k"] + 1, (m,), generator=gen, device="cuda")
            s["top_p"] = 1 - uniform(m) * (1 - case["top_p"]) if case["top_p"] < 1 else torch.ones(m, device="cuda")
            s["min_p"] = uniform(m) * case["min_p"]
    elif op in ("pack", "linear4"):
        n, k = case["out"], case["in"]
        s["w"] = normal(n, k, scale=k ** -0.5, kind=kind)
        if op == "linear4":
            m = case["rows"]
            s["x"] = normal(m, k, kind=kind)
            s["b"] = normal(n, scale=0.1, kind=kind) if case["bias"] else None
            s["residual"] = normal(m, n, kind=kind) if case["residual"] else None
    else:
        shapes = _shapes(case)
        gkind = _TYPES[case.get("grad", case["type"])]
        # Entries of a gradient differ by orders of magnitude between rows.
        s["grads"] = [normal(*p, scale=1e-2).mul_(torch.exp(normal(p[0], *[1] * (len(p) - 1)))).to(gkind) for p in shapes]
        # The limit in units of what such a gradient's norm is expected to be.
        s["max_norm"] = case["limit"] * 1e-2 * math.e * math.sqrt(sum(math.prod(p) for p in shapes))
        if op == "clip":
            s["out"] = [torch.empty_like(g) for g in s["grads"]]
        else:
            s["params"] = [normal(*p, scale=p[-1] ** -0.5 if len(p) == 2 else 0.1, kind=kind) for p in shapes]
            s["decay"] = [_DECAY if len(p) == 2 else 0.0 for p in shapes]
            sizes = [math.prod(p) for p in shapes]
            padded = [-(-c // _BLOCK) * _BLOCK for c in sizes]
            s["offsets"] = [sum(padded[:i]) for i in range(len(padded))]
            s["total"] = sum(padded)
            s["step"] = _STEPS
            # Moments as earlier steps with such gradients leave them.
            live = torch.cat([torch.nn.functional.pad(torch.ones(c, device="cuda"), (0, p - c)) for c, p in zip(sizes, padded)])
            m = normal(s["total"], scale=3e-3) * live
            r = (normal(s["total"]).abs() * 1e-2 + 1e-3) * live
            s["m"], s["v"] = m, r * r
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear4":
        # The packed layer that a program keeps.
        if own:
            import virtual_noise_perturbed_gb300 as vn
            s["packed"] = vn.pack4(s["w"], group=case["group"])
        else:
            s["codes"], s["scales"] = _pack4(s["w"], case["group"])
        del s["w"]
    elif case["op"] == "step" and own:
        # The handle that a program keeps, over these same tensors.
        import virtual_noise_perturbed_gb300 as vn
        s["opt"] = vn.AdamW(s["params"], lr=_LR, betas=(_BETA1, _BETA2), eps=_EPS, weight_decay=s["decay"],
                            maximize=case["maximize"], state={"m": s["m"], "v": s["v"]}, step=_STEPS)
    return s


# ---------------------------------------------------------------- the plain forms
def _column(v, rows, kind):
    """A number, or one for each row, as a column in 64 bits."""
    return (v if isinstance(v, torch.Tensor) else torch.full((rows,), v, dtype=kind, device="cuda")).to(kind)[:, None]


def _plain_sample(s):
    # In 64 bits: a random number next to a border of two actions, or an action next to a filter's.
    x, u = s["x"].double(), s["u"].double()
    m, n = x.shape
    t, p, lowest = (_column(s[k], m, torch.float64) for k in ("temperature", "top_p", "min_p"))
    k = _column(s["top_k"], m, torch.int64)
    d = x - x.amax(1, keepdim=True)
    w = torch.where(t > 0, torch.exp(d / torch.where(t > 0, t, torch.ones_like(t))), (d == 0).double())
    k = torch.where(t > 0, torch.where((k <= 0) | (k > n), n, k), 1)
    _, order = torch.sort(x, dim=1, descending=True, stable=True)
    ws = torch.gather(w, 1, order)
    at = torch.arange(n, device=x.device)[None, :]
    ws = torch.where(at < k, ws, torch.zeros_like(ws))
    c = torch.cumsum(ws, 1)
    before = torch.cat([torch.zeros_like(c[:, :1]), c[:, :-1]], 1)
    keep = (at < k) & (ws >= lowest) & ((p >= 1) | (before < p * c[:, -1:]) | (at == 0))
    w = w * torch.zeros_like(keep).scatter_(1, order, keep)
    c = torch.cumsum(w, 1)
    i = (c <= u[:, None] * c[:, -1:]).sum(1, keepdim=True)
    i = torch.minimum(i, (c < c[:, -1:]).sum(1, keepdim=True))
    out = [i[:, 0]]
    if s["case"]["logprobs"]:
        out.append(torch.log(torch.gather(w, 1, i) / c[:, -1:])[:, 0].float())
    return out


def _pack4(w, group):
    """Codes of -7..7 and the scales that they are in units of, for each group of a row."""
    n, k = w.shape
    padded = torch.nn.functional.pad(w.float(), (0, -k % group)).view(n, -1, group)
    # In 64 bits: a weight next to the border of two codes.
    scales = (padded.abs().amax(2).double() / 7).to(w.dtype)
    unit = scales.double()[:, :, None]
    codes = torch.where(unit == 0, torch.zeros_like(unit), torch.round(padded.double() / unit).clamp(-7, 7))
    return codes.view(n, -1)[:, :k].to(torch.int8), scales


def _values4(codes, scales, group):
    return codes.float() * scales.float().repeat_interleave(group, 1)[:, :codes.shape[1]]


def _plain_pack(s):
    codes, scales = _pack4(s["w"], s["case"]["group"])
    return [_values4(codes, scales, s["case"]["group"]).to(s["w"].dtype), scales]


def _act(z, act):
    if act == "tanh":
        return torch.tanh(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain_linear4(s):
    z = s["x"].float() @ _values4(s["codes"], s["scales"], s["case"]["group"]).t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(s["x"].dtype)]


def _factor(s):
    """The norm, and what a gradient is multiplied by: a long sum, in 64 bits."""
    norm = torch.sqrt(sum((g.double() ** 2).sum() for g in s["grads"]))
    return norm.float(), torch.where(norm <= s["max_norm"], torch.ones_like(norm), s["max_norm"] / norm).float()


def _plain_clip(s):
    norm, factor = _factor(s)
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * factor)
    return s["out"] + [norm]


def _plain_step(s):
    s["step"] += 1
    t, case = s["step"], s["case"]
    norm, factor = _factor(s)
    m, v = s["m"], s["v"]
    g = torch.zeros_like(m)
    for o, q in zip(s["offsets"], s["grads"]):
        g[o:o + q.numel()] = q.float().reshape(-1) * factor
    g = -g if case["maximize"] else g
    m = m * _BETA1 + g * (1 - _BETA1)
    v = v * _BETA2 + (g * g) * (1 - _BETA2)
    move = m / (torch.sqrt(v) * (1 / math.sqrt(1 - _BETA2 ** t)) + _EPS) * (_LR / (1 - _BETA1 ** t))
    for o, p, decay in zip(s["offsets"], s["params"], s["decay"]):
        p.copy_(p.float() * (1 - _LR * decay) - move[o:o + p.numel()].view(p.shape))
    s["m"].copy_(m)
    s["v"].copy_(v)
    return s["params"] + [s["m"], s["v"], norm]


_PLAIN = {"sample": _plain_sample, "clip": _plain_clip, "step": _plain_step, "pack": _plain_pack, "linear4": _plain_linear4}


# ---------------------------------------------------------------- the package's operators
def _own(s):
    import virtual_noise_perturbed_gb300 as vn
    case = s["case"]
    op = case["op"]
    if op == "sample":
        out = vn.sample(s["x"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                        logprobs=case["logprobs"])
        return list(out) if case["logprobs"] else [out]
    if op == "clip":
        return s["out"] + [vn.clip_gradients(s["grads"], s["max_norm"], out=s["out"])]
    if op == "step":
        norm = s["opt"].step(s["grads"], max_norm=s["max_norm"])
        return s["params"] + list(s["opt"].moments()) + [norm]
    if op == "pack":
        packed = vn.pack4(s["w"], group=case["group"])
        return [packed.dequantize(), packed.scales]
    return [vn.linear4(s["x"], s["packed"], s["b"], activation=case["act"], residual=s["residual"])]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_sample(case, s):
    """Prefixes of the descending order are counted, then a random number is looked up in the sums of what is left."""
    x, u = s["x"].double(), s["u"].double()
    rows, n = x.shape
    full = lambda v: v.double() if isinstance(v, torch.Tensor) else torch.full((rows,), float(v), dtype=torch.float64, device=x.device)  # noqa: E731
    t, k, p, lowest = (full(s[name]) for name in ("temperature", "top_k", "top_p", "min_p"))
    index = torch.empty(rows, dtype=torch.int64, device=x.device)
    logp = torch.empty(rows, dtype=torch.float64, device=x.device)
    step = max(1, 2 ** 24 // n)
    for a in range(0, rows, step):
        e = slice(a, min(rows, a + step))
        order = torch.argsort(-x[e], dim=1, stable=True)
        z = x[e].gather(1, order) / torch.where(t[e] > 0, t[e], 1.0)[:, None]
        z = z - z[:, :1]
        prob = torch.softmax(z, 1)
        count = torch.where((k[e] < 1) | (k[e] > n), n, k[e].long())
        count = torch.where(t[e] > 0, count, 1)
        sums = torch.cumsum(prob, 1)
        total = sums.gather(1, count[:, None] - 1)
        # An action stays while those before it have not reached the nucleus: one more than the sums below it.
        nucleus = torch.searchsorted(sums, p[e, None] * total)[:, 0] + 1
        count = torch.where(p[e] < 1, torch.minimum(count, nucleus), count)
        floor = (z >= torch.log(lowest[e, None])).sum(1)
        count = torch.minimum(count, floor)
        place = torch.empty_like(order).scatter_(1, order, torch.arange(n, device=x.device).expand_as(order))
        prob = torch.where(place < count[:, None], torch.empty_like(prob).scatter_(1, order, prob), 0.0)
        sums = torch.cumsum(prob, 1)
        last = torch.searchsorted(sums, sums[:, -1:].contiguous())
        i = torch.minimum(torch.searchsorted(sums, u[e, None] * sums[:, -1:], right=True), last)
        index[e] = i[:, 0]
        logp[e] = (prob.gather(1, i).log() - sums[:, -1:].log())[:, 0]
    return [index, logp] if case["logprobs"] else [index]


def _exact_pack(w, group):
    scales, codes = [], []
    for part in w.split(group, 1):
        scale = (part.abs().max(1, keepdim=True).values.double() / 7).to(w.dtype).double()
        q = torch.nan_to_num(part.double() / scale, nan=0.0, posinf=0.0, neginf=0.0)
        codes.append(torch.clamp(torch.round(q), -7, 7) * scale)
        scales.append(scale)
    return torch.cat(codes, 1), torch.cat(scales, 1)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "sample":
        return _exact_sample(case, s)
    if op == "pack":
        return list(_exact_pack(s["w"], case["group"]))
    if op == "linear4":
        z = torch.einsum("mk,nk->mn", s["x"].double(), _exact_pack(s["w"], case["group"])[0])
        z = z + s["b"].double() if case["bias"] else z
        y = {"none": lambda: z, "tanh": lambda: torch.tanh(z), "relu": lambda: z.clamp(min=0),
             "gelu": lambda: z * 0.5 * torch.special.erfc(-z / math.sqrt(2)), "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
        return [y + s["residual"].double() if case["residual"] else y]
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]]))
    scale = min(1.0, s["max_norm"] / norm.item())
    if op == "clip":
        return [g.double() * scale for g in s["grads"]] + [norm]
    sign, t = -scale if case["maximize"] else scale, _STEPS + 1
    m, v = s["m"].double(), s["v"].double()
    g = torch.zeros_like(m)
    for o, q in zip(s["offsets"], s["grads"]):
        g[o:o + q.numel()] = sign * q.double().flatten()
    m = _BETA1 * m + (1 - _BETA1) * g
    v = _BETA2 * v + (1 - _BETA2) * g ** 2
    out = []
    for o, p, d in zip(s["offsets"], s["params"], s["decay"]):
        e = slice(o, o + p.numel())
        hat_m, hat_v = m[e] / (1 - _BETA1 ** t), v[e] / (1 - _BETA2 ** t)
        q = p.double().flatten()
        out.append((q - _LR * d * q - _LR * hat_m / (hat_v ** 0.5 + _EPS)).view(p.shape))
    return out + [m, v, norm]
