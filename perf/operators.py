"""What is measured of the operators around the evolution-strategies step: the linear layer with its
epilogue and its gradients, layer norm with its gradients, and the AdamW step over many tensors.

The population step perturbs a centre network; these operators run that network itself: acting with
the centre policy (one observation, or one for every environment), fitting it to targets by its
gradients before the search starts, and turning any gradient, the population's estimate included,
into a parameter step. Sizes are those of the package's workloads (widths 8, 64, 256, 1024 and 4096,
populations of 1,024 to 16,384) and odd neighbours of them.

``run`` computes each operator in elementary torch operations in 32 bits where ``own`` is false, and
through the package's entry points where it is true.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ACTS = ("none", "tanh", "relu", "gelu", "silu")
_BLOCK = 256                 # elements that share a scale of an 8-bit moment
_TOP = 448.0                 # largest finite e4m3 value
_TINY = 1e-30                # a block whose largest magnitude is below this is stored as zeros
_BETA1, _BETA2, _EPS, _LR, _DECAY, _STEPS = 0.9, 0.999, 1e-8, 1e-3, 0.01, 37


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # Acting with a wide centre network on one observation: the weight is read once, latency counts.
        {"name": "linear one observation", "op": "linear", "rows": 1, "in": 4096, "out": 4096, "type": "bf16",
         "act": "gelu", "bias": True, "residual": True, "preact": False},
        # The policy's hidden layer over one observation for each of 1,024 environments.
        {"name": "linear policy layer", "op": "linear", "rows": 1024, "in": 256, "out": 256, "type": "fp32",
         "act": "tanh", "bias": True, "residual": False, "preact": False},
        # A residual layer of the large network in training: the pre-activation is kept for the gradients.
        {"name": "linear training layer", "op": "linear", "rows": 8192, "in": 4096, "out": 4096, "type": "bf16",
         "act": "gelu", "bias": True, "residual": True, "preact": True},
        # Fitting the policy to targets over a ragged batch.
        {"name": "linear grads policy", "op": "linear_grads", "rows": 1021, "in": 256, "out": 256, "type": "fp32",
         "act": "tanh", "bias": True},
        # The large network's layer: all three gradients.
        {"name": "linear grads training", "op": "linear_grads", "rows": 8192, "in": 4096, "out": 4096, "type": "bf16",
         "act": "gelu", "bias": True},
        # Normalising the policy's observations' features.
        {"name": "norm policy", "op": "norm", "rows": 1024, "n": 256, "type": "fp32", "weight": "fp32"},
        # A long batch of the large network.
        {"name": "norm large", "op": "norm", "rows": 32768, "n": 4096, "type": "bf16", "weight": "bf16"},
        # A ragged batch with an odd width: rows that no vector load divides.
        {"name": "norm grads odd", "op": "norm_grads", "rows": 4099, "n": 1021, "type": "fp32", "weight": "fp32"},
        {"name": "norm grads large", "op": "norm_grads", "rows": 32768, "n": 4096, "type": "bf16", "weight": "fp32"},
        # The policy's six tensors: a step of 84,488 parameters, where launches count.
        {"name": "adamw policy", "op": "adamw", "layers": 3, "in": 64, "width": 256, "out": 8, "type": "fp32",
         "grad": "fp32", "bits": 32, "maximize": True},
        # The large network's tensors with 32-bit moments, and with 8-bit ones.
        {"name": "adamw large 32 bits", "op": "adamw", "layers": 4, "in": 4096, "width": 4096, "out": 4096,
         "type": "fp32", "grad": "fp32", "bits": 32, "maximize": False},
        {"name": "adamw large 8 bits", "op": "adamw", "layers": 4, "in": 4096, "width": 4096, "out": 1021,
         "type": "bf16", "grad": "bf16", "bits": 8, "maximize": True},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm; odd ones, multiples of 8 and of 64 all occur."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.random()
    if kind < 0.3 and v >= 64:
        v -= v % 64
    elif kind < 0.6 and v >= 8:
        v -= v % 8
    v = max(lo, min(hi, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grads", "linear_grads", "norm", "norm_grads", "adamw", "adamw"))
    kind = rng.choice(("bf16", "bf16", "fp32"))
    if op in ("linear", "linear_grads"):
        most = 4096 if kind == "bf16" else 1024
        c = {"op": op, "rows": _spread(rng, 1, 8192), "in": _spread(rng, 8, most), "out": _spread(rng, 8, most),
             "type": kind, "act": rng.choice(_ACTS), "bias": rng.random() < 0.75}
        if op == "linear":
            c["residual"] = rng.random() < 0.5
            c["preact"] = rng.random() < 0.5
        return c
    if op in ("norm", "norm_grads"):
        n = _spread(rng, 8, 8192)
        rows = _spread(rng, 1, min(65536, 32768 * 4096 // n))
        return {"op": op, "rows": rows, "n": n, "type": kind, "weight": rng.choice(("fp32", kind))}
    width = _spread(rng, 16, 4096)
    return {"op": op, "layers": rng.randint(2, 3 if width > 2048 else 12), "in": _spread(rng, 8, 4096), "width": width,
            "out": _spread(rng, 1, 4096), "type": kind, "grad": rng.choice(("fp32", kind)),
            "bits": rng.choice((8, 32)), "maximize": rng.random() < 0.5}


def _shapes(case):
    """Weight and bias of each layer, as the package lays a policy out."""
    sizes = [case["in"]] + [case["width"]] * (case["layers"] - 1) + [case["out"]]
    return [s for a, b in zip(sizes[:-1], sizes[1:]) for s in ((b, a), (b,))]


def work(case):
    op = case["op"]
    if op in ("linear", "linear_grads"):
        m, k, n, size = case["rows"], case["in"], case["out"], _TYPES[case["type"]].itemsize
        bias = n if case["bias"] else 0
        if op == "linear":
            outs = m * n * (1 + case["residual"] + case["preact"])
            return {"bytes": size * (m * k + n * k + bias + outs), "flops": 2 * m * n * k}
        kept = m * n * (1 + (case["act"] != "none"))
        return {"bytes": size * (kept + 2 * m * k + 2 * n * k + bias), "flops": 4 * m * n * k}
    if op in ("norm", "norm_grads"):
        m, n, size, wsize = case["rows"], case["n"], _TYPES[case["type"]].itemsize, _TYPES[case["weight"]].itemsize
        if op == "norm":
            return {"bytes": 2 * m * n * size + 2 * n * wsize + 8 * m, "flops": 8 * m * n}
        return {"bytes": 3 * m * n * size + 3 * n * wsize + 8 * m, "flops": 14 * m * n}
    count = sum(math.prod(s) for s in _shapes(case))
    per = 2 * _TYPES[case["type"]].itemsize + _TYPES[case["grad"]].itemsize
    # The moments read and written; with 8 bits, one byte each and two scales a block, and their values read out.
    per += 16 if case["bits"] == 32 else 4 + 16 / _BLOCK + 2 + 8
    return {"bytes": int(per * count), "flops": 16 * count}


# ---------------------------------------------------------------- the inputs
def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0, kind=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(kind)

    op, kind = case["op"], _TYPES[case["type"]]
    s = {"case": case}
    if op in ("linear", "linear_grads"):
        m, k, n = case["rows"], case["in"], case["out"]
        s["x"] = normal(m, k, kind=kind)
        s["w"] = normal(n, k, scale=k ** -0.5, kind=kind)
        s["b"] = normal(n, scale=0.1, kind=kind) if case["bias"] else None
        if op == "linear":
            s["residual"] = normal(m, n, kind=kind) if case["residual"] else None
        else:
            s["grad"] = normal(m, n, kind=kind)
            s["preact"] = normal(m, n, kind=kind) if case["act"] != "none" else None
    elif op in ("norm", "norm_grads"):
        m, n, wkind = case["rows"], case["n"], _TYPES[case["weight"]]
        x = normal(m, n) * (0.5 + torch.rand(m, 1, generator=gen, device="cuda")) + normal(m, 1)
        s["x"] = x.to(kind)
        s["w"], s["b"] = normal(n, scale=0.2, shift=1.0, kind=wkind), normal(n, scale=0.1, kind=wkind)
        if op == "norm_grads":
            s["grad"] = normal(m, n, kind=kind)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + 1e-5).rsqrt().float()
    else:
        shapes = _shapes(case)
        s["params"] = [normal(*p, scale=p[-1] ** -0.5 if len(p) == 2 else 0.1, kind=kind) for p in shapes]
        # Entries of a gradient differ by orders of magnitude between rows.
        s["grads"] = [normal(*p, scale=1e-2, kind=torch.float32).mul_(torch.exp(normal(p[0], *[1] * (len(p) - 1)))).to(_TYPES[case["grad"]])
                      for p in shapes]
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
        if case["bits"] == 32:
            s["m"], s["v"] = m, r * r
        else:
            s["m"], s["m_scale"] = _pack(m)
            s["v"], s["v_scale"] = _pack(r, positive=True)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] == "adamw":
        # The handle that a program keeps, over these same tensors.
        import virtual_noise_perturbed_gb300 as vn
        state = {k: s[k] for k in ("m", "v", "m_scale", "v_scale") if k in s}
        s["opt"] = vn.AdamW(s["params"], lr=_LR, betas=(_BETA1, _BETA2), eps=_EPS, weight_decay=s["decay"],
                            state_bits=case["bits"], maximize=case["maximize"], state=state, step=_STEPS)
    return s


# ---------------------------------------------------------------- the plain forms
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


def _slope(z, act):
    if act == "tanh":
        t = torch.tanh(z)
        return 1 - t * t
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        t = 1 / (1 + torch.exp(-z))
        return t * (1 + z * (1 - t))
    return torch.ones_like(z)


def _plain_linear(s):
    case, x, w = s["case"], s["x"], s["w"]
    z = x.float() @ w.float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(x.dtype), z.to(x.dtype)] if case["preact"] else [y.to(x.dtype)]


def _plain_linear_grads(s):
    case, x, w = s["case"], s["x"], s["w"]
    d = s["grad"].float()
    if s["preact"] is not None:
        d = d * _slope(s["preact"].float(), case["act"])
    out = [(d @ w.float()).to(x.dtype), (d.t() @ x.float()).to(w.dtype)]
    return out + [d.sum(0).to(w.dtype)] if case["bias"] else out


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + 1e-5)
    y = c * rstd[:, None] * s["w"].float() + s["b"].float()
    return [y.to(s["x"].dtype), mean, rstd]


def _plain_norm_grads(s):
    d, rstd = s["grad"].float(), s["rstd"][:, None]
    hat = (s["x"].float() - s["mean"][:, None]) * rstd
    t = d * s["w"].float()
    dx = rstd * (t - t.mean(1, keepdim=True) - hat * (t * hat).mean(1, keepdim=True))
    return [dx.to(s["x"].dtype), (d * hat).sum(0).to(s["w"].dtype), d.sum(0).to(s["w"].dtype)]


def _pack(x, positive=False):
    """e4m3 codes of x in blocks, each in units of its block's scale: its largest magnitude over 448."""
    x = x.view(-1, _BLOCK)
    top = x.abs().amax(1, keepdim=True)
    scale = torch.where(top < _TINY, torch.zeros_like(top), top * (1.0 / _TOP))
    q = torch.where(scale == 0, torch.zeros_like(x), x * (torch.ones_like(scale) / scale))
    q = q.clamp(-_TOP, _TOP).to(torch.float8_e4m3fn)
    if positive:  # a positive root never becomes zero: it divides the step
        q = torch.where((q.float() == 0) & (x > 0) & (scale > 0), torch.full_like(x, 2.0 ** -9), q.float()).to(torch.float8_e4m3fn)
    return q.view(-1), scale.view(-1)


def _unpack(q, scale):
    return (q.float().view(-1, _BLOCK) * scale[:, None]).view(-1)


def _plain_adamw_one(s, i, m, v):
    """One tensor's step on its flat moments (in 32 bits), and the new moments."""
    p, g, c = s["params"][i], s["grads"][i].float().reshape(-1), s["case"]
    g = -g if c["maximize"] else g
    m = m * _BETA1 + g * (1 - _BETA1)
    v = v * _BETA2 + (g * g) * (1 - _BETA2)
    root = torch.sqrt(v)
    t = s["step"]
    denom = root * (1 / math.sqrt(1 - _BETA2 ** t)) + _EPS
    new = p.float().reshape(-1) * (1 - _LR * s["decay"][i]) - (m / denom) * (_LR / (1 - _BETA1 ** t))
    p.copy_(new.view(p.shape))
    return m, v, root


def _plain_adamw(s):
    s["step"] += 1
    eight = s["case"]["bits"] == 8
    at = [(o, o + p.numel()) for o, p in zip(s["offsets"], s["params"])]
    m = _unpack(s["m"], s["m_scale"]) if eight else s["m"]
    v = _unpack(s["v"], s["v_scale"]) if eight else s["v"]
    v = v * v if eight else v
    new = [_plain_adamw_one(s, i, m[a:b], v[a:b]) for i, (a, b) in enumerate(at)]
    tails = [b - e[1] for e, b in zip(at, s["offsets"][1:] + [s["total"]])]
    m, v, root = (torch.cat([torch.nn.functional.pad(n[k], (0, t)) for n, t in zip(new, tails)]) for k in range(3))
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return s["params"] + [s["m"], s["v"]]
    s["m"], s["m_scale"] = _pack(m)
    s["v"], s["v_scale"] = _pack(root, positive=True)
    root = _unpack(s["v"], s["v_scale"])
    return s["params"] + [_unpack(s["m"], s["m_scale"]), root * root]


_PLAIN = {"linear": _plain_linear, "linear_grads": _plain_linear_grads, "norm": _plain_norm,
          "norm_grads": _plain_norm_grads, "adamw": _plain_adamw}


# ---------------------------------------------------------------- the package's operators
def _own(s):
    import virtual_noise_perturbed_gb300 as vn
    case = s["case"]
    op = case["op"]
    if op == "linear":
        y = vn.linear(s["x"], s["w"], s["b"], activation=case["act"], residual=s["residual"], preact=case["preact"])
        return list(y) if case["preact"] else [y]
    if op == "linear_grads":
        dx, dw, db = vn.linear_backward(s["grad"], s["x"], s["w"], s["preact"], activation=case["act"], bias=case["bias"])
        return [dx, dw, db] if case["bias"] else [dx, dw]
    if op == "norm":
        return list(vn.layer_norm(s["x"], s["w"], s["b"], eps=1e-5))
    if op == "norm_grads":
        return list(vn.layer_norm_backward(s["grad"], s["x"], s["mean"], s["rstd"], s["w"]))
    s["opt"].step(s["grads"])
    return s["params"] + list(s["opt"].moments())


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _round_e4m3(x):
    """The nearest e4m3 value, ties to even: 4 significant bits, steps of 2^-9 below 2^-6."""
    a = x.abs().clamp(max=_TOP)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 4).clamp(min=-9))
    return torch.round(a / step) * step * torch.sign(x)


def _exact_blocks(x, positive):
    x = x.view(-1, _BLOCK)
    scale = x.abs().max(1, keepdim=True).values / _TOP
    scale = torch.where(scale < _TINY / _TOP, torch.zeros_like(scale), scale)
    q = _round_e4m3(torch.nan_to_num(x / scale, nan=0.0, posinf=0.0, neginf=0.0))
    if positive:
        q = torch.where((q == 0) & (x > 0) & (scale > 0), torch.full_like(q, 2.0 ** -9), q)
    return (q * scale).view(-1)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("linear", "linear_grads"):
        x, w = s["x"].double(), s["w"].double()
        cdf = lambda z: 0.5 * torch.special.erfc(-z / math.sqrt(2))  # noqa: E731
        if op == "linear":
            z = torch.einsum("mk,nk->mn", x, w)
            z = z + s["b"].double() if case["bias"] else z
            y = {"none": lambda: z, "tanh": lambda: torch.tanh(z), "relu": lambda: z.clamp(min=0),
                 "gelu": lambda: z * cdf(z), "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
            y = y + s["residual"].double() if case["residual"] else y
            return [y, z] if case["preact"] else [y]
        d = s["grad"].double()
        if s["preact"] is not None:
            z = s["preact"].double()
            t = torch.sigmoid(z)
            d = d * {"tanh": lambda: 1 / torch.cosh(z) ** 2, "relu": lambda: torch.heaviside(z, torch.zeros_like(z)),
                     "gelu": lambda: cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                     "silu": lambda: t + z * t * (1 - t)}[case["act"]]()
        out = [torch.einsum("mn,nk->mk", d, w), torch.einsum("mn,mk->nk", d, x)]
        return out + [torch.einsum("mn->n", d)] if case["bias"] else out
    if op in ("norm", "norm_grads"):
        x, w = s["x"].double(), s["w"].double()
        if op == "norm":
            mean = x.mean(1)
            rstd = (x.var(1, unbiased=False) + 1e-5) ** -0.5
            return [(x - mean[:, None]) * rstd[:, None] * w + s["b"].double(), mean, rstd]
        d, mean, rstd = s["grad"].double(), s["mean"].double(), s["rstd"].double()
        hat = torch.einsum("mn,m->mn", x - mean[:, None], rstd)
        n = x.shape[1]
        a, c = torch.einsum("mn,n->m", d, w) / n, torch.einsum("mn,mn,n->m", d, hat, w) / n
        dx = torch.einsum("mn,m->mn", d * w - a[:, None] - hat * c[:, None], rstd)
        return [dx, torch.einsum("mn,mn->n", d, hat), torch.einsum("mn->n", d)]
    eight, sign, t = case["bits"] == 8, -1.0 if case["maximize"] else 1.0, _STEPS + 1
    m, r = s["m"].double(), s["v"].double()
    if eight:
        m = m * s["m_scale"].double().repeat_interleave(_BLOCK)
        r = r * s["v_scale"].double().repeat_interleave(_BLOCK)
    v = r * r if eight else r
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
    if eight:
        m, v = _exact_blocks(m, False), _exact_blocks(v ** 0.5, True) ** 2
    return out + [m, v]
