"""The centre network: what the population step perturbs, run unperturbed and trained.

``linear`` and ``layer_norm`` with their gradients, and ``AdamW``, the parameter step for any
gradient: these, or the population's estimate (``virtual_flat_gradient`` and the others).

Like the rest of the package's Python, these functions only check and marshal arguments and
call ``libvn.so`` on the current CUDA stream; all arithmetic runs in the library's kernels.
Tensors must be on a CUDA device; there is no CPU path. Inputs that are not contiguous are
copied first.
"""

from __future__ import annotations

import struct
from array import array
from typing import Optional, Sequence, Tuple, Union

import torch

from . import _lib
from ._lib import check, load
from .api import _DT, _cuda, _device, _dt, device_status

_ACTS = {None: _lib.VN_ACT_NONE, "none": _lib.VN_ACT_NONE, "tanh": _lib.VN_ACT_TANH, "relu": _lib.VN_ACT_RELU,
         "gelu": _lib.VN_ACT_GELU, "silu": _lib.VN_ACT_SILU}


def _act(activation: Optional[str]) -> int:
    try:
        return _ACTS[activation]
    except (KeyError, TypeError):
        raise ValueError("activation must be None, 'tanh', 'relu', 'gelu' or 'silu'") from None


def _at(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _run(device: torch.device, where: str, fn, *args) -> None:
    """fn(*args, stream) with ``device`` current, on its current stream."""
    stream = torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() == device.index:
        check(fn(*args, stream), where)
    else:
        with torch.cuda.device(device):
            check(fn(*args, stream), where)


def _same(t: torch.Tensor, name: str, shape, dtype: torch.dtype) -> torch.Tensor:
    """``t`` contiguous, of this shape and dtype."""
    t = _cuda(t, name)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _workspace(bytes_: int, device: torch.device) -> Optional[torch.Tensor]:
    return torch.empty(bytes_, dtype=torch.uint8, device=device) if bytes_ > 0 else None


def _result(out: Optional[torch.Tensor], shape, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(out, torch.Tensor) or out.shape != shape or out.dtype != dtype or not out.is_contiguous() \
            or out.device != device:
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return out


def _layer(x: torch.Tensor, weight: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor, int, int, int, int]:
    """x and weight checked; rows, in, out and the type of a linear layer on them."""
    x = _cuda(x, "x")
    weight = _cuda(weight, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must be (out_features, in_features)")
    n, k = weight.shape
    if x.dim() < 1 or x.shape[-1] != k:
        raise ValueError(f"x must be (..., {k}), got {tuple(x.shape)}")
    if x.dtype != weight.dtype:
        raise TypeError(f"x and weight must have one dtype, got {x.dtype} and {weight.dtype}")
    rows = 1
    for d in x.shape[:-1]:
        rows *= d
    return x, weight, rows, k, n, _dt(x, "x")


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
           activation: Optional[str] = None, residual: Optional[torch.Tensor] = None, preact: bool = False,
           out: Optional[torch.Tensor] = None,
           check_status: bool = False) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """act(x W^T + b) + residual, shape (..., out), in one epilogue (``vn_linear``).

    x is (..., in), weight (out, in), residual (..., out), all float32 or all bfloat16; bias
    (out,) of either type. ``activation``: None, "tanh", "relu", "gelu" (z times the normal
    distribution function of z) or "silu". With ``preact=True`` the result is (y, z), z the
    value before the activation that ``linear_backward`` needs. ``check_status=True`` calls
    ``device_status()`` before returning (it synchronises): the tensor-core kernels bound
    their waits, and a wait that ran out leaves y unwritten."""
    lib = load()
    x, weight, rows, k, n, dt = _layer(x, weight)
    shape = x.shape[:-1] + (n,)
    if bias is not None:
        bias = _cuda(bias, "bias")
        if bias.shape != (n,):
            raise ValueError(f"bias must have shape ({n},)")
    if residual is not None:
        residual = _same(residual, "residual", shape, x.dtype)
    act = _act(activation)
    dev = _device(x, weight, bias, residual)
    y = _result(out, shape, x.dtype, dev)
    z = torch.empty(shape, dtype=x.dtype, device=dev) if preact else None
    px, pw = x.data_ptr(), weight.data_ptr()
    need = lib.vn_linear_workspace(rows, k, n, dt, not (px | pw) & 15)
    ws = _workspace(need, dev)
    _run(dev, "vn_linear", lib.vn_linear, px, pw, dt, _at(bias), _dt(bias, "bias") if bias is not None else 0,
         _at(residual), rows, k, n, act, y.data_ptr(), _at(z), _at(ws), max(need, 0))
    if check_status:
        device_status(dev)
    return (y, z) if preact else y


def linear_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                    preact: Optional[torch.Tensor] = None, *, activation: Optional[str] = None, bias: bool = True,
                    check_status: bool = False) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(grad_x, grad_weight, grad_bias) of ``linear`` (``vn_linear_backward``).

    grad is the gradient of y, (..., out); preact the z that ``linear(..., preact=True)``
    returned (not needed without an activation). The gradients have their tensors' shapes and
    dtypes, grad_bias the weight's (None with ``bias=False``). The residual's gradient is
    grad."""
    lib = load()
    x, weight, rows, k, n, dt = _layer(x, weight)
    shape = x.shape[:-1] + (n,)
    grad = _same(grad, "grad", shape, x.dtype)
    act = _act(activation)
    if act != _lib.VN_ACT_NONE:
        if preact is None:
            raise ValueError("the gradient through an activation needs preact")
        preact = _same(preact, "preact", shape, x.dtype)
    else:
        preact = None
    dev = _device(grad, x, weight, preact)
    gx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    gw = torch.empty((n, k), dtype=x.dtype, device=dev)
    gb = torch.empty(n, dtype=x.dtype, device=dev) if bias else None
    pg, px, pw = grad.data_ptr(), x.data_ptr(), weight.data_ptr()
    need = lib.vn_linear_backward_workspace(rows, k, n, dt, act, not (pg | px | pw) & 15)
    ws = _workspace(need, dev)
    _run(dev, "vn_linear_backward", lib.vn_linear_backward, pg, px, pw, _at(preact), dt, rows, k, n, act,
         gx.data_ptr(), gw.data_ptr(), _at(gb), dt, _at(ws), max(need, 0))
    if check_status:
        device_status(dev)
    return gx, gw, gb


def _norm_params(weight: Optional[torch.Tensor], bias: Optional[torch.Tensor], n: int):
    """Weight and bias of a norm over n elements, checked, and their one type."""
    dts = []
    out = []
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            t = _cuda(t, name)
            if t.shape != (n,):
                raise ValueError(f"{name} must have shape ({n},)")
            dts.append(_dt(t, name))
        out.append(t)
    if len(set(dts)) > 1:
        raise TypeError("weight and bias must have one dtype")
    return out[0], out[1], dts[0] if dts else _lib.VN_F32


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5,
               out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): each row of x (..., n) to zero mean and unit variance, times weight plus
    bias (``vn_layer_norm``). x is float32 or bfloat16 and y like it; weight and bias (n,) are of
    either type, or None. mean and rstd are float32 of x's leading shape; ``layer_norm_backward``
    takes them."""
    lib = load()
    x = _cuda(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be (..., n) with n >= 1")
    n = x.shape[-1]
    weight, bias, wdt = _norm_params(weight, bias, n)
    dev = _device(x, weight, bias)
    y = _result(out, x.shape, x.dtype, dev)
    lead = x.shape[:-1]
    mean = torch.empty(lead, dtype=torch.float32, device=dev)
    rstd = torch.empty(lead, dtype=torch.float32, device=dev)
    _run(dev, "vn_layer_norm", lib.vn_layer_norm, x.data_ptr(), _dt(x, "x"), _at(weight), _at(bias), wdt,
         mean.numel(), n, float(eps), y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def layer_norm_backward(grad: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None) \
        -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(grad_x, grad_weight, grad_bias) of ``layer_norm`` from its stored mean and rstd
    (``vn_layer_norm_backward``). The last two are (n,) of weight's dtype, None without a weight."""
    lib = load()
    x = _cuda(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be (..., n) with n >= 1")
    n = x.shape[-1]
    grad = _same(grad, "grad", x.shape, x.dtype)
    mean = _same(mean, "mean", x.shape[:-1], torch.float32)
    rstd = _same(rstd, "rstd", x.shape[:-1], torch.float32)
    weight, _, wdt = _norm_params(weight, None, n)
    dev = _device(grad, x, mean, rstd, weight)
    gx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    gw = gb = ws = None
    rows, need = mean.numel(), 0
    if weight is not None:
        gw = torch.empty(n, dtype=weight.dtype, device=dev)
        gb = torch.empty(n, dtype=weight.dtype, device=dev)
        need = lib.vn_layer_norm_backward_workspace(rows, n)
        ws = _workspace(need, dev)
    _run(dev, "vn_layer_norm_backward", lib.vn_layer_norm_backward, grad.data_ptr(), x.data_ptr(), _dt(x, "x"),
         mean.data_ptr(), rstd.data_ptr(), _at(weight), wdt, rows, n, gx.data_ptr(), _at(gw), _at(gb), _at(ws),
         max(need, 0))
    return gx, gw, gb


class AdamW:
    """AdamW over many tensors, one launch a step (``vn_adamw``).

    ``params``: contiguous CUDA tensors of one dtype (float32 or bfloat16) on one device,
    updated in place by ``step``. ``weight_decay``: one number, or one for each tensor.
    ``maximize=True`` ascends: the direction of a fitness gradient. ``state_bits``: 32, or 8 for
    moments held as e4m3 codes with a float32 scale for each 256 elements of a tensor.

    ``state`` holds the moments in flat tensors: "m" and "v", and with 8 bits "m_scale" and
    "v_scale" (v's codes are of its root). Tensor i's moments are the ``params[i].numel()``
    elements from ``offsets[i]`` on, a multiple of 256. To resume, pass the saved ``state`` and
    ``steps``; the tensors passed are used and updated as they are."""

    BLOCK = 256

    def __init__(self, params: Sequence[torch.Tensor], lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.01, *, state_bits: int = 32,
                 maximize: bool = False, state: Optional[dict] = None, step: int = 0):
        self.params = list(params)
        if not self.params:
            raise ValueError("at least one tensor is needed")
        for i, p in enumerate(self.params):
            if not isinstance(p, torch.Tensor) or not p.is_cuda or not p.is_contiguous():
                raise ValueError(f"params[{i}] must be a contiguous CUDA tensor (updated in place)")
            if p.dtype != self.params[0].dtype:
                raise TypeError("the parameters must have one dtype")
        self.device = _device(*self.params)
        self._dt = _dt(self.params[0], "params[0]")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        n = len(self.params)
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(d) for d in weight_decay]
        if len(decay) != n:
            raise ValueError("one weight_decay for each tensor")
        self.lr, self.betas, self.eps, self.maximize = float(lr), (float(betas[0]), float(betas[1])), float(eps), bool(maximize)
        self.state_bits, self.steps = state_bits, int(step)
        self.sizes = [p.numel() for p in self.params]
        self.offsets, total = [], 0
        for s in self.sizes:
            self.offsets.append(total)
            total += -(-s // self.BLOCK) * self.BLOCK
        self.state = self._state(total, state)
        # One row of eight words a tensor, as the library's struct has them.
        self._table = array("Q", bytes(64 * n))
        self._table[6::8] = array("Q", self.sizes)
        self._table[7::8] = array("Q", struct.pack(f"{n}d", *decay))
        starts, at = [], 0
        for s in self.sizes:
            starts.append(at)
            at += s
        self._starts, self.total = starts, at

    def _state(self, total: int, given: Optional[dict]) -> dict:
        kind = torch.float32 if self.state_bits == 32 else torch.float8_e4m3fn
        want = {"m": (total, kind), "v": (total, kind)}
        if self.state_bits == 8:
            want.update(m_scale=(total // self.BLOCK, torch.float32), v_scale=(total // self.BLOCK, torch.float32))
        if given is None:
            return {k: torch.zeros(size, dtype=torch.uint8 if d == torch.float8_e4m3fn else d, device=self.device).view(d)
                    for k, (size, d) in want.items()}
        if set(given) != set(want):
            raise ValueError(f"state must have {sorted(want)}, got {sorted(given)}")
        for k, (size, d) in want.items():
            t = given[k]
            if not isinstance(t, torch.Tensor) or t.shape != (size,) or t.dtype != d or t.device != self.device \
                    or not t.is_contiguous():
                raise ValueError(f"state['{k}'] must be a contiguous {d} tensor of shape ({size},) on {self.device}")
        return dict(given)

    def _grads(self, grads) -> Tuple[list, torch.dtype, list]:
        """Addresses of the tensors' gradients, their dtype, and what has to stay alive."""
        if isinstance(grads, torch.Tensor):
            grads = _cuda(grads, "grads")
            if grads.shape != (self.total,):
                raise ValueError(f"a flat gradient must have shape ({self.total},)")
            _device(grads, self.params[0])
            base, size = grads.data_ptr(), grads.element_size()
            return [base + o * size for o in self._starts], grads.dtype, [grads]
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(self.params)} tensors but {len(grads)} gradients")
        kept, kind = [], None
        for i, (g, p) in enumerate(zip(grads, self.params)):
            if not isinstance(g, torch.Tensor) or g.shape != p.shape or g.device != p.device:
                raise ValueError(f"grads[{i}] must have params[{i}]'s shape and device")
            if kind is None:
                kind = g.dtype
            elif g.dtype != kind:
                raise TypeError("the gradients must have one dtype")
            kept.append(g if g.is_contiguous() else g.contiguous())
        return [g.data_ptr() for g in kept], kind, kept

    def step(self, grads: Union[torch.Tensor, Sequence[torch.Tensor]], lr: Optional[float] = None) -> None:
        """One step of every tensor. ``grads``: a gradient for each tensor, or one flat tensor with
        all of them one after another (as ``virtual_flat_gradient`` lays them out); float32 or
        bfloat16. ``lr`` replaces the learning rate for this step."""
        lib = load()
        at, kind, kept = self._grads(grads)
        if kind not in _DT:
            raise TypeError(f"grads: dtype {kind} is not supported (float32 or bfloat16)")
        t, s, o = self._table, self.state, self.offsets
        t[0::8] = array("Q", [p.data_ptr() for p in self.params])
        t[1::8] = array("Q", at)
        m, v, size = s["m"].data_ptr(), s["v"].data_ptr(), self.state_bits // 8
        t[2::8] = array("Q", [m + i * size for i in o])
        t[3::8] = array("Q", [v + i * size for i in o])
        if self.state_bits == 8:
            m, v = s["m_scale"].data_ptr(), s["v_scale"].data_ptr()
            t[4::8] = array("Q", [m + i // 64 for i in o])
            t[5::8] = array("Q", [v + i // 64 for i in o])
        _run(self.device, "vn_adamw", lib.vn_adamw, t.buffer_info()[0], len(self.params), self._dt, _DT[kind],
             self.state_bits, self.lr if lr is None else float(lr), self.betas[0], self.betas[1], self.eps,
             self.steps + 1, self.maximize)
        self.steps += 1
        del kept

    def moments(self) -> Tuple[torch.Tensor, torch.Tensor]:
        """The moments (m, v) as flat float32 tensors in ``offsets``' layout: the state itself with
        32 bits, with 8 the values that the codes stand for (``vn_adamw_moments``)."""
        s = self.state
        if self.state_bits == 32:
            return s["m"], s["v"]
        lib = load()
        n = s["m"].numel()
        m = torch.empty(n, dtype=torch.float32, device=self.device)
        v = torch.empty(n, dtype=torch.float32, device=self.device)
        _run(self.device, "vn_adamw_moments", lib.vn_adamw_moments, s["m"].data_ptr(), s["v"].data_ptr(),
             s["m_scale"].data_ptr(), s["v_scale"].data_ptr(), n, m.data_ptr(), v.data_ptr())
        return m, v


__all__ = ["AdamW", "layer_norm", "layer_norm_backward", "linear", "linear_backward"]
