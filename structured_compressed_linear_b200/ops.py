"""Binding of the operators around a projection: layer norm, low-rank adapters, AdamW.

The arithmetic runs in the CUDA library (include/ss1.h); this module checks tensors, allocates
outputs and workspaces, and passes pointers, sizes and the stream. Every call runs on the device
of its tensors, on `stream` or that device's current stream, and never falls back to another
implementation. Tensors are contiguous CUDA tensors, bf16 or float32. For a CUDA graph, capture these
functions; a backward pass through autograd is captured only while no eager graph of the same leaves
is alive (autograd ties a leaf to the stream of its first use).
"""

from __future__ import annotations

import array
import ctypes
import functools
import inspect
import struct
from operator import attrgetter
from typing import List, Optional, Sequence, Tuple

import numpy as np
import torch
from torch.autograd.function import once_differentiable

from . import ss1
from .ss1 import _check, _dtype_code, lib

#: Limits of the adapters (SS1_ADAPTER_MAX_RANK, SS1_ADAPTER_MAX_COUNT in include/ss1.h).
ADAPTER_MAX_RANK = 128
ADAPTER_MAX_COUNT = 1024
#: Elements that share one scale of an 8-bit AdamW state, the last step that rounds such states to the nearest
#: code, and the step's factors (SS1_ADAMW_*).
ADAMW_BLOCK = 256
ADAMW_NEAREST = 10
ADAMW_FACTORS = 9


def _tensor(name: str, t: torch.Tensor, shape=None, dtype=None, device=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, not {t.device}")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return t.data_ptr() if t is not None else None


def _call(device: int, fn, *args):
    """fn(*args, the device's current stream) on `device`, made current for the call where it is not."""
    handle = torch._C._cuda_getCurrentRawStream(device)
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != 0:
        _check(status, fn.__name__)


def _streamed(fn):
    """Adds the argument `stream`: the call, and what it allocates, then belong to that stream. (Memory that another
    stream's allocator handed out could still be in use there.)"""
    name = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream: Optional[torch.cuda.Stream] = None, **kw):
        if stream is None:
            return fn(*args, **kw)
        t = args[0] if args else kw.get(name)
        t = t[0] if isinstance(t, (list, tuple)) and t else t
        if isinstance(t, torch.Tensor) and t.device != stream.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _written(tensors):
    """Tells autograd that `tensors` were changed in place: a backward pass that saved one of them refuses to run on it."""
    torch.autograd.graph.increment_version(tensors)


def _apart(out: torch.Tensor, name: str, **inputs):
    """A given output must not share memory with an input."""
    a, b = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for other, t in inputs.items():
        if t is not None and t.data_ptr() < b and a < t.data_ptr() + t.numel() * t.element_size():
            raise ValueError(f"{name} must not overlap {other}")


# ---- layer norm ------------------------------------------------------------------------------

def _norm_weights(X: torch.Tensor, device: int, weight, bias=None) -> torch.dtype:
    """The weights' type; X's without weights."""
    dt = None
    for name, w in (("weight", weight), ("bias", bias)):
        if w is None:
            continue
        _tensor(name, w, X.shape[1:], None, device)
        t = w.dtype
        if (t != X.dtype and t != torch.float32) or (dt is not None and t != dt):
            raise ValueError(f"{name} must have X's dtype or float32, and weight and bias one dtype")
        dt = t
    return dt if dt is not None else X.dtype


def _norm_rows(X: torch.Tensor) -> Tuple[int, int]:
    _tensor("X", X)
    if X.dim() != 2 or X.shape[1] < 1:
        raise ValueError("X must be [M, K] with K >= 1")
    return X.shape


@functools.lru_cache(maxsize=4096)
def _norm_workspace(L, M: int, K: int) -> int:
    n = ctypes.c_size_t()
    _check(L.ss1_layernorm_backward_workspace(M, K, ctypes.byref(n)), "ss1_layernorm_backward_workspace")
    return n.value


@_streamed
def layernorm_forward(X: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                      eps: float = 1e-5, out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Y, mean, rstd) of X [M, K]: Y in X's dtype, mean and rstd float32 [M] (ss1_layernorm_forward).
    weight and bias [K] in X's dtype, or float32 beside bf16 rows."""
    M, K = _norm_rows(X)
    device = X.get_device()
    wt = _norm_weights(X, device, weight, bias)
    if out is None:
        Y = torch.empty_like(X)
    else:
        Y = _tensor("out", out, X.shape, X.dtype, device)
        _apart(Y, "out", X=X, weight=weight, bias=bias)
    mean, rstd = X.new_empty(M, dtype=torch.float32), X.new_empty(M, dtype=torch.float32)
    _call(device, lib().ss1_layernorm_forward, X.data_ptr(), _ptr(weight),
          _ptr(bias), Y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), M, K, eps, _dtype_code(X.dtype), _dtype_code(wt))
    if out is not None:
        _written(out)
    return Y, mean, rstd


@_streamed
def layernorm_backward(dY: torch.Tensor, X: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                       weight: Optional[torch.Tensor] = None, need: Tuple[bool, bool, bool] = (True, True, True),
                       weight_dtype: Optional[torch.dtype] = None):
    """(dX, dweight, dbias) from dY, the forward's X, mean and rstd (ss1_layernorm_backward). dweight and
    dbias have weight's dtype; without a weight weight_dtype (X's or float32: the bias's), or X's. `need`: which of the
    three to compute (the others are None)."""
    M, K = _norm_rows(X)
    device = X.get_device()
    _tensor("dY", dY, X.shape, X.dtype, device)
    _tensor("mean", mean, X.shape[:1], torch.float32, device)
    _tensor("rstd", rstd, X.shape[:1], torch.float32, device)
    wt = _norm_weights(X, device, weight)
    if weight_dtype is not None and weight_dtype != wt:
        if weight is not None or weight_dtype != torch.float32:
            raise ValueError(f"weight_dtype must be {wt}" + ("" if weight is not None else " or torch.float32"))
        wt = weight_dtype
    L = lib()
    dX = torch.empty_like(X) if need[0] else None
    dw = X.new_empty(K, dtype=wt) if need[1] else None
    db = X.new_empty(K, dtype=wt) if need[2] else None
    size = _norm_workspace(L, M, K) if need[1] or need[2] else 0
    ws = X.new_empty(size, dtype=torch.uint8) if size else None
    _call(device, L.ss1_layernorm_backward, dY.data_ptr(), X.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), _ptr(weight), _ptr(dX), _ptr(dw), _ptr(db), M, K, _dtype_code(X.dtype), _dtype_code(wt), _ptr(ws),
          size)
    return dX, dw, db


class LayerNormFunction(torch.autograd.Function):
    """Autograd wrapper: Y = LayerNormFunction.apply(X, weight, bias, eps)."""

    @staticmethod
    def forward(ctx, X, weight, bias, eps=1e-5):
        X = X.contiguous()
        Y, mean, rstd = layernorm_forward(X, weight, bias, eps)
        ctx.save_for_backward(X, mean, rstd, weight)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, mean, rstd, weight = ctx.saved_tensors
        # a bias without a weight may be float32 beside bf16 rows
        return *layernorm_backward(dY.contiguous(), X, mean, rstd, weight, tuple(ctx.needs_input_grad[:3]), ctx.bias_dtype), None


# ---- low-rank adapters -----------------------------------------------------------------------

#: ss1_adapters of include/ss1.h: A, B, scale, index, plan; K, N; R, count, dtype.
_ADAPTERS = struct.Struct("@5P2q3i4x")


class AdapterPlan:
    """The rows of a batch sorted by adapter, made once for all layers that run on the batch."""

    def __init__(self, data: torch.Tensor, M: int, count: int):
        self.data, self.M, self.count = data, M, count


@functools.lru_cache(maxsize=4096)
def _plan_bytes(L, M: int, count: int) -> int:
    n = ctypes.c_size_t()
    _check(L.ss1_adapter_plan_bytes(M, count, ctypes.byref(n)), "ss1_adapter_plan_bytes")
    return n.value


@_streamed
def adapter_plan(index: torch.Tensor, count: int) -> AdapterPlan:
    """Plan of `index` (int32 [M]; outside [0, count): no adapter) for adapter_forward and adapter_backward."""
    _tensor("index", index, dtype=torch.int32)
    if index.dim() != 1:
        raise ValueError("index must be [M]")
    M, L = index.shape[0], lib()
    size = _plan_bytes(L, M, count)
    data = index.new_empty(size, dtype=torch.uint8)
    _call(index.get_device(), L.ss1_adapter_plan, index.data_ptr(), M, count, data.data_ptr(), size)
    return AdapterPlan(data, M, count)


@functools.lru_cache(maxsize=4096)
def _adapter_workspace(L, M: int, K: int, N: int, R: int, n: int, dtype: int, backward: bool) -> int:
    size = ctypes.c_size_t()
    fwd, bwd = (None, ctypes.byref(size)) if backward else (ctypes.byref(size), None)
    _check(L.ss1_adapter_workspace(M, K, N, R, n, dtype, fwd, bwd), "ss1_adapter_workspace")
    return max(size.value, 1)


def _adapters(X, A, B, index, scale, plan):
    """(device, M, K, N, R, the packed ss1_adapters, dtype code, count) of checked arguments."""
    if X.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("X must be [M, K], A [count, R, K] and B [count, N, R]")
    M, K = X.shape
    n, R, _ = A.shape
    N = B.shape[1]
    device, t = X.get_device(), X.dtype
    _tensor("X", X)
    _tensor("A", A, (n, R, K), t, device)
    _tensor("B", B, (n, N, R), t, device)
    if not 1 <= R <= ADAPTER_MAX_RANK or not 1 <= n <= ADAPTER_MAX_COUNT:
        raise ValueError(f"ranks 1 .. {ADAPTER_MAX_RANK} and 1 .. {ADAPTER_MAX_COUNT} adapters, not {R} and {n}")
    if index is not None:
        _tensor("index", index, (M,), torch.int32, device)
    elif n != 1:
        raise ValueError("several adapters need an index")
    if scale is not None:
        _tensor("scale", scale, (n,), torch.float32, device)
    if plan is not None and (index is None or plan.M != M or plan.count != n or plan.data.get_device() != device):
        raise ValueError("the plan was made for another batch, count or device")
    code = int(_dtype_code(t))
    packed = _ADAPTERS.pack(A.data_ptr(), B.data_ptr(), _ptr(scale) or 0, _ptr(index) or 0,
                            plan.data.data_ptr() if plan is not None else 0, K, N, R, n, code)
    return device, M, K, N, R, packed, code, n


@_streamed
def adapter_forward(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, Y: torch.Tensor, index: Optional[torch.Tensor] = None,
                    scale: Optional[torch.Tensor] = None, keep: bool = False, plan: Optional[AdapterPlan] = None,
                    out: Optional[torch.Tensor] = None):
    """Y[m] + scale[a] (X[m] A[a]^T) B[a]^T with a = index[m] (ss1_adapter_forward): X [M, K] and the
    projection's output Y [M, N], A [count, R, K], B [count, N, R], scale float32 [count]. index int32
    [M]; an entry outside [0, count) leaves its row as it is; None: every row uses the one adapter.
    `out` may be Y itself. keep: returns (out, H) with H = X A^T, float32 [M, R], for the backward pass."""
    device, M, K, N, R, ad, code, n = _adapters(X, A, B, index, scale, plan)
    _tensor("Y", Y, (M, N), X.dtype, device)
    given = out is not None
    if not given:
        out = torch.empty_like(Y)
    else:
        _tensor("out", out, Y.shape, Y.dtype, device)
        _apart(out, "out", X=X, A=A, B=B, Y=Y if out.data_ptr() != Y.data_ptr() else None)
    H = X.new_empty((M, R), dtype=torch.float32) if keep else None
    L = lib()
    size = _adapter_workspace(L, M, K, N, R, n, code, False)
    ws = X.new_empty(size, dtype=torch.uint8)
    _call(device, L.ss1_adapter_forward, ad, X.data_ptr(), Y.data_ptr(), out.data_ptr(), _ptr(H), M,
          ws.data_ptr(), size)
    if given:
        _written(out)
    return (out, H) if keep else out


@_streamed
def adapter_backward(dY: torch.Tensor, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, H: Optional[torch.Tensor],
                     dX: Optional[torch.Tensor] = None, index: Optional[torch.Tensor] = None,
                     scale: Optional[torch.Tensor] = None, plan: Optional[AdapterPlan] = None,
                     need: Tuple[bool, bool, bool] = (True, True, True)):
    """(dX, dA, dB) of adapter_forward for dY, the gradient of its output (ss1_adapter_backward). H is what
    the forward kept (needed for dB); `dX`, if given, is the projection's input gradient, which the
    result includes. `need`: which of the three to compute (the others are None)."""
    device, M, K, N, R, ad, code, n = _adapters(X, A, B, index, scale, plan)
    _tensor("dY", dY, (M, N), X.dtype, device)
    if need[2]:
        if H is None:
            raise ValueError("dB needs H, which adapter_forward(keep=True) returns")
        _tensor("H", H, (M, R), torch.float32, device)
    if dX is not None:
        _tensor("dX", dX, X.shape, X.dtype, device)
    out = torch.empty_like(X) if need[0] else None
    dA = torch.empty_like(A) if need[1] else None
    dB = torch.empty_like(B) if need[2] else None
    L = lib()
    size = _adapter_workspace(L, M, K, N, R, n, code, True)
    ws = X.new_empty(size, dtype=torch.uint8)
    _call(device, L.ss1_adapter_backward, ad, dY.data_ptr(), X.data_ptr(),
          H.data_ptr() if need[2] else None, _ptr(dX) if need[0] else None, _ptr(out), _ptr(dA), _ptr(dB), M, ws.data_ptr(), size)
    return out, dA, dB


def adapter_status(device: Optional[int] = None) -> Tuple[int, int]:
    """(status, detail) of `device` (the current one): whether a bounded wait of adapter_backward ran out since the last look
    (ss1_adapter_status; its results are NaN then). Call after synchronising."""
    detail = ctypes.c_int32()
    with torch.cuda.device(device):
        status = lib().ss1_adapter_status(ctypes.byref(detail))
    return status, detail.value


class AdaptedSS1Function(torch.autograd.Function):
    """Autograd wrapper of an SS1 layer with low-rank adapters beside it:
    Y = AdaptedSS1Function.apply(X, Wc, layer, A, B, index, scale, plan), the last three as in adapter_forward. `scale` has
    no gradient: the backward pass refuses one that asks for it."""

    @staticmethod
    def forward(ctx, X, Wc, layer, A, B, index=None, scale=None, plan=None):
        X, Wc, A, B = X.contiguous(), Wc.contiguous(), A.contiguous(), B.contiguous()
        Y = layer.forward(X, Wc)
        Y, H = adapter_forward(X, A, B, Y, index, scale, keep=True, plan=plan, out=Y)
        ctx.layer, ctx.plan = layer, plan
        ctx.save_for_backward(X, Wc, A, B, H, index, scale)
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        if any(ctx.needs_input_grad[6:7]):
            raise ValueError("scale has no gradient here: pass scale.detach()")
        X, Wc, A, B, H, index, scale = ctx.saved_tensors
        dY = dY.contiguous()
        nx, nw, _, na, nb = ctx.needs_input_grad[:5]
        dX = ctx.layer.backward_input(dY, Wc) if nx else None
        dWc = ctx.layer.backward_weight(X, dY) if nw else None
        dA = dB = None
        if nx or na or nb:
            dX, dA, dB = adapter_backward(dY, X, A, B, H, dX, index, scale, ctx.plan, (nx, na, nb))
        return dX, dWc, None, dA, dB, None, None, None


# ---- AdamW -----------------------------------------------------------------------------------

class _AdamWHyper(ctypes.Structure):
    """ss1_adamw_hyper of include/ss1.h."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double), ("step", ctypes.c_int64)]


#: ss1_adamw_tensor of include/ss1.h.
_ADAMW_TENSOR = np.dtype([("param", "u8"), ("grad", "u8"), ("master", "u8"), ("exp_avg", "u8"), ("exp_avg_sq", "u8"),
                          ("avg_scale", "u8"), ("sq_scale", "u8"), ("numel", "i8"), ("param_dtype", "i4"),
                          ("grad_dtype", "i4")])


def adamw_factors(step: int, lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                  weight_decay: float = 0.01, grad_scale: float = 1.0) -> torch.Tensor:
    """The factors of one step as a float32 CPU tensor [ADAMW_FACTORS] (ss1_adamw_factors). On the device,
    they are adamw_step's `factors`: a captured step reads them when it is replayed."""
    out = torch.empty(ADAMW_FACTORS, dtype=torch.float32)
    h = _AdamWHyper(lr, betas[0], betas[1], eps, weight_decay, grad_scale, step)
    _check(lib().ss1_adamw_factors(ctypes.byref(h), out.data_ptr()), "ss1_adamw_factors")
    return out


_POINTER, _NUMEL, _CONTIGUOUS, _DEVICE = (torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous,
                                          torch.Tensor.get_device)
_DTYPE = attrgetter("dtype")


def _like(name: str, ts: Sequence[torch.Tensor], sizes: List[int], device: int, dtypes):
    """(the tensors' addresses, their types), after the checks."""
    if list(map(_NUMEL, ts)) != sizes:
        raise ValueError(f"{name}: one tensor for each parameter, of its size")
    kinds = set(map(_DTYPE, ts))
    if set(map(_DEVICE, ts)) - {device} or not all(map(_CONTIGUOUS, ts)) or not kinds <= dtypes:
        raise ValueError(f"{name} must be contiguous, on cuda:{device} and of " + " or ".join(map(str, dtypes)))
    return array.array("Q", map(_POINTER, ts)), kinds


_WEIGHTS, _F32, _U8 = {torch.bfloat16, torch.float32}, {torch.float32}, {torch.uint8}


@_streamed
def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], exp_avg: Sequence[torch.Tensor],
               exp_avg_sq: Sequence[torch.Tensor], step: int = 1, lr: float = 1e-3,
               betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale: float = 1.0, master: Optional[Sequence[Optional[torch.Tensor]]] = None,
               scales: Optional[Tuple[Sequence[torch.Tensor], Sequence[torch.Tensor]]] = None,
               factors: Optional[torch.Tensor] = None, device_step: Optional[torch.Tensor] = None) -> None:
    """One AdamW step over all tensors, in place (ss1_adamw_step). params and grads: bf16 or float32, each
    tensor by itself. exp_avg and exp_avg_sq: float32; with `scales` = (of the first moment, of the
    root of the second one), float32 [ceil(numel / ADAMW_BLOCK)] each, uint8 E4M3 codes instead. `step` numbers
    the parameters' steps from 1 on: past ADAMW_NEAREST, codes are rounded up or down by a hash of it.
    master: float32 copies of bf16 params, which the step then reads and writes (None: has none). factors: float32
    CUDA tensor of adamw_factors, read on the device in place of step .. grad_scale. No tensor that is written may overlap
    another one of the call (but a gradient may be its parameter itself). device_step: int64 CUDA tensor [1],
    the step's number beside `factors`, read on the device too; 8-bit states with factors need it."""
    _adamw(params, grads, exp_avg, exp_avg_sq, 0 if device_step is not None else step, lr, betas, eps, weight_decay, grad_scale,
           master, scales, factors, device_step)


def _adamw(params, grads, exp_avg, exp_avg_sq, step, lr, betas, eps, weight_decay, grad_scale, master, scales, factors, device_step):
    """adamw_step; with a device_step, `step` is added to it."""
    n = len(params)
    if n == 0:
        return
    device = params[0].get_device()
    if device < 0:
        raise ValueError("params must be CUDA tensors")
    bits = 32 if scales is None else 8
    sizes = list(map(_NUMEL, params))
    table = np.zeros(n, _ADAMW_TENSOR)
    state = _F32 if bits == 32 else _U8
    changed = [*params, *exp_avg, *exp_avg_sq]
    table["param"], pt = _like("params", params, sizes, device, _WEIGHTS)
    table["grad"], gt = _like("grads", grads, sizes, device, _WEIGHTS)
    table["exp_avg"], _ = _like("exp_avg", exp_avg, sizes, device, state)
    table["exp_avg_sq"], _ = _like("exp_avg_sq", exp_avg_sq, sizes, device, state)
    table["param_dtype"] = _dtype_code(pt.pop()) if len(pt) == 1 else [_dtype_code(t.dtype) for t in params]
    table["grad_dtype"] = _dtype_code(gt.pop()) if len(gt) == 1 else [_dtype_code(t.dtype) for t in grads]
    table["numel"] = sizes
    if master is not None:
        if len(master) != n:
            raise ValueError(f"master: {len(master)} tensors for {n} parameters")
        if all(map(torch.is_tensor, master)):
            table["master"], _ = _like("master", master, sizes, device, _F32)
            changed += master
        else:
            some = [i for i, t in enumerate(master) if t is not None]
            if some:
                mine = [master[i] for i in some]
                table["master"][some], _ = _like("master", mine, [sizes[i] for i in some], device, _F32)
                changed += mine
    if scales is not None:
        blocks = [-(-size // ADAMW_BLOCK) for size in sizes]
        for k, name in enumerate(("avg_scale", "sq_scale")):
            table[name], _ = _like(f"scales[{k}]", scales[k], blocks, device, _F32)
            changed += scales[k]
    if factors is not None:
        _tensor("factors", factors, (ADAMW_FACTORS,), torch.float32, device)
    if device_step is not None:
        _tensor("device_step", device_step, (1,), torch.int64, device)
    if (device_step is not None) > (factors is not None) or (bits == 8 and factors is not None and device_step is None):
        raise ValueError("device_step goes with factors, and 8-bit states with factors need it")
    hyper = _AdamWHyper(lr, betas[0], betas[1], eps, weight_decay, grad_scale, step)
    try:
        _call(device, lib().ss1_adamw_step_ex, table.ctypes.data, n, bits, ctypes.byref(hyper), _ptr(factors), _ptr(device_step))
    except ss1.SS1Error as e:
        if e.status == -9:
            raise ValueError("a tensor is given twice, or overlaps another: parameters, moments, scales and master copies are "
                             "written at the same time") from None
        raise
    _written(changed)


class AdamW:
    """AdamW over a list of parameters: holds the states and calls adamw_step with each parameter's .grad
    (parameters without one are left as they are). Every parameter has a step number of its own, so one that
    gets its first gradient late starts with the bias corrections of step 1.

    state_bits: 32 or 8. master: float32 copies of the bf16 parameters.

    In a CUDA graph: capture step(factors=...) and write adamw_factors of the next step number to `factors`
    before each replay. The captured steps count their replays on the device."""

    def __init__(self, params, lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, master: bool = False):
        self.params: List[torch.Tensor] = list(params)
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        for i, p in enumerate(self.params):
            _tensor(f"params[{i}]", p, device=self.params[0].get_device())
            _dtype_code(p.dtype)
            if any(q is p for q in self.params[:i]):
                raise ValueError(f"params[{i}] is in the list twice")
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits = state_bits
        # steps that were run by the host, and replays of captured steps (of the parameters in _captured)
        self._counts = [0] * len(self.params)
        self._captured: Optional[List[int]] = None
        self._replays = self.params[0].new_zeros(1, dtype=torch.int64, requires_grad=False) if self.params else None
        state = torch.float32 if state_bits == 32 else torch.uint8
        self.exp_avg = [torch.zeros_like(p, dtype=state) for p in self.params]
        self.exp_avg_sq = [torch.zeros_like(p, dtype=state) for p in self.params]
        self.scales = None
        if state_bits == 8:
            self.scales = tuple([torch.zeros(-(-p.numel() // ADAMW_BLOCK), dtype=torch.float32, device=p.device)
                                 for p in self.params] for _ in range(2))
        self.master = [p.detach().float() if master and p.dtype == torch.bfloat16 else None for p in self.params]

    def zero_grad(self):
        for p in self.params:
            p.grad = None

    def counts(self) -> List[int]:
        """Each parameter's number of steps. Waits for the device once a step was captured."""
        if self._captured is None:
            return list(self._counts)
        torch.cuda.synchronize(self._replays.device)       # a replay may run on any stream
        replays, captured = int(self._replays), set(self._captured)
        return [c + replays if i in captured else c for i, c in enumerate(self._counts)]

    @property
    def steps(self) -> int:
        """The largest of the parameters' step numbers."""
        return max(self.counts(), default=0)

    @torch.no_grad()
    def step(self, grad_scale: float = 1.0, factors: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
        """One step; the step numbers of the parameters that have a gradient go up by one. `factors` as in
        adamw_step, for parameters that share a step number; a captured step needs them, and every captured step has to
        update the same parameters."""
        who = [i for i, p in enumerate(self.params) if p.grad is not None]
        if not who:
            return
        device = self.params[0].device
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the parameters on {device}")
        if stream is not None or torch.cuda.current_device() != device.index:
            with torch.cuda.device(device), torch.cuda.stream(stream):
                self._step(who, grad_scale, factors)
        else:
            self._step(who, grad_scale, factors)

    def _step(self, who: List[int], grad_scale: float, factors: Optional[torch.Tensor]):
        """step on the current device and stream, of the parameters `who`."""
        capturing = torch.cuda.is_current_stream_capturing()
        counts = self._counts if capturing or self._captured is None else self.counts()
        grads = [p.grad for p in self.params]
        if len({counts[i] for i in who}) == 1:
            groups = {counts[who[0]]: who}
        else:
            groups = {}
            for i in who:
                groups.setdefault(counts[i], []).append(i)
            if factors is not None:
                raise ValueError(f"factors are of one step number, the parameters are at {sorted(groups)}")
            # all gradients are checked before the first group's step
            _like("grads", [grads[i] for i in who], [self.params[i].numel() for i in who], self.params[0].get_device(), _WEIGHTS)
        if capturing:
            if factors is None:
                raise ValueError("a captured step needs factors: without them each replay would repeat one step number")
            if self._captured not in (None, who):
                raise ValueError("another captured step updates other parameters: load this state into a new AdamW for that")
            self._replays.add_(1)
        for count, group in groups.items():
            def of(ts):
                return ts if len(group) == len(ts) else [ts[i] for i in group]
            # with factors the number that 8-bit states round by is read on the device: the host's steps and the replays
            number = self._counts[group[0]] + (0 if capturing else 1) if factors is not None else count + 1
            _adamw(of(self.params), of(grads), of(self.exp_avg), of(self.exp_avg_sq), number, self.lr, self.betas, self.eps,
                   self.weight_decay, grad_scale, of(self.master),
                   None if self.scales is None else (of(self.scales[0]), of(self.scales[1])), factors,
                   self._replays if factors is not None else None)
        if capturing:
            self._captured = who
        else:
            for i in who:
                self._counts[i] += 1

    def state_dict(self) -> dict:
        """States and step numbers, for a checkpoint (tensors are the live ones)."""
        counts = self.counts()
        return {"steps": max(counts, default=0), "counts": counts, "state_bits": self.state_bits, "exp_avg": self.exp_avg,
                "exp_avg_sq": self.exp_avg_sq, "scales": self.scales, "master": self.master}

    def load_state_dict(self, state: dict):
        """Copies a state_dict of the same parameters and state_bits back in. One without "counts" has "steps" for all."""
        if state["state_bits"] != self.state_bits:
            raise ValueError(f"the state has {state['state_bits']} bits, this optimizer {self.state_bits}")
        counts = list(state.get("counts") or [state["steps"]] * len(self.params))
        if len(counts) != len(self.params):
            raise ValueError("the state is of other parameters")
        pairs = [(name, getattr(self, name), state[name]) for name in ("exp_avg", "exp_avg_sq", "master")]
        if self.scales is not None:
            pairs += [("scales", mine, theirs) for mine, theirs in zip(self.scales, state["scales"] or ((), ()))]
        for name, mine, theirs in pairs:       # everything is checked before anything is written
            if len(mine) != len(theirs) or any((a is None) != (b is None) for a, b in zip(mine, theirs)):
                raise ValueError(f"{name}: the state is of other parameters or master copies")
            if any(a is not None and (a.shape != b.shape or a.dtype != b.dtype) for a, b in zip(mine, theirs)):
                raise ValueError(f"{name}: a tensor of the state has another shape or type")
        with torch.no_grad():
            for _, mine, theirs in pairs:
                for a, b in zip(mine, theirs):
                    if a is not None:
                        a.copy_(b)
        replayed = [a - b for a, b in zip(self.counts(), self._counts)]
        self._counts = [c - r for c, r in zip(counts, replayed)]
