"""PyTorch functions and modules around the sublayer operators (argument marshalling only).

The operators of a pre-LN block outside the sharded MLP: LayerNorm with weight and bias, the linear layer
with bias, activation and residual, and causal attention over packed sequences with grouped heads.  The
first two have plain functions that allocate their outputs and call the C ABI (`layer_norm_fwd`,
`layer_norm_bwd`, `linear_fwd`, `linear_bwd`), a differentiable function (`layer_norm`, `linear`) and a
module (`DominoLayerNorm`, `DominoLinear`); the attention (`packed_attention`) is forward only.  The operators run in the library's kernels;
what PyTorch does beside them is to copy tensors that the library cannot stride over, to round the fp32 gradients of bf16
parameters, and to take the sequences' lengths from `cu_q` where they are not given.  Tensors must be on one CUDA device,
matrices bf16.

Calls run on the current stream of the tensors' device.  Workspaces come from PyTorch's allocator for each
call, so calls on several streams, and several captured graphs, share none.  One library handle per device
serves all threads; a lock is held while a call enqueues its kernels.
"""
from __future__ import annotations

import functools
import threading

import torch
import torch.autograd.forward_ad as forward_ad

from . import domino as dm

_handles: dict[int, int] = {}
_lock = threading.Lock()
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
# The current stream's handle as an integer and the current device, without the objects that torch.cuda builds
# around them (3 us a call on a Grace core).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# workspace sizes, functions of the shapes alone (a call through ctypes takes 1.3 us)
_norm_scratch, _linear_scratch, _packed_scratch = (functools.lru_cache(4096)(f) for f in (
    dm.domino_layernorm_bwd_workspace_size, dm.domino_linear_bwd_workspace_size, dm.domino_attn_packed_workspace_size))


# A workspace straight from PyTorch's allocator, on a stream as a tensor's memory would be, without a tensor around it
# (2 - 3 us a call less): given back as soon as the call is enqueued, it is reused in the stream's order.
_take = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_give = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)
if _take is None or _give is None:
    _take, _give = torch.cuda.caching_allocator_alloc, torch.cuda.caching_allocator_delete
    _take = functools.partial(lambda alloc, size, stream: alloc(size, stream=stream), _take)


def _call(fn, x: torch.Tensor, *args, scratch: int | None = None) -> None:
    """fn(handle, *args, stream) on the device of `x` and its current stream, under the lock; with `scratch`, a
    workspace of so many bytes and its size follow the arguments."""
    index = x.get_device()
    if _device() != index:
        with torch.cuda.device(index):
            return _call(fn, x, *args, scratch=scratch)
    with _lock:
        handle = _handles.get(index)
        if handle is None:
            handle = _handles[index] = dm.domino_create()
        stream = _raw_stream(index)
        if scratch is None:
            fn(handle, *args, stream=stream)
        elif scratch == 0:
            fn(handle, *args, None, 0, stream=stream)
        else:
            ws = _take(scratch, stream)
            try:
                fn(handle, *args, ws, scratch, stream=stream)
            finally:
                _give(ws)


def _check(name: str, x: torch.Tensor, like: torch.Tensor | None = None, shape=None, dtype=_BF16) -> None:
    """Refuses a tensor that is not on the GPU (that of `like`), or not of the shape or type."""
    if (isinstance(x, torch.Tensor) and x.dtype is dtype and x.is_cuda and (shape is None or x.shape == shape)
            and (like is None or x.get_device() == like.get_device())):
        return
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {x.dtype}")
    if like is not None and x.device != like.device:
        raise ValueError(f"{name} is on {x.device}, not on {like.device}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(x.shape)}")


def _rows(x: torch.Tensor) -> tuple[torch.Tensor, int]:
    """A 2-D tensor whose rows the library can stride over, and that stride: `x` itself where its rows
    are contiguous, 16-byte aligned and do not overlap, else a copy."""
    n, c = x.shape
    if x.is_contiguous() and x.data_ptr() % 16 == 0:
        return x, c
    ld, one = x.stride()
    if (one == 1 or c <= 1) and x.data_ptr() % 16 == 0:
        if n <= 1:
            return x, c
        if ld >= c and ld % 8 == 0:
            return x, ld
    return x.clone(memory_format=torch.contiguous_format), c


def _vec(x: torch.Tensor | None) -> torch.Tensor | None:
    """A vector the library can read: contiguous and 16-byte aligned."""
    if x is None or (x.is_contiguous() and x.data_ptr() % 16 == 0):
        return x
    return x.clone(memory_format=torch.contiguous_format)


def _no_tangent(what: str, *tensors: torch.Tensor | None) -> None:
    """Refuses tensors that carry a tangent: it would be lost, since the result is computed outside of autograd."""
    if getattr(forward_ad, "_current_level", 0) < 0:  # outside of every dual level
        return
    if any(isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError(f"{what} has no derivative in forward mode")


def _matrix(name: str, x: torch.Tensor) -> None:
    _check(name, x)
    if x.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {x.dim()}")


# ---- LayerNorm -----------------------------------------------------------------------------------

def _differentiated(*tensors: torch.Tensor | None) -> bool:
    """Whether a backward pass may follow."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5,
                   stats: bool = True):
    """LayerNorm of each row of x [rows, h] (bf16) with weight and bias (bf16): (y, mean, rstd), the last
    two fp32, for `layer_norm_bwd` (None without `stats`)."""
    _matrix("x", x)
    rows, h = x.shape
    _check("weight", weight, x, (h,))
    if bias is not None:
        _check("bias", bias, x, (h,))
    x, ld = _rows(x)
    weight, bias = _vec(weight), _vec(bias)
    y = torch.empty((rows, h), dtype=_BF16, device=x.device)
    mean = torch.empty(rows, dtype=_F32, device=x.device) if stats else None
    rstd = torch.empty(rows, dtype=_F32, device=x.device) if stats else None
    _call(dm.domino_layernorm_fwd, x, x, ld, weight, bias, eps, y, h, mean, rstd, rows, h)
    return y, mean, rstd


def layer_norm_bwd(gy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   gres: torch.Tensor | None = None, grads: tuple | None = None, bias_grad: bool = True):
    """Gradients of `layer_norm_fwd`: (gx, gweight, gbias), gx bf16 (with `gres`, the gradient of a
    residual connection around the LayerNorm, added before its rounding), the others fp32.  `grads`, a
    pair of fp32 buffers, is added to instead of allocated (main_grad accumulation)."""
    _matrix("gy", gy)
    _matrix("x", x)
    rows, h = x.shape
    _check("gy", gy, x, (rows, h))
    _check("weight", weight, x, (h,))
    _check("mean", mean, x, (rows,), torch.float32)
    _check("rstd", rstd, x, (rows,), torch.float32)
    if gres is not None:
        _check("gres", gres, x, (rows, h))
    if grads is not None:
        gw, gb = grads
        for name, g in (("weight", gw), ("bias", gb)):
            if g is None and name == "bias":
                continue
            _check(f"the {name}'s gradient buffer", g, x, (h,), torch.float32)
            if not g.is_contiguous() or g.data_ptr() % 16:
                raise ValueError(f"the {name}'s gradient buffer must be contiguous and 16-byte aligned")
    else:
        gw = torch.empty(h, dtype=_F32, device=x.device)
        gb = torch.empty(h, dtype=_F32, device=x.device) if bias_grad else None
    gy, ld_gy = _rows(gy)
    x, ld_x = _rows(x)
    ld_r = h
    if gres is not None:
        gres, ld_r = _rows(gres)
    weight, mean, rstd = _vec(weight), _vec(mean), _vec(rstd)
    gx = torch.empty((rows, h), dtype=_BF16, device=x.device)
    _call(dm.domino_layernorm_bwd, x, gy, ld_gy, x, ld_x, weight, mean, rstd, gres, ld_r, gx, h, gw, gb,
          int(grads is not None), rows, h, scratch=_norm_scratch(rows, h))
    return gx, gw, gb


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias = bias is not None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        x, weight, mean, rstd = ctx.saved_tensors
        gx, gw, gb = layer_norm_bwd(gy, x, weight, mean, rstd, bias_grad=ctx.bias)
        return gx, gw.to(weight.dtype), gb.to(weight.dtype) if ctx.bias else None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5):
    """Differentiable LayerNorm over the last dimension of x [..., h] (bf16); not in forward mode."""
    _no_tangent("layer_norm", x, weight, bias)
    _check("x", x)
    if x.dim() == 0:
        raise ValueError("x must have at least one dimension")
    if not _differentiated(x, weight, bias):
        return layer_norm_fwd(x.reshape(-1, x.shape[-1]), weight, bias, eps, stats=False)[0].view(x.shape)
    return _LayerNorm.apply(x.reshape(-1, x.shape[-1]), weight, bias, eps).view(x.shape)


class DominoLayerNorm(torch.nn.Module):
    """LayerNorm over the last dimension with bf16 weight and bias."""

    def __init__(self, h: int, eps: float = 1e-5, bias: bool = True, device: str | torch.device = "cuda"):
        super().__init__()
        self.h, self.eps = h, eps
        self.weight = torch.nn.Parameter(torch.ones(h, dtype=torch.bfloat16, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(h, dtype=torch.bfloat16, device=device)) if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.dim() == 0 or x.shape[-1] != self.h:
            raise ValueError(f"x must have {self.h} columns")
        return layer_norm(x, self.weight, self.bias, self.eps)


# ---- linear layer ----------------------------------------------------------------------------------

ACTS = {"none": dm.ACT_NONE, "relu": dm.ACT_RELU, "gelu": dm.ACT_GELU}


def _act(act) -> int:
    code = ACTS.get(act, act)
    if code not in ACTS.values():
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    return code


def _linear_shapes(x: torch.Tensor, weight: torch.Tensor) -> tuple[int, int, int]:
    _matrix("x", x)
    _matrix("weight", weight)
    n, k = weight.shape
    _check("weight", weight, x, (n, x.shape[1]))
    return x.shape[0], n, k


def linear_fwd(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, act="none",
               residual: torch.Tensor | None = None, save: bool = False):
    """y = act(x weight^T + bias) + residual for x [m, k], weight [n, k] (bf16): (y, z), z the
    pre-activation that `linear_bwd` needs, or None without `save`."""
    m, n, k = _linear_shapes(x, weight)
    act = _act(act)
    if bias is not None:
        _check("bias", bias, x, (n,))
    ld_r = n
    if residual is not None:
        _check("residual", residual, x, (m, n))
        residual, ld_r = _rows(residual)
    x, ld_x = _rows(x)
    weight, bias = _vec(weight), _vec(bias)
    y = torch.empty((m, n), dtype=_BF16, device=x.device)
    z = torch.empty_like(y) if save else None
    _call(dm.domino_linear_fwd, x, x, ld_x, weight, bias, act, residual, ld_r, y, n, z, n, m, n, k)
    return y, z


def linear_bwd(gy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, z: torch.Tensor | None = None, act="none",
               x_grad: bool = True, weight_grad: bool = True, bias_grad: bool = True, main_grad: torch.Tensor | None = None,
               bias_main_grad: torch.Tensor | None = None):
    """Gradients of `linear_fwd`: (gx, gweight, gbias), gx and gweight bf16, gbias fp32; None where not
    asked for.  With `main_grad` (fp32, like weight) the weight's gradient is added to it instead of
    returned; with `bias_main_grad` the bias's.  `z`: what the forward kept (act "none" needs none)."""
    m, n, k = _linear_shapes(x, weight)
    act = _act(act)
    _check("gy", gy, x, (m, n))
    ld_z = n
    if act != dm.ACT_NONE:
        if z is None:
            raise ValueError("the activation's gradient needs z")
        _check("z", z, x, (m, n))
        z, ld_z = _rows(z)
    else:
        z = None
    for name, g, shape in (("main_grad", main_grad, (n, k)), ("bias_main_grad", bias_main_grad, (n,))):
        if g is not None:
            _check(name, g, x, shape, torch.float32)
            if not g.is_contiguous() or g.data_ptr() % 16:
                raise ValueError(f"{name} must be contiguous and 16-byte aligned")
    gy, ld_gy = _rows(gy)
    x, ld_x = _rows(x)
    weight = _vec(weight)
    gx = torch.empty((m, k), dtype=_BF16, device=x.device) if x_grad else None
    gw = torch.empty((n, k), dtype=_BF16, device=x.device) if weight_grad and main_grad is None else None
    gb = bias_main_grad
    if gb is None and bias_grad:
        gb = torch.empty(n, dtype=_F32, device=x.device)
    _call(dm.domino_linear_bwd, x, gy, ld_gy, x, ld_x, weight, z, ld_z, act, gx, k, gw,
          main_grad if weight_grad else None, gb, int(bias_main_grad is not None), m, n, k,
          scratch=_linear_scratch(m, n, k, act))
    return gx, gw, gb


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, act, main_grad, bias_main_grad):
        y, z = linear_fwd(x, weight, bias, act, residual, save=act != dm.ACT_NONE)
        ctx.save_for_backward(x, weight, z)
        ctx.act, ctx.bias, ctx.main = act, bias is not None, (main_grad, bias_main_grad)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        x, weight, z = ctx.saved_tensors
        need = ctx.needs_input_grad
        main, bias_main = ctx.main
        gx, gw, gb = linear_bwd(gy, x, weight, z, ctx.act, need[0], need[1], ctx.bias and need[2], main if need[1] else None,
                                bias_main if ctx.bias and need[2] else None)
        if bias_main is not None:
            gb = None
        return gx, gw, gb.to(weight.dtype) if gb is not None else None, gy if need[3] else None, None, None, None


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, act="none",
           residual: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable y = act(x weight^T + bias) + residual for x [..., k] (bf16), the residual in y's shape or as its
    rows.  Where weight (bias) has an fp32 `main_grad`, its gradient is accumulated there and its `.grad` stays None.
    Where no gradient is asked for, the pre-activation is not kept.  Not differentiable in forward mode."""
    _no_tangent("linear", x, weight, bias, residual)
    _check("x", x)
    if x.dim() == 0:
        raise ValueError("x must have at least one dimension")
    _matrix("weight", weight)
    x2, r = x.reshape(-1, x.shape[-1]), residual
    if r is not None:
        _check("residual", r, x)
        rows = (x2.shape[0], weight.shape[0])
        if r.shape != rows:
            if r.shape != (*x.shape[:-1], weight.shape[0]):
                raise ValueError(f"residual must have the output's shape {(*x.shape[:-1], weight.shape[0])}, not {tuple(r.shape)}")
            r = r.reshape(rows)
    if not _differentiated(x, weight, bias, residual):
        y, _ = linear_fwd(x2, weight, bias, act, r)
    else:
        y = _Linear.apply(x2, weight, bias, r, _act(act), getattr(weight, "main_grad", None), getattr(bias, "main_grad", None))
    return y.view(*x.shape[:-1], weight.shape[0])


class DominoLinear(torch.nn.Module):
    """y = act(x weight^T + bias) + residual with bf16 parameters; with `fuse_wgrad` their gradients are
    accumulated in fp32 `main_grad` buffers, as in `DominoMLP`."""

    def __init__(self, k: int, n: int, bias: bool = True, act="none", fuse_wgrad: bool = False, init_std: float = 0.02,
                 device: str | torch.device = "cuda"):
        super().__init__()
        self.act = _act(act)
        self.weight = torch.nn.Parameter(torch.empty((n, k), dtype=torch.bfloat16, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(n, dtype=torch.bfloat16, device=device)) if bias else None
        with torch.no_grad():
            self.weight.normal_(0.0, init_std)
        if fuse_wgrad:
            for p in self.parameters():
                p.main_grad = torch.zeros(p.shape, dtype=torch.float32, device=device)

    def zero_main_grad(self) -> None:
        for p in self.parameters():
            if hasattr(p, "main_grad"):
                p.main_grad.zero_()

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        return linear(x, self.weight, self.bias, self.act, residual)


# ---- attention over packed sequences ---------------------------------------------------------------

HEAD_DIM = 128


def _heads(name: str, x: torch.Tensor) -> tuple[torch.Tensor, int]:
    """A [tokens, heads, 128] tensor with its heads one after the other, and its token stride."""
    t, h, d = x.shape
    if x.is_contiguous() and x.data_ptr() % 16 == 0:
        return x, h * d
    if x.data_ptr() % 16 == 0 and x.stride(2) == 1 and (h <= 1 or x.stride(1) == d):
        if t <= 1:
            return x, h * d
        if x.stride(0) >= h * d and x.stride(0) % 8 == 0:
            return x, x.stride(0)
    return x.clone(memory_format=torch.contiguous_format), h * d


def packed_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                     k_start: torch.Tensor | None = None, k_len: torch.Tensor | None = None, scale: float | None = None,
                     return_lse: bool = False, out: torch.Tensor | None = None):
    """Causal attention of n packed sequences, q [tq, heads, 128], k and v [tk, kv_heads, 128] (bf16).

    Sequence s has the queries cu_q[s] .. cu_q[s + 1] - 1 and the k_len[s] keys from row k_start[s]; its last
    query sees all of them, the one before all but the last, and so on (int32 tensors on the device, of n + 1,
    n and n values).  Without k_start and k_len the keys are the sequence's own rows, as in prompts.  The scale
    is 1 / sqrt(128) unless given.  Returns o, or (o, lse) with lse [tq, heads] fp32.  Rows that belong to no
    sequence are left as they were in `out` (undefined without it), which may not overlap q, k or v.  Lengths that leave the tensors are not
    raised here: they are read on the device, and `device_status` reports them.  Forward only."""
    _no_tangent("packed_attention", q, k, v)
    for name, x in (("q", q), ("k", k), ("v", v)):
        _check(name, x, q)
        if x.dim() != 3 or x.shape[2] != HEAD_DIM:
            raise ValueError(f"{name} must have shape [tokens, heads, {HEAD_DIM}], not {tuple(x.shape)}")
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        raise ValueError("packed_attention has no backward: call it under torch.no_grad(), or detach its inputs")
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    tq, hq, _ = q.shape
    tk, hkv, _ = k.shape
    if hkv == 0 or hq == 0 or hq % hkv:
        raise ValueError("the query heads must be a multiple of the key heads")
    _check("cu_q", cu_q, q, None, torch.int32)
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be a vector of n + 1 values")
    n = cu_q.numel() - 1
    if (k_start is None) != (k_len is None):
        raise ValueError("k_start and k_len go together")
    if k_start is None:
        if tk != tq:
            raise ValueError("without k_start and k_len, q and k must have the same rows")
        k_start, k_len = cu_q[:-1], cu_q.diff()
    _check("k_start", k_start, q, (n,), torch.int32)
    _check("k_len", k_len, q, (n,), torch.int32)
    q, ld_q = _heads("q", q)
    k, ld_k = _heads("k", k)
    v, ld_v = _heads("v", v)
    cu_q, k_start, k_len = (t.contiguous() for t in (cu_q, k_start, k_len))
    if out is None:
        out = torch.empty((tq, hq, HEAD_DIM), dtype=torch.bfloat16, device=q.device)
        ld_o = hq * HEAD_DIM
    else:
        _check("out", out, q, (tq, hq, HEAD_DIM))
        same, ld_o = _heads("out", out)
        if same is not out:
            raise ValueError("out must have contiguous, 16-byte aligned tokens that do not overlap")
    lse = torch.empty((tq, hq), dtype=torch.float32, device=q.device) if return_lse else None
    _call(dm.domino_attn_packed_fwd, q, q, ld_q, k, ld_k, v, ld_v, cu_q, k_start, k_len,
          HEAD_DIM ** -0.5 if scale is None else scale, out, ld_o, lse, tq, n, hq, hkv, tk,
          scratch=_packed_scratch(tq, n, hq, hkv, tk))
    return (out, lse) if return_lse else out


def device_status(device: torch.device | int | None = None) -> None:
    """Synchronises the device and raises DominoError if a call of this module's since the last look ran out
    of a wait or met lengths that leave their tensors."""
    x = torch.empty(0, device="cuda" if device is None else device)
    status, site = 0, 0

    def read(handle, stream):
        nonlocal status, site
        status, site = dm.domino_device_status(handle)

    _call(read, x)
    if status != dm.DOMINO_OK:
        what = "packed_attention met lengths that leave its tensors" if site == dm.BAD_LENGTHS_SITE else \
            f"a device-side wait ran out (site {site:#x})"
        raise dm.DominoError(status, what)
