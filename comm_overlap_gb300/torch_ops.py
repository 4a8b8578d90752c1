"""PyTorch functions and modules around the sublayer operators (argument marshalling only).

The operators of a pre-LN block outside the sharded MLP: LayerNorm with weight and bias, the linear layer
with bias, activation and residual, and causal attention over packed sequences with grouped heads.  The
first two have plain functions that allocate their outputs and call the C ABI (`layer_norm_fwd`,
`layer_norm_bwd`, `linear_fwd`, `linear_bwd`), a differentiable function (`layer_norm`, `linear`) and a
module (`DominoLayerNorm`, `DominoLinear`); the attention (`packed_attention`) is forward only.  Between the
projection and the attention stand the norm and rotation of query and key heads (`qk_rotary_fwd`, `qk_rotary_bwd`,
`qk_rotary`, `DominoQKRotary`); for serving, `cache_write` does the same and writes keys and values to an 8-bit cache
(`QuantizedCache`), which `cached_attention` reads for single tokens and drafts and `cache_read` gives back in bf16 for
`packed_attention`.  The operators run in the library's kernels;
what PyTorch does beside them is to copy tensors that the library cannot stride over, to round the fp32 gradients of bf16
parameters, and to take the sequences' lengths from `cu_q` where they are not given.  Tensors must be on one CUDA device,
matrices bf16.

Calls run on the current stream of the tensors' device.  Workspaces come from PyTorch's allocator for each
call, so calls on several streams, and several captured graphs, share none.  One library handle per device
serves all threads; a lock is held while a call enqueues its kernels.
"""
from __future__ import annotations

import ctypes
import functools
import math
import re
import threading
import warnings
from typing import NamedTuple

import torch
import torch.autograd.forward_ad as forward_ad

from . import domino as dm

_handles: dict[int, int] = {}
_lock = threading.Lock()
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_F64, _U8, _FP8 = torch.float64, torch.uint8, torch.float8_e4m3fn
# The current stream's handle as an integer and the current device, without the objects that torch.cuda builds
# around them (3 us a call on a Grace core).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# workspace sizes, functions of the shapes alone (a call through ctypes takes 1.3 us)
_norm_scratch, _linear_scratch, _packed_scratch, _rotary_scratch, _cached_scratch = (functools.lru_cache(4096)(f) for f in (
    dm.domino_layernorm_bwd_workspace_size, dm.domino_linear_bwd_workspace_size, dm.domino_attn_packed_workspace_size,
    dm.domino_qk_rotary_bwd_workspace_size, dm.domino_attn_cached_workspace_size))


# A workspace straight from PyTorch's allocator, on a stream as a tensor's memory would be, without a tensor around it
# (2 - 3 us a call less): given back as soon as the call is enqueued, it is reused in the stream's order.
_take = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_give = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)
if _take is None or _give is None:
    _take, _give = torch.cuda.caching_allocator_alloc, torch.cuda.caching_allocator_delete
    _take = functools.partial(lambda alloc, size, stream: alloc(size, stream=stream), _take)


# The short way of the last section's functions (csrc/torch_calls.cpp): outputs, or None where something is not of the plain
# form or is to be refused.  There from a device's first call on, if it could be built.
_short = None


def _shorten(index: int, handle: int) -> None:
    global _short
    try:
        from . import torch_calls
        built = torch_calls.built_for  # three numbers; what follows them here names the build
        if re.match(r"\d+\.\d+\.\d+", torch.__version__).group() != built:  # it reads tensors as that version lays them out
            raise ImportError(f"it was built for PyTorch {built}, this is {torch.__version__}")
    except (ImportError, AttributeError) as e:
        warnings.warn(f"calls of the rotation and the 8-bit cache take 10 us longer each: torch_calls is not there ({e})", stacklevel=4)
        return
    torch_calls.use_handle(index, handle)
    if _short is None:
        L = dm.lib()
        torch_calls.use(*(ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in (
            "domino_qk_rotary_fwd", "domino_qk_rotary_bwd", "domino_qk_rotary_bwd_workspace_size", "domino_cache_write",
            "domino_cache_read", "domino_attn_cached_fwd", "domino_attn_cached_workspace_size")), _lock)
        _short = torch_calls


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
            _shorten(index, handle)
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


# ---- norm and rotation of query and key heads -------------------------------------------------------

LAYOUTS = {"half": dm.ROTARY_HALF, "interleaved": dm.ROTARY_INTERLEAVED}


def rotary_frequencies(rot: int, base: float = 10000.0, factor: float = 1.0, original: int | None = None, slow: float = 1.0,
                       fast: float = 4.0, device: str | torch.device = "cuda") -> torch.Tensor:
    """Radians a position of the rot / 2 rotated pairs, base^(-2 i / rot), for `qk_rotary` and `cache_write` (fp64).  For
    contexts `factor` times longer they are all divided by it; with `original`, the length trained on, only those
    that turn fewer than `slow` times over it, while those that turn more than `fast` times stay, with a linear
    ramp between."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not (base > 0 and factor > 0 and fast > slow):
        raise ValueError("need base > 0, factor > 0 and fast > slow")
    f = base ** (-torch.arange(rot // 2, dtype=_F64) * 2 / rot)
    if original is None:
        f = f / factor
    else:
        keep = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f.to(device)


# The functions below try the short way first.  What it leaves is checked here, each property of a tensor looked at once: a Grace
# core takes 0.1 - 0.4 us for one.

def _device_index(name: str, x: torch.Tensor) -> int:
    if not isinstance(x, torch.Tensor) or x.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return x.get_device()


def _head_tensor(name: str, x: torch.Tensor, like: torch.Tensor, index: int, tokens: int | None = None, copy: bool = True):
    """(tensor, address, tokens, heads, token stride) of [tokens, heads, 128] bf16 heads one after the other, of a copy where
    they are not (with `copy`; else refused).  Hold the tensor until the call is enqueued."""
    if isinstance(x, torch.Tensor) and x.dtype is _BF16 and x.get_device() == index:
        shape = x.shape
        if len(shape) == 3 and shape[2] == HEAD_DIM and (tokens is None or shape[0] == tokens) and shape[1]:
            t, h, d = shape
            a, b, c = x.stride()
            p = x.data_ptr()
            if c == 1 and not p & 15 and (b == d or h == 1):
                if t <= 1:
                    return x, p, t, h, h * d
                if a >= h * d and not a & 7:
                    return x, p, t, h, a
            if not copy:
                if t == 0:
                    return x, p, t, h, h * d
                raise ValueError(f"{name} must have contiguous, 16-byte aligned tokens that do not overlap")
            x = x.clone(memory_format=torch.contiguous_format)
            return x, x.data_ptr(), t, h, h * d
    _check(name, x, like)
    raise ValueError(f"{name} must have shape [{'tokens' if tokens is None else tokens}, heads, {HEAD_DIM}], not {tuple(x.shape)}")


def _list(name: str, x: torch.Tensor, like: torch.Tensor, index: int, n: int, dtype) -> tuple[torch.Tensor, int]:
    """(tensor, address) of a contiguous vector of n values, a copy where it is not."""
    if not (isinstance(x, torch.Tensor) and x.dtype is dtype and x.get_device() == index and x.shape == (n,)):
        _check(name, x, like, (n,), dtype)
    if not x.is_contiguous():
        x = x.contiguous()
    return x, x.data_ptr()


def _rotation(x: torch.Tensor, index: int, tokens: int, positions, frequencies, layout, q_weight, k_weight, heads: int, kv_heads: int):
    """Checked arguments of a norm and rotation: addresses of positions, frequencies and the weights, rot, the layout's code, and
    the tensors to hold."""
    code = LAYOUTS.get(layout, layout)
    if code not in (dm.ROTARY_HALF, dm.ROTARY_INTERLEAVED):
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
    rot, at, by, wq, wk = 0, None, None, None, None
    if frequencies is not None and positions is not None:
        _check("frequencies", frequencies, x, None, _F64)
        if frequencies.dim() != 1:
            raise ValueError("frequencies must be a vector")
        rot = 2 * frequencies.shape[0]
        if rot > HEAD_DIM or rot % 16:
            raise ValueError(f"there must be a multiple of 8 frequencies, at most {HEAD_DIM // 2}, not {rot // 2}")
        frequencies, by = _list("frequencies", frequencies, x, index, rot // 2, _F64)
        positions, at = _list("positions", positions, x, index, tokens, _I32)
    elif frequencies is not None or positions is not None:
        raise ValueError("positions and frequencies go together")
    if q_weight is not None or k_weight is not None:
        if heads and kv_heads and (q_weight is None or k_weight is None):
            raise ValueError("q_weight and k_weight go together")
        if q_weight is not None and not heads or k_weight is not None and not kv_heads:
            raise ValueError("a weight needs its heads")
        if q_weight is not None:
            _check("q_weight", q_weight, x, _WEIGHT)
            q_weight = _vec(q_weight)
            wq = q_weight.data_ptr()
        if k_weight is not None:
            _check("k_weight", k_weight, x, _WEIGHT)
            k_weight = _vec(k_weight)
            wk = k_weight.data_ptr()
    return at, by, rot, code, wq, wk, (positions, frequencies, q_weight, k_weight)


_WEIGHT = (HEAD_DIM,)


def qk_rotary_fwd(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None, frequencies: torch.Tensor | None,
                  q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, layout="half", eps: float = 1e-6,
                  amplitude: float = 1.0, out: tuple | None = None):
    """RMS norm of each head of q [tokens, heads, 128] and k [tokens, kv_heads, 128] (bf16), with q_weight and k_weight
    (128 values, bf16; no norm without them), and the rotation of the first 2 x len(frequencies) values of each head by
    position x frequency, in one pass: (q', k').  positions: int32, one a token; frequencies: fp64 (`rotary_frequencies`),
    or None for no rotation.  layout: "half" (value i pairs with i + len(frequencies)) or "interleaved" (2 i with 2 i + 1);
    the rotated values are multiplied by `amplitude`.  q and k may be slices of a fused projection; k may be None.  `out`:
    tensors for (q', k'), which may be q and k."""
    if _short is not None and out is None:
        y = _short.qk_rotary_fwd(q, k, positions, frequencies, q_weight, k_weight, LAYOUTS.get(layout, layout), eps, amplitude)
        if y is not None:
            return y
    index = _device_index("q", q)
    q, pq, tokens, hq, ld_q = _head_tensor("q", q, q, index)
    pk, hkv, ld_k, yk, pyk, ld_yk = None, 0, 0, None, None, 0
    if k is not None:
        k, pk, _, hkv, ld_k = _head_tensor("k", k, q, index, tokens)
    at, by, rot, code, wq, wk, held = _rotation(q, index, tokens, positions, frequencies, layout, q_weight, k_weight, hq, hkv)
    if out is None:
        yq = torch.empty((tokens, hq, HEAD_DIM), dtype=_BF16, device=q.device)
        pyq, ld_yq = yq.data_ptr(), hq * HEAD_DIM
        if hkv:
            yk = torch.empty((tokens, hkv, HEAD_DIM), dtype=_BF16, device=q.device)
            pyk, ld_yk = yk.data_ptr(), hkv * HEAD_DIM
    else:
        yq, pyq, _, h, ld_yq = _head_tensor("out[0]", out[0], q, index, tokens, copy=False)
        if hkv:
            yk, pyk, _, h2, ld_yk = _head_tensor("out[1]", out[1], q, index, tokens, copy=False)
        if h != hq or hkv and h2 != hkv:
            raise ValueError("out must have as many heads as q and k")
    _call(dm.domino_qk_rotary_fwd, q, pq, ld_q, pk, ld_k, at, by, rot, code, amplitude, wq, wk, eps, pyq, ld_yq, pyk, ld_yk, tokens,
          hq, hkv)
    return yq, yk


def qk_rotary_bwd(gq: torch.Tensor, gk: torch.Tensor | None, q: torch.Tensor | None, k: torch.Tensor | None,
                  positions: torch.Tensor | None, frequencies: torch.Tensor | None, q_weight: torch.Tensor | None = None,
                  k_weight: torch.Tensor | None = None, layout="half", eps: float = 1e-6, amplitude: float = 1.0,
                  grads: tuple | None = None):
    """Gradients of `qk_rotary_fwd` from those of its outputs: (gq, gk, gq_weight, gk_weight), the first two bf16, the others
    fp32 (None without weights).  q and k, the forward's inputs, are needed with weights only.  `grads`, a pair of fp32
    buffers for the weights' gradients, is added to instead of allocated."""
    if _short is not None and grads is None:
        g = _short.qk_rotary_bwd(gq, gk, q, k, positions, frequencies, q_weight, k_weight, LAYOUTS.get(layout, layout), eps, amplitude)
        if g is not None:
            return g
    index = _device_index("gq", gq)
    gq, pgq, tokens, hq, ld_gyq = _head_tensor("gq", gq, gq, index)
    pgk, hkv, ld_gyk, yk, pyk = None, 0, 0, None, None
    if gk is not None:
        gk, pgk, _, hkv, ld_gyk = _head_tensor("gk", gk, gq, index, tokens)
    at, by, rot, code, wq, wk, held = _rotation(gq, index, tokens, positions, frequencies, layout, q_weight, k_weight, hq, hkv)
    gwq = gwk = pq = pk = None
    ld_q = ld_k = 0
    if wq is not None:
        if q is None or (k is None) != (gk is None):
            raise ValueError("the norm's gradient needs q and k")
        q, pq, _, h, ld_q = _head_tensor("q", q, gq, index, tokens)
        h2 = hkv
        if hkv:
            k, pk, _, h2, ld_k = _head_tensor("k", k, gq, index, tokens)
        if h != hq or h2 != hkv:
            raise ValueError("q and k must have as many heads as their gradients")
        if grads is not None:
            gwq, gwk = grads
            for name, g in (("gq_weight", gwq), ("gk_weight", gwk)):
                if name == "gk_weight" and not hkv:
                    continue
                _check(f"the buffer of {name}", g, gq, _WEIGHT, _F32)
                if not g.is_contiguous() or g.data_ptr() % 16:
                    raise ValueError(f"the buffer of {name} must be contiguous and 16-byte aligned")
        else:
            gwq = torch.empty(HEAD_DIM, dtype=_F32, device=gq.device)
            gwk = torch.empty(HEAD_DIM, dtype=_F32, device=gq.device) if hkv else None
    yq = torch.empty((tokens, hq, HEAD_DIM), dtype=_BF16, device=gq.device)
    if hkv:
        yk = torch.empty((tokens, hkv, HEAD_DIM), dtype=_BF16, device=gq.device)
        pyk = yk.data_ptr()
    _call(dm.domino_qk_rotary_bwd, gq, pgq, ld_gyq, pgk, ld_gyk, pq, ld_q, pk, ld_k, at, by, rot, code, amplitude, wq, wk, eps,
          yq.data_ptr(), hq * HEAD_DIM, pyk, hkv * HEAD_DIM, gwq, gwk, int(grads is not None), tokens, hq, hkv,
          scratch=_rotary_scratch(tokens, hq, hkv) if wq is not None else 0)
    return yq, yk, gwq, gwk


class _QKRotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, frequencies, q_weight, k_weight, layout, eps, amplitude):
        y = qk_rotary_fwd(q, k, positions, frequencies, q_weight, k_weight, layout, eps, amplitude)
        norm = q_weight is not None
        ctx.save_for_backward(q if norm else None, k if norm else None, positions, frequencies, q_weight, k_weight)
        ctx.how = layout, eps, amplitude
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        q, k, positions, frequencies, wq, wk = ctx.saved_tensors
        gq, gk, gwq, gwk = qk_rotary_bwd(gq, gk, q, k, positions, frequencies, wq, wk, *ctx.how)
        return (gq, gk, None, None, gwq.to(wq.dtype) if gwq is not None else None, gwk.to(wk.dtype) if gwk is not None else None, None,
                None, None)


def qk_rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None, frequencies: torch.Tensor | None,
              q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, layout="half", eps: float = 1e-6,
              amplitude: float = 1.0):
    """Differentiable `qk_rotary_fwd`: (q', k'); not in forward mode, and not by the frequencies."""
    _no_tangent("qk_rotary", q, k, q_weight, k_weight)
    if not _differentiated(q, k, q_weight, k_weight):
        return qk_rotary_fwd(q, k, positions, frequencies, q_weight, k_weight, layout, eps, amplitude)
    return _QKRotary.apply(q, k, positions, frequencies, q_weight, k_weight, layout, eps, amplitude)


class DominoQKRotary(torch.nn.Module):
    """Norm of query and key heads (with `norm`: bf16 weights) and rotation of their first `rot` values; `scaling`: what
    `rotary_frequencies` takes beyond rot and base."""

    def __init__(self, rot: int = HEAD_DIM, base: float = 10000.0, layout="half", norm: bool = True, eps: float = 1e-6,
                 amplitude: float = 1.0, device: str | torch.device = "cuda", **scaling):
        super().__init__()
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
        self.layout, self.eps, self.amplitude = layout, eps, amplitude
        self._how = rot, base, scaling
        self.frequencies = rotary_frequencies(rot, base, device=device, **scaling)  # fp64 whatever the module is cast to
        self.q_weight, self.k_weight = (
            torch.nn.Parameter(torch.ones(HEAD_DIM, dtype=_BF16, device=device)) if norm else None for _ in range(2))

    def _apply(self, fn, recurse=True):
        super()._apply(fn, recurse)
        device = fn(self.frequencies).device
        if self.frequencies.is_meta and device.type != "meta":  # built without memory, which it gets now
            rot, base, scaling = self._how
            self.frequencies = rotary_frequencies(rot, base, device=device, **scaling)
        else:
            self.frequencies = self.frequencies.to(device)
        return self

    def forward(self, q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor):
        return qk_rotary(q, k, positions, self.frequencies, self.q_weight, self.k_weight, self.layout, self.eps, self.amplitude)

    def write(self, cache: "QuantizedCache", rows: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              positions: torch.Tensor) -> torch.Tensor:
        """The same for serving: k and v into the cache (`cache_write`), q' returned."""
        return cache_write(cache, rows, k, v, q, positions, self.frequencies, self.q_weight, self.k_weight, self.layout, self.eps,
                           self.amplitude)


# ---- the 8-bit cache of keys and values ---------------------------------------------------------------

EXP_BIAS = 127


class QuantizedCache(NamedTuple):
    """Keys and values as E4M3 codes [rows, kv_heads, 128], each row and head with a power of two: its exponent + 127 in
    k_exp and v_exp [kv_heads, rows].  Sequences lie in ranges of rows, as in the caches of `packed_attention`."""
    k: torch.Tensor
    v: torch.Tensor
    k_exp: torch.Tensor
    v_exp: torch.Tensor

    @staticmethod
    def empty(rows: int, kv_heads: int, device: str | torch.device = "cuda") -> "QuantizedCache":
        codes = [torch.zeros((rows, kv_heads, HEAD_DIM), dtype=_U8, device=device).view(_FP8) for _ in range(2)]
        return QuantizedCache(*codes, *(torch.full((kv_heads, rows), EXP_BIAS, dtype=_U8, device=device) for _ in range(2)))


def _cache(cache: tuple, like: torch.Tensor, index: int):
    """(k, v, k_exp, v_exp) addresses of a cache, the row stride of its exponents, its rows and its heads."""
    k, v, ke, ve = cache
    shape = k.shape if isinstance(k, torch.Tensor) else ()
    if not (len(shape) == 3 and k.dtype is _FP8 and k.get_device() == index and shape[2] == HEAD_DIM and shape[1]):
        _check("the cache's k", k, like, None, _FP8)
        raise ValueError(f"the cache's k must have shape [rows, kv_heads, {HEAD_DIM}], not {tuple(shape)}")
    rows, hkv, _ = shape
    _check("the cache's v", v, like, shape, _FP8)
    _check("the cache's k_exp", ke, like, (hkv, rows), _U8)
    _check("the cache's v_exp", ve, like, (hkv, rows), _U8)
    pk, pv = k.data_ptr(), v.data_ptr()
    if not (k.is_contiguous() and v.is_contiguous()) or pk & 15 or pv & 15:
        raise ValueError("the cache's k and v must be contiguous and 16-byte aligned")
    ld = rows
    if not (ke.is_contiguous() and ve.is_contiguous()):
        ld = ke.stride(0)
        if ke.stride() != ve.stride() or (rows > 1 and ke.stride(1) != 1) or (hkv > 1 and ld < rows):
            raise ValueError("the cache's k_exp and v_exp must have contiguous rows that do not overlap, and the same strides")
        ld = max(ld, rows)
    return (pk, pv, ke.data_ptr(), ve.data_ptr()), ld, rows, hkv


def cache_write(cache: tuple, rows: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
                positions: torch.Tensor | None = None, frequencies: torch.Tensor | None = None,
                q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, layout="half", eps: float = 1e-6,
                amplitude: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Writes the tokens of k and v [tokens, kv_heads, 128] (bf16) to the rows `rows` (int32, one a token) of the cache,
    quantised: for each token and head the least power of two at which the largest value fits E4M3.  With weights or
    frequencies the keys are normed and rotated before, as in `qk_rotary_fwd`, and so is q [tokens, heads, 128] in the same
    pass, which is returned (`out`: a tensor for it, which may be q).  Negative rows are not written; rows beyond the cache
    neither, and `device_status` reports them; a row must not be given twice.  No gradients."""
    _no_tangent("cache_write", q, k, v, q_weight, k_weight)
    if _short is not None and out is None:
        y = _short.cache_write(cache, rows, k, v, q, positions, frequencies, q_weight, k_weight, LAYOUTS.get(layout, layout), eps, amplitude)
        if y is not None:
            return y[0]
    if _differentiated(q, k, v, q_weight, k_weight):
        raise ValueError("cache_write has no backward: call it under torch.no_grad(), or detach its inputs")
    index = _device_index("k", k)
    k, pk, tokens, hkv, ld_k = _head_tensor("k", k, k, index)
    v, pv, _, h, ld_v = _head_tensor("v", v, k, index, tokens)
    if h != hkv:
        raise ValueError(f"v has {h} heads, k {hkv}")
    codes, ld_exp, cache_rows, h = _cache(cache, k, index)
    if h != hkv:
        raise ValueError(f"k has {hkv} heads, the cache {h}")
    rows, at_rows = _list("rows", rows, k, index, tokens, _I32)
    pq, hq, ld_q, y, py, ld_y = None, 0, 0, None, None, 0
    if q is not None:
        q, pq, _, hq, ld_q = _head_tensor("q", q, k, index, tokens)
    at, by, rot, code, wq, wk, held = _rotation(k, index, tokens, positions, frequencies, layout, q_weight, k_weight, hq, hkv)
    if hq and out is None:
        y = torch.empty((tokens, hq, HEAD_DIM), dtype=_BF16, device=k.device)
        py, ld_y = y.data_ptr(), hq * HEAD_DIM
    elif hq:
        y, py, _, h, ld_y = _head_tensor("out", out, k, index, tokens, copy=False)
        if h != hq:
            raise ValueError("out must have as many heads as q")
    _call(dm.domino_cache_write, k, pq, ld_q, pk, ld_k, pv, ld_v, at, by, rot, code, amplitude, wq, wk, eps, py, ld_y, at_rows, *codes,
          ld_exp, cache_rows, tokens, hq, hkv)
    return y


def cache_read(cache: tuple, rows: torch.Tensor, out: tuple | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """What the cache holds in the rows `rows` (int32): (k, v), each [len(rows), kv_heads, 128] in bf16, exact; zeros where a
    row is negative, or beyond the cache, which `device_status` reports.  `out`: tensors for them."""
    if _short is not None and out is None:
        x = _short.cache_read(cache, rows)
        if x is not None:
            return x
    index = _device_index("rows", rows)
    if rows.dim() != 1:
        raise ValueError("rows must be a vector")
    tokens = rows.shape[0]
    rows, at_rows = _list("rows", rows, rows, index, tokens, _I32)
    codes, ld_exp, cache_rows, hkv = _cache(cache, rows, index)
    if out is None:
        k, v = (torch.empty((tokens, hkv, HEAD_DIM), dtype=_BF16, device=rows.device) for _ in range(2))
        pk, pv, ld_k, ld_v = k.data_ptr(), v.data_ptr(), hkv * HEAD_DIM, hkv * HEAD_DIM
    else:
        k, pk, _, h, ld_k = _head_tensor("out[0]", out[0], rows, index, tokens, copy=False)
        v, pv, _, h2, ld_v = _head_tensor("out[1]", out[1], rows, index, tokens, copy=False)
        if h != hkv or h2 != hkv:
            raise ValueError("out must have as many heads as the cache")
    _call(dm.domino_cache_read, rows, *codes, ld_exp, cache_rows, at_rows, pk, ld_k, pv, ld_v, tokens, hkv)
    return k, v


def cached_attention(q: torch.Tensor, cache: tuple, k_start: torch.Tensor, k_len: torch.Tensor,
                     prefix: torch.Tensor | None = None, scale: float | None = None, return_lse: bool = False,
                     out: torch.Tensor | None = None):
    """Attention of the last tokens of n sequences over the 8-bit cache: q [n, heads, 128], one token a sequence, or
    [n, t, heads, 128] (bf16).

    Sequence s has the k_len[s] keys from cache row k_start[s] (int32, n each, on the device); its query i of t sees the
    first k_len[s] - t + i + 1 of them.  `prefix`: int32 [first row, rows] on the device, keys that every query of every
    sequence sees before its own; they are read once for all.  The scale is 1 / sqrt(128) unless given.  Returns o like q,
    or (o, lse) with lse fp32, q without its last dimension.  A query that sees no key gets zeros and -inf.  `out` may not
    overlap q.  Lengths that leave the cache are not raised here: they are read on the device, such a sequence has no keys,
    and `device_status` reports them.  Forward only.  Made for few tokens a sequence: for long chunks, `cache_read` and
    `packed_attention`."""
    _no_tangent("cached_attention", q)
    if scale is None:
        scale = HEAD_DIM ** -0.5
    if _short is not None and out is None:
        y = _short.cached_attention(q, cache, k_start, k_len, prefix, scale, bool(return_lse))
        if y is not None:
            return y if return_lse else y[0]
    index = _device_index("q", q)
    shape = q.shape
    if len(shape) not in (3, 4) or shape[-1] != HEAD_DIM:
        raise ValueError(f"q must have shape [n, heads, {HEAD_DIM}] or [n, t, heads, {HEAD_DIM}], not {tuple(shape)}")
    if q.requires_grad and torch.is_grad_enabled():
        raise ValueError("cached_attention has no backward: call it under torch.no_grad(), or detach its inputs")
    codes, ld_exp, cache_rows, hkv = _cache(cache, q, index)
    n, t = shape[0], 1
    if len(shape) == 4:
        t = shape[1]
        q = q.reshape(n * t, shape[2], HEAD_DIM)
    q, pq, tokens, hq, ld_q = _head_tensor("q", q, q, index)
    if hq % hkv:
        raise ValueError("the query heads must be a multiple of the cache's heads")
    k_start, at_start = _list("k_start", k_start, q, index, n, _I32)
    k_len, at_len = _list("k_len", k_len, q, index, n, _I32)
    at_prefix = None
    if prefix is not None:
        prefix, at_prefix = _list("prefix", prefix, q, index, 2, _I32)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
        po, ld_o = out.data_ptr(), hq * HEAD_DIM
    else:
        _check("out", out, q, shape)
        try:
            o = out.view(tokens, hq, HEAD_DIM)
        except RuntimeError:
            raise ValueError("out must have tokens at one stride") from None
        _, po, _, _, ld_o = _head_tensor("out", o, q, index, tokens, copy=False)
    lse = torch.empty(shape[:-1], dtype=_F32, device=q.device) if return_lse else None
    _call(dm.domino_attn_cached_fwd, q, pq, ld_q, *codes, ld_exp, cache_rows, at_start, at_len, at_prefix,
          scale, po, ld_o, lse, n, t, hq, hkv,
          scratch=_cached_scratch(n, t, hq, hkv, int(prefix is not None)))
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
        what = "a call met lengths or rows that leave its tensors" if site == dm.BAD_LENGTHS_SITE else \
            f"a device-side wait ran out (site {site:#x})"
        raise dm.DominoError(status, what)
