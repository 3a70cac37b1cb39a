"""Layers on 4-bit codes (include/bakron_q4.h): packing, the linear layer, its
input gradient and a mixture-of-experts layer.

As in the rest of the binding, arguments are checked here, every arithmetic
step runs in the library's HIP kernels, and there is no fallback.  The
calls are made once per layer and token, so the checks are kept to
attribute reads (no tensor is looked into: no copy, no synchronisation).
"""
from __future__ import annotations

import contextlib
import ctypes

import torch
from torch.autograd import forward_ad as _forward

from . import _binding as _b

BAKRON_Q4_BF16 = 0
BAKRON_Q4_FP16 = 1
BAKRON_Q4_MAX_TOKENS = 16777216
BAKRON_Q4_MAX_LAYERS = 256
BAKRON_Q4_MOE_MAX_TOKENS = 64
BAKRON_Q4_MOE_MAX_TOP_K = 16

_VP, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_LINEAR = [_VP, _I64, _I64, _I32, _VP, _I64, _I64, _I64, _VP, _I64, _VP, _SZ, _VP]
_b.SIGNATURES.update({
    "bakron_q4_packed_bytes": (_SZ, [_I64] * 4),
    "bakron_q4_pack": (ctypes.c_int, [_VP, _VP, _VP, _I64, _I64, _I64, _I64, _VP, _VP]),
    "bakron_q4_linear_workspace_bytes": (_SZ, [_I64] * 4),
    "bakron_q4_linear": (ctypes.c_int, _LINEAR),
    "bakron_q4_linear_grad_workspace_bytes": (_SZ, [_I64] * 4),
    "bakron_q4_linear_grad": (ctypes.c_int, _LINEAR),
    "bakron_q4_moe_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I32, _I64]),
    "bakron_q4_moe": (ctypes.c_int, [_VP, _I64, _I64, _I32, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _I32, _I64, _VP, _I64,
                                     _VP, _VP, _VP, _SZ, _VP]),
})

_TYPES = {torch.bfloat16: BAKRON_Q4_BF16, torch.float16: BAKRON_Q4_FP16}


class Q4Weight:
    """One layer (count 1) or a stack of ``count`` layers of m x n in the
    packed layout, with group_size columns per grid (None: one grid per row).
    ``data`` is the device buffer (uint8) that holds it, as q4_pack makes it (its size is
    not checked again by every call).  ``w[e]`` is layer e of
    a stack alone, on the same memory: what q4_linear takes (q4_experts takes the
    stack as it is)."""

    __slots__ = ("data", "count", "m", "n", "group_size", "_group")

    def __init__(self, data, count, m, n, group_size):
        self.data, self.count, self.m, self.n, self.group_size = data, count, m, n, group_size
        self._group = group_size or 0

    @property
    def device(self):
        return self.data.device

    def __len__(self):
        return self.count

    def __getitem__(self, e):
        if not 0 <= e < self.count:
            raise IndexError(f"layer {e} of {self.count}")
        size = _b.lib().bakron_q4_packed_bytes(1, self.m, self.n, self._group)
        return Q4Weight(self.data[e * size:(e + 1) * size], 1, self.m, self.n, self.group_size)

    def __repr__(self):
        return f"Q4Weight(count={self.count}, m={self.m}, n={self.n}, group_size={self.group_size})"


def _group(group_size):
    if group_size is None:
        return 0
    if group_size <= 0 or group_size % 64:
        raise ValueError("group_size must be a positive multiple of 64")
    return int(group_size)


def q4_pack(codes, scale, zero, *, group_size=None, stream=None, check=True):
    """bakron_q4_pack: the packed form of a rounded layer (codes m x n, grids m
    or m x ceil(n / group_size)) or of a stack of layers (one more dimension
    in front): codes uint8 in [0, 15], scale and zero float32, as solve() and
    gptq() take and return them.  ``check``: raise GridError if a code is
    above 15, a scale neither 0 nor of magnitude 2^-100 .. 2^100 or a zero
    point not finite (reads them back to the host on ``stream``, which waits
    for the work there that makes them)."""
    g = _group(group_size)
    if not isinstance(codes, torch.Tensor) or codes.dim() not in (2, 3):
        raise ValueError("codes must be an m x n or count x m x n tensor")
    lead, (m, n) = tuple(codes.shape[:-2]), codes.shape[-2:]
    count = lead[0] if lead else 1
    _b._check_dev("codes", codes, torch.uint8, lead + (m, n))
    gshape = lead + ((m, -(-n // g)) if g else (m,))
    if not g and isinstance(scale, torch.Tensor) and scale.dim() == len(lead) + 2:
        gshape = lead + (m, 1)
    _b._check_dev("scale", scale, torch.float32, gshape)
    _b._check_dev("zero", zero, torch.float32, gshape)
    index = codes.get_device()
    _one_device(index, stream, scale=scale, zero=zero)
    if _device() != index:
        with torch.cuda.device(index):
            return q4_pack(codes, scale, zero, group_size=group_size, stream=stream, check=check)
    if check and codes.numel():
        with _on(stream):
            size = scale.abs()
            steps = (((size >= 2.0**-100) & (size <= 2.0**100)) | (size == 0)).all()   # False for NaN
            high, finite = torch.stack((codes.max() > 15, steps & torch.isfinite(zero).all())).tolist()
        if high:
            raise _b.GridError("codes must lie in [0, 15]")
        if not finite:
            raise _b.GridError("scale must be 0 or of magnitude 2^-100 .. 2^100, zero finite")
    data, = _made(stream, lambda: (_b.workspace(_b.lib().bakron_q4_packed_bytes(count, m, n, g), codes.device),))
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    call = "bakron_q4_pack"
    _check(_calls[call](codes.data_ptr(), scale.data_ptr(), zero.data_ptr(), count, m, n, g, data.data_ptr(), s), call)
    return Q4Weight(data, count, m, n, group_size)


def q4_linear_workspace_bytes(tokens: int, w: Q4Weight) -> int:
    return _b.lib().bakron_q4_linear_workspace_bytes(tokens, w.m, w.n, w._group)


def q4_linear_grad_workspace_bytes(tokens: int, w: Q4Weight) -> int:
    return _b.lib().bakron_q4_linear_grad_workspace_bytes(tokens, w.m, w.n, w._group)


def q4_moe_workspace_bytes(tokens: int, w_gate: Q4Weight, top_k: int) -> int:
    return _b.lib().bakron_q4_moe_workspace_bytes(tokens, w_gate.n, w_gate.m, w_gate.count, top_k, w_gate._group)


def _no_tangent(name, t):
    """Refuses a dual tensor of forward-mode autograd, whose tangent the calls would drop."""
    if _forward.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} has a forward-mode tangent, and the call has no derivative in forward mode")


def _rows(name, t, cols, like=None):
    """Leading dimension of a tokens x cols matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if _forward._current_level >= 0:   # (inside a dual_level)
        _no_tangent(name, t)
    if t.dtype not in _TYPES or (like is not None and t.dtype != like):
        raise TypeError(f"{name} must be {like or 'torch.bfloat16 or torch.float16'}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols:
        raise ValueError(f"{name} must have shape (tokens, {cols}), got {tuple(shape)}")
    ld, inner = t.stride()
    if cols > 1 and inner != 1 and shape[0]:   # (no rows: any strides, as autograd's are)
        raise ValueError(f"{name} must have contiguous rows")
    if shape[0] <= 1 or cols == 0:
        return cols
    if ld < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    return ld


def _one(name, w, index, count=1):
    if not isinstance(w, Q4Weight):
        raise TypeError(f"{name} must be a Q4Weight (q4_pack)")
    if w.count != count:
        raise ValueError(f"{name} must hold {count} layer(s), got {w.count}")
    if w.data.get_device() != index:
        raise ValueError(f"{name} is on {w.device}, not on cuda:{index}")


def _workspace(need, device, stream):
    if not need:
        return None
    with _on(stream):
        return _b.workspace(need, device)


def _refuse(ws, index):
    if ws.get_device() != index:
        raise ValueError(f"ws is on {ws.device}, not on cuda:{index}")
    raise ValueError("ws must be contiguous")   # its bytes are counted as if each were its own


# The current stream's handle without a Stream object around it (a call of
# one token's layer takes less time than making that).
_raw_stream = torch._C._cuda_getCurrentRawStream


_HERE = contextlib.nullcontext()


def _one_device(index, stream, **tensors):
    """Every tensor and the stream have to be on the device of the first one."""
    for name, t in tensors.items():
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if stream is not None and stream.device_index != index:
        raise ValueError(f"stream is on cuda:{stream.device_index}, not on cuda:{index}")


_device = torch._C._cuda_getDevice
_grad_on = torch.is_grad_enabled


def _check(rc, call):
    if rc != _b.BAKRON_SUCCESS:
        raise _b.BakronError(rc, call)


def _on(stream):
    """Where results and workspaces of a call on ``stream`` are made: in that
    stream's memory pool.  A block of the current stream's could still be in
    use there, by work that is only ordered before the current stream's own
    next use of it."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _made(stream, make):
    """Results of a call on ``stream``, made there, that the caller will use on
    the current one: torch's allocator has to wait for that too before it
    hands them out again."""
    if stream is None:
        return make()
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        results = make()
    for t in results:
        t.record_stream(here)
    return results


_increment = torch._C._increment_version


def _plain_outputs(*tensors):
    """Given outputs that require a gradient would keep the one of what they held before."""
    for t in tensors:
        if t.requires_grad and _grad_on():
            raise ValueError("out must not require a gradient")


def _written(*tensors):
    """Given outputs count as changed in place, as torch's own do: autograd then refuses
    a backward pass that would read what was saved there before."""
    try:
        _increment(tensors)
    except RuntimeError:                     # (inference tensors, which have no version, among them)
        _increment([t for t in tensors if not t.is_inference()])


class _Calls(dict):
    """The library's functions by name (an attribute of it is looked up anew
    each time)."""

    def __missing__(self, name):
        f = self[name] = getattr(_b.lib(), name)
        return f


_calls = _Calls()


def _linear(call, size, name, x, w, out, ws, stream):
    if not isinstance(w, Q4Weight):
        raise TypeError("w must be a Q4Weight (q4_pack)")
    in_cols, out_cols = (w.n, w.m) if name == "x" else (w.m, w.n)
    ldx = _rows(name, x, in_cols)
    index, T, data = x.get_device(), x.shape[0], w.data
    if w.count != 1 or data.get_device() != index:
        _one("w", w, index)
    if _device() != index:
        # kernels go to the current device, and the default stream's handle
        # names none
        with torch.cuda.device(index):
            return _linear(call, size, name, x, w, out, ws, stream)
    if stream is None:
        s = _raw_stream(index)
    else:
        _one_device(index, stream)
        s = stream.cuda_stream
    if x.requires_grad and _grad_on():
        if out is not None:
            raise ValueError(f"out cannot be given where {name} requires a gradient")
        both = (q4_linear, q4_linear_grad) if name == "x" else (q4_linear_grad, q4_linear)
        return _Differentiable.apply(x, w, *both, ws, stream)
    given = out is not None
    if not given:
        out = x.new_empty((T, out_cols)) if stream is None else _made(stream, lambda: (x.new_empty((T, out_cols)),))[0]
        ldo = out_cols
    else:
        ldo = _rows("out", out, out_cols, x.dtype)
        if out.shape[0] != T or out.get_device() != index:
            raise ValueError(f"out must be a ({T}, {out_cols}) tensor on {x.device}")
        _plain_outputs(out)
    if ws is None:
        ws = _workspace(size(T, w), x.device, stream)
    elif ws.get_device() != index or not ws.is_contiguous():
        _refuse(ws, index)
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)
    rc = _calls[call](x.data_ptr(), ldx, T, _TYPES[x.dtype], data.data_ptr(), w.m, w.n, w._group, out.data_ptr(), ldo, wp, wn, s)
    if rc:
        _check(rc, call)
    if given:
        _written(out)
    return out


class _Differentiable(torch.autograd.Function):
    """q4_linear and q4_linear_grad, each the other's derivative (the codes and
    grids have none)."""

    @staticmethod
    def forward(ctx, v, w, call, back, ws, stream):
        ctx.w, ctx.back = w, back
        return call(v, w, ws=ws, stream=stream)

    @staticmethod
    def backward(ctx, g):
        # (a sum's gradient, say, is one value expanded)
        return ctx.back(g.contiguous(), ctx.w), None, None, None, None, None


def q4_linear(x, w, *, out=None, ws=None, stream=None):
    """bakron_q4_linear: y = x W^T (tokens x m) of one packed layer, x tokens x n
    in bfloat16 or float16 (rows contiguous, any row stride).  ``out``: where
    to write y; ``ws``: a workspace of q4_linear_workspace_bytes.  Where x
    requires a gradient (and ``out`` is not given), autograd takes it with
    q4_linear_grad."""
    return _linear("bakron_q4_linear", q4_linear_workspace_bytes, "x", x, w, out, ws, stream)


def q4_linear_grad(dy, w, *, out=None, ws=None, stream=None):
    """bakron_q4_linear_grad: dx = dy W (tokens x n), the gradient of q4_linear
    with respect to x.  ``out``, ``ws`` (q4_linear_grad_workspace_bytes) and
    autograd: as there."""
    return _linear("bakron_q4_linear_grad", q4_linear_grad_workspace_bytes, "dy", dy, w, out, ws, stream)


def q4_moe(x, router, w_gate, w_up, w_down, top_k, *, out=None, ws=None, stream=None):
    """bakron_q4_moe: a mixture-of-experts layer for up to 64 tokens.  x tokens x
    hidden; router experts x hidden; w_gate and w_up stacks of ffn x hidden,
    w_down a stack of hidden x ffn layers.  Returns dict(y, ids, weights): the
    layer's output, the chosen experts (int32 tokens x top_k, largest logit
    first) and their shares (float32).  ``out``: a dict of the three to write
    to; ``ws``: a workspace of q4_moe_workspace_bytes.  It has no gradient:
    x and router that require one are refused unless under torch.no_grad()
    (q4_moe_layer: any number of tokens, with gradients)."""
    if not isinstance(w_gate, Q4Weight):
        raise TypeError("w_gate must be a Q4Weight (q4_pack)")
    f, h, E = w_gate.m, w_gate.n, w_gate.count
    ldx = _rows("x", x, h)
    index, T, dtype = x.get_device(), x.shape[0], x.dtype
    if w_gate.data.get_device() != index:
        _one("w_gate", w_gate, index, E)
    group = w_gate._group
    for name, w, m, n in (("w_up", w_up, f, h), ("w_down", w_down, h, f)):
        if not isinstance(w, Q4Weight) or w.count != E or w.data.get_device() != index:
            _one(name, w, index, E)
        if w.m != m or w.n != n:
            raise ValueError(f"{name} must be {(m, n)}, got {(w.m, w.n)}")
        if w._group != group:
            raise ValueError("the three stacks must have one group_size")
    if not (isinstance(router, torch.Tensor) and router.dtype == dtype and router.get_device() == index and
            router.shape == (E, h) and router.is_contiguous()):
        _b._check_dev("router", router, dtype, (E, h))
        _one_device(index, None, router=router)
    if _forward._current_level >= 0:
        _no_tangent("router", router)
    if _device() != index:
        with torch.cuda.device(index):
            return q4_moe(x, router, w_gate, w_up, w_down, top_k, out=out, ws=ws, stream=stream)
    if stream is None:
        s = _raw_stream(index)
    else:
        _one_device(index, stream)
        s = stream.cuda_stream
    if (x.requires_grad or router.requires_grad) and _grad_on():
        raise ValueError("q4_moe has no gradient: call it under torch.no_grad() or with detached tensors")
    if out is None:
        y, ids, weights = _made(stream, lambda: (x.new_empty((T, h)), x.new_empty((T, top_k), dtype=torch.int32),
                                                 x.new_empty((T, top_k), dtype=torch.float32)))
        out, ldy = {"y": y, "ids": ids, "weights": weights}, h
    else:
        y, ids, weights = out["y"], out["ids"], out["weights"]
        ldy = _rows("out['y']", y, h, dtype)
        if y.shape[0] != T:
            raise ValueError(f"out['y'] must have shape ({T}, {h}), got {tuple(y.shape)}")
        _b._check_dev("out['ids']", ids, torch.int32, (T, top_k))
        _b._check_dev("out['weights']", weights, torch.float32, (T, top_k))
        _one_device(index, None, **{"out['y']": y, "out['ids']": ids, "out['weights']": weights})
        _plain_outputs(y, weights)
    if ws is None:
        ws = _workspace(q4_moe_workspace_bytes(T, w_gate, top_k), x.device, stream)
    elif ws.get_device() != index or not ws.is_contiguous():
        _refuse(ws, index)
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)
    call = "bakron_q4_moe"
    rc = _calls[call](x.data_ptr(), ldx, T, _TYPES[dtype], router.data_ptr(), w_gate.data.data_ptr(), w_up.data.data_ptr(),
                      w_down.data.data_ptr(), h, f, E, top_k, group, y.data_ptr(), ldy, ids.data_ptr(),
                      weights.data_ptr(), wp, wn, s)
    if rc:
        _check(rc, call)
    _written(y, ids, weights)
    return out
