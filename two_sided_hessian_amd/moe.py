"""The expert layer for any number of tokens, forward and backward, on packed
4-bit experts (include/bakron_moe.h): the choice of experts and its sorted
order, rows there and back, the experts' products, their inner activation with
8-bit checkpoints, and the whole layer.

Arguments are checked as in q4.py: no tensor is looked into, the calls' arithmetic runs
in the library's HIP kernels, and there is no fallback (q4_moe_layer's backward pass makes
a second set of places with three of torch's operators).  Calls whose
outputs are given (decoding steps, captured or not) are tried by _fast first,
which checks and enqueues them in native code (csrc/fast_calls.cpp) and leaves
everything else, refusals among it, to the code here.

Given outputs count as changed in place, as torch's own do.

Autograd: moe_route (weights), moe_gather, moe_combine, q4_experts, gated_act
and q4_moe_layer take part in it where an input requires a gradient and ``out``
is not given.  Gradients with respect to sorted rows that no choice has are
zeros.  moe_gather, q4_experts and moe_combine without weights are linear and can be
differentiated again; the others have first derivatives only, and a second one that
reaches them raises.  There are no derivatives in forward mode: dual tensors are refused.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from . import q4 as _q
from .q4 import Q4Weight, _calls, _check, _device, _grad_on, _made, _on, _one_device, _plain_outputs, _raw_stream, _rows, \
    _written

BAKRON_MOE_F32 = 2
BAKRON_MOE_SILU = 0
BAKRON_MOE_GELU = 1
BAKRON_MOE_MAX_ROWS = 16777216
BAKRON_MOE_MAX_TOP_K = 16
BAKRON_MOE_MAX_PLACES = 32
BAKRON_MOE_MAX_EXPERTS = 256

_VP, _I64, _I32, _SZ, _INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
_EXPERTS = [_VP, _I64, _I64, _I32, _VP, _I64, _I64, _I64, _I64, _VP, _VP, _I64, _VP, _SZ, _VP]
_b.SIGNATURES.update({
    "bakron_moe_route_workspace_bytes": (_SZ, [_I64, _I64, _I32]),
    "bakron_moe_route": (_INT, [_VP, _I64, _I64, _I32, _I64, _I32] + [_VP] * 6 + [_SZ, _VP]),
    "bakron_moe_route_grad": (_INT, [_VP, _VP, _VP, _I64, _I64, _I32, _VP, _I64, _I32, _VP]),
    "bakron_moe_gather": (_INT, [_VP, _I64, _I64, _I32, _I64, _I32, _VP, _VP, _I64, _I64, _VP]),
    "bakron_moe_combine": (_INT, [_VP, _I64, _I64, _I32, _I64, _I32, _VP, _VP, _I64, _VP, _I64, _VP]),
    "bakron_moe_combine_grad": (_INT, [_VP, _I64, _VP, _I64, _I64, _I32, _I64, _I32, _VP, _VP, _I64, _VP, _I64, _VP, _VP]),
    "bakron_q4_experts_workspace_bytes": (_SZ, [_I64] * 5),
    "bakron_q4_experts": (_INT, _EXPERTS),
    "bakron_q4_experts_grad_workspace_bytes": (_SZ, [_I64] * 5),
    "bakron_q4_experts_grad": (_INT, _EXPERTS),
    "bakron_ck8_bytes": (_SZ, [_I64, _I64]),
    "bakron_ck8_pack": (_INT, [_VP, _I64, _I64, _I32, _I64, _VP, _VP]),
    "bakron_ck8_unpack": (_INT, [_VP, _I64, _I64, _I32, _VP, _I64, _VP]),
    "bakron_gated_act": (_INT, [_VP, _I64, _VP, _I64, _I64, _I32, _I64, _I32, _VP, _VP, _I64, _VP, _VP, _VP]),
    "bakron_gated_act_grad": (_INT, [_VP, _I64, _VP, _VP, _I64, _I32, _I64, _I32, _VP, _VP, _I64, _VP, _I64, _VP]),
})

_TYPES = dict(_q._TYPES)
_TYPES3 = _TYPES | {torch.float32: BAKRON_MOE_F32}
_ACTS = {"silu": BAKRON_MOE_SILU, "gelu": BAKRON_MOE_GELU}


try:
    from . import _fast
except ImportError:                      # not built: the same calls through ctypes, 4 us each on the host
    _fast = None


def _not_here(*_):
    return False


def _native(name):
    return getattr(_fast, name, _not_here)


_route_at, _route_grad_at, _gather_at, _combine_at, _combine_grad_at, _experts_at, _experts_grad_at, _pack_at, _gated_at, \
    _gated_grad_at = map(_native, ("route", "route_grad", "gather", "combine", "combine_grad", "experts", "experts_grad", "pack",
                                   "gated", "gated_grad"))
_ready = _fast is None


def _get_ready():
    """The library's functions for _fast, which declines every call until then."""
    global _ready
    _b.lib()
    _fast.load(_b.LIB_PATH, Q4Weight, Checkpoint8, _b.BakronError)
    _ready = True


def _type_of(name, dtype):
    if dtype not in _TYPES3:
        raise TypeError(f"{name} must be torch.float32, torch.bfloat16 or torch.float16, got {dtype}")
    return _TYPES3[dtype]


def _matrix(name, t, cols=None):
    """Leading dimension of a matrix of one of the three types whose rows are
    contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    _type_of(name, t.dtype)
    if _q._forward._current_level >= 0:
        _q._no_tangent(name, t)
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must have shape (rows, {'columns' if cols is None else cols}), got {tuple(t.shape)}")
    rows, cols = t.shape
    ld, inner = t.stride()
    if cols > 1 and inner != 1 and rows:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1 or cols == 0:
        return cols
    if ld < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    return ld


def _flat(name, t, dtype, shape, index):
    """A contiguous tensor of that type and shape on that device."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.is_contiguous() and
            t.get_device() == index):
        _b._check_dev(name, t, dtype, shape)
        _one_device(index, None, **{name: t})
    if _q._forward._current_level >= 0:
        _q._no_tangent(name, t)
    return t.data_ptr()


def _output(name, t, rows, cols, dtype, index):
    """Leading dimension of a given output."""
    ld = _rows(name, t, cols, dtype)
    if t.shape[0] != rows:
        raise ValueError(f"{name} must have shape ({rows}, {cols}), got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    return ld


def _stream_of(index, stream):
    if stream is None:
        return _raw_stream(index)
    _one_device(index, stream)
    return stream.cuda_stream


def _run(call, *args):
    rc = _calls[call](*args)
    if not _ready:
        _get_ready()
    if rc:
        _check(rc, call)


def _space(ws, need, device, index, stream):
    """The workspace: the given one, or a new one where one is needed."""
    if ws is None:
        return _q._workspace(need, device, stream)
    if ws.get_device() != index or not ws.is_contiguous():
        _q._refuse(ws, index)
    return ws


def _without_out(out, what):
    if out is not None:
        raise ValueError(f"out cannot be given where {what} requires a gradient")


def _no_gradient(call, *tensors):
    """For calls whose results are not differentiable."""
    if _grad_on() and any(t.requires_grad for t in tensors):
        raise ValueError(f"{call} has no gradient: call it under torch.no_grad() or with detached tensors")


def _top_k(top_k):
    if not 1 <= top_k <= BAKRON_MOE_MAX_TOP_K:
        raise ValueError(f"top_k must be 1 .. {BAKRON_MOE_MAX_TOP_K}")
    return int(top_k)


class _Refusing(torch.autograd.Function):
    """Gradients as they are, whose own derivative is refused."""

    @staticmethod
    def forward(ctx, name, count, *tensors):
        ctx.name = name
        return tuple(t.detach() for t in tensors[:count])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has no second derivative")


def _plainly(back, *args):
    """A backward pass whose calls are not recorded in a kept graph."""
    if not _grad_on():
        return back(*args)
    with torch.no_grad():
        return back(*args)


def _once(name, gradients, *causes):
    """The gradients that a backward pass of ``name`` made, None among them.  In a kept
    graph (create_graph) they depend on ``causes``, and a derivative that reaches them
    raises: without that they would count as constants."""
    if not _grad_on() or not any(t.requires_grad for t in causes):
        return gradients
    made = [t for t in gradients if t is not None]
    refusing = iter(_Refusing.apply(name, len(made), *made, *causes))
    return tuple(None if t is None else next(refusing) for t in gradients)


# A function whose backward pass keeps no tensor that leads to its inputs in the graph
# returns an empty one beside its results (`lead`), and gives that to _once.

# -------------------------------------------------------------------- route

def moe_route_workspace_bytes(tokens: int, experts: int, top_k: int) -> int:
    return _b.lib().bakron_moe_route_workspace_bytes(tokens, experts, top_k)


_ROUTE = ("ids", "weights", "place", "order", "offsets")


def _route_results(logits, k):
    (T, E), e, i32 = logits.shape, logits.new_empty, torch.int32
    return (e((T, k), dtype=i32), e((T, k), dtype=torch.float32), e((T, k), dtype=i32), e((T * k,), dtype=i32),
            e((E + 1,), dtype=i32))


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, ws, stream):
        r = moe_route(logits.detach(), top_k, ws=ws, stream=stream)
        ctx.experts, ctx.dtype = logits.shape[1], logits.dtype
        ctx.save_for_backward(r["weights"], r["ids"])
        ctx.mark_non_differentiable(*(r[name] for name in _ROUTE if name != "weights"))
        return tuple(r[name] for name in _ROUTE)

    @staticmethod
    def backward(ctx, _ids, dweights, *_):
        weights, ids = ctx.saved_tensors
        dlogits = _plainly(lambda: moe_route_grad(dweights.contiguous(), weights, ids, ctx.experts, dtype=ctx.dtype))
        return _once("moe_route", (dlogits, None, None, None), dweights, weights)


def moe_route(logits, top_k, *, out=None, ws=None, stream=None):
    """bakron_moe_route: the choice of top_k experts per token and the choices
    sorted by expert.  logits: tokens x experts in float32, bfloat16 or float16
    (rows contiguous); -inf and NaN are never chosen.  Returns dict(ids, weights,
    place, order, offsets): the chosen experts (int32 tokens x top_k, largest
    logit first, -1: none), their shares (float32), the sorted row of each
    choice (int32 tokens x top_k, -1: none), the choice at each sorted row (int32
    tokens * top_k, -1 behind the last) and each expert's first row (int32
    experts + 1).  ``out``: a dict of the five to write to; ``ws``: a workspace of
    moe_route_workspace_bytes.  Autograd: the weights' gradient is taken with
    moe_route_grad."""
    if out is not None and stream is None and _route_at(logits, top_k, out, ws):
        return out
    ld = _matrix("logits", logits)
    T, E = logits.shape
    k, index = _top_k(top_k), logits.get_device()
    if _device() != index:
        with torch.cuda.device(index):
            return moe_route(logits, top_k, out=out, ws=ws, stream=stream)
    s = _stream_of(index, stream)
    if logits.requires_grad and _grad_on():
        _without_out(out, "logits")
        return dict(zip(_ROUTE, _Route.apply(logits, k, ws, stream)))
    i32 = torch.int32
    if out is None:
        out = dict(zip(_ROUTE, _made(stream, lambda: _route_results(logits, k))))
    at = [_flat(f"out['{name}']", out[name], torch.float32 if name == "weights" else i32,
                (T * k,) if name == "order" else (E + 1,) if name == "offsets" else (T, k), index) for name in _ROUTE]
    _plain_outputs(out["weights"])
    ws = _space(ws, moe_route_workspace_bytes(T, E, k), logits.device, index, stream)
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)
    _run("bakron_moe_route", logits.data_ptr(), ld, T, _TYPES3[logits.dtype], E, k, *at, wp, wn, s)
    _written(*(out[name] for name in _ROUTE))
    return out


def moe_route_grad(dweights, weights, ids, experts, *, dtype=torch.float32, out=None, stream=None):
    """bakron_moe_route_grad: the gradient of moe_route's weights with respect to
    the logits, tokens x experts of ``dtype`` (or of out's), zero where an expert
    was not chosen.  It has no gradient itself: tensors that require one are refused
    unless under torch.no_grad()."""
    if out is not None and stream is None and _route_grad_at(dweights, weights, ids, experts, out):
        return out
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda or ids.dim() != 2:
        raise TypeError("ids must be a CUDA (HIP) tensor, tokens x top_k")
    (T, k), index, E = ids.shape, ids.get_device(), int(experts)
    k = _top_k(k)
    at = [_flat("dweights", dweights, torch.float32, (T, k), index), _flat("weights", weights, torch.float32, (T, k), index),
          _flat("ids", ids, torch.int32, (T, k), index)]
    if not k <= E <= BAKRON_MOE_MAX_EXPERTS:
        raise ValueError(f"experts must be {k} .. {BAKRON_MOE_MAX_EXPERTS}")
    _no_gradient("moe_route_grad", dweights, weights)
    if _device() != index:
        with torch.cuda.device(index):
            return moe_route_grad(dweights, weights, ids, experts, dtype=dtype, out=out, stream=stream)
    s = _stream_of(index, stream)
    if out is None:
        _type_of("dtype", dtype)
        out = _made(stream, lambda: (weights.new_empty((T, E), dtype=dtype),))[0]
    ld = _matrix("out", out, E)
    if out.shape[0] != T or out.get_device() != index:
        raise ValueError(f"out must be a ({T}, {E}) tensor on cuda:{index}")
    _plain_outputs(out)
    _run("bakron_moe_route_grad", *at, T, E, k, out.data_ptr(), ld, _TYPES3[out.dtype], s)
    _written(out)
    return out


# ------------------------------------------------------- rows there and back

def _places(place, index):
    if not isinstance(place, torch.Tensor) or not place.is_cuda or place.dim() != 2:
        raise TypeError("place must be a CUDA (HIP) tensor, tokens x top_k")
    T, k = place.shape
    if not 1 <= k <= BAKRON_MOE_MAX_PLACES:
        raise ValueError(f"place must have 1 .. {BAKRON_MOE_MAX_PLACES} columns, got {k}")
    return T, k, _flat("place", place, torch.int32, (T, k), index)


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, place, stream):
        ctx.save_for_backward(place)
        return moe_gather(x.detach(), place, stream=stream)

    @staticmethod
    def backward(ctx, g):
        return moe_combine(g.contiguous(), ctx.saved_tensors[0]), None, None


def moe_gather(x, place, *, out=None, stream=None):
    """bakron_moe_gather: tokens' rows into the sorted order, xs[place[t, j]] =
    x[t].  x: tokens x columns in bfloat16 or float16; place: int32 tokens x top_k
    (moe_route).  Returns tokens * top_k x columns; ``out``: where to write it (any
    number of rows).  Rows that no choice has stay as they are (in a new result:
    undefined); a row that two choices share ends as some mixture of theirs.  Autograd:
    its gradient is moe_combine without weights."""
    if out is not None and stream is None and _gather_at(x, place, out):
        return out
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a CUDA (HIP) tensor, tokens x columns")
    n = x.shape[1]
    ldx, index = _rows("x", x, n), x.get_device()
    T, k, at = _places(place, index)
    if x.shape[0] != T:
        raise ValueError(f"place must have {x.shape[0]} rows, got {T}")
    if _device() != index:
        with torch.cuda.device(index):
            return moe_gather(x, place, out=out, stream=stream)
    s = _stream_of(index, stream)
    if x.requires_grad and _grad_on():
        _without_out(out, "x")
        return _Gather.apply(x, place, stream)
    if out is None:
        out = _made(stream, lambda: (x.new_empty((T * k, n)),))[0]
    ldo = _output("out", out, out.shape[0] if isinstance(out, torch.Tensor) and out.dim() else 0, n, x.dtype, index)
    _plain_outputs(out)
    _run("bakron_moe_gather", x.data_ptr(), ldx, T, _TYPES[x.dtype], n, k, at, out.data_ptr(), ldo, out.shape[0], s)
    _written(out)
    return out


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, place, weights, stream):
        # without weights the gradient needs no rows
        ctx.save_for_backward(place, weights, None if weights is None else ys)
        ctx.rows = ys.shape[0]
        return moe_combine(ys.detach(), place, None if weights is None else weights.detach(), stream=stream)

    @staticmethod
    def backward(ctx, g):
        place, weights, ys = ctx.saved_tensors
        g = g.contiguous()
        if weights is None:
            dys = _Spread.apply(g, place, ctx.rows) if g.requires_grad else _spread(g, place, ctx.rows)
            return dys, None, None, None
        return _combine_back(g, ys, place, weights) + (None,)


def _spread(g, place, rows):
    return moe_gather(g, place, out=g.new_zeros((rows, g.shape[1])))


class _Spread(torch.autograd.Function):
    """moe_gather into zeros, for second derivatives of moe_combine without
    weights."""

    @staticmethod
    def forward(ctx, g, place, rows):
        ctx.save_for_backward(place)
        return _spread(g.detach(), place, rows)

    @staticmethod
    def backward(ctx, gg):
        return moe_combine(gg.contiguous(), ctx.saved_tensors[0]), None, None


def _combine_back(g, ys, place, weights):
    if g.requires_grad and _grad_on():
        raise RuntimeError("moe_combine with weights has no second derivative")

    def back():
        out = {"dys": torch.zeros(ys.shape, dtype=ys.dtype, device=ys.device), "dweights": torch.empty_like(weights)}
        return moe_combine_grad(g, ys, place, weights, out=out)
    r = _plainly(back)
    return _once("moe_combine with weights", (r["dys"], None, r["dweights"]), ys, weights)


def moe_combine(ys, place, weights=None, *, out=None, stream=None):
    """bakron_moe_combine: sorted rows back to their tokens, y[t] = sum_j
    weights[t, j] ys[place[t, j]] (weights None: all 1; a choice without a row adds
    nothing).  ys: rows x columns in bfloat16 or float16; weights: float32 tokens x
    top_k.  ``out``: where to write y.  Autograd: the gradients are those of
    moe_combine_grad (without weights: moe_gather), for places that name each row once at
    most, as moe_route's do (of a row that two choices share, the gradient ends as some
    mixture of theirs and not as their sum)."""
    if out is not None and stream is None and _combine_at(ys, place, weights, out):
        return out
    if not isinstance(ys, torch.Tensor) or ys.dim() != 2:
        raise TypeError("ys must be a CUDA (HIP) tensor, rows x columns")
    rows, n = ys.shape
    ldys, index = _rows("ys", ys, n), ys.get_device()
    T, k, at = _places(place, index)
    wp = None if weights is None else _flat("weights", weights, torch.float32, (T, k), index)
    if _device() != index:
        with torch.cuda.device(index):
            return moe_combine(ys, place, weights, out=out, stream=stream)
    s = _stream_of(index, stream)
    if (ys.requires_grad or (weights is not None and weights.requires_grad)) and _grad_on():
        _without_out(out, "ys or weights")
        return _Combine.apply(ys, place, weights, stream)
    if out is None:
        out, ldo = _made(stream, lambda: (ys.new_empty((T, n)),))[0], n
    else:
        ldo = _output("out", out, T, n, ys.dtype, index)
    _plain_outputs(out)
    _run("bakron_moe_combine", ys.data_ptr(), ldys, rows, _TYPES[ys.dtype], n, k, at, wp, T, out.data_ptr(), ldo, s)
    _written(out)
    return out


def moe_combine_grad(dy, ys, place, weights, *, out=None, stream=None):
    """bakron_moe_combine_grad: moe_combine's gradients, dict(dys, dweights):
    dys[place[t, j]] = weights[t, j] dy[t] and dweights[t, j] = dy[t] . ys[place[t, j]].
    ``out``: a dict of the two to write to.  Rows of dys that no choice has stay as
    they are (in a new result: undefined).  It has no gradient itself: tensors that
    require one are refused unless under torch.no_grad()."""
    if out is not None and stream is None and _combine_grad_at(dy, ys, place, weights, out):
        return out
    if not isinstance(ys, torch.Tensor) or ys.dim() != 2:
        raise TypeError("ys must be a CUDA (HIP) tensor, rows x columns")
    rows, n = ys.shape
    ldys, index = _rows("ys", ys, n), ys.get_device()
    T, k, at = _places(place, index)
    lddy = _output("dy", dy, T, n, ys.dtype, index)
    wp = _flat("weights", weights, torch.float32, (T, k), index)
    _no_gradient("moe_combine_grad", dy, ys, weights)
    if _device() != index:
        with torch.cuda.device(index):
            return moe_combine_grad(dy, ys, place, weights, out=out, stream=stream)
    s = _stream_of(index, stream)
    if out is None:
        dys, dw = _made(stream, lambda: (ys.new_empty((rows, n)), weights.new_empty((T, k))))
        out = {"dys": dys, "dweights": dw}
    dys = out["dys"]
    ldo, dw = _output("out['dys']", dys, rows, n, ys.dtype, index), _flat("out['dweights']", out["dweights"], torch.float32, (T, k), index)
    _plain_outputs(dys, out["dweights"])
    _run("bakron_moe_combine_grad", dy.data_ptr(), lddy, ys.data_ptr(), ldys, rows, _TYPES[ys.dtype], n, k, at, wp, T,
         dys.data_ptr(), ldo, dw, s)
    _written(out["dys"], out["dweights"])
    return out


# ------------------------------------------------------------------ products

def q4_experts_workspace_bytes(rows: int, w: Q4Weight) -> int:
    return _b.lib().bakron_q4_experts_workspace_bytes(rows, w.count, w.m, w.n, w._group)


def q4_experts_grad_workspace_bytes(rows: int, w: Q4Weight) -> int:
    return _b.lib().bakron_q4_experts_grad_workspace_bytes(rows, w.count, w.m, w.n, w._group)


class _Experts(torch.autograd.Function):
    """q4_experts and q4_experts_grad, each the other's derivative."""

    @staticmethod
    def forward(ctx, v, w, offsets, call, back, ws, stream, gradient):
        ctx.w, ctx.call, ctx.back = w, call, back
        ctx.save_for_backward(offsets)
        v, out = v.detach(), None
        if gradient:   # zeros in the rows that no expert has
            out = v.new_zeros((v.shape[0], w.n if call is q4_experts_grad else w.m))
        return call(v, w, offsets, out=out, ws=ws, stream=stream)

    @staticmethod
    def backward(ctx, g):
        offsets, = ctx.saved_tensors
        return (_Experts.apply(g.contiguous(), ctx.w, offsets, ctx.back, ctx.call, None, None, True),) + 7 * (None,)


def _experts(call, size, name, x, w, offsets, out, ws, stream):
    if not isinstance(w, Q4Weight):
        raise TypeError("w must be a Q4Weight (q4_pack)")
    in_cols, out_cols = (w.n, w.m) if name == "x" else (w.m, w.n)
    ldx, index = _rows(name, x, in_cols), x.get_device()
    R, data = x.shape[0], w.data
    if data.get_device() != index:
        _q._one("w", w, index, w.count)
    at = _flat("offsets", offsets, torch.int32, (w.count + 1,), index)
    if _device() != index:
        with torch.cuda.device(index):
            return _experts(call, size, name, x, w, offsets, out, ws, stream)
    s = _stream_of(index, stream)
    if x.requires_grad and _grad_on():
        _without_out(out, name)
        both = (q4_experts, q4_experts_grad) if name == "x" else (q4_experts_grad, q4_experts)
        return _Experts.apply(x, w, offsets, *both, ws, stream, False)
    if out is None:
        out, ldo = _made(stream, lambda: (x.new_empty((R, out_cols)),))[0], out_cols
    else:
        ldo = _output("out", out, R, out_cols, x.dtype, index)
    _plain_outputs(out)
    ws = _space(ws, size(R, w), x.device, index, stream)
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)
    _run(call, x.data_ptr(), ldx, R, _TYPES[x.dtype], data.data_ptr(), w.count, w.m, w.n, w._group, at, out.data_ptr(), ldo,
         wp, wn, s)
    _written(out)
    return out


def q4_experts(x, w, offsets, *, out=None, ws=None, stream=None):
    """bakron_q4_experts: each expert's rows times its layer of a packed stack,
    y[p] = W_e x[p] for offsets[e] <= p < offsets[e + 1].  x: rows x n in bfloat16
    or float16 (rows contiguous, any row stride); offsets: int32 count + 1 on the
    device (moe_route).  Rows from offsets[-1] on stay as they are (in a new
    result: undefined).  ``ws``: a workspace of q4_experts_workspace_bytes.
    Autograd: with respect to x, by q4_experts_grad."""
    if out is not None and stream is None and _experts_at(x, w, offsets, out, ws):
        return out
    return _experts("bakron_q4_experts", q4_experts_workspace_bytes, "x", x, w, offsets, out, ws, stream)


def q4_experts_grad(dy, w, offsets, *, out=None, ws=None, stream=None):
    """bakron_q4_experts_grad: dx[p] = dy[p] W_e, the gradient of q4_experts with
    respect to x.  ``out``, ``ws`` (q4_experts_grad_workspace_bytes) and autograd: as
    there."""
    if out is not None and stream is None and _experts_grad_at(dy, w, offsets, out, ws):
        return out
    return _experts("bakron_q4_experts_grad", q4_experts_grad_workspace_bytes, "dy", dy, w, offsets, out, ws, stream)


# ------------------------------------------------------------- 8-bit checkpoints

class Checkpoint8:
    """rows x cols values kept in 8 bits with a power of two per row and 32
    columns (include/bakron_moe.h).  ``data`` is the device buffer (uint8) that
    holds it, ``dtype`` the type of the values that went in."""

    __slots__ = ("data", "rows", "cols", "dtype")

    def __init__(self, data, rows, cols, dtype):
        self.data, self.rows, self.cols, self.dtype = data, rows, cols, dtype

    @staticmethod
    def empty(rows, cols, dtype, device):
        """Room for a checkpoint (what it stands for is undefined)."""
        if dtype not in _TYPES:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        if not 0 <= rows <= BAKRON_MOE_MAX_ROWS or not 0 <= cols <= _b.BAKRON_MAX_DIM:
            raise ValueError(f"no checkpoint of {rows} x {cols}")
        return Checkpoint8(_b.workspace(_b.lib().bakron_ck8_bytes(rows, cols), device), rows, cols, dtype)

    @property
    def device(self):
        return self.data.device

    def __repr__(self):
        return f"Checkpoint8(rows={self.rows}, cols={self.cols}, dtype={self.dtype})"


def _checkpoint(name, ck, rows, cols, dtype, index):
    if not isinstance(ck, Checkpoint8):
        raise TypeError(f"{name} must be a Checkpoint8")
    if (ck.rows, ck.cols) != (rows, cols) or ck.dtype != dtype:
        raise ValueError(f"{name} must be a checkpoint of {rows} x {cols} values of {dtype}, got {ck!r}")
    data = ck.data
    if data.get_device() != index:
        raise ValueError(f"{name} is on {ck.device}, not on cuda:{index}")
    if not data.is_contiguous() or data.nbytes < _b.lib().bakron_ck8_bytes(rows, cols):
        raise ValueError(f"{name} must have the bytes of {rows} x {cols} values, one after the other")
    return data.data_ptr()


def ck8_pack(x, *, out=None, stream=None):
    """bakron_ck8_pack: the 8-bit checkpoint of a matrix in bfloat16 or float16
    (rows contiguous).  ``out``: a Checkpoint8 of its size and type to write to.  It has
    no gradient: x that requires one is refused unless under torch.no_grad()."""
    if out is not None and stream is None and _pack_at(x, out):
        return out
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a CUDA (HIP) tensor, rows x columns")
    rows, n = x.shape
    ldx, index = _rows("x", x, n), x.get_device()
    _no_gradient("ck8_pack", x)
    if _device() != index:
        with torch.cuda.device(index):
            return ck8_pack(x, out=out, stream=stream)
    s = _stream_of(index, stream)
    if out is None:
        data, = _made(stream, lambda: (Checkpoint8.empty(rows, n, x.dtype, x.device).data,))
        out = Checkpoint8(data, rows, n, x.dtype)
    at = _checkpoint("out", out, rows, n, x.dtype, index)
    _run("bakron_ck8_pack", x.data_ptr(), ldx, rows, _TYPES[x.dtype], n, at, s)
    _written(out.data)
    return out


def ck8_unpack(ck, *, dtype=None, out=None, stream=None):
    """bakron_ck8_unpack: the values that a checkpoint stands for, in ``dtype``
    (float32, bfloat16 or float16; None: that of the values that went in), or in
    ``out``."""
    if not isinstance(ck, Checkpoint8):
        raise TypeError("ck must be a Checkpoint8")
    index = ck.data.get_device()
    if index < 0:
        raise TypeError("ck must be on a CUDA (HIP) device")
    at = _checkpoint("ck", ck, ck.rows, ck.cols, ck.dtype, index)
    if _device() != index:
        with torch.cuda.device(index):
            return ck8_unpack(ck, dtype=dtype, out=out, stream=stream)
    s = _stream_of(index, stream)
    if out is None:
        dtype = dtype or ck.dtype
        _type_of("dtype", dtype)
        out = _made(stream, lambda: (torch.empty((ck.rows, ck.cols), dtype=dtype, device=ck.device),))[0]
    ld = _matrix("out", out, ck.cols)
    if out.shape[0] != ck.rows or out.get_device() != index:
        raise ValueError(f"out must be a ({ck.rows}, {ck.cols}) tensor on cuda:{index}")
    _plain_outputs(out)
    _run("bakron_ck8_unpack", at, ck.rows, ck.cols, _TYPES3[out.dtype], out.data_ptr(), ld, s)
    _written(out)
    return out


# ---------------------------------------------------------- inner activation

def _act(act):
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return _ACTS[act]


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, b, act, count, stream):
        h, ca, cb = gated_act(a.detach(), b.detach(), act=act, checkpoint=True, count=count, stream=stream)
        lead = h.new_empty(0)
        ctx.act, ctx.like = act, (ca.rows, ca.cols, ca.dtype)
        ctx.save_for_backward(ca.data, cb.data, count, lead)
        ctx.set_materialize_grads(False)   # (lead has no gradient)
        return h, lead

    @staticmethod
    def backward(ctx, dh, _):
        ca, cb, count, lead = ctx.saved_tensors
        if dh is None:
            return 5 * (None,)

        def back():
            g = dh.contiguous()
            out = None if count is None else (torch.zeros_like(g), torch.zeros_like(g))
            return gated_act_grad(g, Checkpoint8(ca, *ctx.like), Checkpoint8(cb, *ctx.like), act=ctx.act,
                                  count=count, out=out)
        return _once("gated_act", (*_plainly(back), None, None, None), dh, lead)


def gated_act(a, b, *, act="silu", checkpoint=False, count=None, out=None, stream=None):
    """bakron_gated_act: h = act(a) * b, a and b rows x columns in bfloat16 or
    float16 (rows contiguous, any row strides); act "silu" or "gelu" (its tanh
    form).  ``checkpoint``: True, or a pair of Checkpoint8 to write to: returns (h,
    checkpoint of a, checkpoint of b) for gated_act_grad instead of h.  ``count``:
    int32 of one element on the device, rows from it on are left as they are
    (moe_route's offsets[-1:]).  ``out``: where to write h.  Autograd keeps a and b as
    checkpoints: the gradient is gated_act_grad's."""
    if out is not None and stream is None and _gated_at(a, b, _ACTS.get(act, -1), checkpoint or None, count, out):
        return (out, *checkpoint) if checkpoint else out
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise TypeError("a must be a CUDA (HIP) tensor, rows x columns")
    rows, n = a.shape
    lda, index, kind = _rows("a", a, n), a.get_device(), _act(act)
    ldb = _output("b", b, rows, n, a.dtype, index)
    cp = None if count is None else _flat("count", count, torch.int32, (1,), index)
    if _device() != index:
        with torch.cuda.device(index):
            return gated_act(a, b, act=act, checkpoint=checkpoint, count=count, out=out, stream=stream)
    s = _stream_of(index, stream)
    if (a.requires_grad or b.requires_grad) and _grad_on():
        _without_out(out, "a or b")
        if checkpoint is not False:
            raise ValueError("checkpoint cannot be given where a or b requires a gradient: autograd keeps its own")
        return _Gated.apply(a, b, act, count, stream)[0]
    if out is None:
        out, ldo = _made(stream, lambda: (a.new_empty((rows, n)),))[0], n
    else:
        ldo = _output("out", out, rows, n, a.dtype, index)
    if checkpoint is False:
        ca = cb = None
    else:
        if checkpoint is True:
            checkpoint = [Checkpoint8(data, rows, n, a.dtype) for data in
                          _made(stream, lambda: [Checkpoint8.empty(rows, n, a.dtype, a.device).data for _ in range(2)])]
        ca, cb = (_checkpoint("checkpoint", c, rows, n, a.dtype, index) for c in checkpoint)
    _plain_outputs(out)
    _run("bakron_gated_act", a.data_ptr(), lda, b.data_ptr(), ldb, rows, _TYPES[a.dtype], n, kind, cp, out.data_ptr(), ldo,
         ca, cb, s)
    if checkpoint is False:
        _written(out)
        return out
    _written(out, *(c.data for c in checkpoint))
    return (out, *checkpoint)


def gated_act_grad(dh, ck_a, ck_b, *, act="silu", count=None, out=None, stream=None):
    """bakron_gated_act_grad: (da, db), the gradients of gated_act from the
    checkpoints of a and b.  ``out``: a pair to write to; ``count``: as there.  It has no
    gradient itself: dh that requires one is refused unless under torch.no_grad()."""
    if out is not None and stream is None and _gated_grad_at(dh, ck_a, ck_b, _ACTS.get(act, -1), count, *out):
        return tuple(out)
    if not isinstance(dh, torch.Tensor) or dh.dim() != 2:
        raise TypeError("dh must be a CUDA (HIP) tensor, rows x columns")
    rows, n = dh.shape
    lddh, index, kind = _rows("dh", dh, n), dh.get_device(), _act(act)
    pa, pb = _checkpoint("ck_a", ck_a, rows, n, dh.dtype, index), _checkpoint("ck_b", ck_b, rows, n, dh.dtype, index)
    cp = None if count is None else _flat("count", count, torch.int32, (1,), index)
    _no_gradient("gated_act_grad", dh)
    if _device() != index:
        with torch.cuda.device(index):
            return gated_act_grad(dh, ck_a, ck_b, act=act, count=count, out=out, stream=stream)
    s = _stream_of(index, stream)
    if out is None:
        out = tuple(_made(stream, lambda: (dh.new_empty((rows, n)), dh.new_empty((rows, n)))))
    da, db = out
    lda, ldb = _output("out[0]", da, rows, n, dh.dtype, index), _output("out[1]", db, rows, n, dh.dtype, index)
    _plain_outputs(da, db)
    _run("bakron_gated_act_grad", dh.data_ptr(), lddh, pa, pb, rows, _TYPES[dh.dtype], n, kind, cp, da.data_ptr(), lda,
         db.data_ptr(), ldb, s)
    _written(da, db)
    return da, db


# ------------------------------------------------------------ the whole layer

def _shared(sizes, like):
    """One workspace for calls that follow each other, or None."""
    need = max(sizes)
    return _b.workspace(need, like.device) if need else None


def _forward(x, logits, w_gate, w_up, w_down, k, act, keep):
    # outputs are given everywhere, which is what the native calls take
    (T, n), f, e = x.shape, w_gate.m, x.new_empty
    R = T * k
    ws = _shared((moe_route_workspace_bytes(T, w_gate.count, k), q4_experts_workspace_bytes(R, w_gate),
                  q4_experts_workspace_bytes(R, w_down)), x)
    r = moe_route(logits, k, out=dict(zip(_ROUTE, _route_results(logits, k))), ws=ws)
    place, offsets = r["place"], r["offsets"]
    count = offsets[-1:]
    xs = moe_gather(x, place, out=e((R, n)))
    a, b = (q4_experts(xs, w, offsets, out=e((R, f)), ws=ws) for w in (w_gate, w_up))
    if keep:
        h, *cks = gated_act(a, b, act=act, count=count, out=e((R, f)),
                            checkpoint=tuple(Checkpoint8.empty(R, f, x.dtype, x.device) for _ in range(2)))
    else:
        h, cks = gated_act(a, b, act=act, count=count, out=e((R, f))), None
    ys = q4_experts(h, w_down, offsets, out=e((R, n)), ws=ws)
    return moe_combine(ys, place, r["weights"], out=e((T, n))), r, ys, cks


class _Layer(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, logits, w_gate, w_up, w_down, k, act):
        y, r, ys, (ca, cb) = _forward(x.detach(), logits.detach(), w_gate, w_up, w_down, k, act, True)
        ctx.layers, ctx.act, ctx.like = (w_gate, w_up, w_down), act, (ca.rows, ca.cols, ca.dtype)
        ctx.logits = logits.shape[1], logits.dtype
        lead = y.new_empty(0)
        ctx.save_for_backward(r["ids"], r["weights"], r["place"], r["offsets"], ys, ca.data, cb.data, lead)
        ctx.set_materialize_grads(False)   # (lead has no gradient)
        return y, lead

    @staticmethod
    def backward(ctx, dy, _):
        *saved, lead = ctx.saved_tensors
        if dy is None:
            return 7 * (None,)
        return _once("q4_moe_layer", _plainly(_layer_back, ctx, dy, *saved) + 5 * (None,), dy, lead)


def _layer_back(ctx, dy, ids, weights, place, offsets, ys, ca, cb):
    """The gradients of x and of the logits, None where one is not needed."""
    w_gate, w_up, w_down = ctx.layers
    (R, n), f, e = ys.shape, w_gate.m, ys.new_empty
    back = moe_combine_grad(dy.contiguous(), ys, place, weights,
                            out={"dys": e((R, n)), "dweights": torch.empty_like(weights)})
    dlogits = dx = None
    if ctx.needs_input_grad[1]:
        E, dtype = ctx.logits
        dlogits = moe_route_grad(back["dweights"], weights, ids, E, out=e((weights.shape[0], E), dtype=dtype))
    if ctx.needs_input_grad[0]:
        ws = _shared((q4_experts_grad_workspace_bytes(R, w_down), q4_experts_grad_workspace_bytes(R, w_gate)), ys)
        dh = q4_experts_grad(back["dys"], w_down, offsets, out=e((R, f)), ws=ws)
        da, db = gated_act_grad(dh, Checkpoint8(ca, *ctx.like), Checkpoint8(cb, *ctx.like), act=ctx.act,
                                count=offsets[-1:], out=(e((R, f)), e((R, f))))
        # both halves of the rows' gradient in one sum: a token's places in the first
        # and in the second
        dxs = e((2 * R, n))
        q4_experts_grad(da, w_gate, offsets, out=dxs[:R], ws=ws)
        q4_experts_grad(db, w_up, offsets, out=dxs[R:], ws=ws)
        both = torch.cat((place, torch.where(place < 0, place, place + R)), 1)
        dx = moe_combine(dxs, both, out=e((place.shape[0], n)))
    return dx, dlogits


def q4_moe_layer(x, logits, w_gate, w_up, w_down, top_k, *, act="silu"):
    """A mixture-of-experts layer for any number of tokens: moe_route, moe_gather,
    the gate and up products (q4_experts), gated_act, the down product and
    moe_combine,
        y[t] = sum_k weights[t, k] down_e (act(gate_e x_t) * (up_e x_t)),   e = ids[t, k].
    x: tokens x hidden in bfloat16 or float16; logits: tokens x experts in
    float32, bfloat16 or float16 (tokens without a logit above -inf get zeros);
    w_gate, w_up, w_down: stacks as q4_moe takes them.  Between the calls values
    are rounded to x's type.  Autograd: with respect to x and logits, the inner
    activations kept in 8 bits.  (q4_moe has its router inside, three launches and no
    gradient: for one token, 2 of 8 experts of 14336 x 4096, 46 us and 54 here; 16: 185 and
    173; 64: 335 and 232.)"""
    if not all(isinstance(w, Q4Weight) for w in (w_gate, w_up, w_down)):
        raise TypeError("w_gate, w_up and w_down must be Q4Weights (q4_pack)")
    E, f, h = w_gate.count, w_gate.m, w_gate.n
    for name, w, m, n in (("w_up", w_up, f, h), ("w_down", w_down, h, f)):
        if w.count != E or (w.m, w.n) != (m, n):
            raise ValueError(f"{name} must be {E} layers of {(m, n)}, got {w!r}")
    _rows("x", x, h)
    _matrix("logits", logits, E)
    if logits.shape[0] != x.shape[0] or logits.get_device() != x.get_device():
        raise ValueError(f"logits must be a ({x.shape[0]}, {E}) tensor on {x.device}")
    k = _top_k(top_k)
    if k > E:
        raise ValueError(f"top_k must be {E} at most, the number of experts")
    _act(act)
    if (x.requires_grad or logits.requires_grad) and _grad_on():
        return _Layer.apply(x, logits, w_gate, w_up, w_down, k, act)[0]
    return _forward(x, logits, w_gate, w_up, w_down, k, act, False)[0]
