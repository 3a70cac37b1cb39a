"""The measured cases of the expert layer for many tokens, forward and backward.

A mixture-of-experts layer on packed 4-bit experts, for any number of tokens
and for calibration, which passes gradients back through rounded layers:

* "route"    the choice of top_k experts per token, their shares, and the
             choices sorted by expert; as a step, the logits' gradient too;
* "rows"     tokens' rows brought into that order and back, weighted; as a
             step, the gradients of both;
* "experts"  each expert's rows times its 4-bit layer;
* "grad"     the gradient of that with respect to the rows;
* "gated"    the experts' inner activation act(a) b; as a step, a and b kept in
             8 bits for the backward pass, and their gradients from those.

listed() names the cases, draw() draws others of the same ranges, prepare()
makes a case's inputs and what a program keeps between calls, run() is one
call (or a step's calls), exact() the same from the definition in float64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"

# Ranges: 1 .. 16384 tokens, 4 .. 256 experts, 1 .. 8 of them chosen, sides up to
# 14336; no rows case above ROWS_MOST sorted values, no experts or grad case above
# EXPERTS_MOST multiply-adds or STACK_MOST weights, no gated case above GATED_MOST
# values (the largest listed ones).
ROWS_MOST = 8192 * 2 * 4096
EXPERTS_MOST = 8192 * 2 * 4096 * 14336
STACK_MOST = 8 * 4096 * 14336
GATED_MOST = 16384 * 14336


def listed():
    return [
        # one decoding token's choice among eight experts: latency
        dict(name="route 1 8/2", op="route", T=1, E=8, k=2, dtype="fp32", masked=False, step=False),
        # a prompt batch's choice among many experts in training, some experts switched off, padded tokens without any
        dict(name="route 8192 64/6 step", op="route", T=8192, E=64, k=6, dtype="bf16", masked=True, step=True),
        # sixteen sequences decoding together: rows to their experts and back
        dict(name="rows 16x2048 64/6", op="rows", T=16, h=2048, E=64, k=6, dtype="fp16", pad=0, step=False),
        # a long batch forward and backward
        dict(name="rows 8192x4096 8/2 step", op="rows", T=8192, h=4096, E=8, k=2, dtype="bf16", pad=0, step=True),
        # an odd batch, odd rows that are slices of a wider buffer
        dict(name="rows 777x1003 5/2 step ragged", op="rows", T=777, h=1003, E=5, k=2, dtype="fp16", pad=5, step=True),
        # sixteen decoding tokens through the up-projections of many small experts: one or two rows each
        dict(name="experts 16x1024x2048 64/6", op="experts", T=16, m=1024, n=2048, E=64, k=6, group=64, dtype="fp16", pad=0,
             bits=4),
        # the largest: a long batch through the up-projections of eight large experts
        dict(name="experts 8192x14336x4096 8/2", op="experts", T=8192, m=14336, n=4096, E=8, k=2, group=128, dtype="bf16",
             pad=0, bits=4),
        # a short odd batch, odd layers, one grid per row
        dict(name="experts 777x1501x1003 5/2 ragged", op="experts", T=777, m=1501, n=1003, E=5, k=2, group=0, dtype="bf16",
             pad=3, bits=3),
        # calibration: a batch's gradient back through the up-projections of eight large experts
        dict(name="grad 2048x14336x4096 8/2", op="grad", T=2048, m=14336, n=4096, E=8, k=2, group=128, dtype="bf16", pad=0,
             bits=4),
        # the same through many small experts' down-projections
        dict(name="grad 1024x2048x1024 64/6", op="grad", T=1024, m=2048, n=1024, E=64, k=6, group=64, dtype="fp16", pad=0,
             bits=4),
        # the inner activation of sixteen decoding tokens, six experts each
        dict(name="gated 96x1024", op="gated", R=96, f=1024, act="silu", dtype="fp16", pad=0, step=False),
        # a long batch's, forward with checkpoints and backward from them
        dict(name="gated 16384x14336 step", op="gated", R=16384, f=14336, act="silu", dtype="bf16", pad=0, step=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _side(rng, lo, hi):
    """A side: half of them multiples of 64, half any number."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["route", "rows", "rows", "experts", "experts", "experts", "grad", "grad", "gated"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    pad = rng.choice([0, 0, 0, 8, rng.randint(1, 63)])
    if op == "gated":
        while True:
            c |= {"R": _log(rng, 1, 65536), "f": _side(rng, 64, 14336), "act": rng.choice(["silu", "gelu"]), "pad": pad,
                  "step": rng.random() < 0.7}
            if c["R"] * c["f"] <= GATED_MOST:
                return c
    while True:
        E = _log(rng, 4, 256)
        c |= {"T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E))}
        if op == "route":
            return c | {"dtype": rng.choice(["fp32", "bf16", "fp16"]), "masked": rng.random() < 0.5, "step": rng.random() < 0.5}
        if op == "rows":
            c |= {"h": _side(rng, 64, 8192), "pad": pad, "step": rng.random() < 0.7}
            if c["T"] * c["k"] * c["h"] <= ROWS_MOST:
                return c
            continue
        c |= {"m": _side(rng, 256, 14336), "n": _side(rng, 256, 14336), "group": rng.choice([0, 64, 128, 128, 256]),
              "pad": pad, "bits": rng.choice([3, 4])}
        if E * c["m"] * c["n"] <= STACK_MOST and c["T"] * c["k"] * c["m"] * c["n"] <= EXPERTS_MOST:
            return c


# ------------------------------------------------------------------- inputs

def _logits(gen, T, E):
    """Router outputs: some experts are more in demand than others."""
    return torch.randn((T, E), generator=gen, device=DEV) + 0.5 * torch.randn((1, E), generator=gen, device=DEV)


def _values(gen, rows, cols, pad, dtype):
    """rows x cols (a slice of a buffer cols + pad wide) with a few channels far
    larger than the others, as activations and gradients have."""
    x = torch.empty((rows, cols + pad), dtype=dtype, device=DEV)
    ch = torch.exp(0.7 * torch.randn((1, cols + pad), generator=gen, device=DEV))
    for r in range(0, rows, 4096):
        x[r:r + 4096] = torch.randn((min(4096, rows - r), cols + pad), generator=gen, device=DEV) * ch
    return x[:, :cols]


def _groups(n, group):
    return (n, 1) if group == 0 else (group, -(-n // group))


def _layer(gen, m, n, group, bits):
    """Normal weights with a scale per row, rounded to nearest on the min-max
    grid of each (row, group): codes uint8 m x n, scale and zero m x G."""
    g, G = _groups(n, group)
    maxq = 2 ** bits - 1
    w = torch.randn((m, n), generator=gen, device=DEV)
    w *= 0.02 * torch.exp(0.3 * torch.randn((m, 1), generator=gen, device=DEV))
    lo, hi = torch.empty((m, G), device=DEV), torch.empty((m, G), device=DEV)
    full = n // g
    if full:
        v = w[:, :full * g].reshape(m, full, g)
        lo[:, :full], hi[:, :full] = v.amin(2), v.amax(2)
    if full < G:
        lo[:, full:], hi[:, full:] = w[:, full * g:].amin(1, keepdim=True), w[:, full * g:].amax(1, keepdim=True)
    scale = ((hi - lo) / maxq).clamp_min(1e-6)
    zero = -lo / scale
    col = torch.arange(n, device=DEV) // g
    codes = (w / scale[:, col] + zero[:, col]).round_().clamp_(0, maxq).to(torch.uint8)
    return codes, scale, zero


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "gated":
        R, f, pad = case["R"], case["f"], case["pad"]
        s = {"a": _values(gen, R, f, pad, dtype), "b": _values(gen, R, f, pad, dtype)}
        if case["step"]:
            s["dh"] = _values(gen, R, f, pad, dtype)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    logits = _logits(gen, T, E)
    if op == "route":
        if case["masked"]:
            # an eighth of the experts off, a sixteenth of the tokens padding
            logits.masked_fill_(torch.rand((1, E), generator=gen, device=DEV) < 0.125, -math.inf)
            logits.masked_fill_(torch.rand((T, 1), generator=gen, device=DEV) < 0.0625, -math.inf)
        s = {"logits": logits.to(dtype)}
        if case["step"]:
            s["dweights"] = torch.randn((T, k), generator=gen, device=DEV)
        return s
    r = _plain_route(logits, k)
    if op == "rows":
        h, pad = case["h"], case["pad"]
        s = {"place": r["place"], "weights": r["weights"], "x": _values(gen, T, h, pad, dtype),
             "ys": _values(gen, T * k, h, pad, dtype)}
        if case["step"]:
            s["dy"], s["dxs"] = _values(gen, T, h, pad, dtype), _values(gen, T * k, h, pad, dtype)
        return s
    m, n = case["m"], case["n"]
    layers = [_layer(gen, m, n, case["group"], case["bits"]) for _ in range(E)]
    at = r["offsets"].tolist()
    return {"x": _values(gen, T * k, n if op == "experts" else m, case["pad"], dtype), "offsets": r["offsets"],
            "rows": [(e, at[e], at[e + 1]) for e in range(E) if at[e] < at[e + 1]],
            "w": tuple(torch.stack([v[i] for v in layers]) for i in range(3))}


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if not own:
        return s
    # what a program keeps: packed layers, outputs, checkpoints, the workspace
    import two_sided_hessian_amd as B
    op, dtype = case["op"], DTYPES[case["dtype"]]

    def out(*shape, dtype=dtype):
        return torch.zeros(shape, dtype=dtype, device=DEV)
    if op == "gated":
        R, f = case["R"], case["f"]
        s["h"] = out(R, f)
        if case["step"]:
            s["ck"] = B.Checkpoint8.empty(R, f, dtype, DEV), B.Checkpoint8.empty(R, f, dtype, DEV)
            s["out"] = out(R, f), out(R, f)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    i32 = torch.int32
    if op == "route":
        s["out"] = {"ids": out(T, k, dtype=i32), "weights": out(T, k, dtype=torch.float32), "place": out(T, k, dtype=i32),
                    "order": out(T * k, dtype=i32), "offsets": out(E + 1, dtype=i32)}
        s["ws"] = B.workspace(B.moe_route_workspace_bytes(T, E, k), DEV)
        if case["step"]:
            s["dlogits"] = out(T, E)
    elif op == "rows":
        h = case["h"]
        s["xs"], s["y"] = out(T * k, h), out(T, h)
        if case["step"]:
            s["back"], s["dx"] = {"dys": out(T * k, h), "dweights": out(T, k, dtype=torch.float32)}, out(T, h)
    else:
        s["w"] = B.q4_pack(*s["w"], group_size=case["group"] or None)
        size = B.q4_experts_workspace_bytes if op == "experts" else B.q4_experts_grad_workspace_bytes
        s["ws"] = B.workspace(size(T * k, s["w"]), DEV)
        s["out"] = out(T * k, case["m"] if op == "experts" else case["n"])
    return s


# -------------------------------------------------------- the plain operators

def _plain_route(logits, k):
    T, E = logits.shape
    l = logits.to(torch.float32)
    l = torch.where(torch.isnan(l), -math.inf, l)
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)       # equal logits: the lowest index first
    top, ids = top[:, :k], ids[:, :k]
    live = top > -math.inf
    e = torch.where(live, torch.exp(torch.where(top == top[:, :1], 0.0, top - top[:, :1])), 0.0)
    weights = e / e.sum(1, keepdim=True).clamp_min(1e-30)
    expert = torch.where(live, ids, E).reshape(-1)                      # no choice: behind the last expert
    expert, order = torch.sort(expert, stable=True)
    offsets = torch.searchsorted(expert, torch.arange(E + 1, device=expert.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=order.device)
    return {"ids": torch.where(live, ids, -1).to(torch.int32), "weights": weights,
            "place": torch.where(live, place.reshape(T, k), -1).to(torch.int32),
            "order": torch.where(expert < E, order, -1).to(torch.int32), "offsets": offsets.to(torch.int32)}


def _plain_route_grad(dweights, weights, ids, logits):
    g = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
    E = logits.shape[1]
    dlogits = torch.zeros((ids.shape[0], E + 1), device=ids.device)     # the last column: no choice
    dlogits.scatter_(1, torch.where(ids < 0, E, ids).long(), g)
    return dlogits[:, :E].to(logits.dtype)


def _plain_rows(s, step):
    x, ys, place, w = s["x"].to(torch.float32), s["ys"].to(torch.float32), s["place"].long(), s["weights"]
    dtype = s["x"].dtype
    xs = torch.empty_like(ys)
    xs[place] = x[:, None, :]
    back = ys[place]                                                    # T x k x h
    out = {"xs": xs.to(dtype), "y": (w[:, :, None] * back).sum(1).to(dtype)}
    if step:
        dy = s["dy"].to(torch.float32)
        dys = torch.empty_like(ys)
        dys[place] = w[:, :, None] * dy[:, None, :]
        out |= {"dys": dys.to(dtype), "dweights": (dy[:, None, :] * back).sum(2),
                "dx": s["dxs"].to(torch.float32)[place].sum(1).to(dtype)}
    return out


def _weights(layer, e, group):
    """s (c - z) of expert e in float32."""
    codes, scale, zero = (v[e] for v in layer)
    col = torch.arange(codes.shape[1], device=codes.device) // _groups(codes.shape[1], group)[0]
    return scale[:, col] * (codes.to(torch.float32) - zero[:, col])


def _plain_experts(s, case):
    grad = case["op"] == "grad"
    y = torch.zeros((s["x"].shape[0], case["n"] if grad else case["m"]), dtype=s["x"].dtype, device=s["x"].device)
    for e, p, q in s["rows"]:
        w = _weights(s["w"], e, case["group"])
        y[p:q] = (s["x"][p:q].to(torch.float32) @ (w if grad else w.t())).to(y.dtype)
    return y


def _slope(a, act):
    """s with act(a) = a sigmoid(s), and ds/da."""
    if act == "silu":
        return a, torch.ones_like(a)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    return c * (a + 0.044715 * a * a * a), c * (1.0 + 3.0 * 0.044715 * a * a)


def _eight_bits(x):
    """What the 8-bit checkpoint of x stands for: in each row's blocks of 32
    columns, whole multiples (-127 .. 127) of the smallest power of two that
    reaches the block's largest value."""
    R, f = x.shape
    v = torch.zeros((R, -(-f // 32) * 32), device=x.device)
    v[:, :f] = x
    v = v.reshape(R, -1, 32)
    top = v.abs().amax(2, keepdim=True)
    step = torch.exp2(torch.frexp(top)[1].to(torch.float32) - 7.0)      # top / step in [64, 128)
    step = torch.where(torch.round(top / step) > 127.0, 2.0 * step, step)
    return (torch.round(v / step) * step).reshape(R, -1)[:, :f]


def _plain_gated(s, case):
    act, dtype = case["act"], s["a"].dtype
    a, b = s["a"].to(torch.float32), s["b"].to(torch.float32)
    h = (a / (1.0 + torch.exp(-_slope(a, act)[0])) * b).to(dtype)
    if not case["step"]:
        return {"h": h}
    a, b, dh = _eight_bits(a), _eight_bits(b), s["dh"].to(torch.float32)
    t, dt = _slope(a, act)
    p = 1.0 / (1.0 + torch.exp(-t))
    return {"h": h, "da": (dh * b * (p + a * p * (1.0 - p) * dt)).to(dtype), "db": (dh * (a * p)).to(dtype)}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import two_sided_hessian_amd as B
        if op == "route":
            r = B.moe_route(state["logits"], case["k"], out=state["out"], ws=state["ws"])
            if not case["step"]:
                return r
            return r | {"dlogits": B.moe_route_grad(state["dweights"], r["weights"], r["ids"], case["E"], out=state["dlogits"])}
        if op == "rows":
            place, w = state["place"], state["weights"]
            out = {"xs": B.moe_gather(state["x"], place, out=state["xs"]),
                   "y": B.moe_combine(state["ys"], place, w, out=state["y"])}
            if case["step"]:
                out |= B.moe_combine_grad(state["dy"], state["ys"], place, w, out=state["back"])
                out["dx"] = B.moe_combine(state["dxs"], place, out=state["dx"])
            return out
        if op == "gated":
            if not case["step"]:
                return {"h": B.gated_act(state["a"], state["b"], act=case["act"], out=state["h"])}
            h, ca, cb = B.gated_act(state["a"], state["b"], act=case["act"], checkpoint=state["ck"], out=state["h"])
            da, db = B.gated_act_grad(state["dh"], ca, cb, act=case["act"], out=state["out"])
            return {"h": h, "da": da, "db": db}
        call = B.q4_experts if op == "experts" else B.q4_experts_grad
        return call(state["x"], state["w"], state["offsets"], out=state["out"], ws=state["ws"])
    if op == "route":
        r = _plain_route(state["logits"], case["k"])
        if case["step"]:
            r["dlogits"] = _plain_route_grad(state["dweights"], r["weights"], r["ids"], state["logits"])
        return r
    if op == "rows":
        return _plain_rows(state, case["step"])
    return _plain_gated(state, case) if op == "gated" else _plain_experts(state, case)


def work(case):
    """2 bytes a value, 4 bits a code, 8 bytes a (scale, zero) pair."""
    op = case["op"]
    if op == "gated":
        values = case["R"] * case["f"]
        return {"bytes": 12.0 * values, "flops": 25.0 * values} if case["step"] else {"bytes": 6.0 * values, "flops": 8.0 * values}
    T, E, k = case["T"], case["E"], case["k"]
    pairs = T * k
    if op == "route":
        size = 4 if case["dtype"] == "fp32" else 2
        once = T * E * size + 16 * pairs + 4 * (E + 1)
        return {"bytes": once + (T * E * size + 4 * pairs if case["step"] else 0.0), "flops": 2.0 * T * E + 4.0 * pairs}
    if op == "rows":
        h = case["h"]
        once = 4.0 * h * (T + pairs) + 8 * pairs
        # back: dy and dxs read, dys, dweights and dx written (ys, place and weights have been read)
        return {"bytes": once + (4.0 * h * (T + pairs) + 4 * pairs if case["step"] else 0.0),
                "flops": (6.0 if case["step"] else 2.0) * pairs * h}
    m, n = case["m"], case["n"]
    # experts that T tokens of k choices each reach, were the choices even
    used = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": used * (m * n / 2 + 8 * m * _groups(n, case["group"])[1]) + 2.0 * pairs * (m + n),
            "flops": 2.0 * pairs * m * n}


# ------------------------------------------------------------------ in 64 bits

def _exact_route(case, s):
    l, k = s["logits"].double(), case["k"]
    T, E = l.shape
    index = torch.arange(E, device=l.device)
    weights = torch.zeros((T, k), dtype=torch.float64, device=l.device)
    dlogits = torch.zeros((T, E), dtype=torch.float64, device=l.device) if case["step"] else None
    for t in range(0, T, 512):
        v = l[t:t + 512]
        # an expert's rank: how many logits are larger, or equal with a lower index
        above = (v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & (index[None, None, :] < index[None, :, None]))
        rank = above.sum(2)
        chosen = (rank < k) & (v > -math.inf)
        some = chosen.any(1, keepdim=True)
        share = torch.where(chosen, v, -math.inf)
        share = torch.softmax(torch.where(some, share, 0.0), 1) * chosen
        full = torch.zeros((v.shape[0], max(k, E)), dtype=torch.float64, device=l.device)
        full.scatter_(1, rank, share)
        weights[t:t + 512] = full[:, :k]
        if case["step"]:
            d = torch.gather(s["dweights"][t:t + 512].double(), 1, rank.clamp_max(k - 1)) * chosen
            dlogits[t:t + 512] = share * (d - (share * d).sum(1, keepdim=True))
    out = {"ids": None, "weights": weights, "place": None, "order": None, "offsets": None}
    return out | {"dlogits": dlogits} if case["step"] else out


def _exact_rows(case, s):
    T, k, h = case["T"], case["k"], case["h"]
    place, w = s["place"].long(), s["weights"].double()
    token = torch.empty(T * k, dtype=torch.long, device=DEV)            # of each sorted row
    share = torch.empty(T * k, dtype=torch.float64, device=DEV)
    for j in range(k):
        token[place[:, j]] = torch.arange(T, device=DEV)
        share[place[:, j]] = w[:, j]

    def summed(v):
        return torch.zeros((T, h), dtype=torch.float64, device=DEV).index_add_(0, token, v)
    ys = s["ys"].double()
    out = {"xs": s["x"].double()[token], "y": summed(ys * share[:, None])}
    if case["step"]:
        dy = s["dy"].double()[token]
        out |= {"dys": dy * share[:, None], "dweights": (dy * ys).sum(1)[place], "dx": summed(s["dxs"].double())}
    return out


def _exact_experts(case, s):
    grad = case["op"] == "grad"
    g, G = _groups(case["n"], case["group"])
    y = torch.zeros((s["x"].shape[0], case["n"] if grad else case["m"]), dtype=torch.float64, device=DEV)
    for e, p, q in s["rows"]:
        codes, scale, zero = (v[e].double() for v in s["w"])
        w = torch.cat([scale[:, i:i + 1] * (codes[:, i * g:(i + 1) * g] - zero[:, i:i + 1]) for i in range(G)], dim=1)
        y[p:q] = torch.mm(s["x"][p:q].double(), w if grad else w.T.contiguous())
    return y


def _exact_checkpoint(x):
    """Block by block: the step is 2^e, e the least with round(top / 2^e) <= 127."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], 32):
        v = x[:, c:c + 32]
        top = v.abs().amax(1, keepdim=True)
        e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 8.0
        for _ in range(4):
            e = torch.where(torch.round(top * torch.exp2(-e)) > 127.0, e + 1.0, e)
        out[:, c:c + 32] = torch.round(v * torch.exp2(-e)) * torch.exp2(e)
    return out


def _exact_gated(case, s):
    silu = case["act"] == "silu"

    def act(v):
        return v * torch.sigmoid(v) if silu else 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))

    def slope(v):
        if silu:
            p = torch.sigmoid(v)
            return p + v * p * (1.0 - p)
        u = torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
        return 0.5 * (1.0 + u) + 0.5 * v * (1.0 - u * u) * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * v * v)
    parts = {"h": [], "da": [], "db": []}
    for r in range(0, case["R"], 2048):
        a, b = s["a"][r:r + 2048].double(), s["b"][r:r + 2048].double()
        parts["h"].append(act(a) * b)
        if case["step"]:
            a, b, dh = _exact_checkpoint(a), _exact_checkpoint(b), s["dh"][r:r + 2048].double()
            parts["da"].append(dh * b * slope(a))
            parts["db"].append(dh * act(a))
    return {name: torch.cat(v) for name, v in parts.items() if v}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "rows":
        return _exact_rows(case, s)
    return _exact_gated(case, s) if case["op"] == "gated" else _exact_experts(case, s)
