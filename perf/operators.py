"""The measured cases of the 4-bit layer operators.

A layer that the solver has rounded is codes c (0 .. 15), a step s and a zero
point z per (output row, group of input columns); its weights are s (c - z).
The operators compute with such layers without writing the weights out:

* "linear"  y = x W^T for a few tokens (one decoding step) or a whole prompt;
* "grad"    dx = dy W, the gradient that passes back through a rounded layer;
* "moe"     a mixture-of-experts layer for a few tokens: router, top-k,
            gated feed-forward of the chosen experts, weighted sum.

listed() names the cases, draw() draws others of the same ranges, prepare()
makes a case's inputs and what a program keeps between calls, run() is one
call, exact() the same from the definition in float64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"

# Ranges: a few tokens are 1 .. 64, a prompt 65 .. 8192; no side above 16384,
# no linear or grad case above LINEAR_MOST multiply-adds (the largest listed),
# no expert stack above MOE_MOST weights (the largest listed).
LINEAR_MOST = 8192 ** 3
MOE_MOST = 8 * 4096 * 14336


def listed():
    return [
        # one decoding step of a small square layer: latency
        dict(name="few 1x1024x1024", op="linear", T=1, m=1024, n=1024, group=128, dtype="bf16", pad=0, bits=3),
        # one decoding step of the widest projection of a 4096 / 14336 gated MLP
        dict(name="few 1x4096x14336", op="linear", T=1, m=4096, n=14336, group=128, dtype="bf16", pad=0, bits=4),
        # sixteen sequences decoding together, small groups
        dict(name="few 16x14336x4096", op="linear", T=16, m=14336, n=4096, group=64, dtype="fp16", pad=0, bits=4),
        # five tokens, no side a multiple of anything, one grid per row, x a slice of a wider buffer
        dict(name="few 5x1001x4099 ragged", op="linear", T=5, m=1001, n=4099, group=0, dtype="bf16", pad=7, bits=4),
        # a prompt through a square attention projection
        dict(name="prompt 2048x4096x4096", op="linear", T=2048, m=4096, n=4096, group=128, dtype="bf16", pad=0, bits=4),
        # the largest: a long prompt through an 8192 x 8192 layer, one grid per row
        dict(name="prompt 8192x8192x8192", op="linear", T=8192, m=8192, n=8192, group=0, dtype="bf16", pad=0, bits=3),
        # a short odd prompt, odd layer, small groups, half precision
        dict(name="prompt 777x4099x2050 ragged", op="linear", T=777, m=4099, n=2050, group=64, dtype="fp16", pad=3, bits=4),
        # calibration: a sequence's gradient back through a rounded up-projection
        dict(name="grad 2048x4096x14336", op="grad", T=2048, m=4096, n=14336, group=128, dtype="bf16", pad=0, bits=4),
        # an odd short sequence's gradient through an odd layer
        dict(name="grad 300x1000x1531 ragged", op="grad", T=300, m=1000, n=1531, group=64, dtype="fp16", pad=5, bits=3),
        # one token through eight large experts, two chosen
        dict(name="moe 1x4096x14336 8/2", op="moe", T=1, h=4096, f=14336, E=8, k=2, group=128, dtype="bf16", bits=4),
        # sixteen tokens through many small experts
        dict(name="moe 16x2048x1024 64/6", op="moe", T=16, h=2048, f=1024, E=64, k=6, group=64, dtype="fp16", bits=4),
        # three tokens, odd sides, one grid per row
        dict(name="moe 3x1003x1501 5/2 ragged", op="moe", T=3, h=1003, f=1501, E=5, k=2, group=0, dtype="bf16", bits=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _side(rng, lo, hi):
    """A side: half of them multiples of 64, half any number."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    kind = rng.choice(["few", "few", "prompt", "prompt", "grad", "moe", "moe"])
    c = {"group": rng.choice([0, 64, 128, 128, 256]), "dtype": rng.choice(["bf16", "bf16", "fp16"]),
         "bits": rng.choice([3, 4])}
    if kind == "moe":
        while True:
            c |= {"op": "moe", "T": _log(rng, 1, 64), "h": _side(rng, 256, 4096), "f": _side(rng, 256, 14336),
                  "E": _log(rng, 4, 64)}
            c["k"] = rng.randint(1, min(8, c["E"]))
            if c["E"] * c["h"] * c["f"] <= MOE_MOST and 3072 not in (c["h"], c["f"]):
                return c
    while True:
        T = _log(rng, 1, 64) if kind == "few" else _log(rng, 65, 8192) if kind == "prompt" else _log(rng, 1, 8192)
        c |= {"op": "grad" if kind == "grad" else "linear", "T": T, "m": _side(rng, 256, 16384),
              "n": _side(rng, 256, 16384), "pad": rng.choice([0, 0, 0, 8, rng.randint(1, 63)])}
        if T * c["m"] * c["n"] <= LINEAR_MOST and 3072 not in (T, c["m"], c["n"]):
            return c


# ------------------------------------------------------------------- inputs

def _groups(n, group):
    return (n, 1) if group == 0 else (group, -(-n // group))


def _layer(gen, m, n, group, bits):
    """Normal weights with a scale per row, rounded to nearest on the min-max
    grid of each (row, group): codes uint8 m x n, scale and zero m x G, the
    zero point fractional."""
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


def _stack(gen, E, m, n, group, bits):
    """E layers: codes E x m x n, scale and zero E x m x G."""
    G = _groups(n, group)[1]
    codes = torch.empty((E, m, n), dtype=torch.uint8, device=DEV)
    scale, zero = torch.empty((E, m, G), device=DEV), torch.empty((E, m, G), device=DEV)
    for e in range(E):
        codes[e], scale[e], zero[e] = _layer(gen, m, n, group, bits)
    return codes, scale, zero


def _tokens(gen, T, n, pad, dtype):
    """T rows of n values (a slice of a buffer n + pad wide) with a few
    channels far larger than the others, as activations and gradients have."""
    x = torch.randn((T, n + pad), generator=gen, device=DEV)
    x *= torch.exp(0.7 * torch.randn((1, n + pad), generator=gen, device=DEV))
    return x.to(dtype)[:, :n]


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "moe":
        h, f, E = case["h"], case["f"], case["E"]
        return {"x": _tokens(gen, case["T"], h, 0, dtype),
                "router": (torch.randn((E, h), generator=gen, device=DEV) * (2.0 / math.sqrt(h))).to(dtype),
                "gate": _stack(gen, E, f, h, case["group"], case["bits"]),
                "up": _stack(gen, E, f, h, case["group"], case["bits"]),
                "down": _stack(gen, E, h, f, case["group"], case["bits"])}
    m, n = case["m"], case["n"]
    return {"x": _tokens(gen, case["T"], n if case["op"] == "linear" else m, case["pad"], dtype),
            "w": _layer(gen, m, n, case["group"], case["bits"])}


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if own:
        # what a program keeps: the packed layer, the output, the workspace
        import two_sided_hessian_amd as B
        T, g = case["T"], case["group"] or None
        if case["op"] == "moe":
            for key in ("gate", "up", "down"):
                s[key] = B.q4_pack(*s[key], group_size=g)
            s["ws"] = B.workspace(B.q4_moe_workspace_bytes(T, s["gate"], case["k"]), DEV)
        else:
            s["w"] = B.q4_pack(*s["w"], group_size=g)
            size = B.q4_linear_workspace_bytes if case["op"] == "linear" else B.q4_linear_grad_workspace_bytes
            s["ws"] = B.workspace(size(T, s["w"]), DEV)
            s["out"] = torch.empty((T, case["m"] if case["op"] == "linear" else case["n"]),
                                   dtype=s["x"].dtype, device=DEV)
    return s


# -------------------------------------------------------- the plain operators

def _weights(layer, group):
    """s (c - z) in float32, of one layer or of a stack."""
    codes, scale, zero = layer
    n = codes.shape[-1]
    col = torch.arange(n, device=codes.device) // _groups(n, group)[0]
    return scale[..., col] * (codes.to(torch.float32) - zero[..., col])


def _plain_linear(x, layer, group):
    return (x.to(torch.float32) @ _weights(layer, group).t()).to(x.dtype)


def _plain_grad(dy, layer, group):
    return (dy.to(torch.float32) @ _weights(layer, group)).to(dy.dtype)


def _plain_moe(s, case):
    x, group = s["x"].to(torch.float32), case["group"]
    logits = x @ s["router"].to(torch.float32).t()                      # T x E
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)  # equal logits: the lowest index first
    top, ids = top[:, :case["k"]], ids[:, :case["k"]]
    e = torch.exp(top - top[:, :1])
    p = e / e.sum(1, keepdim=True)
    if ids.numel() <= case["E"]:
        # fewer choices than experts: the chosen layers, one per choice
        pick = ids.reshape(-1)
        xt = x.repeat_interleave(case["k"], dim=0)[:, :, None]         # Tk x h x 1
        gate, up, down = ([v[pick] for v in s[key]] for key in ("gate", "up", "down"))
    else:
        # every layer on every token
        xt = x.t().contiguous()                                        # h x T
        gate, up, down = s["gate"], s["up"], s["down"]
    a = torch.matmul(_weights(gate, group), xt)
    b = torch.matmul(_weights(up, group), xt)
    y = torch.matmul(_weights(down, group), a / (1.0 + torch.exp(-a)) * b)
    if ids.numel() <= case["E"]:
        y = (y.reshape(case["T"], case["k"], case["h"]) * p[:, :, None]).sum(1)
    else:
        share = torch.zeros_like(logits).scatter_(1, ids, p)           # T x E, zero where not chosen
        y = (y * share.t()[:, None, :]).sum(0).t().contiguous()
    return {"y": y.to(s["x"].dtype), "ids": ids.to(torch.int32), "weights": p}


def run(state):
    case = state["case"]
    if own:
        import two_sided_hessian_amd as B
        if case["op"] == "moe":
            return B.q4_moe(state["x"], state["router"], state["gate"], state["up"], state["down"], case["k"],
                            ws=state["ws"])
        call = B.q4_linear if case["op"] == "linear" else B.q4_linear_grad
        return call(state["x"], state["w"], out=state["out"], ws=state["ws"])
    if case["op"] == "moe":
        return _plain_moe(state, case)
    return (_plain_linear if case["op"] == "linear" else _plain_grad)(state["x"], state["w"], case["group"])


def work(case):
    """4 bits a code, 8 bytes a (scale, zero) pair, 2 bytes a value."""
    if case["op"] == "moe":
        T, h, f, E, k = (case[i] for i in ("T", "h", "f", "E", "k"))
        # experts that T tokens of k choices each reach, were the choices even
        used = E * (1.0 - (1.0 - k / E) ** T)
        layer = 2 * (f * h / 2 + 8 * f * _groups(h, case["group"])[1]) + h * f / 2 + 8 * h * _groups(f, case["group"])[1]
        return {"bytes": used * layer + 2 * E * h + 4 * T * h + 8 * T * k,
                "flops": 2.0 * T * E * h + 6.0 * T * k * h * f}
    T, m, n = case["T"], case["m"], case["n"]
    return {"bytes": m * n / 2 + 8 * m * _groups(n, case["group"])[1] + 2 * T * (m + n), "flops": 2.0 * T * m * n}


# ------------------------------------------------------------------ in 64 bits

def _exact_layer(layer, group):
    codes, scale, zero = layer
    n = codes.shape[1]
    g, G = _groups(n, group)
    return torch.cat([scale[:, q:q + 1].double() * (codes[:, q * g:(q + 1) * g].double() - zero[:, q:q + 1].double())
                      for q in range(G)], dim=1)


def exact(case, seed):
    s = _inputs(case, seed)
    x = s["x"].double()
    if case["op"] == "linear":
        return torch.mm(x, _exact_layer(s["w"], case["group"]).T.contiguous())
    if case["op"] == "grad":
        return torch.mm(x, _exact_layer(s["w"], case["group"]))
    T, k = case["T"], case["k"]
    logits = torch.mm(x, s["router"].double().T.contiguous())
    lists = logits.tolist()
    y = torch.zeros((T, case["h"]), dtype=torch.float64, device=x.device)
    p = torch.zeros((T, k), dtype=torch.float64, device=x.device)
    chosen = {}                                                          # expert -> [(token, place)]
    for t in range(T):
        order = sorted(range(case["E"]), key=lambda e: (-lists[t][e], e))[:k]
        p[t] = torch.softmax(logits[t, order], 0)
        for j, e in enumerate(order):
            chosen.setdefault(e, []).append((t, j))
    for e, pairs in chosen.items():
        rows, place = [t for t, _ in pairs], [j for _, j in pairs]
        gate, up, down = (_exact_layer([v[e] for v in s[key]], case["group"]) for key in ("gate", "up", "down"))
        a, b = torch.mm(x[rows], gate.T.contiguous()), torch.mm(x[rows], up.T.contiguous())
        y[rows] += p[rows, place][:, None] * torch.mm(a * torch.sigmoid(a) * b, down.T.contiguous())
    return {"y": y, "ids": None, "weights": p}
