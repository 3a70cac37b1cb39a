"""Round the layers of a small gated mixture-of-experts block and run it on
its 4-bit codes.

    python examples/quantize_and_serve.py [--hidden 512] [--ffn 1024] [--experts 8] [--tokens 256]

1. Every expert's gate, up and down projection is rounded to 4 bits with
   per-group grids under its input's second moment (moment, factor, gptq), and
   an attention-output projection two-sidedly (solve with K-FAC factors).
2. q4_pack lays codes and grids out; nothing keeps the weights.
3. A prompt runs through the projection (q4_linear, many tokens), then single
   tokens are decoded through projection and experts (q4_linear, q4_moe).
4. q4_linear_grad takes an output gradient back through the rounded projection:
   what the Kronecker factors of the layers before it are built from.

Random weights and inputs; prints how far the rounded block is from the
float32 one and from the same block with its weights written out.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import two_sided_hessian_amd as B  # noqa: E402

GROUP = 64


def grids(W, group, maxq=15):
    """Min-max grids per (row, group of columns): scale, zero, maxq."""
    m, n = W.shape
    parts = W.split(group, dim=1)
    lo = torch.stack([p.amin(1) for p in parts], 1)
    hi = torch.stack([p.amax(1) for p in parts], 1)
    scale = ((hi - lo) / maxq).clamp_min(1e-8)
    return scale.contiguous(), (-lo / scale).contiguous(), torch.full_like(scale, maxq, dtype=torch.int32)


def written_out(codes, scale, zero, group):
    col = torch.arange(codes.shape[1], device=codes.device) // group
    return scale[:, col] * (codes.float() - zero[:, col])


def round_one_sided(W, X):
    """GPTQ with the input's second moment: codes, scale, zero."""
    A = B.moment(X)
    L, P, info = B.factor(A)
    s, z, q = grids(W, GROUP)
    out = B.gptq(W, L, P, s, z, q, group_size=GROUP)
    assert int(info) == 0
    return out["codes"], s, z


def round_two_sided(W, X, Gy):
    """BaKron with K-FAC factors of inputs X and output gradients Gy."""
    A, Bf = B.kfac_factors(X, Gy)
    LA, PA, ia = B.factor(A)
    LB, PB, ib = B.factor(Bf)
    s, z, q = grids(W, GROUP)
    out = B.solve(W, LA, PA, LB, PB, s, z, q, group_size=GROUP)
    assert int(ia) == 0 and int(ib) == 0
    return out["codes"], s, z


def moe_float(x, router, gate, up, down, k):
    """The expert layer in float32 with its weights written out."""
    top, ids = torch.topk(x @ router.float().t(), k, dim=1)
    p = torch.softmax(top, dim=1)
    y = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(k):
            e = int(ids[t, j])
            y[t] += p[t, j] * (down[e] @ (torch.nn.functional.silu(gate[e] @ x[t]) * (up[e] @ x[t])))
    return y


def rel(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--ffn", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=256)
    a = ap.parse_args(argv)
    h, f, E, k, T = a.hidden, a.ffn, a.experts, a.top_k, a.tokens
    dev = "cuda:0"
    gen = torch.Generator(device=dev)
    gen.manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    X = randn(2048, h) * torch.exp(0.5 * randn(1, h))          # calibration samples
    proj = 0.02 * randn(h, h)
    weights = {name: [0.02 * randn(*s) for _ in range(E)] for name, s in (("gate", (f, h)), ("up", (f, h)), ("down", (h, f)))}
    router = (2.0 / h ** 0.5 * randn(E, h)).bfloat16()

    # 1, 2: round and pack
    c, s, z = round_two_sided(proj, X, randn(2048, h))
    w_proj, proj_q = B.q4_pack(c, s, z, group_size=GROUP), written_out(c, s, z, GROUP)
    packed, rounded = {}, {}
    inner = randn(2048, f)
    for name, layers in weights.items():
        parts = [round_one_sided(W, inner if name == "down" else X) for W in layers]
        packed[name] = B.q4_pack(*(torch.stack(v) for v in zip(*parts)), group_size=GROUP)
        rounded[name] = [written_out(*v, GROUP) for v in parts]

    # 3: a prompt, then four decoding steps of one token each
    prompt = (randn(T, h) * torch.exp(0.5 * randn(1, h))).bfloat16()
    y = B.q4_linear(prompt, w_proj)
    prompt_err = rel(y, prompt.float() @ proj_q.t())
    token, moe_err = y[-1:], 0.0
    for _ in range(4):
        hid = B.q4_linear(token, w_proj)
        out = B.q4_moe(hid, router, packed["gate"], packed["up"], packed["down"], k)
        moe_err = max(moe_err, rel(out["y"], moe_float(hid.float(), router, rounded["gate"], rounded["up"], rounded["down"], k)))
        token = (out["y"].float() + hid.float()).bfloat16()
        token = (token.float() / token.float().pow(2).mean().sqrt()).bfloat16()

    # 4: a gradient back through the rounded projection, and its factor
    dy = randn(T, h).bfloat16()
    dx = B.q4_linear_grad(dy, w_proj)
    grad_err = rel(dx, dy.float() @ proj_q)
    factor = B.moment(dx.float())

    res = {"prompt against the rounded weights": prompt_err, "experts against the rounded weights": moe_err,
           "gradient against the rounded weights": grad_err,
           "rounded prompt against float32": rel(y, prompt.float() @ proj.t())}
    for what, v in res.items():
        print(f"{what}: {v:.2e}")
    print(f"trace of the next layer's output factor: {float(factor.diagonal().sum()):.4g}")
    return res


if __name__ == "__main__":
    main()
