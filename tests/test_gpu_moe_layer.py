"""The expert layer for many tokens as a whole: q4_moe_layer against its formula
and against q4_moe, its gradients against the calls that it is made of, in HIP
graphs, on other streams.

Tolerance of the forward pass: a and b, the activation h and the experts' results
ys are rounded to the type, and so is the sum.  A relative error of u at most in a,
b and h changes h by u |a act'(a) b|, u |h| and u |h|; these roundings are
independent from value to value and meet the down layer's weights d_i, so that
their sum exceeds six times u (sum_i d_i^2 (2 h_i^2 + (a_i act'(a_i) b_i)^2))^(1/2)
with a probability below 2 exp(-18) were each as large as it can be (Hoeffding), 2
exp(-54) at their mean square.  ys adds u |ys| per choice, times its share, the
result u |y|, and the float32 sums what they add to the linear layer."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_q4 import DEV, LINEAR, TINY, U, make_layer, pack, rms, tokens, weights64

pytestmark = pytest.mark.gpu


def make(T, h, f, E, k, group, dtype, seed, masked=False):
    stacks = [make_layer(f, h, group, seed, lead=(E,)), make_layer(f, h, group, seed + 1, lead=(E,)),
              make_layer(h, f, group, seed + 2, lead=(E,))]
    for codes, scale, zero in stacks:                             # results of the order of 1
        scale *= 6.0 / np.sqrt(codes.shape[-1])
        zero[:] = np.random.default_rng(seed).uniform(5.0, 10.0, zero.shape)
    g = torch.Generator().manual_seed(seed)
    logits = 2 * torch.randn((T, E), generator=g)
    if masked:
        logits[torch.rand((T, E), generator=g) < 0.3] = -float("inf")
        logits[torch.rand((T,), generator=g) < 0.2] = -float("inf")
    return tokens(T, h, dtype, seed), logits.to(DEV), stacks, [pack(*s, group) for s in stacks]


def formula(x, r, stacks, group, act="silu"):
    """The layer in float64, the sum over choices of the magnitudes of their results,
    and the squares that its inner roundings go by."""
    x, ids, p = x.double().cpu().numpy(), r["ids"].cpu().numpy(), r["weights"].double().cpu().numpy()
    gate, up, down = (weights64(*s, group) for s in stacks)
    y, size, squares = (np.zeros((x.shape[0], down.shape[1])) for _ in range(3))
    for e in range(gate.shape[0]):
        t, j = np.nonzero(ids == e)
        if len(t):
            share = p[t, j][:, None]
            a, b = x[t] @ gate[e].T, x[t] @ up[e].T
            c = 2 * np.sqrt(2 / np.pi)
            s, ds = (a, 1.0) if act == "silu" else (c * (a + 0.044715 * a ** 3), c * (1 + 3 * 0.044715 * a ** 2))
            q = 1 / (1 + np.exp(-s))
            h = a * q * b
            v = share * (h @ down[e].T)
            np.add.at(y, t, v)
            np.add.at(size, t, np.abs(v))
            np.add.at(squares, t, share ** 2 * ((2 * h ** 2 + (a * (q + a * q * (1 - q) * ds) * b) ** 2) @ (down[e] ** 2).T))
    return y, size, squares


def close_layer(got, ref, dtype, keep=slice(None)):
    y, size, squares = (v[keep] for v in ref)
    u = U[dtype]
    tol = u * 1.02 * (np.abs(y) + size) + 6 * u * np.sqrt(squares) + 2 * LINEAR * rms(y) + TINY[dtype]
    worst = (np.abs(got.double().cpu().numpy() - y) / tol).max()
    assert worst <= 1.0, f"{worst:.2f} times the tolerance"


CASES = [(1, 130, 100, 8, 2, 64), (16, 256, 192, 64, 6, 64), (65, 100, 130, 5, 5, 0), (300, 192, 320, 8, 2, 128),
         (1000, 64, 128, 16, 4, 0), (700, 200, 90, 3, 1, 64)]


@pytest.mark.parametrize("T,h,f,E,k,group", CASES)
def test_the_layer_matches_its_formula(T, h, f, E, k, group):
    for dtype, act, masked in ((torch.bfloat16, "silu", False), (torch.float16, "gelu", True)):
        x, logits, stacks, w = make(T, h, f, E, k, group, dtype, T + h, masked)
        y = B.q4_moe_layer(x, logits, *w, k, act=act)
        ref = formula(x, B.moe_route(logits, k), stacks, group, act)
        close_layer(y, ref, dtype)
        assert (y[torch.isinf(logits).all(1)] == 0).all()
        assert torch.equal(y, B.q4_moe_layer(x, logits, *w, k, act=act))


def test_the_layer_and_the_one_for_few_tokens_agree():
    T, h, f, E, k, group, dtype = 40, 256, 192, 8, 2, 64, torch.bfloat16
    x, _, stacks, w = make(T, h, f, E, k, group, dtype, 3)
    router = tokens(E, h, dtype, 9).contiguous() * 0.1
    few = B.q4_moe(x, router, *w, k)
    logits = x.float() @ router.float().t()
    r = B.moe_route(logits, k)
    same = (r["ids"] == few["ids"]).all(1)
    assert same.float().mean() > 0.9
    y, ref = B.q4_moe_layer(x, logits, *w, k), formula(x, r, stacks, group)
    keep = same.cpu().numpy()
    close_layer(y[same], ref, dtype, keep)
    close_layer(few["y"][same], ref, dtype, keep)


def by_hand(x, logits, w, k, act, dy):
    """Forward and backward by the single calls."""
    r = B.moe_route(logits, k)
    at, R = r["offsets"], x.shape[0] * k
    xs = B.moe_gather(x, r["place"])
    a, b = B.q4_experts(xs, w[0], at), B.q4_experts(xs, w[1], at)
    h, ca, cb = B.gated_act(a, b, act=act, checkpoint=True, count=at[-1:])
    ys = B.q4_experts(h, w[2], at)
    y = B.moe_combine(ys, r["place"], r["weights"])
    back = B.moe_combine_grad(dy, ys, r["place"], r["weights"])
    dlogits = B.moe_route_grad(back["dweights"], r["weights"], r["ids"], logits.shape[1], dtype=logits.dtype)
    da, db = B.gated_act_grad(B.q4_experts_grad(back["dys"], w[2], at), ca, cb, act=act, count=at[-1:])
    dxs = torch.cat((B.q4_experts_grad(da, w[0], at), B.q4_experts_grad(db, w[1], at)))
    place = torch.cat((r["place"], torch.where(r["place"] < 0, -1, r["place"] + R)), 1)
    return y, B.moe_combine(dxs, place), dlogits


@pytest.mark.parametrize("T,h,f,E,k,group", CASES[1:])
def test_gradients_are_those_of_the_calls(T, h, f, E, k, group):
    dtype = torch.bfloat16
    x, logits, _, w = make(T, h, f, E, k, group, dtype, T, masked=True)
    dy = tokens(T, h, dtype, 5)
    for what in ((True, True), (True, False), (False, True)):
        xg, lg = x.clone().requires_grad_(what[0]), logits.clone().requires_grad_(what[1])
        y = B.q4_moe_layer(xg, lg, *w, k)
        y.backward(dy)
        ref, dx, dl = by_hand(x, logits, w, k, "silu", dy)
        assert torch.equal(y, ref)
        assert torch.equal(xg.grad, dx) if what[0] else xg.grad is None
        assert torch.equal(lg.grad, dl) if what[1] else lg.grad is None
        assert torch.isfinite(dx).all() and torch.isfinite(dl).all()


def test_the_single_calls_under_autograd():
    """The same layer written with the differentiable calls gives the same
    gradients: of the logits to the bit, of x but for one more rounding of the two
    halves of its sum."""
    T, h, f, E, k, group, dtype = 200, 192, 130, 6, 2, 64, torch.bfloat16
    x, logits, _, w = make(T, h, f, E, k, group, dtype, 8, masked=True)
    dy = tokens(T, h, dtype, 5)
    xg, lg = x.clone().requires_grad_(), logits.clone().requires_grad_()
    r = B.moe_route(lg, k)
    xs = B.moe_gather(xg, r["place"])
    hs = B.gated_act(B.q4_experts(xs, w[0], r["offsets"]), B.q4_experts(xs, w[1], r["offsets"]), count=r["offsets"][-1:])
    y = B.moe_combine(B.q4_experts(hs, w[2], r["offsets"]), r["place"], r["weights"])
    y.backward(dy)
    ref, dx, dl = by_hand(x, logits, w, k, "silu", dy)
    assert torch.equal(y, ref) and torch.equal(lg.grad, dl)
    # three roundings (the halves' sum per row, the sum over rows twice as large at most)
    assert ((xg.grad.double() - dx.double()).abs() <= 3 * U[dtype] * dx.double().abs() + 6 * U[dtype] * dx.double().square().mean(1, keepdim=True).sqrt()).all()


def test_gradients_by_differences():
    """Along one direction of x and of the logits, over all results at once.  Both
    sides carry 16-bit roundings and the gradient the checkpoints' 8 bits (1 / 254 of
    a block's largest value, some three deviations, at most: 0.7 % in the mean
    square), independent over 8192 results: 2 % of the product of the norms is six
    times what that leaves of a sum of 8192 terms."""
    T, h, f, E, k, group, dtype = 64, 128, 256, 4, 2, 64, torch.float16
    x, logits, _, w = make(T, h, f, E, k, group, dtype, 12)
    dy = tokens(T, h, dtype, 5)
    xg, lg = x.clone().requires_grad_(), logits.clone().requires_grad_()
    B.q4_moe_layer(xg, lg, *w, k).backward(dy)
    ids = B.moe_route(logits, k)["ids"]
    d, g = xg.grad.double(), dy.double()

    def value(x, l):   # per token; a token whose choice the step changes is left out
        same = (B.moe_route(l, k)["ids"].sort(1)[0] == ids.sort(1)[0]).all(1)
        return (B.q4_moe_layer(x, l, *w, k).double() * g).sum(1), same

    def agree(up, down, d):
        (a, p), (b, q) = value(*up), value(*down)
        on = p & q
        assert on.sum() >= T - 4
        moved = up[0].double() - down[0].double() if d is xg.grad else up[1].double() - down[1].double()
        slope, want = (a - b)[on].sum(), (d.double() * moved).sum(1)[on].sum()
        assert abs(slope - want) <= 0.02 * abs(want)
    # along the gradients themselves
    v = (d / d.square().mean().sqrt()).clamp(-3, 3)
    e = 2.0 ** -4
    agree(((x.double() + e * v).to(dtype), logits), ((x.double() - e * v).to(dtype), logits), xg.grad)
    d = lg.grad.double()
    v = (d / d.square().mean().sqrt()).clamp(-3, 3)
    chosen = torch.zeros_like(logits).scatter_(1, ids.long(), 1.0).double()
    e = 2.0 ** -5
    agree((x, (logits.double() + e * v * chosen).float()), (x, (logits.double() - e * v * chosen).float()), lg.grad)


def graph_of(run):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    return g, out


@pytest.mark.parametrize("T", [8, 400])
def test_in_a_graph(T):
    h, f, E, k, group, dtype = 128, 192, 8, 2, 64, torch.bfloat16
    x, logits, _, w = make(T, h, f, E, k, group, dtype, 4)
    dy = tokens(T, h, dtype, 5)
    g, out = graph_of(lambda: by_hand(x, logits, w, k, "silu", dy))
    for i in range(4):
        nx, nl, _, _ = make(T, h, f, E, k, group, dtype, 20 + i, masked=i % 2 == 1)
        x.copy_(nx), logits.copy_(nl)
        ref = [v.clone() for v in by_hand(x, logits, w, k, "silu", dy)]
        for v in out:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for v, want in zip(out, ref):
            assert torch.equal(v, want), i


def test_two_graphs_share_a_workspace():
    E, m, n, group = 4, 200, 328, 64
    w = pack(*make_layer(m, n, group, 1, lead=(E,)), group)
    sizes = (300, 1200)
    ws = B.workspace(max(B.q4_experts_workspace_bytes(R, w) for R in sizes) + B.moe_route_workspace_bytes(1200, E, 1), DEV)
    xs = [tokens(R, n, torch.bfloat16, R) for R in sizes]
    logits = [torch.randn((R, E), generator=torch.Generator().manual_seed(R)).to(DEV) for R in sizes]

    def step(i):
        r = B.moe_route(logits[i], 1, ws=ws)
        xs_ = B.moe_gather(xs[i], r["place"])
        return B.q4_experts(xs_, w, r["offsets"], ws=ws)
    graphs = [graph_of(lambda i=i: step(i)) for i in range(2)]
    for i in (0, 1, 1, 0, 1, 0):
        logits[i].copy_(logits[i].flip(0))
        want = step(i).clone()
        ws.fill_(255)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[i][1], want)


def test_on_another_stream():
    """Calls with stream=, on a stream that nothing orders after the current one,
    beside pending work on that."""
    T, h, f, E, k, group, dtype = 300, 128, 192, 8, 2, 64, torch.bfloat16
    x, logits, _, w = make(T, h, f, E, k, group, dtype, 4)
    dy = tokens(T, h, dtype, 5)
    r = B.moe_route(logits, k)
    at, place, weights = r["offsets"], r["place"], r["weights"]
    xs = B.moe_gather(x, place)
    a, b = B.q4_experts(xs, w[0], at), B.q4_experts(xs, w[1], at)
    hs, ca, cb = B.gated_act(a, b, checkpoint=True)
    calls = [lambda **s: tuple(B.moe_route(logits, k, **s).values()), lambda **s: B.moe_gather(x, place, **s),
             lambda **s: B.q4_experts(xs, w[0], at, **s), lambda **s: B.q4_experts_grad(a, w[0], at, **s),
             lambda **s: B.gated_act(a, b, **s), lambda **s: B.gated_act_grad(hs, ca, cb, **s),
             lambda **s: B.gated_act(a, b, checkpoint=True, **s), lambda **s: (B.ck8_pack(a, **s),),
             lambda **s: B.ck8_unpack(ca, **s), lambda **s: B.moe_combine(xs, place, weights, **s),
             lambda **s: tuple(B.moe_combine_grad(dy, a[:, :h], place, weights, **s).values()),
             lambda **s: B.moe_route_grad(weights, weights, r["ids"], E, **s)]
    for i, call in enumerate(calls):
        want = call()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        torch.cuda._sleep(20_000_000)
        got = call(stream=side)
        side.synchronize()
        for g_, w_ in zip(*(v if isinstance(v, tuple) else (v,) for v in (got, want))):
            if isinstance(g_, B.Checkpoint8):
                g_, w_ = B.ck8_unpack(g_), B.ck8_unpack(w_)
            assert torch.equal(g_, w_), i


def test_a_backward_pass_with_large_numbers_of_choices():
    T, h, f, E, k, group, dtype = 70, 64, 64, 20, 16, 64, torch.float16
    x, logits, _, w = make(T, h, f, E, k, group, dtype, 2)
    dy = tokens(T, h, dtype, 5)
    xg, lg = x.clone().requires_grad_(), logits.clone().requires_grad_()
    B.q4_moe_layer(xg, lg, *w, k).backward(dy)
    _, dx, dl = by_hand(x, logits, w, k, "silu", dy)
    assert torch.equal(xg.grad, dx) and torch.equal(lg.grad, dl)


def test_no_tokens():
    x, logits, _, w = make(5, 64, 128, 4, 2, 64, torch.bfloat16, 1)
    assert B.q4_moe_layer(x[:0], logits[:0], *w, 2).shape == (0, 64)
    xg = x[:0].clone().requires_grad_()
    B.q4_moe_layer(xg, logits[:0], *w, 2).sum().backward()
    assert xg.grad.shape == (0, 64)
