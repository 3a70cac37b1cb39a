"""The choice of experts and its gradient (moe_route, moe_route_grad) against
their definition.

Tolerances.  A share is exp(l - top) / sum in float32.  The difference is rounded
once (2^-24 of |l - top|, which is that relative error of the exponential), the
exponential is good to 2 units in the last place, the sum of up to 16 terms to 16
roundings and the quotient to one: |l - top| 2^-24 + 22 * 2^-24, less than
(|l - top| + 22) 2^-24 relative, and 2^-126 where float32 ends.
The gradient w (g - S), S = sum w g, has 18 roundings of terms up to sum |w g| in
S, one of the difference and one of the product: w 2^-24 (20 sum |w g| + 2 |g|),
and the one of the result to its type, half a step."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def reference(logits, k):
    """ids, weights and each weight's |l - top|, place, order, offsets, one token at a time."""
    l = logits.double().cpu().numpy()
    T, E = l.shape
    key = np.where(np.isnan(l), -np.inf, l)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(key, order, 1)
    live = top > -np.inf
    ids = np.where(live, order, -1)
    d = np.where(live, 0.0, -np.inf)
    with np.errstate(invalid="ignore"):
        d = np.where(live & (top != top[:, :1]), top - top[:, :1], d)
    e = np.exp(d)
    weights = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    pairs = [[] for _ in range(E)]
    for p, i in enumerate(ids.reshape(-1)):
        if i >= 0:
            pairs[i].append(p)
    offsets = np.concatenate(([0], np.cumsum([len(p) for p in pairs])))
    rows = np.full(T * k, -1, dtype=np.int64)
    used = [p for ps in pairs for p in ps]
    rows[:len(used)] = used
    place = np.full(T * k, -1, dtype=np.int64)
    place[used] = np.arange(len(used))
    return ids, weights, np.where(live, np.maximum(d, -1e4), 0.0), place.reshape(T, k), rows, offsets


def check(r, logits, k):
    ids, weights, d, place, order, offsets = reference(logits, k)
    for name, ref in (("ids", ids), ("place", place), ("order", order), ("offsets", offsets)):
        assert r[name].dtype == torch.int32 and np.array_equal(r[name].cpu().numpy(), ref), name
    got = r["weights"].double().cpu().numpy()
    tol = weights * (np.abs(d) + 22) * 2.0 ** -24 + 2.0 ** -126
    assert r["weights"].dtype == torch.float32 and (np.abs(got - weights) <= tol).all()


def make(T, E, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    l = 2.0 * torch.randn((T, E), generator=g)
    if kind == "ties":
        l = l.round() * torch.where(torch.rand((T, E), generator=g) < 0.5, -1.0, 1.0)    # both zeros among them
    elif kind == "masked":
        l[torch.rand((T, E), generator=g) < 0.4] = -np.inf
        l[torch.rand((T, E), generator=g) < 0.1] = np.nan
        l[torch.rand((T, E), generator=g) < 0.02] = np.inf
        l[torch.rand((T, E), generator=g) < 0.1] = torch.finfo(dtype).min
        l[torch.rand((T,), generator=g) < 0.2] = -np.inf
        l[torch.rand((T,), generator=g) < 0.1] = torch.finfo(dtype).min
    return l.to(dtype).to(DEV)


# one workgroup of one to four passes, several of one and more passes; every
# number of logits a lane holds
SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 64, 6), (63, 16, 16), (65, 17, 3), (129, 33, 8), (256, 256, 16), (257, 256, 8),
          (300, 100, 1), (1000, 130, 4), (4097, 128, 8), (9000, 64, 6), (20001, 4, 2)]


@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route_matches_its_definition(T, E, k, kind):
    for i, dtype in enumerate(TYPES):
        logits = make(T, E, dtype, 100 * T + E + i, kind)
        check(B.moe_route(logits, k), logits, k)


def test_nothing_to_choose():
    for T in (1, 70, 300):
        logits = torch.full((T, 9), -np.inf, device=DEV)
        r = B.moe_route(logits, 3)
        check(r, logits, 3)
        assert (r["ids"] == -1).all() and (r["weights"] == 0).all() and (r["offsets"] == 0).all()
        d = B.moe_route_grad(torch.full((T, 3), np.nan, device=DEV), r["weights"], r["ids"], 9)
        assert (d == 0).all()
    r = B.moe_route(torch.empty((0, 9), device=DEV), 3)
    assert r["ids"].shape == (0, 3) and (r["offsets"] == 0).all()
    assert B.moe_route_grad(r["weights"], r["weights"], r["ids"], 9).shape == (0, 9)


def test_all_tokens_choose_one_expert():
    for T in (200, 5000):
        logits = torch.zeros((T, 40), device=DEV)
        logits[:, 17] = 1.0
        check(B.moe_route(logits, 1), logits, 1)
        check(B.moe_route(logits, 3), logits, 3)


@pytest.mark.parametrize("dtype", TYPES)
def test_slices_given_outputs_and_the_same_bits_again(dtype):
    T, E, k = 700, 23, 5
    wide = make(T, E + 6, dtype, 5, "ties")
    logits = wide[:, 3:3 + E]
    out = {"ids": torch.empty((T, k), dtype=torch.int32, device=DEV), "weights": torch.empty((T, k), device=DEV),
           "place": torch.empty((T, k), dtype=torch.int32, device=DEV), "order": torch.empty(T * k, dtype=torch.int32, device=DEV),
           "offsets": torch.empty(E + 1, dtype=torch.int32, device=DEV)}
    ws = B.workspace(B.moe_route_workspace_bytes(T, E, k), DEV)
    assert B.moe_route(logits, k, out=out, ws=ws) is out
    check(out, logits, k)
    again = B.moe_route(logits, k)
    assert all(torch.equal(out[name], again[name]) for name in out)


@pytest.mark.parametrize("kind", ["normal", "masked"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (300, 256, 16), (1000, 31, 5), (70000, 4, 1)])
def test_gradient_matches_its_formula(T, E, k, kind):
    for i, dtype in enumerate(TYPES):
        logits = make(T, E, dtype, T + i, kind)
        r = B.moe_route(logits, k)
        g = torch.randn((T, k), generator=torch.Generator().manual_seed(i)).to(DEV)
        wide = torch.full((T, E + 3), 7.0, dtype=dtype, device=DEV)
        got = B.moe_route_grad(g, r["weights"], r["ids"], E, out=wide[:, 1:1 + E])
        assert (wide[:, 0] == 7).all() and (wide[:, 1 + E:] == 7).all()
        w, v, ids = r["weights"].double(), g.double(), r["ids"].long()
        live = ids >= 0
        wv = torch.where(live, w * v, 0.0)
        d = torch.where(live, w * (v - wv.sum(1, keepdim=True)), 0.0)
        loose = torch.where(live, w * 2.0 ** -24 * (20 * wv.abs().sum(1, keepdim=True) + 2 * v.abs()), 0.0)
        full = torch.zeros((T, E + 1), dtype=torch.float64, device=DEV)
        tol = full.clone()
        at = torch.where(live, ids, E)
        full.scatter_(1, at, d), tol.scatter_(1, at, loose)
        full, tol = full[:, :E], tol[:, :E]
        assert ((got.double() - full).abs() <= tol * 1.01 + U[dtype] * full.abs() + TINY[dtype]).all()


def test_autograd_and_differences():
    T, E, k = 300, 20, 4
    logits = make(T, E, torch.float32, 9).requires_grad_()
    r = B.moe_route(logits, k)
    assert r["weights"].requires_grad and not r["ids"].requires_grad
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).to(DEV)
    r["weights"].backward(g)
    assert torch.equal(logits.grad, B.moe_route_grad(g, r["weights"].detach(), r["ids"], E))
    # along a direction small enough to leave the choice as it is: third
    # derivatives of a share are at most 1, so (2^-7)^2 |v|^3 |g| / 6 over the
    # token's chosen logits, and a share's float32 (2^-19) over 2^-7
    v = torch.randn((T, E), generator=torch.Generator().manual_seed(2)).to(DEV).clamp_(-2, 2)
    h = 2.0 ** -7
    l = logits.detach()
    up, down = B.moe_route(l + h * v, k), B.moe_route(l - h * v, k)
    same = (up["ids"] == r["ids"]).all(1) & (down["ids"] == r["ids"]).all(1)
    assert same.sum() > T // 2
    slope = ((up["weights"].double() - down["weights"].double()) * g.double()).sum(1) / (2 * h)
    want = (logits.grad.double() * v.double()).sum(1)
    tol = (h * h * 8 * 16 / 6 + 2.0 ** -19 / h) * g.double().abs().sum(1)
    assert ((slope - want).abs() <= tol)[same].all()
    with pytest.raises(ValueError, match="out"):
        B.moe_route(logits, k, out=r)
    with torch.no_grad():
        assert not B.moe_route(logits, k)["weights"].requires_grad
