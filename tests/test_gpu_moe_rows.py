"""Rows into the experts' order and back (moe_gather, moe_combine and their
gradients) against their formulas.

Tolerances.  gather moves values: equal bits.  combine is a float32 sum of up to
32 products, a rounding each: 32 * 2^-24 of the sum of the terms' magnitudes, and
half a step of the result's type.  dys is one product, rounded to float32 and to
the type.  dweights sums n products of 16-bit values (exact in float32 but for the
addition): a lane n / 64 of them at most, then 6 + 4 steps over lanes and waves:
(n / 64 + 18) 2^-24 of the sum of the magnitudes."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def values(rows, cols, dtype, seed, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, cols + pad), generator=g).to(dtype).to(DEV)[:, shift:shift + cols]


def places(T, k, rows, seed, some=True):
    """Distinct rows; some choices without one (-1 and numbers outside)."""
    g = torch.Generator().manual_seed(seed)
    p = torch.randperm(rows, generator=g)[:T * k].reshape(T, k).to(torch.int32)
    if some:
        out = torch.tensor([-1, -1, rows, -(2 ** 31), 2 ** 31 - 1], dtype=torch.int32)
        hit = torch.rand((T, k), generator=g) < 0.2
        p = torch.where(hit, out[torch.randint(0, 5, (T, k), generator=g)], p)
    return p.to(DEV)


def used(place, rows):
    """(token, choice, row) of the choices that have a row."""
    t, j = torch.nonzero((place >= 0) & (place < rows), as_tuple=True)
    return t, j, place[t, j].long()


SHAPES = [(1, 1, 1), (1, 8, 16384), (3, 2, 7), (16, 6, 2048), (37, 5, 1003), (64, 3, 64), (65, 16, 513), (130, 1, 4100),
          (20, 32, 300), (5000, 2, 24), (4200, 2, 520), (7, 4, 65536)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,k,n", SHAPES)
def test_rows_there_and_back(T, k, n, dtype):
    rows, pad = T * k + 3, 5 if n % 2 else 0
    place = places(T, k, rows, T)
    t, j, p = used(place, rows)
    x, ys = values(T, n, dtype, 1, pad, 3 if pad else 0), values(rows, n, dtype, 2, pad, 1 if pad else 0)
    weights = torch.rand((T, k), generator=torch.Generator().manual_seed(3)).to(DEV)
    weights[0, 0] = 0.0
    # there
    wide = torch.full((rows, n + 4), 3.0, dtype=dtype, device=DEV)
    ref = torch.full((rows, n), 3.0, dtype=dtype, device=DEV)
    ref[p] = x[t]
    assert B.moe_gather(x, place, out=wide[:, 2:2 + n]).data_ptr() == wide[:, 2:].data_ptr()
    assert torch.equal(wide[:, 2:2 + n], ref) and (wide[:, :2] == 3).all() and (wide[:, 2 + n:] == 3).all()
    # back; rows that no choice has may hold anything
    lost = torch.ones(rows, dtype=torch.bool, device=DEV)
    lost[p] = False
    ys = ys.clone() if not pad else ys
    ys[lost] = float("nan")
    for w in (weights, None):
        term = ys[p].double() * (1.0 if w is None else w[t, j].double()[:, None])
        want = torch.zeros((T, n), dtype=torch.float64, device=DEV).index_add_(0, t, term)
        size = torch.zeros((T, n), dtype=torch.float64, device=DEV).index_add_(0, t, term.abs())
        got = B.moe_combine(ys, place, w)
        assert got.dtype == dtype and got.shape == (T, n)
        tol = 32 * 2.0 ** -24 * size + U[dtype] * want.abs() * 1.001 + TINY[dtype]
        assert ((got.double() - want).abs() <= tol).all()
        assert torch.equal(got, B.moe_combine(ys, place, w))
    # and the gradients
    dy = values(T, n, dtype, 4)
    dys = torch.full((rows, n), 5.0, dtype=dtype, device=DEV)
    r = B.moe_combine_grad(dy, ys, place, weights, out={"dys": dys, "dweights": torch.empty_like(weights)})
    want = weights[t, j].double()[:, None] * dy[t].double()
    assert ((dys[p].double() - want).abs() <= U[dtype] * want.abs() * 1.001 + TINY[dtype]).all()
    assert (dys[lost] == 5).all()
    prod = dy[t].double() * ys[p].double()
    want, tol = torch.zeros((T, k), dtype=torch.float64, device=DEV), torch.zeros((T, k), dtype=torch.float64, device=DEV)
    want[t, j], tol[t, j] = prod.sum(1), prod.abs().sum(1) * (n / 64 + 18) * 2.0 ** -24
    assert ((r["dweights"].double() - want).abs() <= tol).all()
    again = B.moe_combine_grad(dy, ys, place, weights, out={"dys": torch.full_like(dys, 5.0), "dweights": torch.empty_like(weights)})
    assert torch.equal(again["dys"], dys) and torch.equal(again["dweights"], r["dweights"])


def test_nothing_there():
    place, weights = torch.full((4, 2), -1, dtype=torch.int32, device=DEV), torch.ones((4, 2), device=DEV)
    dtype = torch.bfloat16
    x, none = values(4, 100, dtype, 1), torch.empty((0, 100), dtype=dtype, device=DEV)
    full = torch.full((9, 100), float("nan"), dtype=dtype, device=DEV)
    for ys in (none, full):
        assert (B.moe_combine(ys, place, weights) == 0).all() and (B.moe_combine(ys, place) == 0).all()
        assert B.moe_gather(x, place, out=ys.clone()).shape == ys.shape
        r = B.moe_combine_grad(x, ys, place, weights)
        assert (r["dweights"] == 0).all()
        assert torch.isnan(B.moe_combine_grad(x, ys, place, weights, out={"dys": ys.clone(), "dweights": weights.clone()})["dys"]).all()
    some = torch.zeros((4, 2), dtype=torch.int32, device=DEV)     # rows that do not exist
    assert (B.moe_combine(none, some, weights) == 0).all()
    empty = torch.empty((4, 0), dtype=dtype, device=DEV)
    assert B.moe_combine(empty[:0], place).shape == (4, 0)
    r = B.moe_combine_grad(empty, empty, place, weights)
    assert (r["dweights"] == 0).all() and r["dys"].shape == (4, 0)
    assert B.moe_gather(x[:0], place[:0]).shape == (0, 100)


def test_a_row_beyond_two_to_the_31_elements():
    rows, n = 34000, 65536                                        # 2.2e9 values
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * 2 * rows * n:
        pytest.skip("not enough memory")
    ys = torch.empty((rows, n), dtype=torch.bfloat16, device=DEV)
    ys[-2:] = values(2, n, torch.bfloat16, 1)
    place = torch.tensor([[rows - 1], [rows - 2]], dtype=torch.int32, device=DEV)
    y = B.moe_combine(ys, place)
    assert torch.equal(y[0], ys[-1]) and torch.equal(y[1], ys[-2])
    x = values(2, n, torch.bfloat16, 2)
    B.moe_gather(x, place, out=ys)
    assert torch.equal(ys[-1], x[0]) and torch.equal(ys[-2], x[1])


def test_autograd():
    T, k, n, dtype = 50, 3, 200, torch.bfloat16
    rows = T * k
    place = places(T, k, rows, 7)
    t, j, p = used(place, rows)
    x = values(T, n, dtype, 1).requires_grad_()
    g = values(rows, n, dtype, 2)
    xs = B.moe_gather(x, place)
    gx, = torch.autograd.grad(xs, x, g.clone().requires_grad_(), create_graph=True)
    assert torch.equal(gx, B.moe_combine(g, place))
    # the gradient of that: moe_gather, and zeros in the other rows
    v = g.clone().requires_grad_()
    gx, = torch.autograd.grad(B.moe_gather(x, place), x, v, create_graph=True)
    u = values(T, n, dtype, 3)
    gv, = torch.autograd.grad(gx, v, u)
    zeros = torch.zeros((rows, n), dtype=dtype, device=DEV)
    assert torch.equal(gv, B.moe_gather(u, place, out=zeros.clone()))
    # back
    ys, w = g.clone().requires_grad_(), torch.rand((T, k), generator=torch.Generator().manual_seed(3)).to(DEV).requires_grad_()
    B.moe_combine(ys, place, w).backward(u)
    r = B.moe_combine_grad(u, g, place, w.detach(), out={"dys": zeros.clone(), "dweights": torch.empty((T, k), device=DEV)})
    assert torch.equal(ys.grad, r["dys"]) and torch.equal(w.grad, r["dweights"])
    ys.grad = None
    B.moe_combine(ys, place).sum().backward()                     # an expanded gradient
    ones = torch.zeros((rows, n), dtype=dtype, device=DEV)
    ones[p] = 1.0
    assert torch.equal(ys.grad, ones)
    with pytest.raises(RuntimeError):
        a, = torch.autograd.grad(B.moe_combine(ys, place, w), ys, u.clone().requires_grad_(), create_graph=True)
    for call in (lambda: B.moe_gather(x, place, out=g), lambda: B.moe_combine(ys, place, w, out=u)):
        with pytest.raises(ValueError, match="out"):
            call()


def test_gradients_by_differences():
    """combine is linear in rows and in weights: its difference quotient with
    values that bfloat16 holds exactly is the derivative, but for the rounding of
    the sums to that type (2^-8 of the two results)."""
    T, k, n = 40, 3, 64
    place = places(T, k, T * k, 11)
    ys, d, dy = (values(T * k, n, torch.bfloat16, i) if i < 3 else values(T, n, torch.bfloat16, i) for i in (1, 2, 3))
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(3)).to(DEV)
    r = B.moe_combine_grad(dy, ys, place, w, out={"dys": torch.zeros_like(ys), "dweights": torch.empty_like(w)})
    h = 2.0
    a, b = B.moe_combine(h * d, place, w).double(), B.moe_combine(-h * d, place, w).double()
    slope, want = ((a - b) / (2 * h) * dy.double()).sum(), (r["dys"].double() * d.double()).sum()
    size = ((a.abs() + b.abs()) / (2 * h) * dy.double().abs()).sum() + (r["dys"].double() * d.double()).abs().sum()
    assert abs(slope - want) <= 2.0 ** -8 * size
    v = torch.rand((T, k), generator=torch.Generator().manual_seed(4)).to(DEV)
    a, b = B.moe_combine(ys, place, w + v).double(), B.moe_combine(ys, place, w - v).double()
    slope, want = ((a - b) / 2 * dy.double()).sum(), (r["dweights"].double() * v.double()).sum()
    assert abs(slope - want) <= 2.0 ** -8 * ((a.abs() + b.abs()) / 2 * dy.double().abs()).sum()
