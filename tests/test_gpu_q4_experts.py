"""The experts' products on 4-bit stacks (q4_experts, q4_experts_grad) against
their formulas in float64.

Tolerances.  A product's is that of the linear layer (test_gpu_q4.py), whose sums
these are.  A gradient rounds each weight once, by u |w| at most: its error is a
sum of dy_i d_i with |d_i| <= u |w_i|, and the signs of dy are random, so that it
exceeds six times u (sum (dy_i w_i)^2)^(1/2) with a probability below 2 exp(-18) were
every d_i the largest possible (Hoeffding), 2 exp(-54) at their mean square.  That
root is an entry's own: with few terms, of steps that differ, it can be several
times the token's rms.  Sums and the result's rounding add what they add to a
product."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from moe_forms import experts_form, experts_grad_form, tail
from test_gpu_q4 import DEV, LINEAR, TINY, U, close, make_layer, pack, rms, tokens, weights64

pytestmark = pytest.mark.gpu


def close_grad(got, ref, squares, dtype):
    """squares: sum of (dy_i w_i)^2 of each entry."""
    got = got.double().cpu().numpy()
    tol = U[dtype] * (1 + 2.0 ** -6) * np.abs(ref) + 6 * U[dtype] * np.sqrt(squares) + LINEAR * rms(ref) + TINY[dtype]
    assert got.shape == ref.shape and (np.abs(got - ref) <= tol).all()


def spread(R, E, seed, first=0, tail=0):
    """Offsets of E experts over rows first .. R - tail: uneven, some without rows."""
    rng = np.random.default_rng(seed)
    share = rng.exponential(size=E) * (rng.random(E) < 0.8)
    if not share.any():
        share[rng.integers(E)] = 1.0
    n = R - first - tail
    cuts = np.round(np.concatenate(([0.0], np.cumsum(share))) / share.sum() * n).astype(np.int64) + first
    return cuts


def formula(x, offsets, ref, grad):
    """Each row's result in float64 (zeros in rows without an expert)."""
    x = x.double().cpu().numpy()
    y = np.zeros((x.shape[0], ref.shape[2] if grad else ref.shape[1]))
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            y[a:b] = x[a:b] @ (ref[e] if grad else ref[e].T)
    return y


def check(R, E, m, n, group, dtype, grad, seed, offsets=None, pad=0, out_pad=0):
    stack = make_layer(m, n, group, seed, lead=(E,))
    w, ref = pack(*stack, group), weights64(*stack, group)
    offsets = spread(R, E, seed) if offsets is None else np.asarray(offsets)
    cin, cout = (m, n) if grad else (n, m)
    x = tokens(R, cin, dtype, seed, pad=pad, shift=1 if pad else 0)
    call, size = ((B.q4_experts_grad, B.q4_experts_grad_workspace_bytes) if grad else
                  (B.q4_experts, B.q4_experts_workspace_bytes))
    at = torch.from_numpy(offsets.astype(np.int32)).to(DEV)
    first, last = offsets[0], offsets[-1]
    x = x.clone() if not pad else x
    x[:first], x[last:] = float("nan"), float("inf")
    wide = torch.full((R, cout + out_pad), 3.0, dtype=dtype, device=DEV)
    out = wide[:, :cout]
    ws = B.workspace(size(R, w), DEV)
    ws.fill_(255)                                                 # NaN, read as floats
    assert call(x, w, at, out=out, ws=ws) is out
    want = formula(x, offsets, ref, grad)[first:last]
    if grad:
        close_grad(out[first:last], want, formula(x.double().square(), offsets, ref * ref, grad)[first:last], dtype)
    else:
        close(out[first:last], want, dtype, LINEAR)
    assert (out[:first] == 3).all() and (out[last:] == 3).all() and (wide[:, cout:] == 3).all()
    assert torch.equal(call(x, w, at)[first:last], out[first:last])
    return out


TYPES = [torch.bfloat16, torch.float16]
# rows, experts, m, n, group: one row to many per expert, each kernel form
SHAPES = [(1, 1, 1, 1, 0), (1, 8, 130, 300, 64), (6, 64, 33, 515, 192), (16, 5, 100, 64, 0), (96, 3, 64, 130, 64),
          (287, 256, 280, 70, 64), (15, 16, 2244, 72, 0), (150, 2, 100, 1000, 128), (4521, 40, 278, 70, 64), (4485, 40, 259, 128, 0),
          (2497, 40, 34, 1180, 128), (2353, 16, 33, 1472, 0), (6000, 16, 4000, 66, 64), (8000, 16, 4096, 64, 0), (63, 1, 36, 43, 0),
          (50, 1, 70, 64, 64), (58, 1, 70, 927, 128), (49, 1, 70, 768, 64), (700, 9, 260, 640, 0)]
GRADS = [(1, 1, 1, 1, 0), (3, 8, 130, 300, 64), (6, 64, 515, 33, 0), (96, 3, 64, 130, 64), (300, 256, 65, 265, 64), (17, 4, 31, 40, 0),
         (40, 2, 1100, 300, 128), (9, 3, 5000, 70, 64), (200, 8, 2090, 400, 0), (90, 40, 300, 700, 192), (33, 1, 700, 129, 256),
         (4980, 40, 30, 581, 192), (5260, 40, 337, 8, 64), (70, 1, 264, 100, 64), (7801, 3, 49, 483, 192), (2189, 8, 66, 3491, 0), (4000, 16, 300, 2500, 128),
         (1558, 24, 64, 2262, 64), (616, 3, 717, 96, 64), (1200, 3, 1030, 1300, 64), (8004, 24, 40, 1755, 64), (6734, 16, 64, 2242, 0),
         (5559, 3, 14462, 129, 0), (92, 3, 560, 95, 192), (107, 3, 412, 376, 192), (524, 16, 428, 127, 64), (4096, 2, 14336, 130, 128)]


def test_the_shapes_reach_every_form():
    forms = [experts_form(*s[:4]) + (s[3] % 64 == 0,) for s in SHAPES]
    assert {f[1] for f in forms if f[0] == "few"} == {2, 4, 8}
    forms = {(f[0], f[1] > 1, *f[2:]) for f in forms if f[0] != "few"}   # rows, shared out, own sums, aligned
    assert forms >= {(256, False, False, a) for a in (True, False)}
    assert forms >= {(128, shared, False, a) for shared in (True, False) for a in (True, False)}
    assert forms >= {(64, shared, a, a) for shared in (True, False) for a in (True, False)}
    assert {(f, s > 1) for f, s in (experts_grad_form(*s) for s in GRADS)} == {(f, s) for f in ("few", 256, 128) for s in (True, False)}
    # few rows: blocks of up to 16 and 32 of them, grids that end inside a block of columns
    # or do not, an even and an odd number of row tiles, and a last step that is cut
    few = [s for s in GRADS if experts_grad_form(*s)[0] == "few"]
    assert {s[4] // 64 % 2 for s in few} == {0, 1} and {-(-s[2] // 16) % 2 for s in few} == {0, 1} and {s[2] % 32 > 0 for s in few} == {True, False}
    rest = {min((c - 1) % 32 // 16, 1) for R, E, m, n, g in few if g // 64 % 2 == 0 for c in np.diff(spread(R, E, R + n)) if c}
    assert rest == {0, 1}
    # blocks of every number of rows, behind whole ones and alone
    for shapes, most in ((SHAPES, 256), (SHAPES, 128), (SHAPES, 64), (GRADS, 256), (GRADS, 128)):
        rest = set()
        for R, E, m, n, g in shapes:
            if (experts_grad_form(R, E, m, n, g) if shapes is GRADS else experts_form(R, E, m, n))[0] == most:
                c = np.diff(spread(R, E, R + n))
                rest |= {(1 if r <= 64 else 2 if r <= 128 else 4, x >= most) for x in c for r in [x % most] if r}
        assert rest == {(b, more) for b in (1, 2, 4) if 32 * b < most for more in (True, False)}, most


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,E,m,n,group", SHAPES)
def test_products_match_their_formula(R, E, m, n, group, dtype):
    check(R, E, m, n, group, dtype, False, R + n)


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,E,m,n,group", GRADS)
def test_gradients_match_their_formula(R, E, m, n, group, dtype):
    check(R, E, m, n, group, dtype, True, R + n)


@pytest.mark.parametrize("grad", [False, True], ids=["product", "grad"])
@pytest.mark.parametrize("R,E,m,n,group,pad", [(40, 4, 100, 130, 64, 0), (40, 4, 100, 130, 64, 3), (900, 4, 200, 192, 64, 0),
                                               (900, 4, 200, 192, 64, 8), (900, 4, 200, 193, 0, 5), (150, 2, 320, 1000, 128, 1),
                                               (1500, 4, 1280, 1000, 64, 8), (1500, 4, 1300, 1000, 64, 1)])
def test_rows_outside_the_experts_and_slices(R, E, m, n, group, pad, grad):
    for dtype in TYPES:
        check(R, E, m, n, group, dtype, grad, 7, spread(R, E, 3, first=5, tail=11), pad=pad, out_pad=pad)
        check(R, E, m, n, group, dtype, grad, 8, spread(R, E, 4, tail=R // 2), pad=pad)


@pytest.mark.parametrize("grad", [False, True], ids=["product", "grad"])
def test_one_expert_has_all_rows(grad):
    for R, E, m, n in ((100, 256, 40, 70), (600, 30, 40, 70), (3000, 64, 70, 130)):
        for e in (0, 3, 17, E - 1):
            offsets = np.zeros(E + 1, dtype=np.int64)
            offsets[e + 1:] = R
            check(R, E, m, n, 64, torch.bfloat16, grad, e, offsets)


def test_more_blocks_of_rows_than_65535():
    R, E, m, n = 2_200_000, 2, 8, 8
    assert experts_grad_form(R, E, m, n, 0)[0] == "few" and R // 32 > 65535
    for grad in (False, True):
        check(R, E, m, n, 0, torch.bfloat16, grad, 1, np.array([0, 1_500_001, R]))


# experts' rows, columns of the result, depth: whole rounds of 256 tiles, and a rest of
# tiles for 256, 128, and 64 rows; less than a round, which is not worth sharing out
TAILS = [((2200,), 8300, 3500, {256}), ((0, 1900), 8300, 3520, {128}), ((1796, 0), 9300, 3550, {256, 64}), ((7000,), 1700, 3500, {256, 128})]


@pytest.mark.parametrize("grad", [False, True], ids=["product", "grad"])
@pytest.mark.parametrize("case", range(4))
def test_the_last_tiles_are_shared_out(case, grad):
    counts, cols, depth, bodies = TAILS[case]
    m, n = (depth, cols) if grad else (cols, depth)
    R, E = sum(counts) + 3, len(counts)
    assert (experts_grad_form(R, E, m, n, 64) if grad else experts_form(R, E, m, n))[:2] == (256, "tail")
    whole, left, parts, found = tail(counts, cols, (130.0 if grad else 128.0) * depth / 4096,
                                     min(16, -(-depth // 64) // 2) if grad else min(8, -(-depth // 128) // 2))
    assert found == bodies and left and (whole > 0 and parts > 1 if case < 3 else whole == 0 and parts == 1)
    check(R, E, m, n, 64, TYPES[case % 2], grad, case, np.concatenate(([0], np.cumsum(counts))))
    w = pack(*make_layer(m, n, 64, 1, lead=(E,)), 64)
    call = B.q4_experts_grad if grad else B.q4_experts
    x, out = torch.ones((R, depth), dtype=TYPES[0], device=DEV), torch.full((R, cols), 3.0, dtype=TYPES[0], device=DEV)
    call(x, w, torch.zeros(E + 1, dtype=torch.int32, device=DEV), out=out)
    assert (out == 3).all()
    big = torch.tensor([R, 0, 2 ** 31 - 1], dtype=torch.int32, device=DEV)[-E - 1:]   # no offsets: within the rows all the same
    wide = torch.full((R + 2, cols), 3.0, dtype=TYPES[0], device=DEV)
    call(x, w, big, out=wide[1:-1])
    assert (wide[0] == 3).all() and (wide[-1] == 3).all()


@pytest.mark.parametrize("grad", [False, True], ids=["product", "grad"])
@pytest.mark.parametrize("R,E", [(50, 8), (2000, 8)])
def test_no_rows_at_all(R, E, grad):
    for at in (0, R):
        check(R, E, 70, 130, 64, torch.float16, grad, 1, np.full(E + 1, at))
    m, n = 70, 130
    w = pack(*make_layer(m, n, 64, 1, lead=(E,)), 64)
    call = B.q4_experts_grad if grad else B.q4_experts
    x = torch.empty((0, m if grad else n), dtype=torch.bfloat16, device=DEV)
    assert call(x, w, torch.zeros(E + 1, dtype=torch.int32, device=DEV)).shape == (0, n if grad else m)


@pytest.mark.parametrize("grad", [False, True], ids=["product", "grad"])
@pytest.mark.parametrize("R", [50, 2000])
def test_offsets_that_are_no_offsets_stay_within_the_rows(R, grad):
    """What is written is not specified; that it lies in the given rows is."""
    E, m, n = 8, 70, 130
    w = pack(*make_layer(m, n, 64, 1, lead=(E,)), 64)
    cin, cout = (m, n) if grad else (n, m)
    x = tokens(R, cin, torch.bfloat16, 1)
    big = 2 ** 31 - 1
    for offsets in ([0, R, 0, R, 0, R, 0, R, 0], [-5, -3, 2, 9, 1, big, big, -big, 40], [big] * 9, [-big] * 9, list(range(9, 0, -1)),
                    [0, 10 * R, 20 * R, 30 * R, 40 * R, 50 * R, 60 * R, 70 * R, 80 * R]):
        room = torch.full((R + 200, cout), 3.0, dtype=torch.bfloat16, device=DEV)
        at = torch.tensor(offsets, dtype=torch.int64).clamp(-big, big).to(torch.int32).to(DEV)
        (B.q4_experts_grad if grad else B.q4_experts)(x, w, at, out=room[100:100 + R])
        assert (room[:100] == 3).all() and (room[100 + R:] == 3).all()


def test_empty_layers():
    offsets = np.array([1, 4, 4, 9])
    at = torch.from_numpy(offsets.astype(np.int32)).to(DEV)
    for m, n in ((0, 130), (70, 0)):
        w = B.Q4Weight(torch.empty(0, dtype=torch.uint8, device=DEV), 3, m, n, 64)
        for call, cin, cout in ((B.q4_experts, n, m), (B.q4_experts_grad, m, n)):
            out = torch.full((12, cout), 3.0, dtype=torch.bfloat16, device=DEV)
            call(torch.ones((12, cin), dtype=torch.bfloat16, device=DEV), w, at, out=out)
            assert (out[1:9] == 0).all() and (out[:1] == 3).all() and (out[9:] == 3).all()


def test_a_row_with_infinities_and_nan_touches_no_other():
    for R, E in ((40, 4), (900, 4)):
        for grad in (False, True):
            m, n, dtype = 130, 200, torch.bfloat16
            w = pack(*make_layer(m, n, 64, 2, lead=(E,)), 64)
            x = tokens(R, m if grad else n, dtype, 3)
            at = torch.from_numpy(spread(R, E, 5).astype(np.int32)).to(DEV)
            call = B.q4_experts_grad if grad else B.q4_experts
            ref = call(x, w, at)
            x[7, 3], x[21, 70] = float("nan"), float("inf")
            got = call(x, w, at)
            keep = torch.ones(R, dtype=torch.bool, device=DEV)
            keep[[7, 21]] = False
            assert torch.equal(got[keep], ref[keep]) and not torch.isfinite(got[[7, 21]]).any()


def test_an_expert_alone_equals_the_linear_layer():
    m, n, group, E = 300, 520, 128, 3
    w = pack(*make_layer(m, n, group, 9, lead=(E,)), group)
    for R in (20, 400):
        x, dy = tokens(R, n, torch.bfloat16, 1), tokens(R, m, torch.bfloat16, 2)
        at = torch.tensor([0, 0, R, R], dtype=torch.int32, device=DEV)
        ref = weights64(*make_layer(m, n, group, 9, lead=(E,)), group)[1]
        # two results of one formula: each within its tolerance of it
        want = x.double().cpu().numpy() @ ref.T
        close(B.q4_experts(x, w, at), want, torch.bfloat16, LINEAR)
        close(B.q4_linear(x, w[1]), want, torch.bfloat16, LINEAR)
        want, squares = dy.double().cpu().numpy() @ ref, dy.double().square().cpu().numpy() @ (ref * ref)
        close_grad(B.q4_experts_grad(dy, w, at), want, squares, torch.bfloat16)
        close_grad(B.q4_linear_grad(dy, w[1]), want, squares, torch.bfloat16)


def test_autograd():
    R, E, m, n, dtype = 130, 5, 200, 330, torch.bfloat16
    w = pack(*make_layer(m, n, 64, 21, lead=(E,)), 64)
    offsets = spread(R, E, 6, tail=9)
    at, last = torch.from_numpy(offsets.astype(np.int32)).to(DEV), int(offsets[-1])
    for call, back, cin, cout in ((B.q4_experts, B.q4_experts_grad, n, m), (B.q4_experts_grad, B.q4_experts, m, n)):
        plain = tokens(R, cin, dtype, 1, pad=5)
        x = plain.detach().requires_grad_()
        g = tokens(R, cout, dtype, 2)
        y = call(x, w, at)
        assert y.requires_grad and torch.equal(y[:last], call(plain, w, at)[:last])
        y.backward(g)
        zeros = torch.zeros((R, cin), dtype=dtype, device=DEV)
        assert torch.equal(x.grad, back(g, w, at, out=zeros.clone())) and (x.grad[last:] == 0).all()
        v = g.clone().requires_grad_()
        dx, = torch.autograd.grad(call(x, w, at), x, v, create_graph=True)
        dv, = torch.autograd.grad(dx, v, plain)
        assert torch.equal(dv[:last], call(plain, w, at)[:last]) and (dv[last:] == 0).all()
        with pytest.raises(ValueError, match="gradient"):
            call(x, w, at, out=torch.empty_like(y))


def test_gradient_by_differences():
    """The product is linear: the quotient with exact inputs is the derivative, but
    for the two sides' roundings (u of every result, 4 u rms of every gradient)."""
    R, E, m, n, dtype = 60, 4, 90, 140, torch.float16
    w = pack(*make_layer(m, n, 64, 5, lead=(E,)), 64)
    at = torch.from_numpy(spread(R, E, 8).astype(np.int32)).to(DEV)
    v, dy = tokens(R, n, dtype, 1), tokens(R, m, dtype, 2)
    up, down = B.q4_experts(v, w, at).double(), B.q4_experts(-v, w, at).double()
    slope = ((up - down) / 2 * dy.double()).sum(1)
    dx = B.q4_experts_grad(dy, w, at).double()
    want = (dx * v.double()).sum(1)
    tol = U[dtype] * 1.1 * (up.abs() * dy.double().abs()).sum(1) + 5 * U[dtype] * (dx.square().mean(1).sqrt()[:, None] * v.double().abs()).sum(1)
    assert ((slope - want).abs() <= tol).all()
