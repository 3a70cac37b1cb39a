"""8-bit checkpoints and the gated activation that keeps them (ck8_pack,
ck8_unpack, gated_act, gated_act_grad).

Tolerances.  A checkpoint is defined to the bit.  sigmoid(t) is made of an
exponential whose argument -t log2(e) has two roundings (2^-23 |t| of its result)
and two hardware functions and two sums of a unit in the last place (2^-23) each:
(|t| + 5) 2^-23 relative, below 2^-16 for |t| <= 120, and beyond that p or 1 - p is
below 2^-126; t itself, for GELU, has four roundings (2^-22 |t| more).  2^-15
relative covers both; the results' products add less than that.  act' = p + a p
(1 - p) t' is a sum of two terms, each off by that much of itself, and 1 - p by
2^-23 absolutely.  Then the result's own rounding, half a step."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16]
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def values(rows, cols, dtype, seed, pad=0, shift=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn((rows, cols + pad), generator=g) * torch.exp(spread * torch.randn((rows, cols + pad), generator=g))
    return v.to(dtype).to(DEV)[:, shift:shift + cols]


def checkpoint_of(x):
    """What a checkpoint of x stands for, in float64, and its steps' exponents."""
    v = x.double().cpu().numpy()
    R, n = v.shape
    blocks = -(-n // 32)
    full = np.zeros((R, 32 * blocks))
    full[:, :n] = v
    full = full.reshape(R, blocks, 32)
    top = np.abs(full).max(2, keepdims=True)
    bad = ~np.isfinite(full).all(2, keepdims=True)
    top = np.where(bad, 0.0, top)
    s = np.full(top.shape, -126.0)
    for e in range(-126, 128):                                    # the smallest exponent that reaches the top
        s = np.where((np.rint(top / 2.0 ** s) > 127) & (s < e), e, s)
    out = np.rint(np.where(bad, 0.0, full) / 2.0 ** s) * 2.0 ** s
    out = np.where(bad, np.nan, out)
    return out.reshape(R, -1)[:, :n], np.where(bad, 128, s)[:, :, 0]


def same(got, ref):
    got = got.double().cpu().numpy()
    return np.array_equal(got, ref, equal_nan=True)


SHAPES = [(1, 1), (1, 32), (3, 33), (5, 100), (64, 128), (7, 1003), (300, 257), (2, 14336), (1, 65536), (5000, 40)]


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,n", SHAPES)
def test_a_checkpoint_is_what_it_is_defined_to_be(R, n, dtype):
    x = values(R, n, dtype, R + n, pad=3, shift=1, spread=2.0 if dtype == torch.bfloat16 else 1.0)
    ck = B.ck8_pack(x)
    ref, s = checkpoint_of(x)
    assert same(B.ck8_unpack(ck, dtype=torch.float32), ref)
    assert same(B.ck8_unpack(ck), torch.from_numpy(ref).to(dtype).double().numpy())
    # the layout: codes, then steps
    blocks = -(-n // 32)
    data = ck.data.cpu().numpy()
    codes = data[:R * 32 * blocks].view(np.int8).reshape(R, 32 * blocks)
    at = -(-R * 32 * blocks // 256) * 256
    assert np.array_equal(data[at:at + R * blocks].reshape(R, blocks), s + 127)
    assert (codes[:, n:] == 0).all() and codes.min() >= -127
    # a given one, and given values
    again = B.Checkpoint8.empty(R, n, dtype, DEV)
    assert B.ck8_pack(x, out=again) is again
    wide = torch.full((R, n + 5), 9.0, dtype=torch.float32, device=DEV)
    B.ck8_unpack(again, out=wide[:, 2:2 + n])
    assert same(wide[:, 2:2 + n], ref) and (wide[:, :2] == 9).all() and (wide[:, 2 + n:] == 9).all()


def test_values_where_steps_change():
    """Tops at and around the numbers that round to 128, over the whole range of
    exponents; ties; subnormals, infinities and NaN."""
    rows = []
    for e in list(range(-133, -118)) + list(range(-20, 20)) + [100, 120, 126]:
        for top in (1.0, 1.5, 1.984375, 1.9921875):               # 127 and 127.5 times 2^-6
            rows.append([top * 2.0 ** e] + [k * 2.0 ** (e - 7) for k in range(1, 32)])
    x = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16).to(DEV)
    x = torch.cat((x, -x, x * 0), 0)
    x[-3:, 5] = torch.tensor([float("inf"), -float("inf"), float("nan")], dtype=torch.bfloat16)
    assert same(B.ck8_unpack(B.ck8_pack(x), dtype=torch.float32), checkpoint_of(x)[0])
    x = torch.tensor([[65504.0, 1.0], [6e-8, 3e-5], [0.0, -0.0], [float("nan"), 1.0], [-float("inf"), 1.0]], dtype=torch.float16).to(DEV)
    assert same(B.ck8_unpack(B.ck8_pack(x), dtype=torch.float32), checkpoint_of(x)[0])
    # only the block with the NaN is lost
    x = values(4, 96, torch.bfloat16, 1)
    x[2, 40] = float("nan")
    got = B.ck8_unpack(B.ck8_pack(x))
    assert torch.isnan(got[2, 32:64]).all() and torch.isnan(got).sum() == 32


def parts(a, act):
    """act(a), p, a p (1 - p) t' in float64."""
    if act == "silu":
        t, dt = a, torch.ones_like(a)
    else:
        c = 2 * np.sqrt(2 / np.pi)
        t, dt = c * (a + 0.044715 * a ** 3), c * (1 + 3 * 0.044715 * a ** 2)
    p = torch.sigmoid(t)
    return a * p, p, a * p * (1 - p) * dt


def check_forward(h, a, b, act, dtype):
    a, b = a.double(), b.double()
    want = parts(a, act)[0] * b
    tol = (U[dtype] * 1.001 + 2.0 ** -15) * want.abs() + (a * b).abs() * 2.0 ** -124 + TINY[dtype]
    assert ((h.double() - want).abs() <= tol).all()


def check_back(da, db, dh, ca, cb, act, dtype):
    a, b = (B.ck8_unpack(c, dtype=torch.float32).double() for c in (ca, cb))
    g = dh.double()
    v, p, q = parts(a, act)
    want = g * v
    tol = (U[dtype] * 1.001 + 2.0 ** -15) * want.abs() + (g * a).abs() * 2.0 ** -124 + TINY[dtype]
    assert ((db.double() - want).abs() <= tol).all()
    want = g * b * (p + q)
    c = a.abs() if act == "silu" else a.abs().clamp(max=64.0) * (2 + 0.3 * a.clamp(-64, 64) ** 2)
    loose = (g * b).abs() * (2.0 ** -15 * (p + q.abs()) + c * p * 2.0 ** -22 + 2.0 ** -120)
    assert ((da.double() - want).abs() <= loose + U[dtype] * 1.001 * want.abs() + TINY[dtype]).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,n", SHAPES)
def test_forward_and_backward_match_their_formulas(R, n, dtype, act):
    ab = values(R, 2 * n, dtype, R + n, spread=0.7)
    a, b = ab[:, :n], ab[:, n:]                                   # halves of one buffer
    dh = values(R, n, dtype, 3, pad=2, shift=1, spread=0.7)
    check_forward(B.gated_act(a, b, act=act), a, b, act, dtype)
    h, ca, cb = B.gated_act(a, b, act=act, checkpoint=True)
    assert torch.equal(h, B.gated_act(a, b, act=act))
    for c, v in ((ca, a), (cb, b)):
        assert torch.equal(B.ck8_unpack(c), B.ck8_unpack(B.ck8_pack(v)))
    da, db = B.gated_act_grad(dh, ca, cb, act=act)
    check_back(da, db, dh, ca, cb, act, dtype)
    wide = torch.full((2, R, n + 3), 7.0, dtype=dtype, device=DEV)
    out = (wide[0, :, 1:1 + n], wide[1, :, 1:1 + n])
    got = B.gated_act_grad(dh, ca, cb, act=act, out=out)
    assert torch.equal(got[0], da) and torch.equal(got[1], db)
    assert (wide[:, :, 0] == 7).all() and (wide[:, :, 1 + n:] == 7).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_every_value_and_the_ends_of_the_range(act):
    """All of float16 and bfloat16 as a, ones as b; b infinite or NaN passes through."""
    for dtype in TYPES:
        a = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dtype).to(DEV).reshape(256, 256)
        b = torch.ones_like(a)
        h = B.gated_act(a, b, act=act)
        finite = torch.isfinite(a)
        check_forward(h[finite], a[finite], b[finite], act, dtype)
        assert torch.isnan(h[torch.isnan(a)]).all()
        assert (h[a == float("inf")] == float("inf")).all()
        d = torch.ones_like(a)
        for x in (a, a[:, torch.randperm(256, generator=torch.Generator().manual_seed(1)).to(DEV)].contiguous()):
            _, ca, cb = B.gated_act(x, b, act=act, checkpoint=True)
            da, db = B.gated_act_grad(d, ca, cb, act=act)
            ok = torch.isfinite(B.ck8_unpack(ca, dtype=torch.float32))
            v = B.ck8_unpack(ca, dtype=torch.float32).double()
            val, p, q = parts(v, act)
            q = torch.where(v.abs() > 64, torch.where(torch.tensor(act == "silu", device=DEV), q, 0.0), q)
            assert torch.isfinite(da[ok & (v.abs() < 1e38)]).all()
            want = (p + q).nan_to_num(0.0)
            m = ok & (v.abs() < 1e30)
            assert ((da.double() - want).abs()[m] <= 2.0 ** -7).all()
    a = torch.ones((1, 40), dtype=torch.bfloat16, device=DEV)
    b = a.clone()
    b[0, 3], b[0, 4] = float("inf"), float("nan")
    h = B.gated_act(a, b, act=act)
    assert torch.isinf(h[0, 3]) and torch.isnan(h[0, 4]) and torch.isfinite(h[0, 5:]).all()


@pytest.mark.parametrize("count", [-3, 0, 1, 70, 100, 1000])
def test_rows_behind_the_count_stay_as_they_are(count):
    R, n, dtype = 100, 72, torch.bfloat16
    a, b, dh = (values(R, n, dtype, i) for i in (1, 2, 3))
    c = torch.tensor([5, count], dtype=torch.int32, device=DEV)[-1:]
    cks = tuple(B.Checkpoint8(torch.full_like(B.Checkpoint8.empty(R, n, dtype, DEV).data, 77), R, n, dtype) for _ in range(2))
    h = torch.full((R, n), 3.0, dtype=dtype, device=DEV)
    B.gated_act(a, b, count=c, out=h, checkpoint=cks)
    m = min(max(count, 0), R)
    full, ca, cb = B.gated_act(a, b, checkpoint=True)
    assert torch.equal(h[:m], full[:m]) and (h[m:] == 3).all()
    for mine, whole in zip(cks, (ca, cb)):
        codes = mine.data[:R * 96].reshape(R, 96)
        assert torch.equal(codes[:m], whole.data[:R * 96].reshape(R, 96)[:m]) and (codes[m:] == 77).all()
    da, db = (torch.full((R, n), 4.0, dtype=dtype, device=DEV) for _ in range(2))
    B.gated_act_grad(dh, ca, cb, count=c, out=(da, db))
    ra, rb = B.gated_act_grad(dh, ca, cb)
    assert torch.equal(da[:m], ra[:m]) and torch.equal(db[:m], rb[:m]) and (da[m:] == 4).all() and (db[m:] == 4).all()


def test_nothing_there():
    for R, n in ((0, 40), (5, 0)):
        a = torch.empty((R, n), dtype=torch.float16, device=DEV)
        h, ca, cb = B.gated_act(a, a, checkpoint=True)
        assert h.shape == (R, n) and B.ck8_unpack(ca).shape == (R, n)
        assert B.gated_act_grad(a, ca, cb)[1].shape == (R, n) and B.ck8_unpack(B.ck8_pack(a)).shape == (R, n)


def test_autograd():
    R, n, dtype = 60, 100, torch.bfloat16
    plain = [values(R, n, dtype, i) for i in (1, 2, 3)]
    a, b, dh = plain[0].clone().requires_grad_(), plain[1].clone().requires_grad_(), plain[2]
    h = B.gated_act(a, b, act="gelu")
    ref, ca, cb = B.gated_act(*plain[:2], act="gelu", checkpoint=True)
    assert torch.equal(h, ref)
    h.backward(dh)
    da, db = B.gated_act_grad(dh, ca, cb, act="gelu")
    assert torch.equal(a.grad, da) and torch.equal(b.grad, db)
    a.grad = b.grad = None
    B.gated_act(a, b, act="gelu").sum().backward()                # an expanded gradient
    assert torch.equal(a.grad, B.gated_act_grad(torch.ones_like(dh), ca, cb, act="gelu")[0])
    # rows behind the count: zeros
    a.grad = b.grad = None
    B.gated_act(a, b, act="gelu", count=torch.tensor([7], dtype=torch.int32, device=DEV)).backward(dh)
    assert torch.equal(a.grad[:7], da[:7]) and (a.grad[7:] == 0).all() and (b.grad[7:] == 0).all()
    for kw in ({"out": torch.empty_like(dh)}, {"checkpoint": True}):
        with pytest.raises(ValueError, match="gradient"):
            B.gated_act(a, b, **kw)
    with torch.no_grad():
        assert not B.gated_act(a, b).requires_grad


def test_gradients_by_differences():
    """Central differences of the forward call around values that checkpoints hold
    exactly: an entry's quotient is off by the two results' rounding, 2^-11 of the
    result each (float16) over 2 h, and by h^2 / 6 times b times a third derivative
    below 2; the gradient by its own rounding and 2^-15 of terms of the order of 1."""
    R, n, h = 64, 64, 2.0 ** -3
    g = torch.Generator().manual_seed(5)
    a = (torch.randint(-48, 49, (R, n), generator=g) / 16).to(torch.float16).to(DEV)
    b = (torch.randint(-48, 49, (R, n), generator=g) / 16).to(torch.float16).to(DEV)
    dh = torch.ones_like(a)
    for act in ("silu", "gelu"):
        _, ca, cb = B.gated_act(a, b, act=act, checkpoint=True)
        assert torch.equal(B.ck8_unpack(ca), a) and torch.equal(B.ck8_unpack(cb), b)
        da, db = (v.double() for v in B.gated_act_grad(dh, ca, cb, act=act))
        up, down = B.gated_act(a + h, b, act=act).double(), B.gated_act(a - h, b, act=act).double()
        err = ((up - down) / (2 * h) - da).abs()
        assert (err <= h * h / 3 * b.double().abs() + 1.01 * ((up.abs() + down.abs()) * 2.0 ** -11 / (2 * h) + da.abs() * 2.0 ** -11) + 2.0 ** -12).all()
        up, down = B.gated_act(a, b + h, act=act).double(), B.gated_act(a, b - h, act=act).double()
        err = ((up - down) / (2 * h) - db).abs()
        assert (err <= 1.01 * ((up.abs() + down.abs()) * 2.0 ** -11 / (2 * h) + db.abs() * 2.0 ** -11) + 2.0 ** -12).all()
