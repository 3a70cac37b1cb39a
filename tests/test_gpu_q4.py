"""The 4-bit layer operators (q4_pack, q4_linear, q4_linear_grad, q4_moe;
include/bakron_q4.h) against their formulas in float64.

Tolerances.  u is the unit roundoff of the result's type (2^-8 for bfloat16,
2^-11 for float16).
* A result is a float32 sum rounded once: u |ref|, or half the spacing of the
  type's subnormal numbers where that is more.  The float32 sum itself
  keeps 24 bits of terms up to (16 + c) / 5 times a typical one; over n <=
  4096 terms, summed in blocks, its error is a random walk of at most n / 8
  steps of 2^-24 * 10 rms: below 2^-13 rms of the token's results.
* q4_linear_grad may round a weight once to the type (its step and zero point
  differ along the sum): an error of at most u per term, independent from
  term to term, so at most u rms / sqrt(3) in the mean square; six times
  that covers every entry: 4 u rms.
* q4_moe rounds once at the end; its inner activations keep 16 bits.  Their
  error and the router's float32 (2^-20 relative on a share) stay below 2^-11
  rms of the token's results.
"""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def make_layer(m, n, group, seed, lead=(), maxq=15):
    """Random codes and grids (zero points fractional, some outside [0, 15])."""
    rng = np.random.default_rng(seed)
    G = -(-n // group) if group else 1
    codes = rng.integers(0, maxq + 1, lead + (m, n)).astype(np.uint8)
    scale = (0.01 * np.exp(0.5 * rng.standard_normal(lead + (m, G)))).astype(np.float32)
    zero = rng.uniform(-2.0, maxq + 2.0, lead + (m, G)).astype(np.float32)
    return codes, scale, zero


def weights64(codes, scale, zero, group):
    n = codes.shape[-1]
    col = np.arange(n) // group if group else np.zeros(n, dtype=int)
    return scale.astype(np.float64)[..., col] * (codes.astype(np.float64) - zero.astype(np.float64)[..., col])


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def pack(codes, scale, zero, group):
    s, z = (dev(v if group else v[..., 0]) for v in (scale, zero))
    return B.q4_pack(dev(codes), s, z, group_size=group or None)


def tokens(T, n, dtype, seed, pad=0, shift=0):
    """T x n activations, a slice of rows n + pad wide from column `shift`."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, n + pad)).astype(np.float32)).to(dtype).to(DEV)
    return x[:, shift:shift + n]


def rms(a):
    return np.sqrt((a * a).mean(axis=1, keepdims=True)) if a.size else a


def close(got, ref, dtype, loose):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape
    tol = U[dtype] * (1 + 2.0 ** -6) * np.abs(ref) + loose * rms(ref) + TINY[dtype]
    worst = (np.abs(got - ref) / tol).max() if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.2f} times the tolerance"


LINEAR = 2.0 ** -13
SHAPES = [(1, 1, 0), (1, 300, 64), (16, 128, 128), (17, 130, 64), (100, 64, 0), (33, 1000, 128), (257, 515, 64),
          (130, 700, 192), (300, 1025, 256), (64, 4096, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("m,n,group", SHAPES)
@pytest.mark.parametrize("T", [1, 2, 5, 16, 17, 33, 64, 65, 130])
def test_linear_matches_its_formula(T, m, n, group, dtype):
    layer = make_layer(m, n, group, 1000 * m + n)
    w, ref = pack(*layer, group), weights64(*layer, group)
    x = tokens(T, n, dtype, T)
    close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("m,n,group", SHAPES)
@pytest.mark.parametrize("T", [1, 3, 17, 64, 130])
def test_grad_matches_its_formula(T, m, n, group, dtype):
    layer = make_layer(m, n, group, 1000 * m + n + 1)
    w, ref = pack(*layer, group), weights64(*layer, group)
    dy = tokens(T, m, dtype, T + 1)
    close(B.q4_linear_grad(dy, w), dy.double().cpu().numpy() @ ref, dtype, 4 * U[dtype])


@pytest.mark.parametrize("T,m,n,group", [(300, 520, 1030, 128), (513, 1000, 777, 64), (1025, 384, 2048, 0),
                                         (257, 2049, 320, 192)])
def test_prompt_sizes(T, m, n, group):
    for dtype in (torch.bfloat16, torch.float16):
        layer = make_layer(m, n, group, T)
        w, ref = pack(*layer, group), weights64(*layer, group)
        x, dy = tokens(T, n, dtype, 1), tokens(T, m, dtype, 2)
        close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)
        close(B.q4_linear_grad(dy, w), dy.double().cpu().numpy() @ ref, dtype, 4 * U[dtype])


@pytest.mark.parametrize("T,wide,narrow", [(1040, 6200, 200), (2060, 7200, 136)])
@pytest.mark.parametrize("group", [0, 64, 128])
def test_large_tiles(T, wide, narrow, group):
    """Enough tokens and columns of results for tiles of 128 and 256 tokens."""
    dtype = torch.float16 if group == 128 else torch.bfloat16
    layer = make_layer(wide, narrow, group, T)
    w, ref = pack(*layer, group), weights64(*layer, group)
    x = tokens(T, narrow, dtype, 1)
    close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)
    layer = make_layer(narrow, wide, group, T + 1)
    w, ref = pack(*layer, group), weights64(*layer, group)
    dy = tokens(T, narrow, dtype, 2)
    close(B.q4_linear_grad(dy, w), dy.double().cpu().numpy() @ ref, dtype, 4 * U[dtype])


@pytest.mark.parametrize("T,m,n,group", [
    (3498, 3458, 65, 64),       # layer: 256 x 256 tiles
    (261, 6645, 74, 0),         # layer: 128 x 128
    (2730, 143, 1791, 64),      # layer: 128 x 128, columns shared out; gradient: 256, rows not
    (5100, 450, 3200, 128),     # layer: 256 x 256 or 128 x 128, columns shared out
    (322, 64, 11732, 192),      # gradient: 128 tokens
    (1922, 3401, 66, 64),       # gradient: 128 tokens, rows shared out
    (3803, 6723, 68, 0),        # gradient: 256 tokens, rows shared out
])
def test_tiles_and_shared_sums(T, m, n, group):
    dtype = torch.float16 if n % 2 else torch.bfloat16
    layer = make_layer(m, n, group, T)
    w, ref = pack(*layer, group), weights64(*layer, group)
    x, dy = tokens(T, n, dtype, 1, pad=3), tokens(T, m, dtype, 2)
    close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)
    close(B.q4_linear_grad(dy, w), dy.double().cpu().numpy() @ ref, dtype, 4 * U[dtype])


@pytest.mark.parametrize("scale", [2.0**-101, 2.0**101, float("nan"), -float("inf")])
def test_steps_beyond_the_contract_are_refused(scale):
    codes, step, zero = make_layer(40, 128, 64, 3)
    B.q4_pack(dev(codes), dev(-step), dev(zero), group_size=64)
    step[7, 1] = scale
    with pytest.raises(B.GridError):
        B.q4_pack(dev(codes), dev(step), dev(zero), group_size=64)


@pytest.mark.parametrize("T", [3, 70])
def test_offsets_beyond_32_bits(T):
    # rows 80 MB (2 GB at three tokens) apart, of inputs and of results
    m, n, group = 40, 192, 64
    layer = make_layer(m, n, group, 71)
    w, ref = pack(*layer, group), weights64(*layer, group)
    ld = 40_000_004 if T > 3 else 1_000_000_004
    dtype = torch.bfloat16
    far_in = torch.empty((T, ld), dtype=dtype, device=DEV)
    far_out = torch.empty((T, ld), dtype=dtype, device=DEV)
    x, dy = tokens(T, n, dtype, 1), tokens(T, m, dtype, 2)
    far_in[:, :n] = x
    out = B.q4_linear(far_in[:, :n], w, out=far_out[:, :m])
    close(out, x.double().cpu().numpy() @ ref.T, dtype, LINEAR)
    far_in[:, :m] = dy
    out = B.q4_linear_grad(far_in[:, :m], w, out=far_out[:, :n])
    close(out, dy.double().cpu().numpy() @ ref, dtype, 4 * U[dtype])


@pytest.mark.parametrize("T", [2, 100, 300])
def test_groups_of_step_zero(T):
    # a step of 0 makes every weight of the group 0, whatever its codes
    m, n, group = 70, 320, 64
    layer = make_layer(m, n, group, 81)
    layer[1][::3, 1] = 0.0
    layer[1][5] = 0.0
    w, ref = pack(*layer, group), weights64(*layer, group)
    for dtype in (torch.bfloat16, torch.float16):
        x, dy = tokens(T, n, dtype, 1), tokens(T, m, dtype, 2)
        close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)
        close(B.q4_linear_grad(dy, w), dy.double().cpu().numpy() @ ref, dtype, 4 * U[dtype])


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 0), (8, 8), (7, 3), (64, 1)])
def test_rows_of_a_wider_buffer(T, pad, shift):
    # any row stride and any 2-byte alignment, of inputs and of results
    m, n, group = 96, 256, 64
    layer = make_layer(m, n, group, 5)
    w, ref = pack(*layer, group), weights64(*layer, group)
    for dtype in (torch.bfloat16, torch.float16):
        x, dy = tokens(T, n, dtype, 6, pad, shift), tokens(T, m, dtype, 7, pad, shift)
        for call, v, cols, want in ((B.q4_linear, x, m, x.double().cpu().numpy() @ ref.T),
                                    (B.q4_linear_grad, dy, n, dy.double().cpu().numpy() @ ref)):
            wide = torch.full((T, cols + pad), 7.0, dtype=dtype, device=DEV)
            out = wide[:, shift:shift + cols]
            assert call(v, w, out=out) is out
            close(out, want, dtype, 4 * U[dtype] if call is B.q4_linear_grad else LINEAR)
            rest = torch.ones_like(wide, dtype=torch.bool)
            rest[:, shift:shift + cols] = False
            assert bool((wide[rest] == 7.0).all())     # nothing beside the result is written


def test_extreme_grids():
    # zero points far outside the codes, steps from 1e-9 to 1e3 (beyond
    # float16 as weights), a group of equal weights
    m, n, group = 48, 512, 128
    for step in (1e-9, 1e3):
        codes, scale, zero = make_layer(m, n, group, 9)
        scale[:] *= step / 0.01
        zero[0], zero[1] = -200.0, 300.0
        codes[2, :128], zero[2, 0] = 4, 4.0
        layer = (codes, scale, zero)
        w, ref = pack(*layer, group), weights64(*layer, group)
        for dtype in (torch.bfloat16, torch.float16):
            for T in (2, 100):
                k = np.float32(1e-6 if step > 1 and dtype == torch.float16 else 1.0)
                x, dy = (tokens(T, c, dtype, c) * float(k) for c in (n, m))
                if dtype == torch.float16 and step < 1:
                    x, dy = x * 1000, dy * 1000
                for call, v, want in ((B.q4_linear, x, x.double().cpu().numpy() @ ref.T),
                                      (B.q4_linear_grad, dy, dy.double().cpu().numpy() @ ref)):
                    got = call(v, w).double().cpu().numpy()
                    # the zero points of rows 0 and 1 are some 40 times a typical
                    # code: so many times the sum's float32 error; float16
                    # results below its normal range are rounded to 2^-25
                    tol = (2 * U[dtype] * np.abs(want) + (2.0 ** -7 if call is B.q4_linear else 4 * U[dtype])
                           * rms(want) + (2.0 ** -24 if dtype == torch.float16 else 0.0))
                    assert (np.abs(got - want) <= tol).all(), (step, dtype, T, call.__name__)


@pytest.mark.parametrize("T", [4, 100])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_non_finite_token_stays_alone(T, bad):
    m, n = 80, 300
    layer = make_layer(m, n, 64, 11)
    w = pack(*layer, 64)
    for dtype in (torch.bfloat16, torch.float16):
        for call, cols in ((B.q4_linear, n), (B.q4_linear_grad, m)):
            x = tokens(T, cols, dtype, 12).clone()
            clean = call(x, w)
            x[1, cols // 2] = bad
            got = call(x, w)
            others = [t for t in range(T) if t != 1]
            assert torch.equal(got[others], clean[others])
            assert not bool(torch.isfinite(got[1]).any())


def test_no_columns_no_rows_no_tokens():
    for T, m, n in ((3, 5, 0), (0, 5, 7), (3, 0, 7)):
        layer = make_layer(m, n, 0, 1)
        w = pack(*layer, 0)
        for call, cin, cout in ((B.q4_linear, n, m), (B.q4_linear_grad, m, n)):
            x = torch.ones((T, cin), dtype=torch.bfloat16, device=DEV)
            out = torch.full((T, cout), 5.0, dtype=torch.bfloat16, device=DEV)
            call(x, w, out=out)
            torch.cuda.synchronize()
            assert bool((out == 0).all()), (T, m, n, call.__name__)


@pytest.mark.parametrize("T", [1, 40, 200])
def test_gradient_against_differences(T):
    """The layer is linear: <dy, f(x + v) - f(x)> = <dx, v> for any step v.
    Both sides round results: each f to u of itself, dx as above; errors of
    T m (T n) independent terms."""
    m, n, group = 200, 330, 64
    layer = make_layer(m, n, group, 21)
    w = pack(*layer, group)
    dtype = torch.float16
    x, v, dy = tokens(T, n, dtype, 1), tokens(T, n, dtype, 2), tokens(T, m, dtype, 3)
    xv = x + v                                   # rounded to the type: the step taken is xv - x
    step = (xv.double() - x.double()).cpu()
    f0, f1 = B.q4_linear(x, w).double().cpu(), B.q4_linear(xv, w).double().cpu()
    dx = B.q4_linear_grad(dy, w).double().cpu()
    g = dy.double().cpu()
    left, right = float((g * (f1 - f0)).sum()), float((dx * step).sum())
    u = U[dtype]
    err = 6 * u * float((g * g * (f1 * f1 + f0 * f0)).sum().sqrt()) + 6 * 3 * u * float((dx * dx * step * step).sum().sqrt())
    assert abs(left - right) <= err
    assert err < 0.05 * max(1.0, float((dx * dx).sum().sqrt() * (step * step).sum().sqrt()))


def test_same_call_same_bits():
    layer = make_layer(1000, 1500, 128, 31)
    w = pack(*layer, 128)
    for T in (1, 16, 100, 300):
        x, dy = tokens(T, 1500, torch.bfloat16, T), tokens(T, 1000, torch.bfloat16, T)
        a, b = B.q4_linear(x, w), B.q4_linear_grad(dy, w)
        for _ in range(5):
            assert torch.equal(B.q4_linear(x, w), a) and torch.equal(B.q4_linear_grad(dy, w), b)


def test_other_stream_and_kept_buffers():
    layer = make_layer(500, 640, 64, 41)
    w = pack(*layer, 64)
    side = torch.cuda.Stream()
    for T in (2, 200):
        x = tokens(T, 640, torch.bfloat16, T)
        ref = B.q4_linear(x, w)
        ws = torch.full((max(1, B.q4_linear_workspace_bytes(T, w)),), 0xAB, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(ref)
        side.wait_stream(torch.cuda.current_stream())
        B.q4_linear(x, w, out=out, ws=ws, stream=side)
        alone = B.q4_linear(x, w, stream=side)
        side.synchronize()
        assert torch.equal(out, ref) and torch.equal(alone, ref)


# ------------------------------------------------------------- experts

def moe64(x, router, gate, up, down, k):
    """The layer in float64, and the choices."""
    logits = x @ router.T
    T = x.shape[0]
    ids = np.zeros((T, k), dtype=np.int64)
    p = np.zeros((T, k))
    y = np.zeros((T, down.shape[1]))
    for t in range(T):
        ids[t] = sorted(range(router.shape[0]), key=lambda e: (-logits[t, e], e))[:k]
        ex = np.exp(logits[t, ids[t]] - logits[t, ids[t, 0]])
        p[t] = ex / ex.sum()
        for j, e in enumerate(ids[t]):
            a, b = gate[e] @ x[t], up[e] @ x[t]
            y[t] += p[t, j] * (down[e] @ (a / (1 + np.exp(-a)) * b))
    return y, ids, p


def make_moe(T, h, f, E, k, group, dtype, seed):
    rng = np.random.default_rng(seed)
    x = tokens(T, h, dtype, seed)
    router = torch.from_numpy((rng.standard_normal((E, h)) * 2 / np.sqrt(h)).astype(np.float32)).to(dtype).to(DEV)
    layers = [make_layer(f, h, group, seed + 1, (E,)), make_layer(f, h, group, seed + 2, (E,)),
              make_layer(h, f, group, seed + 3, (E,))]
    return x, router, layers


MOE = 2.0 ** -11


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,h,f,E,k,group", [
    (1, 64, 64, 1, 1, 0), (1, 128, 256, 8, 2, 128), (2, 100, 70, 5, 5, 64), (3, 130, 515, 4, 1, 0),
    (16, 256, 200, 16, 4, 64), (17, 192, 130, 3, 2, 128), (40, 96, 100, 8, 8, 64), (64, 320, 128, 64, 6, 64),
    (64, 65, 33, 2, 2, 0), (5, 512, 1025, 70, 16, 192), (9, 1, 1, 3, 2, 0)])
def test_moe_matches_its_formula(T, h, f, E, k, group, dtype):
    x, router, layers = make_moe(T, h, f, E, k, group, dtype, 7 * T + h)
    out = B.q4_moe(x, router, *(pack(*v, group) for v in layers), k)
    y, ids, p = moe64(x.double().cpu().numpy(), router.double().cpu().numpy(), *(weights64(*v, group) for v in layers), k)
    assert np.array_equal(out["ids"].cpu().numpy(), ids)
    assert np.abs(out["weights"].double().cpu().numpy() - p).max() <= 2.0 ** -18
    close(out["y"], y, dtype, MOE)


def test_moe_equal_logits_go_to_the_lower_index():
    x, router, layers = make_moe(6, 96, 64, 12, 4, 0, torch.bfloat16, 3)
    router[:] = router[3]
    router[7] = router[7] * 0.5
    out = B.q4_moe(x, router, *(pack(*v, 0) for v in layers), 4)
    l3 = (x.double() @ router[3].double()).cpu().numpy()
    for t, ids in enumerate(out["ids"].cpu().tolist()):
        assert ids == ([0, 1, 2, 3] if l3[t] > 0 else [7, 0, 1, 2])
        # equal logits, equal shares
        assert len(set(out["weights"][t, (0 if l3[t] > 0 else 1):].tolist())) == 1


def test_moe_reads_only_chosen_experts_and_keeps_tokens_apart():
    T, h, f, E, k = 5, 128, 192, 6, 2
    x, router, layers = make_moe(T, h, f, E, k, 64, torch.bfloat16, 13)
    router[4] = 0
    router[4, 0] = -100
    x = x.clone()
    x[:, 0] = x[:, 0].abs() + 1              # expert 4 is never chosen
    clean = [pack(*v, 64) for v in layers]
    ref = B.q4_moe(x, router, *clean, k)
    assert not bool((ref["ids"] == 4).any())
    for v in layers:
        v[1][4] = np.nan
    dirty = [B.q4_pack(dev(c), dev(s), dev(z), group_size=64, check=False) for c, s, z in layers]
    got = B.q4_moe(x, router, *dirty, k)
    for key in ref:
        assert torch.equal(got[key], ref[key]), key
    x[2, 5] = float("nan")
    got = B.q4_moe(x, router, *clean, k)
    others = [0, 1, 3, 4]
    assert torch.equal(got["y"][others], ref["y"][others]) and torch.equal(got["ids"][others], ref["ids"][others])
    assert not bool(torch.isfinite(got["y"][2]).any())
    assert got["ids"][2].tolist() == [0, 1]  # every logit NaN


def test_moe_kept_buffers_strides_and_empty_sides():
    T, h, f, E, k = 7, 100, 90, 4, 2
    x, router, layers = make_moe(T, h, f, E, k, 0, torch.float16, 17)
    w = [pack(*v, 0) for v in layers]
    ref = B.q4_moe(x, router, *w, k)
    wide = torch.zeros((T, h + 5), dtype=x.dtype, device=DEV)
    wide[:, 3:3 + h] = x
    out = {"y": torch.zeros((T, h + 9), dtype=x.dtype, device=DEV)[:, 1:1 + h],
           "ids": torch.empty((T, k), dtype=torch.int32, device=DEV),
           "weights": torch.empty((T, k), dtype=torch.float32, device=DEV)}
    ws = torch.full((B.q4_moe_workspace_bytes(T, w[0], k),), 0xFF, dtype=torch.uint8, device=DEV)
    assert B.q4_moe(wide[:, 3:3 + h], router, *w, k, out=out, ws=ws) is out
    for key in ref:
        assert torch.equal(out[key], ref[key]), key
    assert B.q4_moe(x[:0], router, *w, k)["y"].shape == (0, h)
    layers = [make_layer(0, h, 0, 1, (E,)), make_layer(0, h, 0, 1, (E,)), make_layer(h, 0, 0, 1, (E,))]
    empty = B.q4_moe(x, router, *(pack(*v, 0) for v in layers), k)
    assert bool((empty["y"] == 0).all()) and torch.equal(empty["ids"], ref["ids"])


def test_calls_in_a_graph():
    """Every call captured into one HIP graph; replays with eager work and
    synchronisations between them give the eager results."""
    lin = make_layer(300, 512, 64, 51)
    w = pack(*lin, 64)
    x, big, dy = tokens(3, 512, torch.bfloat16, 1), tokens(300, 512, torch.bfloat16, 2), tokens(70, 300, torch.bfloat16, 3)
    mx, router, layers = make_moe(6, 128, 256, 8, 2, 64, torch.bfloat16, 4)
    stacks = [pack(*v, 64) for v in layers]

    def calls():
        return [B.q4_linear(x, w), B.q4_linear(big, w), B.q4_linear_grad(dy, w),
                *B.q4_moe(mx, router, *stacks, 2).values()]
    eager = [t.clone() for t in calls()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        calls()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            outs = calls()
    for _ in range(4):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, eager):
            assert torch.equal(o, r)
        calls()


def test_refusals_on_the_device():
    layer = make_layer(64, 128, 64, 61)
    w = pack(*layer, 64)
    x = tokens(2, 128, torch.bfloat16, 1)
    with pytest.raises(TypeError):
        B.q4_linear(x.float(), w)
    with pytest.raises(TypeError):
        B.q4_linear(x.cpu(), w)
    with pytest.raises(TypeError):
        B.q4_linear(x, w.data)
    with pytest.raises(ValueError):
        B.q4_linear(x[:, :64], w)
    with pytest.raises(ValueError):
        B.q4_linear(tokens(128, 2, torch.bfloat16, 1).t(), w)
    with pytest.raises(ValueError):
        B.q4_linear(x, w, out=torch.empty((3, 64), dtype=x.dtype, device=DEV))
    with pytest.raises(TypeError):
        B.q4_linear(x, w, out=torch.empty((2, 64), dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):
        B.q4_linear_grad(x, w)
    with pytest.raises(B.GridError):
        B.q4_pack(dev(layer[0] + 16), dev(layer[1]), dev(layer[2]), group_size=64)
    with pytest.raises(B.GridError):
        B.q4_pack(dev(layer[0]), dev(layer[1] * np.inf), dev(layer[2]), group_size=64)
    with pytest.raises(ValueError):
        B.q4_pack(dev(layer[0]), dev(layer[1]), dev(layer[2]), group_size=96)
    with pytest.raises(ValueError):
        B.q4_pack(dev(layer[0]), dev(layer[1]), dev(layer[2]), group_size=128)
    mx, router, layers = make_moe(2, 128, 64, 4, 2, 64, torch.bfloat16, 4)
    g, u, d = (pack(*v, 64) for v in layers)
    with pytest.raises(ValueError):
        B.q4_moe(mx, router, g, u, w, 2)
    with pytest.raises(ValueError):
        B.q4_moe(mx, router, g, d, d, 2)
    with pytest.raises(ValueError):
        B.q4_moe(mx, router[:3].contiguous(), g, u, d, 2)
    with pytest.raises(B.BakronError):
        B.q4_moe(mx, router, g, u, d, 5)
    with pytest.raises(B.BakronError):
        B.q4_moe(tokens(65, 128, torch.bfloat16, 1), router, g, u, d, 2)
    with pytest.raises(B.BakronError) as e:
        B.q4_moe(mx, router, g, u, d, 2, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.code == B._binding.BAKRON_ERR_WORKSPACE


def test_solve_then_serve():
    """The rounded layer of a solve, packed and applied: V x to float32's own
    rounding of V."""
    from oracle import reference as R
    from workloads import make_problem
    d = make_problem(128, 192, 3, bits=4, group_size=64)
    fa, fb = R.factor(d["A"]), R.factor(d["B"])
    t = [dev(v.astype(np.float32)) for v in (d["W"], fa["L"], fa["P"], fb["L"], fb["P"])]
    s, z = dev(d["scale"]), dev(d["zero"])
    out = B.solve(*t, s, z, dev(d["maxq"]), group_size=64)
    w = B.q4_pack(out["codes"], s, z, group_size=64)
    x = tokens(4, 192, torch.bfloat16, 5)
    close(B.q4_linear(x, w), (x.double() @ out["V"].double().T.contiguous()).cpu().numpy(), torch.bfloat16, LINEAR)
