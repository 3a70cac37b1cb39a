"""4-bit layers (include/bakron_q4.h) whose grids are far from uniform, against
their formulas in float64.  Tolerances as in test_gpu_q4.py: a result is a
float32 sum rounded once, its error below 2^-13 of the token's rms result;
none of it depends on how large the steps are."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from q4_forms import few_form, grad_form, prompt_form
from test_gpu_q4 import DEV, LINEAR, U, close, make_layer, pack, tokens, weights64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("step", [1e-2, 1e-4, 1e-6, 1e-9])
@pytest.mark.parametrize("T,m,form", [
    (3, 300, (1, 1)), (64, 300, (16, 1)), (65, 300, (64, 128, 1)), (300, 120, (64, 128, 1)), (257, 6619, (128, 128, 1)),
    (4755, 778, (128, 256, 1)), (1295, 8920, (256, 256, 1))])
def test_steps_of_zero_beside_small_steps(T, m, form, step):
    """A group of step 0 leaves the rest of its row its precision, whatever the
    row's other steps are and whether or not x has a mean."""
    n, group = 512, 64
    assert (few_form(T, m) if T <= 64 else prompt_form(T, m, n)) == form
    codes, scale, zero = make_layer(m, n, group, 91)
    scale *= step / 0.01
    scale[::2] *= -1.0
    scale[::3, 1] = 0.0
    scale[1::5, 0] = 0.0        # the first of a row,
    scale[1::7, 7] = 0.0        # the last,
    scale[2::9, 2:6] = 0.0      # some in a run
    w, ref = pack(codes, scale, zero, group), weights64(codes, scale, zero, group)
    for dtype in (torch.bfloat16, torch.float16):
        x = tokens(T, n, dtype, 1) * 2.0 ** min(12, int(np.log2(0.01 / step)))   # (results stay in float16's range)
        x = x + x.abs().max() / 4       # a mean of about one deviation
        close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T,m", [(3, 300), (64, 300), (65, 300), (257, 6619), (4755, 778), (1295, 8920)])
def test_rows_of_step_zero(T, m, group):
    """Rows without any step are 0, up to what the smallest normal float32
    number could leave of a sum."""
    n = 512
    codes, scale, zero = make_layer(m, n, group, 92)
    scale[::4] = 0.0
    w = pack(codes, scale, zero, group)
    for dtype in (torch.bfloat16, torch.float16):
        y = B.q4_linear(tokens(T, n, dtype, 1) + 2, w)
        assert float(y[:, ::4].abs().max()) <= 2.0 ** -110
        dx = B.q4_linear_grad(tokens(T, m, dtype, 2), w)
        assert bool(torch.isfinite(dx).all())


@pytest.mark.parametrize("T,m,form", [(1, 300, (64, 256, 2)), (130, 300, (64, 256, 1)), (300, 1500, (64, 256, 7)),
                                      (8000, 700, (128, 256, 1))])
def test_gradient_of_groups_of_very_different_steps(T, m, form):
    """A group's columns of dx come from its own weights alone: they keep their
    precision, 4 u of the rms of that group's part of a token, beside groups
    (and under rows) whose steps are 2^16 times as large."""
    n, group = 700, 64
    assert grad_form(T, m, n) == form
    codes, scale, zero = make_layer(m, n, group, 93)
    scale *= (2.0 ** -np.arange(11.0) * 2.0 ** -6).astype(np.float32)
    scale[:, 3] *= 2.0 ** 10
    w, ref = pack(codes, scale, zero, group), weights64(codes, scale, zero, group)
    for dtype in (torch.bfloat16, torch.float16):
        dy = tokens(T, m, dtype, 2) * 2.0 ** 10
        want, got = dy.double().cpu().numpy() @ ref, B.q4_linear_grad(dy, w)
        for c in range(0, n, group):
            close(got[:, c:c + group], want[:, c:c + group], dtype, 4 * U[dtype])


def test_gradient_under_rows_that_a_token_leaves_out():
    # the rows of large steps have gradients of zero: the others' weights count
    m, n, group = 400, 320, 64
    codes, scale, zero = make_layer(m, n, group, 94)
    scale[5] *= 2.0 ** 17
    scale[300, 2] *= 2.0 ** 19
    w, ref = pack(codes, scale, zero, group), weights64(codes, scale, zero, group)
    for dtype in (torch.bfloat16, torch.float16):
        for T in (1, 130):
            dy = tokens(T, m, dtype, 2).clone()
            dy[:, [5, 300]] = 0
            close(B.q4_linear_grad(dy, w), dy.double().cpu().numpy() @ ref, dtype, 4 * U[dtype])


# x of a mean of two deviations.  Sums of (16 + c) x, about 23 times the mean of
# x per column, grow with the columns, the result with their root.  They are
# not kept beyond two pieces of 512 columns or two groups: a random walk of n /
# 16 roundings of at most 0.42 * 2^-24 of a ramp up to 1024 * 23.5 * 2 steps,
# against a result of 4.6 sqrt(5 n) steps, is 1.9e-5 of it in the rms; six times
# that stays below 2^-13.
@pytest.mark.parametrize("T,m,n,form", [
    (4, 600, 16384, (1, 1)), (64, 600, 16384, (16, 1)), (200, 1000, 65536, (64, 128, 8)), (1030, 2050, 32768, (128, 128, 5)),
    (600, 4096, 32768, (128, 256, 3)), (2048, 2048, 65536, (256, 256, 4)), (2048, 8192, 16384, (256, 256, 1))])
@pytest.mark.parametrize("group", [0, 128])
def test_activations_with_a_mean(T, m, n, group, form):
    assert (few_form(T, m) if T <= 64 else prompt_form(T, m, n)) == form
    gen = torch.Generator(device=DEV)
    gen.manual_seed(n + group)
    G = -(-n // group) if group else 1
    codes = torch.randint(0, 16, (m, n), generator=gen, device=DEV, dtype=torch.uint8)
    scale = 0.01 * torch.exp(0.3 * torch.randn((m, G), generator=gen, device=DEV))
    zero = 7.5 + 0.3 * torch.randn((m, G), generator=gen, device=DEV)
    dtype = torch.float16
    x = (0.02 * (torch.randn((T, n), generator=gen, device=DEV) + 2)).to(dtype)
    y = B.q4_linear(x, B.q4_pack(codes, scale, zero, group_size=group) if group else B.q4_pack(codes, scale, zero))
    some = torch.linspace(0, T - 1, min(T, 12)).long()
    col, xs, ref = torch.arange(n, device=DEV) // (group or n), x[some].double(), []
    for r in range(0, m, 512):
        rows = scale[r:r + 512].double()[:, col] * (codes[r:r + 512].double() - zero[r:r + 512].double()[:, col])
        ref.append(xs @ rows.t().contiguous())
    close(y[some], torch.cat(ref, 1).cpu().numpy(), dtype, LINEAR)


@pytest.mark.parametrize("T,m,n,form", [(130, 300, 3000, (64, 128, 8)), (1105, 555, 1301, (64, 128, 1)), (2730, 143, 5000, (128, 128, 5)),
                                        (2700, 1200, 900, (128, 128, 1)), (4200, 1100, 4000, (256, 256, 3))])
@pytest.mark.parametrize("group", [0, 64, 192, 576, 1088])
def test_groups_and_splits_that_end_in_any_column(T, m, n, group, form):
    assert prompt_form(T, m, n) == form
    layer = make_layer(m, n, group, 95)
    w, ref = pack(*layer, group), weights64(*layer, group)
    dtype = torch.float16 if group else torch.bfloat16
    x = tokens(T, n, dtype, 1) + 2
    close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)
