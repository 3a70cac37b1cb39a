"""4-bit layers (include/bakron_q4.h) whose grids are far from uniform, against
their formulas in float64.  Tolerances as in test_gpu_q4.py: a result is a
float32 sum rounded once, its error below 2^-13 of the token's rms result;
none of it depends on how large the steps are."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from q4_forms import few_form, grad_form, prompt_form
from test_gpu_q4 import LINEAR, U, close, make_layer, pack, tokens, weights64

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
