"""4-bit layers (include/bakron_q4.h) whose grids are far from uniform, against
their formulas in float64.  Tolerances as in test_gpu_q4.py: a result is a
float32 sum rounded once, its error below 2^-13 of the token's rms result;
none of it depends on how large the steps are."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from q4_forms import few_form, prompt_form
from test_gpu_q4 import LINEAR, close, make_layer, pack, tokens, weights64

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
