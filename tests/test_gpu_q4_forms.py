"""4-bit layer calls (include/bakron_q4.h) at sizes that reach each kernel form
and split, named by the rules that choose them (q4_forms.py).  Tolerances and
helpers as in test_gpu_q4.py."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from q4_forms import few_form, grad_form, moe_splits, moe_up_form, prompt_form
from test_gpu_q4 import LINEAR, MOE, U, close, make_layer, make_moe, moe64, pack, tokens, weights64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,form", [(1, (1, 2)), (4, (1, 2)), (5, (2, 2)), (8, (2, 2)), (16, (4, 2)), (32, (8, 2)), (33, (16, 2)),
                                    (64, (16, 2))])
@pytest.mark.parametrize("group", [0, 64, 128, 192])
def test_few_tokens_two_row_tiles(T, form, group):
    # 513 row tiles: the last workgroup's second one is not there
    m, n = 8200, 300
    assert few_form(T, m) == form
    layer = make_layer(m, n, group, 71)
    w, ref = pack(*layer, group), weights64(*layer, group)
    for dtype in (torch.bfloat16, torch.float16):
        x = tokens(T, n, dtype, T, pad=T % 3)
        close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)


@pytest.mark.parametrize("T,m,n,form", [
    (1100, 2048, 8192, (128, 256, 3)), (600, 4090, 6100, (128, 256, 3)), (1030, 4096, 4999, (256, 256, 3)),
    (300, 300, 5000, (64, 128, 8))])
@pytest.mark.parametrize("group", [0, 64, 128, 192])
def test_prompt_tiles_whose_columns_are_shared_out(T, m, n, form, group):
    assert prompt_form(T, m, n) == form
    layer = make_layer(m, n, group, 72)
    w, ref = pack(*layer, group), weights64(*layer, group)
    dtype = torch.float16 if group % 128 else torch.bfloat16
    x = tokens(T, n, dtype, 1)
    close(B.q4_linear(x, w), x.double().cpu().numpy() @ ref.T, dtype, LINEAR)


@pytest.mark.parametrize("T,m,n,form", [(3, 2100, 700, (64, 256, 16)), (900, 3000, 2600, (128, 256, 2)),
                                        (1500, 3000, 2600, (256, 256, 3)), (2000, 4000, 1400, (256, 256, 5))])
@pytest.mark.parametrize("group", [0, 64, 192])
def test_gradient_tiles_whose_rows_are_shared_out(T, m, n, form, group):
    assert grad_form(T, m, n) == form
    layer = make_layer(m, n, group, 73)
    w, ref = pack(*layer, group), weights64(*layer, group)
    dtype = torch.float16 if group % 128 else torch.bfloat16
    dy = tokens(T, m, dtype, 2)
    close(B.q4_linear_grad(dy, w), dy.double().cpu().numpy() @ ref, dtype, 4 * U[dtype])


@pytest.mark.parametrize("T,h,f,E,k,waves,splits", [
    (3, 300, 1100, 5, 2, 8, 1), (10, 300, 1100, 16, 3, 4, 4), (20, 300, 1100, 24, 6, 4, 4), (40, 300, 1100, 48, 4, 2, 4),
    (64, 520, 700, 64, 6, 2, 4), (20, 4200, 300, 64, 4, 4, 1), (17, 1100, 1200, 12, 2, 8, 3)])
@pytest.mark.parametrize("group", [0, 64, 128, 192])
def test_expert_waves_and_splits(T, h, f, E, k, waves, splits, group):
    assert (moe_up_form(T, f, E, k), moe_splits(T, h, f, E, k)) == (waves, splits)
    dtype = torch.float16 if group % 128 else torch.bfloat16
    x, router, layers = make_moe(T, h, f, E, k, group, dtype, 74)
    out = B.q4_moe(x, router, *(pack(*v, group) for v in layers), k)
    y, ids, p = moe64(x.double().cpu().numpy(), router.double().cpu().numpy(), *(weights64(*v, group) for v in layers), k)
    assert np.array_equal(out["ids"].cpu().numpy(), ids)
    assert np.abs(out["weights"].double().cpu().numpy() - p).max() <= 2.0 ** -18
    close(out["y"], y, dtype, MOE)


@pytest.mark.parametrize("T", [2, 16, 50])
@pytest.mark.parametrize("group", [0, 64, 128])
def test_experts_of_activations_with_a_mean(T, group):
    # x of a mean of two deviations, long rows
    h, f, E, k, dtype = 8200, 200, 6, 2, torch.float16
    x, router, layers = make_moe(T, h, f, E, k, group, dtype, 75)
    x = x / 8 + 0.25
    out = B.q4_moe(x, router, *(pack(*v, group) for v in layers), k)
    y, ids, p = moe64(x.double().cpu().numpy(), router.double().cpu().numpy(), *(weights64(*v, group) for v in layers), k)
    assert np.array_equal(out["ids"].cpu().numpy(), ids)
    # (a result beyond the type's largest value, 65504, is infinite)
    far = np.abs(y) > 65504 + 16
    got = out["y"].double().cpu().numpy()
    assert np.array_equal(got[far], np.copysign(np.inf, y[far])) and far.mean() < 0.1
    y[far] = 0.0
    close(out["y"].masked_fill(torch.from_numpy(far).to(x.device), 0.0), y, dtype, MOE)
