"""The experts' gradient for few rows where rows of W are alike: roundings of dy times
the step then add up instead of averaging out.

a = dy s is kept in two bfloat16 terms.  Here a = 1 + 2^-9 + r in every row (times a power
of two), r just below 2^-17: the terms are 1 and 2^-9, and r is what they leave.  With
zero points of 7.5 every product and every sum of those terms is a multiple of 2^-10 below
2^14, exact in float32.  What is left is r sum_i (c_i - z_i), 2^-17 of the result, and the
result's own rounding."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from moe_forms import experts_grad_form
from test_gpu_q4 import DEV, TINY, U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,R,m,n,group", [(4, 16, 14336, 256, 128), (4, 16, 14336, 192, 64), (3, 48, 9001, 130, 0),
                                           (8, 32, 14336, 4096, 128)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_that_are_alike(E, R, m, n, group, dtype):
    assert experts_grad_form(R, E, m, n, group)[0] == "few"
    G = -(-n // group) if group else 1
    step, z = 2.0 ** -5 * (1 + 2.0 ** -9 + 2.0 ** -17 - 2.0 ** -23), 7.5
    assert float(np.float32(step)) == step
    codes = np.random.default_rng(m + n).integers(0, 16, (E, m, n), dtype=np.uint8)
    scale = torch.full((E, m, G), step, dtype=torch.float32, device=DEV)
    w = B.q4_pack(torch.from_numpy(codes).to(DEV), scale, torch.full_like(scale, z), group_size=group or None)
    each = R // E
    at = torch.arange(E + 1, dtype=torch.int32, device=DEV) * each
    signs = np.where(np.arange(R) % 2, -1.0, 1.0)
    dy = torch.from_numpy(signs).to(DEV, dtype)[:, None].expand(R, m).contiguous()
    got = B.q4_experts_grad(dy, w, at).double().cpu().numpy()
    sums = codes.astype(np.float64).sum(1) - z * m                # sum_i (c_i - z), exact
    assert np.abs(sums).max() < 2.0 ** 13
    want = signs[:, None] * step * np.repeat(sums, each, axis=0)
    tol = (U[dtype] + 2.0 ** -17 + 2.0 ** -22) * np.abs(want) + TINY[dtype]
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1.0, f"{worst:.2f} times the tolerance"
