"""Packing (include/bakron_q4.h) of codes and grids at any address."""
import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_q4 import DEV, dev, make_layer, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [33, 128, 129, 300])
@pytest.mark.parametrize("at", [0, 1, 2, 3, 7, 16])
def test_codes_that_start_at_any_byte(n, at):
    E, m, group = 3, 37, 64
    codes, scale, zero = make_layer(m, n, group, 61, (E,))
    x = tokens(5, n, torch.float16, 1)
    room = torch.full((E * m * n + 64,), 255, dtype=torch.uint8, device=DEV)
    moved = room[at:at + E * m * n].view(E, m, n)
    moved.copy_(dev(codes))
    w = B.q4_pack(dev(codes), dev(scale), dev(zero), group_size=group)
    v = B.q4_pack(moved, dev(scale), dev(zero), group_size=group)
    for e in range(E):
        assert torch.equal(B.q4_linear(x, w[e]), B.q4_linear(x, v[e]))
