"""Packing (include/bakron_q4.h) of codes and grids at any address."""
import numpy as np
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


@pytest.mark.parametrize("m,n,group", [(40, 130, 0), (1000, 64, 64), (8500, 128, 64), (300, 300, 64), (77, 512, 64), (530, 700, 64),
                                       (8300, 1100, 64), (33, 65536, 64)])
def test_grids_of_any_number_of_groups(m, n, group):
    """The steps that a layer of codes 0 and 1 puts out, one column of a group
    at a time, are the ones that went in; steps of 0 give 0."""
    G = -(-n // group) if group else 1
    rng = np.random.default_rng(m)
    scale = (2.0 ** rng.integers(-8, 8, (m, G))).astype(np.float32)
    scale[rng.random((m, G)) < 0.1] = 0.0
    zero = np.zeros((m, G), np.float32)
    codes = np.ones((m, n), np.uint8)
    s, z = (dev(v if group else v[:, 0]) for v in (scale, zero))
    w = B.q4_pack(dev(codes), s, z, group_size=group or None)
    for dtype in (torch.bfloat16, torch.float16):
        some = np.unique(np.linspace(0, G - 1, min(G, 60)).astype(int))
        x = torch.zeros((len(some), n), dtype=dtype, device=DEV)
        for t, g in enumerate(some):
            x[t, g * (group or n)] = 1
        assert torch.equal(B.q4_linear(x, w).float(), dev(scale[:, some].T))
        # and so do the rows, through the gradient: a power of two is exact in either type
        rows = np.unique(np.linspace(0, m - 1, 60).astype(int))
        dy = torch.zeros((len(rows), m), dtype=dtype, device=DEV)
        dy[torch.arange(len(rows)), torch.from_numpy(rows)] = 1
        assert torch.equal(B.q4_linear_grad(dy, w).float(), dev(scale[rows][:, np.arange(n) // (group or n)]))
