"""Autograd of the expert layer's calls where a graph is kept of the backward pass
itself: what its results hold, and what cannot be differentiated twice."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_q4 import DEV, make_layer, pack, tokens
from test_gpu_q4_experts import spread

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def stale(*shapes):
    """Freed blocks of these sizes hold NaN, which a new tensor of that size then begins with."""
    for t in [torch.full(s, float("nan"), dtype=BF16, device=DEV) for s in shapes for _ in range(4)]:
        del t


def test_gradients_of_rows_that_no_expert_has_are_zeros_in_a_kept_graph():
    """First derivatives taken with create_graph, and the derivative of those, in both
    directions: sorted rows before the first expert's and behind the last one's."""
    R, E, m, n = 130, 5, 200, 330
    w = pack(*make_layer(m, n, 64, 21, lead=(E,)), 64)
    offsets = spread(R, E, 6, tail=9).astype(np.int32)
    for at in (offsets, np.maximum(offsets, 7)):
        at, first, last = torch.from_numpy(at).to(DEV), int(at[0]), int(at[-1])
        for call, back, cin, cout in ((B.q4_experts, B.q4_experts_grad, n, m), (B.q4_experts_grad, B.q4_experts, m, n)):
            x = tokens(R, cin, BF16, 1).requires_grad_()
            v = tokens(R, cout, BF16, 2).requires_grad_()
            y = call(x, w, at)
            stale((R, cin), (R, cout))
            dx, = torch.autograd.grad(y, x, v, create_graph=True)
            assert dx.requires_grad
            assert torch.equal(dx, back(v.detach(), w, at, out=torch.zeros_like(x)))
            assert (dx[:first] == 0).all() and (dx[last:] == 0).all()
            g = tokens(R, cin, BF16, 3).requires_grad_()
            stale((R, cin), (R, cout))
            dv, = torch.autograd.grad(dx, v, g, create_graph=True)
            assert torch.equal(dv, call(g.detach(), w, at, out=torch.zeros_like(v)))
            stale((R, cin), (R, cout))
            dg, = torch.autograd.grad(dv, g, v.detach())
            assert torch.equal(dg, dx)
