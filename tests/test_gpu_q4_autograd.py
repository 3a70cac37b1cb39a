"""Autograd through the 4-bit linear layer: its gradient is q4_linear_grad, that
one's q4_linear; what has no gradient says so."""
import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_q4 import make_layer, make_moe, pack, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40, 130])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradients_of_the_layer_and_of_its_gradient(T, dtype):
    m, n, group = 200, 330, 64
    w = pack(*make_layer(m, n, group, 21), group)
    for call, back, cin, cout in ((B.q4_linear, B.q4_linear_grad, n, m), (B.q4_linear_grad, B.q4_linear, m, n)):
        plain = tokens(T, cin, dtype, 1, pad=5)
        x = plain.detach().requires_grad_()
        g = tokens(T, cout, dtype, 2)
        y = call(x, w)
        assert y.requires_grad and torch.equal(y, call(plain, w))
        y.backward(g)
        assert torch.equal(x.grad, back(g, w))
        # through other operators, with an expanded gradient
        x.grad = None
        (2 * call(x * 1, w)).sum().backward()
        assert torch.equal(x.grad, back(torch.full((T, cout), 2.0, dtype=dtype, device=x.device), w))
        # the derivative of the derivative
        v = g.clone().requires_grad_()
        dx, = torch.autograd.grad(call(x, w), x, v, create_graph=True)
        dv, = torch.autograd.grad(dx, v, plain)
        assert torch.equal(dv, call(plain, w))
        with torch.no_grad():
            out = torch.empty_like(y)
            assert not call(x, w).requires_grad and call(x, w, out=out) is out
        with pytest.raises(ValueError, match="gradient"):
            call(x, w, out=torch.empty_like(y))


def test_experts_have_no_gradient():
    x, router, layers = make_moe(3, 128, 64, 4, 2, 64, torch.bfloat16, 4)
    w = [pack(*v, 64) for v in layers]
    ref = B.q4_moe(x, router, *w, 2)["y"]
    for a, b in ((x.detach().requires_grad_(), router), (x, router.detach().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            B.q4_moe(a, b, *w, 2)
        with torch.no_grad():
            assert torch.equal(B.q4_moe(a, b, *w, 2)["y"], ref)
