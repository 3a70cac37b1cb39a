"""A stack's layers one by one: an expert layer for more tokens than q4_moe
takes, expert by expert through q4_linear."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_q4 import LINEAR, close, make_layer, make_moe, moe64, pack, rms, tokens, weights64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [0, 64])
def test_a_layer_of_a_stack(group):
    m, n, E = 33, 200, 5
    stack = make_layer(m, n, group, 51, (E,))
    w, ref = pack(*stack, group), weights64(*stack, group)
    x = tokens(70, n, torch.float16, 1)
    assert len(w) == E
    for e in range(E):
        one = w[e]
        assert (one.count, one.m, one.n, one.group_size) == (1, m, n, w.group_size)
        close(B.q4_linear(x, one), x.double().cpu().numpy() @ ref[e].T, torch.float16, LINEAR)
        assert torch.equal(B.q4_linear(x[:3], one), B.q4_linear(x[:3], pack(*(v[e] for v in stack), group)))
    for e in (-1, E):
        with pytest.raises(IndexError):
            w[e]
    assert [v.m for v in w] == [m] * E


def test_experts_for_a_prompt():
    T, h, f, E, k, group = 150, 128, 192, 6, 2, 64
    dtype = torch.bfloat16
    x, router, layers = make_moe(T, h, f, E, k, group, dtype, 52)
    gate, up, down = (pack(*v, group) for v in layers)
    logits = x.float() @ router.float().t()
    top, ids = logits.sort(dim=1, descending=True, stable=True)
    p, ids = torch.softmax(top[:, :k], 1), ids[:, :k]
    y = torch.zeros((T, h), device=x.device)
    for e in range(E):
        t, j = torch.where(ids == e)
        if len(t):
            a = torch.nn.functional.silu(B.q4_linear(x[t], gate[e]).float()) * B.q4_linear(x[t], up[e]).float()
            y[t] += p[t, j, None] * B.q4_linear(a.to(dtype), down[e]).float()
    ref, want, _ = moe64(x.double().cpu().numpy(), router.double().cpu().numpy(), *(weights64(*v, group) for v in layers), k)
    assert np.array_equal(ids.cpu().numpy(), want)
    # gate and up are rounded to 2^-8 of themselves, their product once more, and
    # every down product: four roundings of at most 2^-8, each independent from
    # term to term, the root of the sum of their squares six times
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= 6 * 2 * 2.0 ** -8 * rms(ref)).all()
