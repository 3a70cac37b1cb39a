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


def kept(call, inputs, out_grad=None):
    """The gradients of a call's result, or of its sum, in a kept graph."""
    y = call(*inputs)
    return torch.autograd.grad(y.sum() if out_grad is None else y, inputs, out_grad, create_graph=True)


def single_calls():
    """Each call that has a first derivative only, its inputs, and the gradients of its sum."""
    T, E, k, n = 40, 8, 2, 96
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(1)).to(DEV)
    r = B.moe_route(logits, k)
    a, b, ys = (tokens(T * k, n, BF16, i) for i in (1, 2, 3))
    ones, rows = torch.ones((T, k), device=DEV), torch.ones((T, n), dtype=BF16, device=DEV)
    out = {"dys": torch.zeros_like(ys), "dweights": torch.empty_like(r["weights"])}
    yield "moe_route", lambda l: B.moe_route(l, k)["weights"], [logits], [B.moe_route_grad(ones, r["weights"], r["ids"], E)]
    yield ("moe_combine", lambda y, w: B.moe_combine(y, r["place"], w), [ys, r["weights"]],
           list(B.moe_combine_grad(rows, ys, r["place"], r["weights"], out=out).values()))
    yield "gated_act", lambda a, b: B.gated_act(a, b), [a, b], list(B.gated_act_grad(torch.ones_like(a), *B.gated_act(a, b, checkpoint=True)[1:]))
    w = [pack(*make_layer(*v, 64, i, lead=(E,)), 64) for i, v in enumerate(((64, n), (64, n), (n, 64)))]
    x = tokens(T, n, BF16, 4)
    p = [x.clone().requires_grad_(), logits.clone().requires_grad_()]
    B.q4_moe_layer(*p, *w, k).sum().backward()
    yield "q4_moe_layer", lambda x, l: B.q4_moe_layer(x, l, *w, k), [x, logits], [v.grad for v in p]


def test_second_derivatives_are_refused_where_the_graph_is_kept():
    """A loss that is linear in the result brings a gradient that requires none itself,
    and the call's gradients depend on its inputs all the same."""
    for name, call, plain, want in single_calls():
        inputs = [v.clone().requires_grad_() for v in plain]
        got = kept(call, inputs)
        for a, b in zip(got, want):                               # the first derivative is what it is without the graph
            assert torch.equal(a.detach(), b), name
        other = sum(v.float().square().sum() for v in inputs)     # a term that has its own way to every input
        for i, v in enumerate(got):
            assert v.requires_grad, (name, i)
            for x in inputs:
                with pytest.raises(RuntimeError, match=f"{name}.* no second derivative"):
                    torch.autograd.grad(v.float().square().sum() + other, x, retain_graph=True)
            with pytest.raises(RuntimeError, match="no second derivative"):
                (v.float().square().sum() + other).backward(retain_graph=True)
        other.backward()                                          # what does not go through them is there
        for x in inputs:
            assert torch.equal(x.grad, 2 * x.detach())


def test_second_derivatives_are_refused_where_the_gradient_requires_one():
    for name, call, plain, want in single_calls():
        inputs = [v.clone().requires_grad_() for v in plain]
        y = call(*inputs)
        g = torch.ones_like(y).requires_grad_()
        with pytest.raises(RuntimeError, match="second derivative"):
            got = torch.autograd.grad(y, inputs, g, create_graph=True)
            torch.autograd.grad(sum(v.float().sum() for v in got), g)


def test_gradients_that_are_not_needed_are_none_in_a_kept_graph():
    for name, call, plain, want in single_calls():
        for i in range(len(plain)):
            inputs = [v.clone().requires_grad_(i == j) for j, v in enumerate(plain)]
            got, = torch.autograd.grad(call(*inputs).sum(), inputs[i], create_graph=True)
            assert torch.equal(got.detach(), want[i]), name


def test_calls_without_a_gradient_refuse_tensors_that_require_one():
    """New results and given ones (the native way), every floating input in turn."""
    T, E, k, n = 40, 8, 2, 96
    r = B.moe_route(torch.randn((T, E), generator=torch.Generator().manual_seed(1)).to(DEV), k)
    x, ys, dy, g = tokens(T * k, n, BF16, 1), tokens(T * k, n, BF16, 2), tokens(T, n, BF16, 3), torch.rand((T, k), device=DEV)
    ck = B.ck8_pack(x)
    e = torch.empty_like
    calls = [
        (lambda v, out: B.moe_route_grad(*v, r["ids"], E, out=out), [g, r["weights"]], lambda: torch.empty((T, E), device=DEV)),
        (lambda v, out: B.moe_combine_grad(v[0], v[1], r["place"], v[2], out=out), [dy, ys, r["weights"]],
         lambda: {"dys": e(ys), "dweights": e(g)}),
        (lambda v, out: B.gated_act_grad(v[0], ck, ck, out=out), [x], lambda: (e(x), e(x))),
        (lambda v, out: B.ck8_pack(v[0], out=out), [x], lambda: B.Checkpoint8.empty(T * k, n, BF16, DEV)),
    ]
    for call, inputs, out in calls:
        for given in (lambda: None, out):
            call(inputs, given())
            for i in range(len(inputs)):
                v = [t.clone().requires_grad_(i == j) for j, t in enumerate(inputs)]
                with pytest.raises(ValueError, match="has no gradient"):
                    call(v, given())
                with torch.no_grad():
                    call(v, given())


class Cut(torch.autograd.Function):
    """Its input as it is, and no gradient for it."""

    @staticmethod
    def forward(ctx, x):
        return x.clone()

    @staticmethod
    def backward(ctx, g):
        return None


def test_a_result_without_a_gradient():
    for name, call, plain, _ in single_calls():
        inputs = [v.clone().requires_grad_() for v in plain]
        other = sum(v.float().square().sum() for v in inputs)
        (Cut.apply(call(*inputs)).sum() + other).backward()
        for x in inputs:
            assert torch.equal(x.grad, 2 * x.detach()), name


def test_saved_tensors_kept_elsewhere_or_made_again():
    """Under activation checkpointing, with saved tensors moved to the host, and for a graph
    that is gone through twice."""
    from torch.utils.checkpoint import checkpoint
    for name, call, plain, want in single_calls():
        def gradients(run, times=1):
            inputs = [v.clone().requires_grad_() for v in plain]
            loss = run(*inputs).sum()
            for i in range(times):
                got = torch.autograd.grad(loss, inputs, retain_graph=i + 1 < times)
                for a, b in zip(got, want):
                    assert torch.equal(a, b), name
        gradients(lambda *v: checkpoint(call, *v, use_reentrant=False))
        gradients(call, 2)
        with torch.autograd.graph.save_on_cpu():
            gradients(call)
            inputs = [v.clone().requires_grad_() for v in plain]
            got = torch.autograd.grad(call(*inputs).sum(), inputs, create_graph=True)
        with pytest.raises(RuntimeError, match="no second derivative"):
            torch.autograd.grad(got[0].float().square().sum(), inputs[0])
