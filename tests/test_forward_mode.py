"""Forward-mode autograd: the layers' calls have no derivative there, and refuse dual
tensors instead of dropping their tangents."""
import pytest
import torch
from torch.autograd import forward_ad

import two_sided_hessian_amd as B
from two_sided_hessian_amd import moe

I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16
T, E, K, N, M = 3, 8, 2, 128, 64
R = T * K


def layer_calls(t, w, w_down, ck):
    """Every public call with floating inputs: (name, function of those, the inputs).  t(name, *shape,
    dtype) makes a tensor, w and w_down are stacks, ck a checkpoint of R x N."""
    place, ids, offsets = (t("ints", *s, dtype=I32) for s in ((T, K), (T, K), (E + 1,)))
    x, ys, dm, logits, weights = t("x", T, N), t("ys", R, N), t("dm", R, M), t("logits", T, E, dtype=F32), t("weights", T, K, dtype=F32)
    five = {"ids": ids, "weights": t("out", T, K, dtype=F32), "place": place, "order": t("ints", R, dtype=I32), "offsets": offsets}
    return [
        ("q4_linear", lambda x: B.q4_linear(x, w[0]), [x]), ("q4_linear_grad", lambda x: B.q4_linear_grad(x, w[0]), [dm]),
        ("q4_moe", lambda x, r: B.q4_moe(x, r, w, w, w_down, K), [x, t("router", E, N)]),
        ("moe_route", lambda l: B.moe_route(l, K), [logits]),
        ("moe_route, given", lambda l: B.moe_route(l, K, out=five), [logits]),
        ("moe_route_grad", lambda g, p: B.moe_route_grad(g, p, ids, E), [t("g", T, K, dtype=F32), weights]),
        ("moe_route_grad, given", lambda g, p: B.moe_route_grad(g, p, ids, E, out=t("out", T, E)), [t("g", T, K, dtype=F32), weights]),
        ("moe_gather", lambda x: B.moe_gather(x, place), [x]),
        ("moe_gather, given", lambda x: B.moe_gather(x, place, out=t("out", R, N)), [x]),
        ("moe_combine", lambda y, p: B.moe_combine(y, place, p), [ys, weights]),
        ("moe_combine, given", lambda y, p: B.moe_combine(y, place, p, out=t("out", T, N)), [ys, weights]),
        ("moe_combine_grad", lambda g, y, p: B.moe_combine_grad(g, y, place, p), [x, ys, weights]),
        ("moe_combine_grad, given", lambda g, y, p: B.moe_combine_grad(g, y, place, p, out={"dys": t("out", R, N), "dweights": t("out", T, K, dtype=F32)}),
         [x, ys, weights]),
        ("q4_experts", lambda x: B.q4_experts(x, w, offsets), [ys]),
        ("q4_experts, given", lambda x: B.q4_experts(x, w, offsets, out=t("out", R, M)), [ys]),
        ("q4_experts_grad", lambda x: B.q4_experts_grad(x, w, offsets), [dm]),
        ("q4_experts_grad, given", lambda x: B.q4_experts_grad(x, w, offsets, out=t("out", R, N)), [dm]),
        ("ck8_pack", lambda x: B.ck8_pack(x), [ys]), ("ck8_pack, given", lambda x: B.ck8_pack(x, out=ck), [ys]),
        ("gated_act", lambda a, b: B.gated_act(a, b), [ys, t("b", R, N)]),
        ("gated_act, given", lambda a, b: B.gated_act(a, b, out=t("out", R, N)), [ys, t("b", R, N)]),
        ("gated_act_grad", lambda g: B.gated_act_grad(g, ck, ck), [ys]),
        ("gated_act_grad, given", lambda g: B.gated_act_grad(g, ck, ck, out=(t("out", R, N), t("out", R, N))), [ys]),
        ("q4_moe_layer", lambda x, l: B.q4_moe_layer(x, l, w, w, w_down, K), [x, logits]),
    ]


def refused(calls):
    for name, call, inputs in calls:
        for i in range(len(inputs)):
            with forward_ad.dual_level():
                v = [forward_ad.make_dual(x, torch.ones_like(x)) if i == j else x for j, x in enumerate(inputs)]
                for grad in (True, False):                        # torch.no_grad does not switch forward mode off
                    with torch.set_grad_enabled(grad), pytest.raises(ValueError, match="forward-mode"):
                        call(*v)
                        pytest.fail(f"{name}: input {i} was not refused")


def test_dual_tensors_are_refused_before_anything_is_enqueued(monkeypatch):
    from test_moe_binding import Calls, checkpoint, layer, on
    calls = Calls(monkeypatch)
    ck = checkpoint(0, R, N)
    each = layer_calls(lambda _, *shape, dtype=BF16: on(0, *shape, dtype=dtype), layer(0, M, N, E), layer(0, N, M, E), ck)
    refused([c for c in each if not c[0].startswith("q4_linear")])   # (one layer of a stack: with its bytes, below)
    assert not calls.made


@pytest.mark.gpu
def test_dual_tensors_are_refused_by_every_call():
    from test_gpu_q4 import DEV, make_layer, pack
    w, w_down = (pack(*make_layer(*s, 64, 1, lead=(E,)), 64) for s in ((M, N), (N, M)))

    def t(name, *shape, dtype=BF16):
        if name == "ints":   # a choice that exists: expert, place and offset 0
            return torch.zeros(shape, dtype=dtype, device=DEV)
        return torch.rand(shape, generator=torch.Generator().manual_seed(1)).to(DEV, dtype)
    calls = layer_calls(t, w, w_down, B.ck8_pack(t("ck", R, N)))
    refused(calls)
    with forward_ad.dual_level():                                 # inside a level, tensors without a tangent are taken
        for name, call, inputs in calls:
            call(*inputs)
    for name, call, inputs in calls:
        call(*inputs)
    x, place, out = t("x", T, N), t("ints", T, K, dtype=I32), t("out", R, N)
    with forward_ad.dual_level():
        assert moe._fast.gather(forward_ad.make_dual(x, x), place, out) is False
        assert moe._fast.gather(x, place, out) is True
