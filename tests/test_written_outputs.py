"""Given outputs count as changed in place: autograd refuses a backward pass that would
read what was saved in them before."""
import pytest
import torch

import two_sided_hessian_amd as B

I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16


def versions(outputs):
    return [t._version for t in outputs]


def test_outputs_given_to_the_checks_in_python(monkeypatch):
    from test_moe_binding import Calls, checkpoint, layer, on
    from test_q4_binding import Calls as LinearCalls
    calls, _ = Calls(monkeypatch), LinearCalls(monkeypatch)
    T, E, k, n, m = 3, 8, 2, 128, 64
    R = T * k
    place, ids, offsets, p = on(0, T, k, dtype=I32), on(0, T, k, dtype=I32), on(0, E + 1, dtype=I32), on(0, T, k, dtype=F32)
    x, ys, dm, w, w1 = on(0, T, n), on(0, R, n), on(0, R, m), layer(0, m, n, E), layer(0, m, n)
    ck = checkpoint(0, R, n)
    five = [on(0, *s, dtype=d) for s, d in (((T, k), I32), ((T, k), F32), ((T, k), I32), ((R,), I32), ((E + 1,), I32))]
    names = ("ids", "weights", "place", "order", "offsets")
    o = {name: on(0, *shape) for name, shape in (("T", (T, n)), ("R", (R, n)), ("R2", (R, n)), ("M", (R, m)), ("L", (T, E)), ("TM", (T, m)))}
    dw, data = on(0, T, k, dtype=F32), [checkpoint(0, R, n) for _ in range(2)]
    ws = on(0, 1 << 20, dtype=torch.uint8)
    for outputs, call in (
            (five, lambda: B.moe_route(on(0, T, E), k, out=dict(zip(names, five)), ws=ws)),
            ([o["L"]], lambda: B.moe_route_grad(p, p, ids, E, out=o["L"])),
            ([o["R"]], lambda: B.moe_gather(x, place, out=o["R"])),
            ([o["T"]], lambda: B.moe_combine(ys, place, p, out=o["T"])),
            ([o["R"], dw], lambda: B.moe_combine_grad(x, ys, place, p, out={"dys": o["R"], "dweights": dw})),
            ([o["M"]], lambda: B.q4_experts(ys, w, offsets, out=o["M"], ws=ws)),
            ([o["R"]], lambda: B.q4_experts_grad(dm, w, offsets, out=o["R"], ws=ws)),
            ([data[0].data], lambda: B.ck8_pack(ys, out=data[0])),
            ([o["R"]], lambda: B.ck8_unpack(ck, out=o["R"])),
            ([o["R"]], lambda: B.gated_act(ys, ys, out=o["R"])),
            ([o["R"], data[0].data, data[1].data], lambda: B.gated_act(ys, ys, out=o["R"], checkpoint=tuple(data))),
            ([o["R"], o["R2"]], lambda: B.gated_act_grad(ys, ck, ck, out=(o["R"], o["R2"]))),
            ([o["TM"]], lambda: B.q4_linear(x, w1, out=o["TM"])), ([o["T"]], lambda: B.q4_linear_grad(o["TM"], w1, out=o["T"])),
            ([o["T"], ids, p], lambda: B.q4_moe(x, on(0, E, n), w, w, layer(0, n, m, E), k, out={"y": o["T"], "ids": ids, "weights": p}, ws=ws))):
        before = versions(outputs)
        call()
        assert versions(outputs) == [v + 1 for v in before]
    assert calls.made


@pytest.mark.gpu
def test_outputs_given_to_every_call():
    from test_gpu_moe_native import calls, outputs, state
    v = state()

    def tensors(o):
        if isinstance(o, B.Checkpoint8):
            return [o.data]
        return [o] if isinstance(o, torch.Tensor) else [t for u in (o.values() if isinstance(o, dict) else o) for t in tensors(u)]
    for kw in ({}, {"stream": torch.cuda.current_stream()}):     # the native way, and that through Python
        o = outputs(v)
        for name, (_, call) in calls(v, o, **kw).items():
            before = versions(tensors(o[name]))
            call()
            assert versions(tensors(o[name])) == [u + 1 for u in before], name
    with torch.inference_mode():                                  # tensors without a count of changes
        for kw in ({}, {"stream": torch.cuda.current_stream()}):
            o = outputs(v)
            for _, call in calls(v, o, **kw).values():
                call()
    for _, call in calls(v, o).values():                          # and written to after it
        call()


@pytest.mark.gpu
def test_a_choice_written_over_before_its_backward_pass_is_refused():
    """Two batches through one set of buffers: the first one's gradient would be taken with
    the second one's choice."""
    from test_gpu_q4 import DEV, tokens
    T, E, k, n = 40, 8, 2, 96
    first, second = (torch.randn((T, E), generator=torch.Generator().manual_seed(i)).to(DEV) for i in (1, 2))
    x, dxs = tokens(T, n, BF16, 1).requires_grad_(), tokens(T * k, n, BF16, 2)
    r = B.moe_route(first, k)
    want, = torch.autograd.grad(B.moe_gather(x, r["place"]), x, dxs)
    for kw in ({}, {"stream": torch.cuda.current_stream()}):
        B.moe_route(first, k, out=r)
        xs = B.moe_gather(x, r["place"])
        B.moe_route(second, k, out=r, **kw)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            xs.backward(dxs)
        B.moe_route(first, k, out=r, **kw)
        got, = torch.autograd.grad(B.moe_gather(x, r["place"]), x, dxs)
        assert torch.equal(got, want)


def test_outputs_that_require_a_gradient_are_refused(monkeypatch):
    from test_moe_binding import Calls, checkpoint, on
    from test_q4_binding import Calls as LinearCalls, layer
    calls, linear = Calls(monkeypatch), LinearCalls(monkeypatch)
    T, E, k, n, m = 3, 8, 2, 128, 64
    place, p = on(0, T, k, dtype=I32), on(0, T, k, dtype=F32)
    x, ys, dm, w, w1 = on(0, T, n), on(0, T * k, n), on(0, T * k, m), layer(0, m, n, E), layer(0, m, n)
    offsets, ws = on(0, E + 1, dtype=I32), on(0, 1 << 20, dtype=torch.uint8)
    ck = checkpoint(0, T * k, n)

    def five(weights):
        return {"ids": on(0, T, k, dtype=I32), "weights": weights, "place": place, "order": on(0, T * k, dtype=I32), "offsets": offsets}
    for shape, dtype, call in (
            ((T, k), F32, lambda o: B.moe_route(on(0, T, E), k, out=five(o), ws=ws)),
            ((T, E), BF16, lambda o: B.moe_route_grad(p, p, place, E, out=o)),
            ((T * k, n), BF16, lambda o: B.moe_gather(x, place, out=o)), ((T, n), BF16, lambda o: B.moe_combine(ys, place, p, out=o)),
            ((T * k, n), BF16, lambda o: B.moe_combine_grad(x, ys, place, p, out={"dys": o, "dweights": on(0, T, k, dtype=F32)})),
            ((T, k), F32, lambda o: B.moe_combine_grad(x, ys, place, p, out={"dys": on(0, T * k, n), "dweights": o})),
            ((T * k, m), BF16, lambda o: B.q4_experts(ys, w, offsets, out=o, ws=ws)),
            ((T * k, n), BF16, lambda o: B.q4_experts_grad(dm, w, offsets, out=o, ws=ws)),
            ((T * k, n), BF16, lambda o: B.ck8_unpack(ck, out=o)), ((T * k, n), BF16, lambda o: B.gated_act(ys, ys, out=o)),
            ((T * k, n), BF16, lambda o: B.gated_act_grad(ys, ck, ck, out=(o, on(0, T * k, n)))),
            ((T * k, n), BF16, lambda o: B.gated_act_grad(ys, ck, ck, out=(on(0, T * k, n), o))),
            ((T, m), BF16, lambda o: B.q4_linear(x, w1, out=o)),
            ((T, n), BF16, lambda o: B.q4_moe(x, on(0, E, n), w, w, layer(0, n, m, E), k, ws=ws, out={"y": o, "ids": place, "weights": p}))):
        out = on(0, *shape, dtype=dtype).requires_grad_()
        with pytest.raises(ValueError, match="out must not require a gradient"):
            call(out)
        assert not calls.made and not linear.made
        with torch.no_grad():
            call(out)
        calls.made.clear(), linear.made.clear()
