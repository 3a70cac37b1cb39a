"""The Python side of the expert layer for many tokens on the CPU: what it
refuses and what it hands to the library."""
import copy
import pickle

import pytest
import torch

import two_sided_hessian_amd as B
from test_q4_binding import OnDevice, layer
from two_sided_hessian_amd import moe, q4

I32, F32, BF16, FP16 = torch.int32, torch.float32, torch.bfloat16, torch.float16
NAMES = ["bakron_moe_route", "bakron_moe_route_grad", "bakron_moe_gather", "bakron_moe_combine", "bakron_moe_combine_grad",
         "bakron_q4_experts", "bakron_q4_experts_grad", "bakron_ck8_pack", "bakron_ck8_unpack", "bakron_gated_act",
         "bakron_gated_act_grad"]


class Calls:
    """What reaches the library, and the device that is current then."""

    def __init__(self, monkeypatch, current=0):
        self.made, self.current = [], current
        for name in NAMES:
            monkeypatch.setitem(q4._calls, name, self.call(name))
        monkeypatch.setattr(moe, "_raw_stream", lambda index: 1000 + index)
        monkeypatch.setattr(moe, "_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", self.device)

    def call(self, name):
        return lambda *args: self.made.append((name, self.current, args[-1])) or 0

    def device(self, index):
        calls = self

        class Guard:
            def __enter__(self):
                self.before, calls.current = calls.current, index

            def __exit__(self, *_):
                calls.current = self.before
        return Guard()


def on(at, *shape, dtype=BF16):
    return OnDevice.make(at, *shape, dtype=dtype)


def checkpoint(at, rows, cols, dtype=BF16):
    return moe.Checkpoint8(on(at, B.lib().bakron_ck8_bytes(rows, cols), dtype=torch.uint8), rows, cols, dtype)


def every_call(at, **other):
    """Each public call on tensors of device `at` (those named in `other`: on
    that one), as (name in the library, function)."""
    def t(name, *shape, dtype=BF16):
        return on(other.get(name, at), *shape, dtype=dtype)
    T, E, k, n, R = 3, 8, 2, 128, 6
    place, weights, ids = t("place", T, k, dtype=I32), t("weights", T, k, dtype=F32), t("ids", T, k, dtype=I32)
    x, ys = t("x", T, n), t("ys", R, n)
    ws = t("ws", 1 << 20, dtype=torch.uint8)
    w = layer(other.get("w", at), 64, n, E)
    ck = checkpoint(other.get("ck", at), R, n)
    offsets = t("offsets", E + 1, dtype=I32)
    five = {"ids": ids, "weights": weights, "place": place, "order": t("order", T * k, dtype=I32), "offsets": offsets}
    return [
        ("bakron_moe_route", lambda: B.moe_route(on(at, T, E, dtype=F32), k, out=five, ws=ws)),
        ("bakron_moe_route_grad", lambda: B.moe_route_grad(on(at, T, k, dtype=F32), weights, on(at, T, k, dtype=I32), E,
                                                           out=t("out", T, E))),
        ("bakron_moe_gather", lambda: B.moe_gather(on(at, T, n), place, out=ys)),
        ("bakron_moe_combine", lambda: B.moe_combine(on(at, R, n), place, weights, out=x)),
        ("bakron_moe_combine_grad", lambda: B.moe_combine_grad(x, on(at, R, n), place, weights, out={
            "dys": ys, "dweights": t("dweights", T, k, dtype=F32)})),
        ("bakron_q4_experts", lambda: B.q4_experts(on(at, R, n), w, offsets, out=t("out", R, 64), ws=ws)),
        ("bakron_q4_experts_grad", lambda: B.q4_experts_grad(on(at, R, 64), w, offsets, out=t("out", R, n), ws=ws)),
        ("bakron_ck8_pack", lambda: B.ck8_pack(on(at, R, n), out=ck)),
        ("bakron_ck8_unpack", lambda: B.ck8_unpack(checkpoint(at, R, n), out=t("out", R, n))),
        ("bakron_gated_act", lambda: B.gated_act(on(at, R, n), t("b", R, n), count=t("count", 1, dtype=I32), out=t("out", R, n),
                                                 checkpoint=(ck, ck))),
        ("bakron_gated_act_grad", lambda: B.gated_act_grad(on(at, R, n), ck, ck, count=t("count", 1, dtype=I32),
                                                           out=(t("out", R, n), on(at, R, n)))),
    ]


def test_kernels_go_to_their_tensors_device(monkeypatch):
    calls = Calls(monkeypatch)
    for at in (0, 1):
        for _, call in every_call(at):
            call()
        assert calls.current == 0
    assert calls.made == [(name, at, 1000 + at) for at in (0, 1) for name in NAMES]


TAKES = {
    "bakron_moe_route": ("ids", "weights", "place", "order", "offsets", "ws"), "bakron_moe_route_grad": ("weights", "out"),
    "bakron_moe_gather": ("place", "ys"), "bakron_moe_combine": ("place", "weights", "x"),
    "bakron_moe_combine_grad": ("place", "weights", "x", "ys", "dweights"), "bakron_q4_experts": ("w", "offsets", "out", "ws"),
    "bakron_q4_experts_grad": ("w", "offsets", "out", "ws"), "bakron_ck8_pack": ("ck",), "bakron_ck8_unpack": ("out",),
    "bakron_gated_act": ("b", "count", "out", "ck"), "bakron_gated_act_grad": ("ck", "count", "out"),
}


def test_tensors_of_two_devices_are_refused(monkeypatch):
    calls = Calls(monkeypatch)
    for name in NAMES:
        for tensor in TAKES[name]:
            with pytest.raises(ValueError, match="on"):
                dict(every_call(0, **{tensor: 1}))[name]()
    assert not calls.made


def test_a_stream_of_another_device_is_refused(monkeypatch):
    calls = Calls(monkeypatch)

    class Stream:
        device_index, cuda_stream = 1, 5
    s = Stream()
    place, weights = on(0, 3, 2, dtype=I32), on(0, 3, 2, dtype=F32)
    x, ys, w, ck = on(0, 3, 128), on(0, 6, 128), layer(0, 64, 128, 8), checkpoint(0, 6, 128)
    for call, args in ((B.moe_route, (on(0, 3, 8), 2)), (B.moe_route_grad, (weights, weights, place, 8)), (B.moe_gather, (x, place)),
                       (B.moe_combine, (ys, place)), (B.moe_combine_grad, (x, ys, place, weights)),
                       (B.q4_experts, (ys, w, on(0, 9, dtype=I32))), (B.q4_experts_grad, (on(0, 6, 64), w, on(0, 9, dtype=I32))),
                       (B.ck8_pack, (ys,)), (B.ck8_unpack, (ck,)), (B.gated_act, (ys, ys)), (B.gated_act_grad, (ys, ck, ck))):
        with pytest.raises(ValueError, match="stream is on"):
            call(*args, stream=s)
    assert not calls.made


def test_shapes_and_types_are_refused(monkeypatch):
    calls = Calls(monkeypatch)
    place, weights = on(0, 3, 2, dtype=I32), on(0, 3, 2, dtype=F32)
    x, ys, w, ck = on(0, 3, 128), on(0, 6, 128), layer(0, 64, 128, 8), checkpoint(0, 6, 128)
    offsets = on(0, 9, dtype=I32)
    wide = OnDevice.make(0, 6, 256)
    bad = [
        lambda: B.moe_route(on(0, 3, 8, dtype=torch.float64), 2), lambda: B.moe_route(on(0, 3, 8), 0),
        lambda: B.moe_route(on(0, 3, 8), 17), lambda: B.moe_route(on(0, 24), 2), lambda: B.moe_route(torch.zeros(3, 8), 2),
        lambda: B.moe_route_grad(weights, weights, place, 1), lambda: B.moe_route_grad(weights, weights, place, 257),
        lambda: B.moe_route_grad(weights, on(0, 3, 3, dtype=F32), place, 8),
        lambda: B.moe_route_grad(weights, weights, place, 8, dtype=torch.float64),
        lambda: B.moe_gather(x, on(0, 4, 2, dtype=I32)), lambda: B.moe_gather(x, on(0, 3, 33, dtype=I32)),
        lambda: B.moe_gather(x, on(0, 3, 2, dtype=torch.int64)), lambda: B.moe_gather(x, place, out=on(0, 6, 127)),
        lambda: B.moe_gather(x, place, out=on(0, 6, 128, dtype=FP16)), lambda: B.moe_gather(on(0, 3, 128, dtype=F32), place),
        lambda: B.moe_combine(ys, place, on(0, 3, 1, dtype=F32)), lambda: B.moe_combine(ys, place, on(0, 3, 2)),
        lambda: B.moe_combine(ys, place, weights, out=on(0, 4, 128)),
        lambda: B.moe_combine(ys.t(), place, weights),
        lambda: B.moe_combine_grad(on(0, 4, 128), ys, place, weights),
        lambda: B.moe_combine_grad(x, ys, place, weights, out={"dys": on(0, 5, 128), "dweights": weights}),
        lambda: B.q4_experts(ys, w, on(0, 8, dtype=I32)), lambda: B.q4_experts(ys, w, on(0, 9, dtype=torch.int64)),
        lambda: B.q4_experts(on(0, 6, 127), w, offsets), lambda: B.q4_experts(ys, "w", offsets),
        lambda: B.q4_experts(ys, w, offsets, out=on(0, 5, 64)), lambda: B.q4_experts_grad(ys, w, offsets),
        lambda: B.ck8_pack(on(0, 6, 128, dtype=F32)), lambda: B.ck8_pack(ys, out=checkpoint(0, 6, 96)),
        lambda: B.ck8_pack(ys, out=checkpoint(0, 6, 128, FP16)), lambda: B.ck8_unpack(ys),
        lambda: B.ck8_unpack(ck, out=on(0, 6, 127)), lambda: B.ck8_unpack(ck, dtype=torch.float64),
        lambda: B.gated_act(ys, on(0, 6, 127)), lambda: B.gated_act(ys, on(0, 6, 128, dtype=FP16)),
        lambda: B.gated_act(ys, ys, act="relu"), lambda: B.gated_act(ys, ys, count=on(0, 2, dtype=I32)),
        lambda: B.gated_act(ys, ys, checkpoint=(ck, checkpoint(0, 5, 128))),
        lambda: B.gated_act_grad(ys, ck, checkpoint(0, 6, 128, FP16)), lambda: B.gated_act_grad(ys, ck, ys),
        lambda: B.gated_act_grad(ys, ck, ck, out=(ys, on(0, 6, 127))),
        lambda: B.gated_act(wide[:, ::2], ys), lambda: B.Checkpoint8.empty(5, 65537, BF16, "cpu"),
        lambda: B.Checkpoint8.empty(5, 64, F32, "cpu"),
        lambda: B.q4_moe_layer(x, on(0, 3, 7), w, w, layer(0, 128, 64, 8), 2),
        lambda: B.q4_moe_layer(x, on(0, 4, 8), w, w, layer(0, 128, 64, 8), 2),
        lambda: B.q4_moe_layer(x, on(0, 3, 8), w, w, layer(0, 128, 63, 8), 2),
        lambda: B.q4_moe_layer(x, on(0, 3, 8), w, layer(0, 64, 128, 7), layer(0, 128, 64, 8), 2),
        lambda: B.q4_moe_layer(x, on(0, 3, 8), w, w, layer(0, 128, 64, 8), 9),
        lambda: B.q4_moe_layer(x, on(0, 3, 8), w, w, layer(0, 128, 64, 8), 2, act="tanh"),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} was not refused")
    assert not calls.made


def test_a_workspace_has_all_the_bytes_that_it_counts(monkeypatch):
    calls = Calls(monkeypatch)
    w, offsets = layer(0, 64, 128, 8), on(0, 9, dtype=I32)
    for call in (lambda ws: B.q4_experts(on(0, 3000, 128), w, offsets, ws=ws), lambda ws: B.moe_route(on(0, 3000, 8), 2, ws=ws),
                 lambda ws: B.q4_experts_grad(on(0, 3000, 64), w, offsets, ws=ws)):
        for ws in (on(0, 1, dtype=torch.uint8).expand(1 << 20), on(0, 1 << 20, dtype=torch.uint8)[::2]):
            ws.at = 0
            with pytest.raises(ValueError, match="contiguous"):
                call(ws)
    assert not calls.made


def test_a_checkpoint_has_all_the_bytes_that_it_counts(monkeypatch):
    calls = Calls(monkeypatch)
    x, whole = on(0, 6, 128), checkpoint(0, 6, 128)
    need = whole.data.numel()
    apart = on(0, 2 * need, dtype=torch.uint8)[::2]
    apart.at = 0
    for data in (on(0, need - 1, dtype=torch.uint8), on(0, 0, dtype=torch.uint8), apart, on(1, need, dtype=torch.uint8),
                 torch.zeros(need, dtype=torch.uint8)):
        bad = B.Checkpoint8(data, 6, 128, BF16)
        for call in (lambda: B.ck8_pack(x, out=bad), lambda: B.gated_act(x, x, checkpoint=(whole, bad)),
                     lambda: B.gated_act_grad(x, bad, whole), lambda: B.gated_act_grad(x, whole, bad, out=(x, x))):
            with pytest.raises(ValueError):
                call()
        if data.get_device() != 1:
            with pytest.raises((ValueError, TypeError)):
                B.ck8_unpack(bad)
    assert not calls.made


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))])
def test_a_copied_checkpoint_has_its_own_data(again):
    c = B.Checkpoint8(torch.arange(64, dtype=torch.uint8), 2, 20, BF16)
    v = again(c)
    assert torch.equal(v.data, c.data) and (v.rows, v.cols, v.dtype) == (2, 20, BF16) and repr(v) == repr(c)
