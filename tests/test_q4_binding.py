"""The Python side of the 4-bit layer calls on the CPU: what it holds and what
it hands to the library."""
import copy
import pickle

import pytest
import torch

from two_sided_hessian_amd import q4


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda w: pickle.loads(pickle.dumps(w))])
def test_a_copied_layer_points_at_its_own_data(again):
    w = q4.Q4Weight(torch.arange(1024, dtype=torch.uint8), 1, 16, 128, 64)
    v = again(w)
    assert torch.equal(v.data, w.data) and (v.count, v.m, v.n, v.group_size) == (1, 16, 128, 64)
    assert v.device == w.device and repr(v) == repr(w)
    # no address or device beside the data's: nothing of the original's is used for the copy
    assert not any(getattr(v, k) == w.data.data_ptr() for k in v.__slots__ if isinstance(getattr(v, k), int))
    v.data = v.data.clone().to(torch.device("meta"))
    assert v.device.type == "meta"


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on GPU `at`; the library's calls, which
    would take its address, are replaced."""
    at = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.at

    @staticmethod
    def make(at, *shape, dtype=torch.bfloat16):
        t = torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)
        t.at = at
        return t

    def new_empty(self, shape, dtype=None):
        return OnDevice.make(self.at, *shape, dtype=dtype or self.dtype)


def layer(at, m, n, count=1):
    data = OnDevice.make(at, 16, dtype=torch.uint8)
    return q4.Q4Weight(data, count, m, n, 64)


class Calls:
    """What reaches the library, and the device that is current then."""

    def __init__(self, monkeypatch, current=0):
        self.made, self.current = [], current
        for name in ("bakron_q4_pack", "bakron_q4_linear", "bakron_q4_linear_grad", "bakron_q4_moe"):
            monkeypatch.setitem(q4._calls, name, self.call(name))
        monkeypatch.setattr(q4, "_raw_stream", lambda index: 1000 + index)
        monkeypatch.setattr(q4, "_device", lambda: self.current, raising=False)
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


def test_kernels_go_to_their_tensors_device(monkeypatch):
    calls = Calls(monkeypatch)
    for at in (0, 1):
        x, w = OnDevice.make(at, 3, 128), layer(at, 64, 128)
        ws = OnDevice.make(at, 1 << 20, dtype=torch.uint8)
        q4.q4_linear(x, w, ws=ws)
        q4.q4_linear_grad(OnDevice.make(at, 3, 64), w, ws=ws)
        gate, up, down = layer(at, 64, 128, 4), layer(at, 64, 128, 4), layer(at, 128, 64, 4)
        q4.q4_moe(x, OnDevice.make(at, 4, 128), gate, up, down, 2, ws=ws)
        assert calls.current == 0
    names = ["bakron_q4_linear", "bakron_q4_linear_grad", "bakron_q4_moe"]
    assert calls.made == [(name, at, 1000 + at) for at in (0, 1) for name in names]


def test_tensors_of_two_devices_are_refused(monkeypatch):
    calls = Calls(monkeypatch)
    x, w = OnDevice.make(0, 3, 128), layer(0, 64, 128)
    ws = OnDevice.make(0, 1 << 20, dtype=torch.uint8)
    router, gate, up, down = OnDevice.make(0, 4, 128), layer(0, 64, 128, 4), layer(0, 64, 128, 4), layer(0, 128, 64, 4)

    def out(**at):
        return {"y": OnDevice.make(at.get("y", 0), 3, 128), "ids": OnDevice.make(at.get("ids", 0), 3, 2, dtype=torch.int32),
                "weights": OnDevice.make(at.get("weights", 0), 3, 2, dtype=torch.float32)}
    q4.q4_moe(x, router, gate, up, down, 2, ws=ws, out=out())
    assert len(calls.made) == 1
    for bad in ("y", "ids", "weights"):
        with pytest.raises(ValueError, match="cuda:0"):
            q4.q4_moe(x, router, gate, up, down, 2, ws=ws, out=out(**{bad: 1}))
    with pytest.raises(ValueError, match="router"):
        q4.q4_moe(x, OnDevice.make(1, 4, 128), gate, up, down, 2, ws=ws)
    with pytest.raises(ValueError):
        q4.q4_linear(x, layer(1, 64, 128), ws=ws)
    with pytest.raises(ValueError):
        q4.q4_linear(x, w, ws=ws, out=OnDevice.make(1, 3, 64))
    codes, grid = OnDevice.make(0, 64, 128, dtype=torch.uint8), OnDevice.make(0, 64, 2, dtype=torch.float32)
    for scale, zero in ((OnDevice.make(1, 64, 2, dtype=torch.float32), grid), (grid, OnDevice.make(1, 64, 2, dtype=torch.float32))):
        with pytest.raises(ValueError, match="is on"):
            q4.q4_pack(codes, scale, zero, group_size=64, check=False)

    class Stream:
        device_index, cuda_stream = 1, 5
    for call, args in ((q4.q4_linear, (x, w)), (q4.q4_linear_grad, (OnDevice.make(0, 3, 64), w)),
                       (q4.q4_moe, (x, router, gate, up, down, 2)), (q4.q4_pack, (codes, grid, grid))):
        kw = {"group_size": 64, "check": False} if call is q4.q4_pack else {"ws": ws}
        with pytest.raises(ValueError, match="stream is on"):
            call(*args, stream=Stream(), **kw)
    assert len(calls.made) == 1


def test_a_workspace_has_all_the_bytes_that_it_counts(monkeypatch):
    calls = Calls(monkeypatch)
    x, w = OnDevice.make(0, 300, 128), layer(0, 64, 128)
    for call, v in ((q4.q4_linear, x), (q4.q4_linear_grad, OnDevice.make(0, 300, 64))):
        for ws in (OnDevice.make(0, 1, dtype=torch.uint8).expand(1 << 20), OnDevice.make(0, 1 << 20, dtype=torch.uint8)[::2]):
            ws.at = 0
            with pytest.raises(ValueError, match="contiguous"):
                call(v, w, ws=ws)
    assert not calls.made
