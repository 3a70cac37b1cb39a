"""The native way of the expert layer's calls with given outputs
(csrc/fast_calls.cpp): it takes what is in order, to the same results and on the
current stream, and leaves everything else alone."""
import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_q4 import DEV, make_layer, pack, tokens
from two_sided_hessian_amd import moe

pytestmark = pytest.mark.gpu
I32, F32, BF16, FP16 = torch.int32, torch.float32, torch.bfloat16, torch.float16


def state(T=40, E=8, k=2, n=128, m=64):
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(1)).to(DEV)
    r = B.moe_route(logits, k)
    w = pack(*make_layer(m, n, 64, 1, lead=(E,)), 64)
    R = T * k
    v = {"x": tokens(T, n, BF16, 1), "ys": tokens(R, n, BF16, 2), "dy": tokens(T, n, BF16, 3), "dm": tokens(R, m, BF16, 4),
         "b": tokens(R, n, BF16, 5), "g": torch.rand((T, k), device=DEV), "logits": logits, "w": w, "r": r}
    v["ck"] = (B.ck8_pack(v["ys"]), B.ck8_pack(v["b"]))
    return v


def outputs(v):
    """Fresh outputs of every call."""
    def e(*shape, dtype=BF16):
        return torch.full(shape, 7, dtype=dtype, device=DEV)
    (T, n), (R, m), E, k = v["x"].shape, v["dm"].shape, 8, 2
    cks = tuple(B.Checkpoint8(torch.zeros_like(v["ck"][0].data), R, n, BF16) for _ in range(2))
    return {"route": {name: e(*t.shape, dtype=t.dtype) for name, t in v["r"].items()}, "route_grad": e(T, E), "gather": e(R, n),
            "combine": e(T, n), "combine_grad": {"dys": e(R, n), "dweights": e(T, k, dtype=F32)}, "experts": e(R, m),
            "experts_grad": e(R, n), "pack": cks[0], "gated": (e(R, n), cks), "gated_grad": (e(R, n), e(R, n))}


def calls(v, o, **kw):
    """Every call as (native function, its arguments, the public call)."""
    r, w, k = v["r"], v["w"], 2
    count = r["offsets"][-1:]
    return {
        "route": ((v["logits"], k, o["route"], None), lambda: B.moe_route(v["logits"], k, out=o["route"], **kw)),
        "route_grad": ((v["g"], r["weights"], r["ids"], 8, o["route_grad"]),
                       lambda: B.moe_route_grad(v["g"], r["weights"], r["ids"], 8, out=o["route_grad"], **kw)),
        "gather": ((v["x"], r["place"], o["gather"]), lambda: B.moe_gather(v["x"], r["place"], out=o["gather"], **kw)),
        "combine": ((v["ys"], r["place"], r["weights"], o["combine"]),
                    lambda: B.moe_combine(v["ys"], r["place"], r["weights"], out=o["combine"], **kw)),
        "combine_grad": ((v["dy"], v["ys"], r["place"], r["weights"], o["combine_grad"]),
                         lambda: B.moe_combine_grad(v["dy"], v["ys"], r["place"], r["weights"], out=o["combine_grad"], **kw)),
        "experts": ((v["ys"], w, r["offsets"], o["experts"], None), lambda: B.q4_experts(v["ys"], w, r["offsets"], out=o["experts"], **kw)),
        "pack": ((v["ys"], o["pack"]), lambda: B.ck8_pack(v["ys"], out=o["pack"], **kw)),
        "gated": ((v["ys"], v["b"], 0, o["gated"][1], count, o["gated"][0]),
                  lambda: B.gated_act(v["ys"], v["b"], checkpoint=o["gated"][1], count=count, out=o["gated"][0], **kw)),
        "gated_grad": ((v["ys"], *v["ck"], 1, None, *o["gated_grad"]),
                       lambda: B.gated_act_grad(v["ys"], *v["ck"], act="gelu", out=o["gated_grad"], **kw)),
    }


def flat(o):
    if isinstance(o, B.Checkpoint8):
        return [B.ck8_unpack(o)]
    if isinstance(o, torch.Tensor):
        return [o]
    return [t for v in (o.values() if isinstance(o, dict) else o) for t in flat(v)]


def test_it_is_built():
    assert moe._fast is not None


def test_the_same_results():
    v = state()
    native, python = outputs(v), outputs(v)
    for name, (args, _) in calls(v, native).items():
        assert getattr(moe._fast, name)(*args) is True, name
    for _, call in calls(v, python, stream=torch.cuda.current_stream()).values():
        call()
    for name in calls(v, native):
        for a, b in zip(flat(native[name]), flat(python[name])):
            assert torch.equal(a, b), name
    # a call that needs a workspace: declined without one
    x, out = tokens(600, 128, BF16, 6), torch.empty((600, 64), dtype=BF16, device=DEV)
    at = torch.arange(9, dtype=I32, device=DEV) * 75
    need = B.q4_experts_workspace_bytes(600, v["w"])
    args = [x, v["w"], at, out, None]
    assert need and moe._fast.experts(*args) is False
    args[-1] = B.workspace(need, DEV)
    assert moe._fast.experts(*args) is True
    assert torch.equal(out, B.q4_experts(x, v["w"], at))
    args[-1] = B.workspace(need, DEV)[:-256]
    assert moe._fast.experts(*args) is False
    dx = torch.empty_like(v["ys"])
    assert moe._fast.experts_grad(v["dm"], v["w"], v["r"]["offsets"], dx, B.workspace(1 << 20, DEV)) is True
    last = int(v["r"]["offsets"][-1])
    assert torch.equal(dx[:last], B.q4_experts_grad(v["dm"], v["w"], v["r"]["offsets"])[:last])
    # and the public calls return what was given to them
    o = outputs(v)
    got = {name: call() for name, (_, call) in calls(v, o).items()}
    for name in got:
        for a, b in zip(flat(got[name]), flat(native[name])):
            assert torch.equal(a, b), name
    assert got["route"] is o["route"] and got["gather"] is o["gather"] and got["gated"][0] is o["gated"][0]


def spoilt(t):
    """Tensors that a call with t in its place must not take."""
    if t.dim() == 1:
        return [t.cpu(), torch.cat((t, t)), t.double()] + ([torch.stack((t, t), 1)[:, 0]] if t.numel() > 1 else [])
    bad = [t.cpu(), t[:, :-1].contiguous(), t.double(), t[:, None], torch.stack((t, t), 2)[:, :, 0]]
    if t.shape[0] > 1:
        bad += [t[:1].expand(t.shape)]
    if t.is_floating_point():
        bad.append(t.clone().requires_grad_())
        bad.append(t.to(FP16 if t.dtype == BF16 else BF16) if t.dtype != F32 else t.to(torch.float64))
    return bad


def test_it_declines_what_is_not_in_order():
    v = state()
    o = outputs(v)
    for name, (args, _) in calls(v, o).items():
        f = getattr(moe._fast, name)
        assert f(*args) is True and f(*args[:-1]) is False and f(*args, None) is False
        for i, a in enumerate(args):
            if name == "route" and i == 0 or name == "route_grad" and i == 4:
                bad = [a.cpu(), a.double(), a[:, None], a.t()]    # another number of tokens or experts may be what is meant
            elif isinstance(a, torch.Tensor):
                bad = spoilt(a)
                if name == "gather" and i == 1:                   # fewer choices are choices too
                    bad = [b for b in bad if b.shape != (a.shape[0], a.shape[1] - 1)]
            elif isinstance(a, dict):
                bad = [{**a, key: b} for key, t in a.items() for b in spoilt(t)] + [{}, None, tuple(a.values())]
            elif isinstance(a, B.Checkpoint8):
                bad = [B.Checkpoint8(a.data, a.rows - 1, a.cols, a.dtype), B.Checkpoint8(a.data, a.rows, a.cols, FP16), a.data, None,
                       B.Checkpoint8(a.data[:-256], a.rows, a.cols, a.dtype), B.Checkpoint8(a.data.cpu(), a.rows, a.cols, a.dtype)]
            elif isinstance(a, B.Q4Weight):
                bad = [B.Q4Weight(a.data, a.count, a.m, a.n + 1, 64), B.Q4Weight(a.data, a.count, a.m + 1, a.n, 64), a.data, None,
                       B.Q4Weight(a.data.cpu(), a.count, a.m, a.n, 64), B.Q4Weight(a.data, a.count - 1, a.m, a.n, 64)]
            elif isinstance(a, tuple):
                bad = [a[:1], list(a), (a[0], None), True]
            elif isinstance(a, int):
                bad = [-1, "2", 2.0, 1 << 70, 9999]
            else:
                bad = [v["logits"].cpu()]
            for b in bad:
                got = f(*args[:i], b, *args[i + 1:])
                assert got is False, (name, i, getattr(b, "shape", b), getattr(b, "dtype", None))


def test_it_goes_to_the_current_stream_and_into_graphs():
    v = state()
    want = outputs(v)
    for args, call in calls(v, want).values():
        call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = outputs(v)
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)                                 # the default stream is busy
    with torch.cuda.stream(side):
        for name, (args, _) in calls(v, o).items():
            assert getattr(moe._fast, name)(*args) is True
    side.synchronize()
    got = [t.clone() for name in calls(v, o) if name not in ("pack", "gated") for t in flat(o[name])]
    torch.cuda.synchronize()
    for a, b in zip(got, [t for name in calls(v, o) if name not in ("pack", "gated") for t in flat(want[name])]):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for name, (args, _) in calls(v, o).items():
            assert getattr(moe._fast, name)(*args) is True
    for _ in range(3):
        for name in calls(v, o):
            for t in flat(o[name]):
                t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for name in calls(v, o):
            for a, b in zip(flat(o[name]), flat(want[name])):
                assert torch.equal(a, b), name


def test_gradients_go_to_autograd():
    v = state()
    x = v["x"].clone().requires_grad_()
    out = torch.empty_like(v["ys"])
    assert moe._fast.gather(x, v["r"]["place"], out) is False
    with torch.no_grad():
        assert moe._fast.gather(x, v["r"]["place"], out) is True
