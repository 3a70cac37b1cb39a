"""4-bit layer calls with stream=, on a stream that nothing orders after the
current one: what the calls allocate is never memory that work pending on the
current stream still uses, and q4_pack looks at its inputs in the order of
the stream that makes them."""
import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_q4 import DEV, dev, make_layer, make_moe, pack, tokens

pytestmark = pytest.mark.gpu
BUSY = 100_000_000          # clock cycles: tens of milliseconds


@pytest.mark.parametrize("call,T", [("linear", 3), ("linear", 200), ("grad", 200), ("moe", 40)])
def test_results_and_workspaces_are_not_those_of_pending_work(call, T):
    layer = make_layer(500, 640, 64, 41)
    x, router, layers = make_moe(T, 640, 500, 4, 2, 64, torch.bfloat16, 42)
    if call == "moe":
        w = [pack(*v, 64) for v in layers]

        def run(**kw):
            return B.q4_moe(x, router, *w, 2, **kw)["y"]
    else:
        w = pack(*layer, 64)
        x = tokens(T, 640 if call == "linear" else 500, torch.bfloat16, T)
        f = B.q4_linear if call == "linear" else B.q4_linear_grad

        def run(**kw):
            return f(x, w, **kw)
    ref = run()
    size = ref.numel()
    need = (B.q4_moe_workspace_bytes(T, w[0], 2) if call == "moe" else
            (B.q4_linear_workspace_bytes if call == "linear" else B.q4_linear_grad_workspace_bytes)(T, w))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # blocks of the sizes that the call needs, read by pending work and let go
    old = [torch.full((size,), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    old += [torch.full((max(need, 1),), 7, dtype=torch.uint8, device=DEV) for _ in range(3)]
    torch.cuda._sleep(BUSY)
    kept = [t.clone() for t in old]
    spans = [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in old]
    del old
    got = run(stream=side)
    assert all(got.data_ptr() + got.nbytes <= a or got.data_ptr() >= b for a, b in spans)
    torch.cuda.synchronize()
    assert torch.equal(got, ref)
    for t, v in zip(kept, [3.0] * 3 + [7] * 3):
        assert bool((t == v).all())


def test_a_result_let_go_is_not_handed_out_while_the_current_stream_reads_it():
    layer = make_layer(500, 640, 64, 43)
    w, x = pack(*layer, 64), tokens(200, 640, torch.bfloat16, 1)
    ref = B.q4_linear(x, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = B.q4_linear(x, w, stream=side)
    side.synchronize()
    torch.cuda._sleep(BUSY)
    kept = y.clone()                   # waits behind the sleep
    at = y.data_ptr()
    del y
    again = B.q4_linear(x * 2, w, stream=side)
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(kept, ref)


@pytest.mark.parametrize("before,after", [(20, 4), (4, 20)])
def test_pack_checks_what_its_stream_makes(before, after):
    codes, scale, zero = make_layer(64, 128, 64, 44)
    scale, zero = dev(scale), dev(zero)
    c = torch.full((64, 128), before, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        c.fill_(after)
    if after > 15:
        with pytest.raises(B.GridError):
            B.q4_pack(c, scale, zero, group_size=64, stream=side)
        return
    w = B.q4_pack(c, scale, zero, group_size=64, stream=side)
    side.synchronize()
    x = tokens(5, 128, torch.float16, 1)
    assert torch.equal(B.q4_linear(x, w), B.q4_linear(x, B.q4_pack(c, scale, zero, group_size=64)))
