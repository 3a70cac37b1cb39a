"""Errors of HIP on the native way of the expert layer's calls (csrc/fast_calls.cpp)."""
import ctypes

import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_moe_native import calls, flat, outputs, state
from two_sided_hessian_amd import moe

pytestmark = pytest.mark.gpu
BAD_DEVICE = 9999
ERR_HIP = -5


def hip():
    """The HIP runtime that this process has loaded."""
    with open("/proc/self/maps") as f:
        return ctypes.CDLL(next(line.split()[-1] for line in f if "libamdhip64" in line))


def test_a_launch_error_is_raised_and_the_call_not_made_again():
    """An error that HIP has pending (a device that does not exist, asked for on the host) is
    what a call finds after its launch: the call raises it, as it does without the native way,
    instead of being made a second time with the error taken away."""
    v, lib = state(), hip()
    want, o = outputs(v), outputs(v)
    for args, call in calls(v, want).values():
        call()
    torch.cuda.synchronize()
    for name, (args, call) in calls(v, o).items():
        for run in (call, lambda: getattr(moe._fast, name)(*args)):
            assert lib.hipSetDevice(BAD_DEVICE) != 0
            with pytest.raises(B.BakronError, match="bakron_") as e:
                run()
            assert e.value.code == ERR_HIP, name
            call()                                                # the error is gone with it
        for a, b in zip(flat(o[name]), flat(want[name])):
            assert torch.equal(a, b), name
    torch.cuda.synchronize()


def test_refusals_are_still_left_to_the_checks_in_python():
    v = state()
    o = outputs(v)
    logits, k = v["logits"], 2
    assert moe._fast.route(logits, k, o["route"], None) is True
    assert moe._fast.route(logits, -1, o["route"], None) is False
    assert moe._fast.gated_grad(v["ys"], *v["ck"], 9, None, *o["gated_grad"]) is False
    with pytest.raises(ValueError, match="act"):
        B.gated_act_grad(v["ys"], *v["ck"], act="relu", out=o["gated_grad"])
