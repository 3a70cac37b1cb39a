"""Calls of the expert layer without a gradient refuse tensors that require one before
anything reaches the library."""
import pytest
import torch

import two_sided_hessian_amd as B
from test_moe_binding import BF16, F32, I32, Calls, checkpoint, on


def test_calls_without_a_gradient(monkeypatch):
    calls = Calls(monkeypatch)
    T, E, k, n = 3, 8, 2, 128
    R = T * k
    place, ck = on(0, T, k, dtype=I32), checkpoint(0, R, n)

    def t(*shape, dtype=BF16):
        return on(0, *shape, dtype=dtype)
    for shapes, call in (
            ([((T, k), F32), ((T, k), F32)], lambda g, p: B.moe_route_grad(g, p, place, E)),
            ([((T, n), BF16), ((R, n), BF16), ((T, k), F32)], lambda g, y, p: B.moe_combine_grad(g, y, place, p)),
            ([((R, n), BF16)], lambda g: B.gated_act_grad(g, ck, ck)),
            ([((R, n), BF16)], lambda x: B.ck8_pack(x, out=ck))):
        for i in range(len(shapes)):
            v = [t(*s, dtype=d).requires_grad_(i == j) for j, (s, d) in enumerate(shapes)]
            with pytest.raises(ValueError, match="has no gradient"):
                call(*v)
            assert not calls.made
            with torch.no_grad():
                call(*v)
            assert len(calls.made) == 1
            calls.made.clear()
