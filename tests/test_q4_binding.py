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
