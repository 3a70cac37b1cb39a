"""moe_route where a workgroup takes its tokens in several passes: beyond 16384 tokens, with
as many choices a pass as there are threads and fewer, and experts that no one chooses."""
import numpy as np
import pytest
import torch

import two_sided_hessian_amd as B
from test_gpu_moe_route import DEV, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,kind", [(16384, 256, 16, "normal"), (16385, 256, 16, "masked"), (33001, 200, 16, "ties"),
                                        (40000, 256, 5, "masked"), (131073, 7, 3, "ties")])
def test_choices_of_many_tokens(T, E, k, kind):
    logits = make(T, E, torch.bfloat16, T + E, kind)
    r = {name: t.cpu().numpy() for name, t in B.moe_route(logits, k).items()}
    l = logits.double().cpu().numpy()
    l = np.where(np.isnan(l), -np.inf, l)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    ids[np.take_along_axis(l, ids, 1) == -np.inf] = -1
    assert np.array_equal(r["ids"], ids)
    each = np.where(ids < 0, E, ids).reshape(-1)                  # a stable sort by expert, no choice behind
    order = np.argsort(each, kind="stable")
    last = int((each < E).sum())
    assert np.array_equal(r["offsets"], np.searchsorted(each[order], np.arange(E + 1)))
    assert np.array_equal(r["order"][:last], order[:last]) and (r["order"][last:] == -1).all()
    place = np.full(T * k, -1)
    place[order[:last]] = np.arange(last)
    assert np.array_equal(r["place"].reshape(-1), place)
    assert ((r["weights"] == 0) | (ids >= 0)).all()
    assert np.abs(r["weights"].astype(np.float64).sum(1) - (ids >= 0).any(1)).max() <= 40 * 2.0 ** -24   # (k + 22 roundings)
