"""moe_route with biases at the ends of fp32's range, on groups."""
import numpy as np
import pytest
import torch

from oracle import block as O
from tests.helpers import load_lib

pytestmark = pytest.mark.gpu

LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("E,G", [(32, 4), (88, 8), (256, 8), (1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group", ["top2", "max"])
def test_route_groups_of_the_lowest_bias(E, G, score, group):
    # experts put last by a bias of fp32's lowest value can still be chosen once nothing else is left: the sum of
    # two of them is past fp32's range, and their group not an empty one
    M = load_lib()
    gs = E // G
    rng = np.random.default_rng(E)
    lg = rng.standard_normal((7, E)).astype(np.float32)
    bias = np.full(E, LOWEST, np.float32)
    bias[gs:2 * gs] = 0                     # the second group alone is at its usual place
    lg[1, :gs] = -np.inf                    # a group before the others that is empty
    k = min(gs + 2, 32)
    ids, w = M.moe_route(torch.from_numpy(lg).cuda(), k, getattr(M, "MOE_SCORE_" + score.upper()),
                         torch.from_numpy(bias).cuda(), G, 2, getattr(M, "MOE_GROUP_" + group.upper()))
    # s + bias rounds to the bias: among the lowest, ties go to the lower group and the lower expert
    _, s = O.route_scores(lg, score)
    for t in range(7):
        first = gs + np.lexsort((np.arange(gs), -s[t, gs:2 * gs].astype(np.float32)))
        rest = np.arange(gs) if t != 1 else 2 * gs + np.arange(gs)
        assert ids[t].tolist() == np.concatenate([first, rest])[:k].tolist()
    assert torch.isfinite(w).all()


@pytest.mark.parametrize("k", [-1, 0, 17, 33, 2 ** 31 - 1])
def test_route_refuses_a_k_out_of_range_as_the_library_does(k):
    M = load_lib()
    with pytest.raises(M.MoeError, match="k must be"):
        M.moe_route(torch.zeros(4, 16, device="cuda"), k)
