"""Groups whose best experts' biases are infinite with both signs: their sum is no number, the
group counts as one of value +infinity, and as many groups stay as were asked for."""
import numpy as np
import pytest
import torch

from oracle import routing_oracle as R
from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size,groups,top,m,k", [(2, 4, 2, 2, 4), (2, 4, 1, 2, 2), (4, 8, 3, 3, 8), (8, 8, 3, 2, 10),
                                                 (16, 16, 4, 2, 8)])
def test_a_forced_expert_among_banned_ones(scoring, size, groups, top, m, k):
    e = size * groups
    g = torch.Generator().manual_seed(e + m)
    for forced in range(0, groups, 3):
        bias = 0.05 * torch.randn(e, generator=g)
        own = slice(forced * size, (forced + 1) * size)
        bias[own] = -INF
        bias[forced * size + size // 2] = INF
        for t in (40, 5000):
            l = torch.randn(t, e, generator=g)
            idx, _ = M.route(l.cuda(), M.Routing(k, scoring, groups, top, m), bias.cuda())
            want, _ = R.route(l[:300].double().numpy(), k, scoring, groups, top, m, bias=bias.double().numpy())
            idx = idx.cpu().numpy()
            assert np.array_equal(idx[:300], want)
            assert (idx[:, 0] == forced * size + size // 2).all()
            assert max(len(set(row)) for row in idx // size) <= top
