"""Groups compared by logits where sigmoids no longer tell them apart: with no bias and one
expert a group the logits decide, whatever their scores round to. Tolerances as for the
other routing tests: indices equal, weights one rounding."""
import numpy as np
import pytest
import torch

from oracle import routing_oracle as R
from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
INF = float("inf")


def _check(l, r):
    idx, w = M.route(l.cuda(), r)
    want_i, want_w = R.route(l.double().numpy(), r.k, r.scoring, r.num_groups, r.topk_groups, r.group_top,
                             r.renormalize, r.scale)
    assert np.array_equal(idx.cpu().numpy(), want_i)
    assert np.all(np.abs(w.cpu().double().numpy() - want_w) <= U * (1 + 1e-6) * np.abs(want_w) + 2.0 ** -149)
    return idx


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_group_of_the_larger_logit_stays(scoring):
    ulp = 26 * (1 + 2.0 ** -22)
    for row, groups, want in (([40, 1, 50, 1, -INF, -INF], 3, 2), ([40, 1, 50, 1, 0, 0], 3, 2),
                              ([40, 1, 50, 1, -1e38, 3], 3, 2), ([26, 1, ulp, 1], 2, 2), ([ulp, 1, 26, 1], 2, 0),
                              ([50, 1, 50, 60, 3e38, 1], 3, 4), ([700, 800, 900, 1000], 2, 3)):
        l = torch.tensor([row], dtype=torch.float32)
        assert _check(l, M.Routing(1, scoring, groups, 1, 1)).item() == want


@pytest.mark.parametrize("e,groups,top,k", [(16, 4, 2, 4), (64, 8, 3, 6), (64, 16, 4, 8), (66, 3, 1, 5), (128, 8, 4, 8),
                                            (256, 8, 4, 8), (256, 32, 7, 12), (512, 16, 3, 32)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", [50, 5000])
def test_saturated_groups(e, groups, top, k, scoring, t):
    g = torch.Generator().manual_seed(e + t)
    l = torch.randn(t, e, generator=g)
    l += torch.tensor([0.0, 24.0, 40.0, 300.0])[torch.arange(t) % 4, None]
    l[torch.rand(t, groups, generator=g).repeat_interleave(e // groups, 1) < 0.1] = -INF   # masked groups
    _check(l[:200] if t > 200 else l, M.Routing(k, scoring, groups, top, 1))
    if t > 200:      # the same rows, among enough others for the form of many tokens
        idx, w = M.route(l.cuda(), M.Routing(k, scoring, groups, top, 1))
        some, part = M.route(l[:200].cuda(), M.Routing(k, scoring, groups, top, 1))
        assert torch.equal(idx[:200], some) and torch.equal(w[:200], part)
