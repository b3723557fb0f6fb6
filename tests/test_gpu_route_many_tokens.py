"""Routing of more than 4096 tokens, where a lane holds more experts than for fewer: against the
fp64 oracle on some rows, and against the form for few tokens on all of them."""
import numpy as np
import pytest
import torch

from oracle import routing_oracle as R
from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("e,k,groups,top,m", [(65, 8, 1, 1, 1), (100, 6, 1, 1, 1), (128, 8, 1, 1, 1), (128, 8, 8, 4, 2),
                                              (128, 4, 4, 2, 1), (96, 8, 6, 3, 2), (40, 8, 1, 1, 1), (64, 8, 8, 4, 2),
                                              (256, 8, 8, 4, 2), (128, 12, 8, 4, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_against_the_oracle(e, k, groups, top, m, scoring, dtype):
    t = 9001
    g = torch.Generator().manual_seed(e * k + groups)
    l = (1.5 * torch.randn(t, e, generator=g)).to(dtype)
    l[5::50] = torch.randint(-2, 3, (t, e), generator=g)[5::50].to(dtype)       # ties
    l[7::50, :e // 2] = -float("inf")
    r = M.Routing(k, scoring, groups, top, m, True, 2.5)
    pick = torch.cat([torch.arange(0, t, 60), torch.arange(5, t, 500), torch.arange(7, t, 500), torch.tensor([t - 1])])
    for bias in (None, torch.zeros(e), 0.05 * torch.randn(e, generator=g)):
        if bias is not None and scoring == "softmax":
            l[5::50] = l[6::50][:l[5::50].shape[0]]       # sums with a bias of tied rows: near ties in double
        dev = None if bias is None else bias.cuda()
        idx, w = M.route(l.cuda(), r, dev)
        want_i, want_w = R.route(l[pick].double().numpy(), k, scoring, groups, top, m, True, 2.5,
                                 None if bias is None else bias.double().numpy())
        assert np.array_equal(idx.cpu().numpy()[pick], want_i)
        assert np.all(np.abs(w.cpu().double().numpy()[pick] - want_w) <= U * (1 + 1e-6) * np.abs(want_w) + 2.0 ** -149)
        for lo in range(0, t, 4000):
            some, part = M.route(l[lo:lo + 4000].cuda(), r, dev)
            assert torch.equal(idx[lo:lo + 4000], some) and torch.equal(w[lo:lo + 4000], part)
