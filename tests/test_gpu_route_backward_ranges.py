"""The losses and the gradient in the logits where the logits have a common offset, or are so
negative that a sigmoid is below fp32's range: against fp64, with the bounds of the other gradient
tests (u = 2^-24, R the largest |l - max l| that has weight): 128 + 4 R u of the terms' magnitudes
for the gradient, 96 + 2 R u for the mean probabilities. A sigmoid of a logit of -32 to -64 adds half a
step of its exponential's argument to what those count, 22 u; its share of a sum twice that."""
import numpy as np
import pytest
import torch

from oracle import routing_oracle as R
from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
T = 300


def _range(l):
    return min(30.0, float((l.max(1, keepdims=True) - l).max()))


def _compare(l, k, scoring, renorm):
    t, e = l.shape
    g = torch.Generator().manual_seed(e + k)
    r = M.Routing(k, scoring, renormalize=renorm, scale=1.5)
    idx = torch.rand(t, e, generator=g).topk(k, dim=1).indices.int()
    d_w, d_losses = torch.randn(t, k, generator=g), torch.randn(2, generator=g)
    ln, i = l.double().numpy(), idx.numpy()
    bound = (128 + 4 * _range(ln)) * U
    los = M.router_losses(l.cuda(), idx.cuda(), r)
    want = R.losses(ln, i, scoring)
    assert np.array_equal(los.counts.cpu().numpy(), want[1])
    c = (96 + 2 * _range(ln)) * U
    assert np.all(np.abs(los.prob_mean.cpu().numpy() - want[2]) <= c * want[2] + 1e-30)
    assert abs(los.losses[0].item() - want[0][0]) <= c * want[0][0]
    for dw, dl in ((d_w, None), (None, d_losses), (d_w, d_losses)):
        got = M.route_backward(l.cuda(), idx.cuda(), r, None if dw is None else dw.cuda(),
                               None if dl is None else los.counts, None if dl is None else dl.cuda())
        want, size = R.route_backward(ln, i, scoring, renorm, 1.5, None if dw is None else dw.numpy(),
                                      los.counts.cpu().numpy(), None if dl is None else dl.numpy())
        assert np.all(np.abs(got.cpu().double().numpy() - want) <= bound * size + 1e-37)


@pytest.mark.parametrize("e,k", [(8, 2), (16, 8), (64, 6), (100, 12), (256, 8), (512, 32)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("offset", [300.0, -300.0, 1000.0, 30000.0, 1e8])
def test_softmax_with_an_offset(e, k, renorm, offset):
    l = torch.randn(T, e, generator=torch.Generator().manual_seed(e))
    step = max(2.0 ** -20, abs(offset) * 2.0 ** -23)
    _compare(torch.round(l / step) * step + offset, k, "softmax", renorm)


@pytest.mark.parametrize("e,k", [(8, 2), (16, 8), (64, 6), (100, 12), (256, 8), (512, 32)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("offset", [-30.0, -60.0, -84.0, -88.0, -110.0, -650.0, 60.0])
def test_sigmoid_with_an_offset(e, k, renorm, offset):
    _compare(torch.randn(T, e, generator=torch.Generator().manual_seed(e)) + offset, k, "sigmoid", renorm)


@pytest.mark.parametrize("e,k", [(8, 3), (64, 6), (256, 8)])
def test_sigmoid_rows_of_every_size(e, k):
    """Tokens of all offsets in one call, a single ordinary logit among very negative ones."""
    g = torch.Generator().manual_seed(e)
    l = torch.randn(T, e, generator=g) - 300 * torch.rand(T, 1, generator=g)
    l[::5, 1] = 0.5
    _compare(l, k, "sigmoid", True)
    _compare(l, k, "sigmoid", False)
