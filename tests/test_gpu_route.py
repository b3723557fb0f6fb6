"""General routing, router losses and their gradient on the GPU against the fp64 oracle.

Tolerances, derived:
- indices: equal. The kernel decides in double, as the oracle does; inputs hold exact ties
  (small whole logits) and no near ties but by a chance of about 1e-9.
- weights: computed in double and rounded once to fp32: 2^-24 of the value (2^-149 below
  the normal range).
- losses and gradient: fp32 terms. With u = 2^-24 and R the largest |l - max l| that has
  weight: an exponential is off by 4u (2^-22) + 1.5 R u (its argument's rounding), and weighted by
  itself by less than 5u, a sum over E <= 512 experts by (V + 5) u <= 21 u, so a probability by
  4 + 1.5 R + 5 + 21 + 2 <= 32 + 2R u; a gradient term multiplies two such factors and adds k <= 32
  products: 128 + 4R u of the magnitudes that are added up. Sums over tokens are double but for at most 64 fp32
  additions per lane: 64 u more."""
import numpy as np
import pytest
import torch

from oracle import routing_oracle as R
from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _logits(t, e, seed, kind, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(t, e, generator=g) * 1.5
    if kind == "ties":
        l = torch.randint(-2, 3, (t, e), generator=g).float()
    if kind == "special":
        pick = torch.rand(t, e, generator=g)
        l[pick < 0.3] = -float("inf")
        l[(pick >= 0.3) & (pick < 0.4)] = float("nan")
        l[(pick >= 0.4) & (pick < 0.45)] = torch.finfo(torch.float32).min
        l[::7] = -float("inf")                      # rows whose mask leaves nothing
        l[3::11, 0] = float("inf")
    return l.to(dtype)


def _args(r: M.Routing):
    return dict(k=r.k, scoring=r.scoring, num_groups=r.num_groups, topk_groups=r.topk_groups,
                group_top=r.group_top, renormalize=r.renormalize, scale=r.scale)


def _check_route(l, r, bias=None):
    idx, w = M.route(l.cuda(), r, None if bias is None else bias.cuda())
    want_i, want_w = R.route(l.double().numpy(), bias=None if bias is None else bias.double().numpy(),
                             **_args(r))
    assert np.array_equal(idx.cpu().numpy(), want_i)
    err = np.abs(w.cpu().double().numpy() - want_w)
    assert np.all(err <= U * (1 + 1e-6) * np.abs(want_w) + 2.0 ** -149)
    return idx, w


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (33, 8, 1), (65, 16, 4), (257, 17, 8), (40, 32, 32),
          (300, 64, 8), (129, 100, 3), (70, 128, 9), (50, 160, 8), (121, 256, 8), (37, 257, 32),
          (19, 512, 16)]


@pytest.mark.parametrize("t,e,k", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["normal", "ties", "special"])
def test_route_one_group(t, e, k, scoring, kind):
    l = _logits(t, e, 17 * t + e, kind)
    _check_route(l, M.Routing(k, scoring))
    bias = torch.randint(-2, 3, (e,), generator=torch.Generator().manual_seed(e)).float() / 8
    if kind == "special":
        bias[0] = float("nan")
        bias[-1] = -float("inf")
    if not (kind == "ties" and scoring == "softmax"):     # p + b of tied rows: near ties in double
        _check_route(l, M.Routing(k, scoring, renormalize=False, scale=2.5), bias)


@pytest.mark.parametrize("e,groups,top,m,k", [(8, 2, 1, 1, 2), (8, 4, 2, 2, 4), (64, 8, 4, 2, 8),
                                              (88, 8, 3, 2, 6), (96, 32, 5, 3, 7), (66, 3, 2, 4, 8),
                                              (256, 8, 4, 2, 8), (240, 8, 8, 2, 8), (512, 16, 2, 1, 20),
                                              (160, 5, 1, 32, 32), (33, 11, 4, 1, 3), (32, 32, 6, 1, 6),
                                              (12, 12, 3, 1, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_groups(e, groups, top, m, k, scoring):
    for kind in ("normal", "special"):
        l = _logits(101, e, e + groups, kind)
        r = M.Routing(k, scoring, groups, top, m)
        _check_route(l, r)
        bias = 0.1 * torch.randn(e, generator=torch.Generator().manual_seed(e))
        _check_route(l, r, bias)
    _check_route(_logits(101, e, e, "normal", torch.bfloat16), M.Routing(k, scoring, groups, top, m, False, 0.5))


def test_route_bf16_logits_many_ties():
    l = _logits(999, 64, 5, "normal", torch.bfloat16)
    _check_route(l, M.Routing(6, "softmax"))
    _check_route(l, M.Routing(6, "sigmoid"), 0.01 * torch.randn(64, generator=torch.Generator().manual_seed(1)))


def test_route_large_values_and_wide_ranges():
    l = torch.tensor([[3e38, -3e38, 1e30, 0.0], [-1e4, -1e4 + 1, -1e4 + 2, -1e5], [88.0, -88.0, 104.0, -104.0],
                      [-745.0, -800.0, -700.0, -745.1]])
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _check_route(l, M.Routing(3, scoring, renormalize=renorm))


def test_route_signed_zeros_are_equal():
    l = torch.tensor([[-0.0, 0.0, -1.0, -0.0], [0.0, -0.0, 0.0, -2.0]])
    idx, _ = _check_route(l, M.Routing(3))
    assert idx.tolist() == [[0, 1, 3], [0, 1, 2]]


@pytest.mark.parametrize("e,k,groups,top,m", [(8, 3, 1, 1, 1), (64, 8, 8, 4, 1), (256, 8, 8, 4, 1), (64, 6, 16, 4, 1),
                                              (120, 8, 8, 3, 1), (512, 32, 32, 8, 1), (48, 12, 4, 2, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_near_ties_are_decided_exactly(e, k, groups, top, m, scoring):
    """Scores a few fp32 steps apart around the same few values: fp32 sums cannot tell them
    apart, double ones can (differences above 2^-34 against errors of 2^-50). Sums of a
    group's two best are left out: those can tie to within double's error."""
    g = torch.Generator().manual_seed(e + k)
    t = 300
    l = torch.randint(-1, 2, (t, e), generator=g).float() * 0.5
    step = torch.stack([torch.randperm(e, generator=g) for _ in range(t)]).float()
    l = l + step * 2.0 ** -23 * 0.5
    _check_route(l, M.Routing(k, scoring, groups, top, m))
    bias = (torch.randint(-1, 2, (e,), generator=g).float() * 0.25)
    _check_route(l, M.Routing(k, scoring, groups, top, m), bias)


def test_route_huge_biases():
    l = _logits(64, 64, 3, "normal")
    g = torch.Generator().manual_seed(8)
    for size in (1e3, 1e30, 3e38, float("inf")):
        sign = torch.randint(-1, 2, (64,), generator=g).float()
        bias = torch.where(sign == 0, 0.0, sign * size)
        _check_route(l, M.Routing(5, "sigmoid", 8, 3, 2), bias)
        _check_route(l, M.Routing(5, "softmax"), bias)


def test_route_a_single_infinite_bias():
    for t in (50, 5000):
        l = _logits(t, 64, 4, "normal")
        for at in (3, 60):
            bias = 0.05 * torch.randn(64, generator=torch.Generator().manual_seed(at))
            bias[at] = float("inf")
            for scoring in ("sigmoid", "softmax"):
                for top in (1, 2):
                    idx, _ = _check_route(l, M.Routing(4, scoring, 8, 1, top), bias)
                    assert (idx[:, 0] == at).all()


def test_route_zero_bias_and_bf16_ties():
    """A bias of zeros (before its first update) over bf16 logits: exact ties in most rows."""
    for t in (300, 5000):
        l = _logits(t, 64, t, "normal", torch.bfloat16)
        for r in (M.Routing(8, "sigmoid"), M.Routing(6, "softmax"), M.Routing(8, "sigmoid", 8, 4, 2)):
            _check_route(l, r, torch.zeros(64))


def test_route_matches_the_layers_router():
    """The default rule on the layer's own logits is the layer's own routing."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(300, 256, generator=g).bfloat16().cuda()
    wr = (torch.randn(8, 256, generator=g) / 16).bfloat16().cuda()
    idx, w, logits = M.router_topk(x, wr, 2, return_logits=True)
    idx2, w2 = M.route(logits, M.Routing(2))
    assert torch.equal(idx, idx2)
    # fp32 softmax of the layer: 2e-6 covers its (32 + 2R) u with R < 1
    assert (w - w2).abs().max() <= 2e-6


def test_strided_rows_and_misaligned_logits():
    big = _logits(50, 300, 9, "normal")
    for dtype in (torch.float32, torch.bfloat16):
        wide = big.to(dtype).cuda()
        for lo, e in ((0, 64), (1, 64), (3, 8), (5, 257)):
            view = wide[:, lo:lo + e]
            r = M.Routing(4, "sigmoid")
            idx, w = M.route(view, r)
            idx2, w2 = M.route(view.contiguous(), r)
            assert torch.equal(idx, idx2) and torch.equal(w, w2)
            d_w = torch.ones_like(w)
            assert torch.equal(M.route_backward(view, idx, r, d_w), M.route_backward(view.contiguous(), idx, r, d_w))
            for a, b in zip(M.router_losses(view, idx, r), M.router_losses(view.contiguous(), idx, r)):
                assert torch.equal(a, b)


def _range(l, floor=30.0):
    """R: the largest |l - max| that has weight (beyond e^-floor terms vanish in the sums)."""
    l = R.clean(l)
    return floor if np.isinf(l).any() else min(floor, float((l.max(1, keepdims=True) - l).max()))


@pytest.mark.parametrize("t,e,k", SHAPES + [(20011, 8, 2), (5000, 64, 6), (8192, 16, 2), (8193, 8, 2), (7777, 256, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_losses(t, e, k, scoring):
    for kind in ("normal", "special"):
        l = _logits(t, e, t + e, kind)
        idx, _ = M.route(l.cuda(), M.Routing(k))
        for share in (None, 0.3):
            mask = None if share is None else torch.rand(t, generator=torch.Generator().manual_seed(4)) > share
            got = M.router_losses(l.cuda(), idx, M.Routing(k, scoring), None if mask is None else mask.cuda())
            ln = l.double().numpy()
            want = R.losses(ln, idx.cpu().numpy(), scoring, None if mask is None else mask.numpy())
            assert np.array_equal(got.counts.cpu().numpy(), want[1])
            c = (32 + 2 * _range(ln) + 64) * U
            assert np.all(np.abs(got.prob_mean.cpu().numpy() - want[2]) <= c * want[2] + 1e-30)
            assert abs(got.losses[0].item() - want[0][0]) <= c * want[0][0]
            keep = np.ones(t, bool) if mask is None else mask.numpy()
            lse = np.abs(R.logsumexp(R.clean(ln)))[keep]
            with np.errstate(over="ignore"):
                if np.isfinite(np.float32(want[0][1])):
                    size = (2 * lse * np.maximum(1, lse)).sum() / max(keep.sum(), 1)
                    assert abs(got.losses[1].item() - want[0][1]) <= (32 + _range(ln)) * U * size


@pytest.mark.parametrize("t,e,k", [(4096, 64, 6), (4097, 64, 6), (1024, 256, 8), (1025, 256, 8), (8192, 32, 4), (9000, 17, 4),
                                   (600, 512, 8), (30000, 128, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_losses_around_the_change_of_form(t, e, k, scoring):
    test_losses(t, e, k, scoring)


@pytest.mark.parametrize("t,e,k", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward(t, e, k, scoring, renorm):
    g = torch.Generator().manual_seed(t * e)
    for kind in ("normal", "special"):
        for dtype in (torch.float32, torch.bfloat16):
            l = _logits(t, e, t + 3 * e, kind, dtype)
            r = M.Routing(k, scoring, renormalize=renorm, scale=1.5)
            idx, _ = M.route(l.cuda(), r)
            d_w = torch.randn(t, k, generator=g)
            d_losses = torch.randn(2, generator=g)
            mask = torch.rand(t, generator=g) > 0.25
            counts = M.router_losses(l.cuda(), idx, r, mask.cuda()).counts
            ln, i = l.double().numpy(), idx.cpu().numpy()
            for dw, dl, m in ((d_w, None, None), (None, d_losses, mask), (d_w, d_losses, mask), (d_w, d_losses, None)):
                got = M.route_backward(l.cuda(), idx, r, None if dw is None else dw.cuda(),
                                       None if dl is None else counts, None if dl is None else dl.cuda(),
                                       None if m is None else m.cuda())
                want, size = R.route_backward(ln, i, scoring, renorm, 1.5, None if dw is None else dw.numpy(),
                                              counts.cpu().numpy(), None if dl is None else dl.numpy(),
                                              None if m is None else m.numpy())
                assert got.dtype == dtype and got.shape == l.shape
                tol = (128 + 4 * _range(ln)) * U * size + 1e-37
                if dtype == torch.bfloat16:
                    tol = tol * 1.01 + 2.0 ** -8 * np.abs(want)
                with np.errstate(over="ignore", invalid="ignore"):
                    fine = size < 1e37                   # (max float)^2 terms of a z-loss overflow
                    assert np.all(np.abs(got.cpu().double().numpy() - want)[fine] <= tol[fine])


def test_backward_ignores_slots_that_name_no_expert():
    l = _logits(9, 8, 1, "normal").cuda()
    r = M.Routing(3)
    idx, _ = M.route(l, r)
    d_w = torch.ones(9, 3, device="cuda")
    d_w[:, 1] = 2
    idx[::2, 2] = -1
    idx[1::2, 2] = 8
    got = M.route_backward(l, idx, r, d_w).cpu().double().numpy()
    want, size = R.route_backward(l.cpu().double().numpy(), idx.cpu().numpy(), d_w=d_w.cpu().numpy())
    assert np.all(np.abs(got - want) <= 160 * U * size + 1e-37)
    assert M.router_losses(l, idx, r).counts[:8].sum().item() == 18


@pytest.mark.parametrize("e,k", [(8, 3), (16, 8), (64, 6), (128, 7), (40, 24), (256, 8), (512, 32)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_of_repeated_experts(e, k, scoring, renorm):
    """An expert named more than once gets the sum of its slots, the same bits each time (up to
    31 more roundings than distinct slots cost)."""
    t = 700
    g = torch.Generator().manual_seed(e * k)
    l = _logits(t, e, e + k, "normal")
    idx = torch.randint(0, e, (t, k), generator=g, dtype=torch.int32)
    idx[::3] = idx[::3, :1]                              # one expert in every slot
    idx[1::3] %= 3
    d_w = torch.randn(t, k, generator=g)
    r = M.Routing(k, scoring, renormalize=renorm, scale=1.5)
    run = lambda: M.route_backward(l.cuda(), idx.cuda(), r, d_w.cuda())
    got = run()
    want, size = R.route_backward(l.double().numpy(), idx.numpy(), scoring, renorm, 1.5, d_w.numpy())
    tol = (160 + 4 * _range(l.double().numpy())) * U * size + 1e-37
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= tol)
    for _ in range(5):
        assert torch.equal(got, run())


def test_no_tokens():
    l = torch.empty(0, 8, device="cuda")
    r = M.Routing(2)
    idx, w = M.route(l, r)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    got = M.router_losses(l, idx, r)
    assert got.losses.tolist() == [0, 0] and got.counts.tolist() == [0] * 9 and got.prob_mean.tolist() == [0] * 8
    assert M.route_backward(l, idx, r, w, got.counts, got.losses).shape == (0, 8)
    # tokens, but the mask leaves none
    l = torch.randn(5, 8, device="cuda")
    idx, w = M.route(l, r)
    mask = torch.zeros(5, dtype=torch.bool, device="cuda")
    got = M.router_losses(l, idx, r, mask)
    assert got.losses.tolist() == [0, 0] and got.counts.tolist() == [0] * 9
    one = torch.ones(2, device="cuda")
    assert M.route_backward(l, idx, r, None, got.counts, one, mask).abs().max().item() == 0


def test_two_calls_give_the_same_bits():
    l = _logits(30000, 64, 8, "normal").cuda()
    r = M.Routing(6, "sigmoid")
    idx, w = M.route(l, r)
    first = M.router_losses(l, idx, r)
    d = M.route_backward(l, idx, r, w, first.counts, first.losses)
    for _ in range(3):
        again = M.router_losses(l, idx, r)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert torch.equal(d, M.route_backward(l, idx, r, w, again.counts, again.losses))


def test_another_stream_and_a_captured_graph():
    l = _logits(200, 64, 8, "normal").cuda()
    r = M.Routing(6, "sigmoid", 8, 4, 2)
    bias = 0.05 * torch.randn(64, device="cuda")
    idx, w = M.route(l, r, bias)
    los = M.router_losses(l, idx, r)
    d = M.route_backward(l, idx, r, w, los.counts, los.losses)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    idx2, w2 = M.route(l, r, bias, stream=side)
    los2 = M.router_losses(l, idx2, r, stream=side)
    d2 = M.route_backward(l, idx2, r, w2, los2.counts, los2.losses, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(idx, idx2) and torch.equal(w, w2) and torch.equal(d, d2)
    graphs, outs = [], []
    for _ in range(2):                              # two graphs, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, capture_error_mode="thread_local"):
            gi, gw = M.route(l, r, bias)
            gl = M.router_losses(l, gi, r)
            gd = M.route_backward(l, gi, r, gw, gl.counts, gl.losses)
        graphs.append(graph)
        outs.append((gi, gw, gd) + tuple(gl))
    l.copy_(_logits(200, 64, 99, "normal"))
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    idx, w = M.route(l, r, bias)
    los = M.router_losses(l, idx, r)
    want = (idx, w, M.route_backward(l, idx, r, w, los.counts, los.losses)) + tuple(los)
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
