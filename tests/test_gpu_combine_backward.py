"""Gradient of the combine on the GPU against fp64.

Tolerances, derived (u = 2^-24): dy is one product of a bf16 and an fp32 value, rounded
once: u of the value. d_topk_w adds 8 ceil(H / 2048) products per thread in a row, then 5 + 8
partial sums: (8 ceil(H / 2048) + 14) u of the sum of the products' magnitudes."""
import math

import numpy as np
import pytest
import torch

from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _case(t, h, k, e, seed, extra_rows=0):
    """A routing, its permutation and a batch; y holds NaN where no slot points."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(t, e, generator=g).topk(k, dim=1).indices.int().cuda()
    x = torch.zeros(t, 128, dtype=torch.bfloat16, device="cuda")
    shape = M.make_shape(t, 128, 128, e, k)
    perm = M.permute(idx, x, e, 128, M.make_workspace(shape))
    rows = M.max_padded_rows(shape) + extra_rows
    y = torch.full((rows, h), float("nan"))
    named = perm["row_of"].cpu().long().reshape(-1)
    y[named] = torch.randn(t * k, h, generator=g)
    d_out = torch.randn(t, h, generator=g).bfloat16()
    w = torch.rand(t, k, generator=g)
    return perm, y.cuda(), d_out.cuda(), w.cuda()


def _check(perm, y, d_out, w, dy, dw):
    rows = perm["row_of"].cpu().long()
    d, yn, wn = d_out.cpu().double().numpy(), y.cpu().double().numpy(), w.cpu().double().numpy()
    t, k = rows.shape
    if dy is not None:
        want = np.zeros(yn.shape)
        for j in range(k):
            want[rows[:, j].numpy()] = wn[:, j:j + 1] * d
        got = dy.cpu().double().numpy()
        assert np.all(np.abs(got - want) <= U * np.abs(want) + 2.0 ** -149)
    if dw is not None:
        prod = d[:, None, :] * yn[rows.numpy()]
        tol = (8 * math.ceil(d.shape[1] / 2048) + 14) * U * np.abs(prod).sum(2)
        assert np.all(np.abs(dw.cpu().double().numpy() - prod.sum(2)) <= tol)


@pytest.mark.parametrize("t,h,k,e", [(1, 8, 1, 1), (1, 4096, 2, 8), (3, 136, 3, 5), (130, 256, 2, 8),
                                     (77, 4104, 4, 16), (500, 1024, 8, 64), (16, 14336, 5, 8),
                                     (2500, 512, 2, 8), (6000, 128, 1, 64)])
def test_against_fp64(t, h, k, e):
    perm, y, d_out, w = _case(t, h, k, e, t + h)
    dy, dw = M.combine_backward(d_out, y, perm["row_of"], w, perm["counts"], perm["offsets"])
    _check(perm, y, d_out, w, dy, dw)
    dy2, none = M.combine_backward(d_out, y, perm["row_of"], w, perm["counts"], perm["offsets"], need_dw=False)
    assert none is None and torch.equal(dy, dy2)
    none, dw2 = M.combine_backward(d_out, y, perm["row_of"], w, need_dy=False)
    assert none is None and torch.equal(dw, dw2)


def test_rows_past_the_groups_are_zero():
    perm, y, d_out, w = _case(40, 256, 2, 8, 1, extra_rows=301)
    dy, _ = M.combine_backward(d_out, y, perm["row_of"], w, perm["counts"], perm["offsets"])
    _check(perm, y, d_out, w, dy, None)


def test_one_expert_takes_all_and_others_none():
    t, h = 256, 64
    idx = torch.full((t, 1), 3, dtype=torch.int32, device="cuda")
    perm = M.permute(idx, torch.zeros(t, 128, dtype=torch.bfloat16, device="cuda"), 8, 128,
                     M.make_workspace(M.make_shape(t, 128, 128, 8, 1)))
    y = torch.randn(t, h, device="cuda")                 # exactly the routed rows: no pads
    d_out, w = torch.randn(t, h, device="cuda").bfloat16(), torch.rand(t, 1, device="cuda")
    dy, dw = M.combine_backward(d_out, y, perm["row_of"], w, perm["counts"], perm["offsets"])
    _check(perm, y, d_out, w, dy, dw)


def test_rows_outside_the_buffer_are_no_slots():
    perm, y, d_out, w = _case(20, 128, 2, 4, 5)
    row_of = perm["row_of"].clone()
    row_of[::2, 1] = -1
    row_of[1::4, 1] = y.shape[0]
    dy, dw = M.combine_backward(d_out, y, row_of, w, perm["counts"], perm["offsets"])
    ok = (row_of >= 0) & (row_of < y.shape[0])
    assert (dw[~ok] == 0).all() and (dw[ok] != 0).all()
    want = M.combine_backward(d_out, y, perm["row_of"], w, perm["counts"], perm["offsets"])
    assert torch.equal(dy[row_of[ok].long()], want[0][row_of[ok].long()])
    assert torch.equal(dw[ok], want[1][ok])


def test_no_tokens():
    e = 4
    c, o = torch.zeros(e, dtype=torch.int32, device="cuda"), torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    dy, dw = M.combine_backward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                                torch.full((130, 64), float("nan"), device="cuda"),
                                torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                                torch.empty(0, 2, device="cuda"), c, o)
    assert dw.shape == (0, 2) and dy.shape == (130, 64) and (dy == 0).all()


def test_gradient_against_differences_of_the_combine():
    """d(sum(v * combine)) / dw_j is <v, y_j>: the combine is linear in w, so a difference of
    two calls with power-of-two weights is exact but for the output's bf16 rounding."""
    perm, y, _, w = _case(12, 512, 2, 8, 7)
    v = torch.randn(12, 512, device="cuda").bfloat16()
    _, dw = M.combine_backward(v, y, perm["row_of"], w, need_dy=False)
    for j in range(2):
        up = torch.zeros_like(w)
        up[:, j] = 1.0
        out = M.combine(y, perm["row_of"], up).double()          # w = 0 gives exactly 0
        diff = (out * v.double()).sum(1)
        # out is off by at most 2^-8 of each value (one bf16 rounding)
        tol = (2.0 ** -8 * 1.01) * (out.abs() * v.double().abs()).sum(1) + 1e-4
        assert ((diff - dw[:, j].double()).abs() <= tol).all()


def test_another_stream_and_captured():
    perm, y, d_out, w = _case(100, 1024, 2, 8, 9)
    want = M.combine_backward(d_out, y, perm["row_of"], w, perm["counts"], perm["offsets"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = M.combine_backward(d_out, y, perm["row_of"], w, perm["counts"], perm["offsets"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        got = M.combine_backward(d_out, y, perm["row_of"], w, perm["counts"], perm["offsets"])
    d_out.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], 2 * want[0]) and torch.equal(got[1], 2 * want[1])
