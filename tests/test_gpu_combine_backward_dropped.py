"""The combine's gradient where slots were taken out (their row set outside the buffer) or
there are no rows at all: every row that no slot names is zero, whatever the output held."""
import pytest
import torch

from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu


def _case(t, h, k, e, extra):
    g = torch.Generator(device="cuda").manual_seed(t + h)
    idx = torch.rand(t, e, device="cuda", generator=g).topk(k, dim=1).indices.int()
    shape = M.make_shape(t, 128, 128, e, k)
    perm = M.permute(idx, torch.zeros(t, 128, dtype=torch.bfloat16, device="cuda"), e, 128, M.make_workspace(shape))
    y = torch.randn(M.max_padded_rows(shape) + extra, h, device="cuda", generator=g)
    d_out = torch.randn(t, h, device="cuda", generator=g).bfloat16()
    return perm, y, d_out, torch.rand(t, k, device="cuda", generator=g) + 0.5, g


def _call(perm, y, d_out, row_of, w, dy, dw):
    t, k = row_of.shape
    status = M.lib().moe_combine_backward(
        d_out.data_ptr(), y.data_ptr(), row_of.data_ptr(), w.data_ptr(), perm["counts"].data_ptr(),
        perm["offsets"].data_ptr(), dy.data_ptr(), dw.data_ptr(), t, k, d_out.shape[1], perm["counts"].numel(),
        y.shape[0], torch.cuda.current_stream().cuda_stream)
    assert status == 0, M.lib().moe_last_error()


@pytest.mark.parametrize("t,h,k,e,extra", [(1, 8, 1, 1, 0), (1, 4096, 2, 8, 0), (20, 128, 2, 4, 37), (77, 1032, 3, 16, 0),
                                           (500, 64, 8, 64, 1000), (3000, 256, 2, 8, 0), (20000, 8, 2, 512, 0),
                                           (5000, 128, 1, 4, 70000)])
@pytest.mark.parametrize("share", [0.0, 0.02, 0.5, 1.0])
def test_unnamed_rows_are_zero(t, h, k, e, extra, share):
    if e > 64:      # more experts than permute takes: their groups by hand
        perm, y, d_out, w, g = _case(t, h, k, 64, extra)
        counts = torch.zeros(e, dtype=torch.int32, device="cuda")
        counts[::8] = perm["counts"]
        offsets = torch.cat([perm["offsets"][:1], perm["offsets"][1:].repeat_interleave(8)])
        perm = {"row_of": perm["row_of"], "counts": counts, "offsets": offsets}
    else:
        perm, y, d_out, w, g = _case(t, h, k, e, extra)
    row_of = perm["row_of"].clone()
    drop = torch.rand(t, k, device="cuda", generator=g) < share
    out_of = torch.tensor([-1, y.shape[0], -2 ** 31, 2 ** 31 - 1], device="cuda").int()
    row_of[drop] = out_of[torch.randint(0, 4, (int(drop.sum()),), device="cuda", generator=g)]
    dy, dw = torch.full_like(y, float("nan")), torch.full((t, k), float("nan"), device="cuda")
    _call(perm, y, d_out, row_of, w, dy, dw)
    want = torch.zeros_like(y)
    for j in range(k):
        ok = ~drop[:, j]
        want[row_of[ok, j].long()] = w[ok, j:j + 1] * d_out[ok].float()   # one rounding, as in the kernel
    assert torch.equal(dy, want)
    assert (dw[drop] == 0).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("t,k", [(1, 1), (5, 1), (5, 2), (40, 8), (6000, 1), (6000, 2)])
def test_tokens_but_no_rows(t, k):
    d_out = torch.randn(t, 64, device="cuda").bfloat16()
    row_of = torch.full((t, k), -1, dtype=torch.int32, device="cuda")
    row_of[::2] = 0
    w = torch.ones(t, k, device="cuda")
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    guard = torch.full((4, 64), 7.0, device="cuda")
    dw = torch.full((t, k), float("nan"), device="cuda")
    perm = {"counts": none[:3], "offsets": none}
    _call(perm, guard[:0], d_out, row_of, w, guard, dw)       # dy is not NULL, but holds no row
    assert (dw == 0).all() and (guard == 7).all()
