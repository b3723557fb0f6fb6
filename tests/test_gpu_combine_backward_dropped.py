"""The combine's gradient where slots name no row."""
import pytest
import torch

from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu


def _call(perm, y, d_out, row_of, w, dy, dw):
    t, k = row_of.shape
    status = M.lib().moe_combine_backward(
        d_out.data_ptr(), y.data_ptr(), row_of.data_ptr(), w.data_ptr(), perm["counts"].data_ptr(),
        perm["offsets"].data_ptr(), dy.data_ptr(), dw.data_ptr(), t, k, d_out.shape[1], perm["counts"].numel(),
        y.shape[0], torch.cuda.current_stream().cuda_stream)
    assert status == 0, M.lib().moe_last_error()


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
