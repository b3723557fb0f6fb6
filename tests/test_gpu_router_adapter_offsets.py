"""Element offsets past 2^31 in the routing, loss, gradient and adapter operators: the same
values as compact tensors, or the tail's own call, give."""
import pytest
import torch

from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()                             # up to 25 GB a test


def _spread(v, stride):
    """v's rows `stride` elements apart; what lies between them is not written."""
    out = torch.empty(v.shape[0] * stride, dtype=v.dtype, device=v.device)
    out = out.as_strided(v.shape, (stride, 1))
    assert (v.shape[0] - 1) * stride > 2 ** 31
    return out.copy_(v)


@pytest.mark.parametrize("t,stride", [(2200, 2 ** 20 + 8), (40, 2 ** 26)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_logits(t, stride, dtype):
    compact = torch.randn(t, 64, device="cuda").to(dtype)
    wide = _spread(compact, stride)
    r = M.Routing(6, "sigmoid", 8, 4, 2)
    idx, w = M.route(compact, r)
    got = M.route(wide, r)
    assert torch.equal(got[0], idx) and torch.equal(got[1], w)
    want, los = M.router_losses(compact, idx, r), M.router_losses(wide, idx, r)
    assert all(torch.equal(a, b) for a, b in zip(los, want))
    assert torch.equal(M.route_backward(wide, idx, r, w, los.counts, los.losses),
                       M.route_backward(compact, idx, r, w, los.counts, los.losses))


def test_many_tokens():
    t, e = 2 ** 22 + 1000, 512
    l = torch.randn(t, e, device="cuda", dtype=torch.bfloat16)
    r = M.Routing(2)
    idx, w = M.route(l, r)
    los = M.router_losses(l, idx, r)
    assert los.counts[e] == t and los.counts[:e].sum() == 2 * t
    d = M.route_backward(l, idx, r, w, los.counts, los.losses)
    assert d.numel() > 2 ** 31
    for at in (0, 2 ** 21, t - 1000):
        part = slice(at, at + 1000)
        i, v = M.route(l[part], r)
        assert torch.equal(i, idx[part]) and torch.equal(v, w[part])
        assert torch.equal(d[part], M.route_backward(l[part], i, r, v, los.counts, los.losses))


@pytest.mark.parametrize("rows,stride", [(2200, 2 ** 20 + 8), (70, 2 ** 25)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_adapter_rows(rows, stride, dtype):
    h, n, rank = 136, 200, 16
    x = torch.randn(rows, h, device="cuda").bfloat16()
    base = torch.randn(rows, n, device="cuda").to(dtype)
    a, b = (torch.randn(5, rank, h, device="cuda") / 12).bfloat16(), torch.randn(5, n, rank, device="cuda").bfloat16()
    ids = torch.randint(-1, 5, (rows,), device="cuda").int()
    want = M.lora_add(base, x, a, b, ids)
    wide = _spread(base, stride)
    assert torch.equal(M.lora_add(base, _spread(x, stride), a, b, ids), want)
    assert torch.equal(M.lora_add(wide, x, a, b, ids), want)
    assert torch.equal(M.lora_add(wide, x, a, b, ids, out=wide), want)


def test_wide_expert_rows():
    t, k, h = 16500, 2, 65536
    rows = t * k + 100
    assert (rows - 200) * h > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(0)
    row_of = torch.randperm(t * k, device="cuda", generator=g).int().view(t, k)
    y = torch.randn(rows, h, device="cuda", generator=g)
    d_out = torch.randn(t, h, device="cuda", dtype=torch.bfloat16, generator=g)
    w = torch.rand(t, k, device="cuda", generator=g)
    counts = torch.tensor([t * k], device="cuda", dtype=torch.int32)
    offsets = torch.tensor([0, rows - 30], device="cuda", dtype=torch.int32)
    dy, dw = M.combine_backward(d_out, y, row_of, w, counts, offsets)
    assert not dy[t * k:].any()
    of_row = torch.empty(t * k, dtype=torch.long, device="cuda")
    of_row[row_of.view(-1).long()] = torch.arange(t * k, device="cuda")
    for row in (0, 16384, 32768, t * k - 1):
        slot = int(of_row[row])
        d = d_out[slot // k]
        assert torch.equal(dy[row], w.view(-1)[slot] * d.float())
        terms = d.double() * y[row].double()
        # 256 products a thread and slot, then 5 + 8 additions
        assert abs(float(dw.view(-1)[slot]) - float(terms.sum())) <= 270 * 2.0 ** -24 * float(terms.abs().sum())
    del dy, d_out
    act = M.swiglu_rows(y, y, offsets)
    for row in (0, 32768, rows - 31):
        assert torch.equal(act[row:row + 1], M.swiglu_rows(y[row:row + 1], y[row:row + 1],
                                                           torch.tensor([0, 1], device="cuda", dtype=torch.int32)))
