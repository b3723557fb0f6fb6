"""Low-rank adapters of many requests on the GPU against fp64.

Tolerances, derived (u = 2^-24). The shrink adds H products in fp32 in chains: at most
8 ceil(H / 2048) products of one thread and 13 partial sums, or 16-wide matrix products into
fresh sums every 64 features (each at most 2 u off, as an accumulation that truncates) and H / 64
additions of those: H / 64 + 32 covers both with the scale's rounding for H <= 4096, twice that
all H <= 14336; it enters the output through b. The expand adds rank <= 128 products, the parts of
the intermediate hold 2^-24 (fp32 outputs) or 2^-16 (bf16) of it. Then one addition and, for
bf16, one rounding: 2^-8 of the value."""
import numpy as np
import pytest
import torch

from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _case(r, h, n, rank, ad, dtype, order, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, ad, (r,), generator=g)
    if order == "runs":
        ids = ids[torch.sort(torch.randint(0, max(1, min(r, 5)), (r,), generator=g)).values]
    if order == "one":
        ids[:] = ad - 1
    if order == "none":
        ids[:] = -1
    x = torch.randn(r, h, generator=g).bfloat16()
    a = (torch.randn(ad, rank, h, generator=g) / h ** 0.5).bfloat16()
    b = (torch.randn(ad, n, rank, generator=g) / rank ** 0.5).bfloat16()
    scale = torch.randn(ad, generator=g)
    base = torch.randn(r, n, generator=g).to(dtype)
    return base, x, a, b, ids.int(), scale


def _want(base, x, a, b, ids, scale):
    """(fp64 result, tolerance)."""
    out = base.double().clone()
    tol = torch.zeros_like(out)
    h, rank = x.shape[1], a.shape[1]
    for g in torch.unique(ids).tolist():
        if g < 0 or g >= a.shape[0]:
            continue
        at = (ids == g).nonzero()[:, 0]
        xg, ag, bg = x[at].double(), a[g].double(), b[g].double()
        s = 1.0 if scale is None else float(scale[g])
        t = s * (xg @ ag.t())
        t_mag = abs(s) * (xg.abs() @ ag.abs().t())
        out[at] += t @ bg.t()
        parts = 2.0 ** -24 if base.dtype == torch.float32 else 2.0 ** -16
        tol[at] = (2 * (h / 64 + 32) * U * t_mag) @ bg.abs().t() + ((2 * rank + 4) * U + parts) * (t.abs() @ bg.abs().t())
    rnd = 2 * U if base.dtype == torch.float32 else 2.0 ** -8 * 1.01
    tol = tol * 1.01 + rnd * out.abs()
    tol[(ids < 0) | (ids >= a.shape[0])] = 0           # rows without an adapter: copied
    return out, tol


def _check(case, **kw):
    base, x, a, b, ids, scale = case
    got = M.lora_add(base.cuda(), x.cuda(), a.cuda(), b.cuda(), ids.cuda(), None if scale is None else scale.cuda(), **kw)
    want, tol = _want(*case)
    assert got.dtype == base.dtype
    err = (got.cpu().double() - want).abs()
    assert (err <= tol).all(), (err - tol).max()
    return got


SIZES = [(1, 8, 8, 8, 1), (1, 14336, 4096, 16, 4), (2, 4096, 1032, 8, 3), (3, 72, 40, 24, 2), (7, 200, 136, 40, 5),
         (33, 1024, 4104, 64, 9), (61, 512, 256, 16, 128), (64, 136, 264, 128, 2), (100, 96, 1000, 104, 100),
         (130, 2048, 520, 32, 7), (300, 640, 776, 64, 3), (513, 264, 392, 16, 40), (700, 128, 128, 72, 200)]


@pytest.mark.parametrize("r,h,n,rank,ad", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", ["mixed", "runs", "one", "none"])
def test_against_fp64(r, h, n, rank, ad, dtype, order):
    _check(_case(r, h, n, rank, ad, dtype, order, r + n))


@pytest.mark.parametrize("r,h,n,rank,ad", [(159, 264, 200, 16, 2), (160, 264, 200, 16, 20), (160, 264, 200, 16, 21), (300, 136, 264, 8, 200),
                                           (511, 72, 104, 16, 128), (512, 72, 104, 16, 400), (300, 136, 264, 24, 200),
                                           (900, 200, 1032, 128, 3), (260, 328, 40, 128, 17), (400, 96, 168, 104, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_around_the_change_of_form(r, h, n, rank, ad, dtype):
    _check(_case(r, h, n, rank, ad, dtype, "mixed", r + ad))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("r", [5, 190, 1100])
def test_in_place_no_scale_and_into_out(dtype, r):
    base, x, a, b, ids, _ = _case(r, 256, 328, 16, 6, dtype, "mixed", r)
    want = _check((base, x, a, b, ids, None))
    args = [t.cuda() for t in (base, x, a, b, ids)]
    out = torch.full_like(args[0], float("nan"))
    assert M.lora_add(*args, out=out) is out and torch.equal(out, want)
    assert M.lora_add(*args, out=args[0]) is args[0] and torch.equal(args[0], want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("r", [6, 300])
def test_strided_rows(dtype, r):
    base, x, a, b, ids, scale = [t.cuda() for t in _case(r, 264, 328, 16, 6, dtype, "mixed", r)]
    want = M.lora_add(base, x, a, b, ids, scale)
    big_x = torch.full((r, 800), float("nan"), dtype=x.dtype, device="cuda")
    big_b = torch.full((r, 1000), float("nan"), dtype=dtype, device="cuda")
    big_o = torch.full((r + 2, 600), 7.0, dtype=dtype, device="cuda")
    big_x[:, 16:280] = x
    big_b[:, 8:336] = base
    M.lora_add(big_b[:, 8:336], big_x[:, 16:280], a, b, ids, scale, out=big_o[1:-1, 24:352])
    assert torch.equal(big_o[1:-1, 24:352], want)
    big_o[1:-1, 24:352] = 7.0
    assert (big_o == 7.0).all()                       # nothing outside the view was written


@pytest.mark.parametrize("r", [4, 200])
def test_ids_outside_the_adapters_are_none(r):
    base, x, a, b, ids, scale = _case(r, 64, 64, 8, 4, torch.float32, "mixed", 3)
    ids[0], ids[1], ids[2] = 4, -7, 2 ** 31 - 1
    _check((base, x, a, b, ids, scale))


@pytest.mark.parametrize("r", [4, 500])
def test_infinities_stay_in_their_rows(r):
    base, x, a, b, ids, scale = _case(r, 128, 72, 16, 4, torch.float32, "mixed", 3)
    ids[:] = (torch.arange(r) % 3).int()
    ids[1] = -1
    x[1] = float("nan")                               # a row without an adapter: never multiplied
    x[2, 5] = float("inf")
    want, _ = _want(base, x, a, b, ids, scale)
    got = M.lora_add(base.cuda(), x.cuda(), a.cuda(), b.cuda(), ids.cuda(), scale.cuda()).cpu()
    rows = torch.ones(r, dtype=torch.bool)
    rows[2] = False
    assert torch.isfinite(got[rows]).all() and torch.equal(got[1], base[1])
    assert not torch.isfinite(got[2]).any()


def test_no_rows():
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)
    out = M.lora_add(e(0, 64), e(0, 128, dtype=torch.bfloat16), e(2, 8, 128, dtype=torch.bfloat16).zero_(),
                     e(2, 64, 8, dtype=torch.bfloat16).zero_(), e(0, dtype=torch.int32))
    assert out.shape == (0, 64)


def test_many_adapters_few_of_them_used():
    """Thousands of adapters loaded, rows of three of them and of none; sizes past 32 bits in a."""
    r, h, n, rank, ad = 300, 8192, 136, 16, 17000 // 2
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn(ad * 2, rank, h, device="cuda", generator=g, dtype=torch.bfloat16)[:16384].contiguous()
    assert a.numel() > 2 ** 31 - 1
    b = torch.randn(16384, n, rank, device="cuda", generator=g, dtype=torch.bfloat16) / 4
    ids = torch.tensor([16383, 5, -1, 16382], dtype=torch.int32, device="cuda").repeat_interleave(75)
    x = torch.randn(r, h, device="cuda", generator=g, dtype=torch.bfloat16) / 64
    base = torch.randn(r, n, device="cuda", generator=g)
    for k in (r, 9):                                 # as tiles, and a row at a time
        rows = torch.linspace(0, r - 1, k).long().cuda()
        got = M.lora_add(base[rows], x[rows], a, b, ids[rows])
        for i in (0, k // 3, k // 2, k - 1):
            j = int(ids[rows][i])
            want = base[rows][i].double()
            if j >= 0:
                t = a[j].double() @ x[rows][i].double()
                want = want + b[j].double() @ t
                mag = b[j].double().abs() @ (a[j].double().abs() @ x[rows][i].double().abs())
                assert ((got[i].double() - want).abs() <= (h / 32 + 200) * U * (mag + want.abs())).all()
            else:
                assert torch.equal(got[i], base[rows][i])


@pytest.mark.parametrize("r", [16, 600])
def test_repeats_streams_and_graphs_give_the_same_bits(r):
    base, x, a, b, ids, scale = [t.cuda() for t in _case(r, 512, 520, 32, 9, torch.bfloat16, "mixed", r)]
    want = M.lora_add(base, x, a, b, ids, scale)
    for _ in range(3):
        assert torch.equal(want, M.lora_add(base, x, a, b, ids, scale))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = M.lora_add(base, x, a, b, ids, scale, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, capture_error_mode="thread_local"):
            out = M.lora_add(base, x, a, b, ids, scale)
        graphs.append((graph, out))
    ids.copy_(ids.flip(0))
    want = M.lora_add(base, x, a, b, ids, scale)
    for graph, out in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out in graphs)


def test_a_row_does_not_depend_on_the_others():
    """The same row alone and within a batch: equal up to the sums' order (2 x the tolerance)."""
    case = _case(400, 1024, 264, 16, 3, torch.float32, "mixed", 5)
    base, x, a, b, ids, scale = case
    got = _check(case)
    _, tol = _want(*case)
    for r in (0, 63, 64, 399):
        one = M.lora_add(*[t.cuda() for t in (base[r:r + 1], x[r:r + 1], a, b, ids[r:r + 1], scale)])
        assert ((one - got[r:r + 1]).abs().cpu() <= 2 * tol[r:r + 1]).all()
