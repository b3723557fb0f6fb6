"""The combine's gradient and the adapters refuse what they cannot take, on the host
before any CUDA call (so these run without a GPU)."""
import pytest
import torch

from sparse_mixture_experts_09_b200 import build_lib
from sparse_mixture_experts_09_b200 import moe as M


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return M.lib()


def combine(L, d_out=16, y=16, row_of=16, w=16, counts=16, offsets=16, dy=16, dw=16, t=4, k=2, h=64, e=8, rows=2048):
    return L.moe_combine_backward(d_out, y, row_of, w, counts, offsets, dy, dw, t, k, h, e, rows, None)


@pytest.mark.parametrize("bad", [dict(t=-1), dict(rows=-1), dict(rows=1 << 31), dict(k=0), dict(k=9), dict(h=0), dict(h=60),
                                 dict(h=-8), dict(e=0), dict(e=513), dict(t=1 << 30, k=2), dict(d_out=None), dict(d_out=24),
                                 dict(y=None), dict(y=20), dict(row_of=None), dict(w=None), dict(counts=None),
                                 dict(offsets=None), dict(dy=20), dict(dw=2)])
def test_combine_backward_refuses(L, bad):
    assert combine(L, **bad) in (1, 2)
    assert L.moe_last_error()


def test_combine_backward_nothing_wanted(L):
    assert combine(L, dy=None, dw=None) == 0


def lora(**kw):
    a = dict(num_rows=4, x_stride=64, base_stride=32, out_stride=32, in_features=64, out_features=32, rank=16,
             num_adapters=3, out_fp32=1)
    a.update(kw)
    return M._LoraArgs(**a)


def add(L, args, base=16, x=16, a=16, b=16, ids=16, scale=None, out=32, ws=256, size=1 << 30):
    return L.moe_lora_add(args, base, x, a, b, ids, scale, out, ws, size, None)


@pytest.mark.parametrize("bad", [dict(num_rows=-1), dict(num_rows=(1 << 24) + 1), dict(in_features=0), dict(in_features=60),
                                 dict(out_features=0), dict(out_features=20), dict(out_features=-8), dict(rank=0), dict(rank=4),
                                 dict(rank=12), dict(rank=136), dict(num_adapters=0), dict(num_adapters=16385),
                                 dict(x_stride=56), dict(x_stride=68), dict(base_stride=24), dict(out_stride=36),
                                 dict(out_fp32=2), dict(in_features=(1 << 20) + 8, x_stride=1 << 21)])
def test_lora_sizes_are_refused(L, bad):
    assert add(L, lora(**bad)) in (1, 2)
    assert L.moe_last_error()
    assert L.moe_lora_workspace(lora(**bad)) == 0


@pytest.mark.parametrize("bad,status", [(dict(base=None), 1), (dict(base=24), 1), (dict(x=None), 1), (dict(x=8), 1), (dict(a=None), 1),
                                        (dict(b=None), 1), (dict(b=8), 1), (dict(ids=None), 1), (dict(ids=2), 1), (dict(scale=2), 1),
                                        (dict(out=None), 1), (dict(out=8), 1), (dict(ws=None), 3), (dict(ws=128), 3), (dict(size=0), 3)])
def test_lora_pointers_are_refused(L, bad, status):
    assert add(L, lora(num_rows=1000), **bad) == status
    assert L.moe_last_error()


def test_lora_aliases_and_empty(L):
    assert add(L, lora(out_stride=40), base=16, out=16) == 1       # in place with another stride
    assert add(L, None) == 1
    assert add(L, lora(num_rows=0), base=None, x=None, ids=None, out=None, ws=None, size=0) == 0
    # many rows: the sorted row numbers and the rank-wide sums at least
    assert L.moe_lora_workspace(lora(num_rows=1000)) >= 1000 * (4 + 16 * 4)
    assert L.moe_lora_workspace(lora()) == 0 and not L.moe_last_error()   # few rows need none


def test_binding_refuses():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int32)
    for args, match in (((torch.zeros(4, 32), bf(4, 64), bf(3, 16, 64), bf(3, 32, 16), ids), "CUDA"),
                        ((torch.zeros(4, 32), bf(4, 60), bf(3, 16, 64), bf(3, 32, 16), ids), "CUDA|shape"),
                        ((torch.zeros(4, 32), bf(64), bf(3, 16, 64), bf(3, 32, 16), ids), "rows, in"),
                        ((torch.zeros(4, 32), torch.zeros(4, 64), bf(3, 16, 64), bf(3, 32, 16), ids), "bfloat16")):
        with pytest.raises(ValueError, match=match):
            M.lora_add(*args)
    for t, shape, match in ((bf(4, 64), (4, 63), "shape"), (bf(4, 64).float(), (4, 64), "bfloat16")):
        with pytest.raises(ValueError, match=match):
            M._rows(t, "x", (torch.bfloat16,), shape)
    with pytest.raises(ValueError, match="2-D"):
        M.combine_backward(bf(4), torch.zeros(8, 64), ids[:, None], torch.zeros(4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        M.combine_backward(bf(4, 64), torch.zeros(8, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))


def test_layer_entry_points_refuse(L):
    s = M.make_shape(4, 128, 128, 8, 2)
    r = lambda **kw: M._RoutingArgs(**{**dict(num_tokens=4, logits_stride=8, num_experts=8, num_experts_per_tok=2, num_groups=1,
                                              topk_groups=1, group_top=1, renormalize=1, weight_scale=1.0), **kw})
    fwd = lambda routing, ws=256, size=1 << 30, x=16, bias=None: L.moe_forward_routing(
        s, routing, x, 16, None, bias, 16, 16, 16, None, 16, ws, size, None)
    for bad in (dict(num_tokens=5), dict(num_experts=16, logits_stride=16), dict(num_experts_per_tok=3), dict(logits_bf16=1),
                dict(logits_stride=9), dict(num_groups=3), dict(scoring=5)):
        assert fwd(r(**bad)) in (1, 2) and L.moe_last_error()
    assert fwd(None) == 1 and fwd(r(), x=None) == 1 and fwd(r(), bias=8) == 1
    assert fwd(r(), ws=None) == 3 and fwd(r(), size=1) == 3
    rows = lambda tok=16, off=16, ad=16, t=4, n=8, e=8, g=2, out=16: L.moe_lora_rows(tok, off, ad, t, n, e, g, out, None)
    for bad in (dict(tok=None), dict(off=None), dict(ad=None), dict(out=None), dict(t=-1), dict(n=-1), dict(e=0), dict(e=513),
                dict(g=0), dict(g=2049), dict(out=2)):
        assert rows(**bad) in (1, 2) and L.moe_last_error()
    assert rows(n=0, tok=None, off=None, out=None) == 0
    act = lambda g=16, u=16, off=16, e=8, n=4, i=64, h=16: L.moe_swiglu_rows(g, u, off, e, n, i, h, None)
    for bad in (dict(g=None), dict(u=8), dict(off=None), dict(h=None), dict(e=0), dict(n=-1), dict(i=0), dict(i=60)):
        assert act(**bad) in (1, 2) and L.moe_last_error()
    assert act(n=0, g=None, u=None, off=None, h=None) == 0


def test_layer_binding_refuses():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    x, wr, w1, w2 = bf(4, 128), bf(8, 128), bf(8, 256, 128), bf(8, 128, 256)
    ids = torch.zeros(4, dtype=torch.int32)
    a, b = bf(3, 8, 16, 128), bf(3, 8, 256, 16)
    lora = lambda ad, i=ids: M.forward_lora(x, wr, w1, w1, w2, 2, ad, i)
    for ad, match in ((M.LoraExperts(), "no pair"), (M.LoraExperts(a1=a), "go together"), (M.LoraExperts(a1=a, b1=bf(3, 8, 128, 16)), "b1"),
                      (M.LoraExperts(a2=a, b2=b), "a2"), (M.LoraExperts(a1=a, b1=b, scale=torch.ones(2)), "scale"),
                      (M.LoraExperts(a1=a, b1=b, a3=bf(2, 8, 16, 128), b3=bf(2, 8, 256, 16)), "b3")):
        with pytest.raises(ValueError, match=match):
            lora(ad)
    with pytest.raises(ValueError, match="adapter"):
        lora(M.LoraExperts(a1=a, b1=b), ids[:3])
    with pytest.raises(ValueError, match="bias"):
        M.forward_routing(x, wr, w1, w1, w2, M.Routing(2), torch.zeros(9))
    with pytest.raises(ValueError, match="CUDA"):
        M.forward_routing(x, wr, w1, w1, w2, M.Routing(2), torch.zeros(8))
    with pytest.raises(ValueError, match="scoring"):
        M.forward_routing(x, wr, w1, w1, w2, M.Routing(2, "relu"))
