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
