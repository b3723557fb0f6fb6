"""Routing, losses and gradients refuse what they cannot take, on the host before any
CUDA call (so these run without a GPU)."""
import ctypes

import pytest
import torch

from sparse_mixture_experts_09_b200 import build_lib
from sparse_mixture_experts_09_b200 import moe as M


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return M.lib()


def args(**kw):
    a = dict(num_tokens=4, logits_stride=8, num_experts=8, num_experts_per_tok=2, scoring=0, num_groups=1,
             topk_groups=1, group_top=1, renormalize=1, logits_bf16=0, weight_scale=1.0)
    a.update(kw)
    return M._RoutingArgs(**a)


RULE = [dict(num_groups=3), dict(num_groups=0), dict(num_groups=-1), dict(num_experts=66, logits_stride=66, num_groups=33),
        dict(num_groups=4, topk_groups=5), dict(num_groups=4, topk_groups=0), dict(num_groups=4, topk_groups=2, group_top=3),
        dict(num_groups=4, topk_groups=2, group_top=0), dict(group_top=2), dict(num_groups=8, topk_groups=1),
        dict(num_groups=4, topk_groups=1, num_experts_per_tok=3)]
SIZES = [dict(num_tokens=-1), dict(num_tokens=(1 << 30) + 1), dict(num_experts=0), dict(num_experts=513, logits_stride=513),
         dict(num_experts_per_tok=0), dict(num_experts_per_tok=9), dict(num_experts=64, logits_stride=64, num_experts_per_tok=33),
         dict(logits_stride=7), dict(logits_stride=-8), dict(scoring=2), dict(scoring=-1), dict(logits_bf16=2),
         dict(renormalize=3), dict(weight_scale=float("inf")), dict(weight_scale=float("nan"))]


@pytest.mark.parametrize("bad", RULE + SIZES)
def test_bad_rules_are_refused(L, bad):
    assert L.moe_route(args(**bad), 16, None, 16, 16, None) in (1, 2)
    assert L.moe_last_error()
    if bad in SIZES:
        assert L.moe_router_losses_workspace(args(**bad)) == 0
        assert L.moe_router_losses(args(**bad), 16, 16, None, 16, 16, 16, 256, 1 << 30, None) in (1, 2)
        assert L.moe_route_backward(args(**bad), 16, 16, 16, None, None, None, 16, None) in (1, 2)


def test_bad_pointers_are_refused(L):
    assert L.moe_route(None, 16, None, 16, 16, None) == 1
    for call in ((None, None, 16, 16), (18, None, 16, 16), (16, 6, 16, 16), (16, None, None, 16), (16, None, 16, 2)):
        assert L.moe_route(args(), *call, None) == 1
        assert L.moe_last_error()
    assert L.moe_router_losses_workspace(args()) == 0 and not L.moe_last_error()   # few tokens need none
    many = args(num_tokens=100000)
    need = L.moe_router_losses_workspace(many)
    assert need > 0
    assert L.moe_router_losses(many, 16, 16, None, 16, 16, 16, 256, need - 1, None) == 3
    assert L.moe_router_losses(many, 16, 16, None, 16, 16, 16, 128, need, None) == 3
    assert L.moe_router_losses(many, 16, 16, None, 16, 16, 16, None, need, None) == 3
    assert L.moe_router_losses(many, 16, None, None, 16, 16, 16, 256, need, None) == 1
    assert L.moe_router_losses(args(), 16, 16, None, None, 16, 16, None, 0, None) == 1
    assert L.moe_route_backward(args(), 16, 16, 16, 16, None, None, 16, None) == 1
    assert b"go together" in L.moe_last_error()
    assert L.moe_route_backward(args(), 16, 16, 16, None, 16, None, 16, None) == 1
    assert L.moe_route_backward(args(), 16, None, 16, None, None, None, 16, None) == 1
    assert L.moe_route_backward(args(), 16, 16, 16, None, None, None, None, None) == 1


def test_no_tokens_is_a_no_op(L):
    empty = args(num_tokens=0)
    assert L.moe_route(empty, None, None, None, None, None) == 0
    assert L.moe_route_backward(empty, None, None, None, None, None, None, None, None) == 0


def test_binding_refuses(L):
    r = M.Routing(2)
    l = torch.zeros(4, 8)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    for call, match in ((lambda: M.route(l, r), "CUDA"), (lambda: M.route(torch.zeros(8), r), "tokens, experts"),
                        (lambda: M.route(l.double(), r), "float32"), (lambda: M._routing_struct(M.Routing(2, "tanh"), 4, 8, 8, False), "scoring"),
                        (lambda: M.router_losses(l, idx, r), "CUDA"), (lambda: M.route_backward(l, idx, r), "CUDA")):
        with pytest.raises(ValueError, match=match):
            call()
    for t, shape, dtypes, match in ((idx, (4, 3), M._I32, "shape"), (idx.long(), (4, 2), M._I32, "int32"), (idx, (4, 2), M._I32, "CUDA")):
        with pytest.raises(ValueError, match=match):
            M._arg(t, "topk_idx", dtypes, shape)
