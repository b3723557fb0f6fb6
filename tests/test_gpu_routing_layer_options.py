"""The layer with general routing and with adapters under the options that the other tests leave
out: against the layer put together from its parts, on one set of logits."""
import pytest
import torch

from sparse_mixture_experts_09_b200 import moe as M
from tests._cases import assert_layer_close

pytestmark = pytest.mark.gpu


def _inputs(t, h, i, e, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    w = [(n(e, h) / h ** 0.5).bfloat16(), (n(e, i, h) / h ** 0.5).bfloat16(), (n(e, i, h) / h ** 0.5).bfloat16(),
         (n(e, h, i) / i ** 0.5).bfloat16()]
    return n(t, h).bfloat16(), w, 0.3 * n(e), 0.05 * n(e), n(t, h).bfloat16(), g


@pytest.mark.parametrize("t,e,r", [(1, 8, M.Routing(2, "sigmoid")), (250, 64, M.Routing(8, "sigmoid", 8, 4, 2, True, 2.5)),
                                   (3000, 8, M.Routing(2, "softmax", renormalize=False))])
@pytest.mark.parametrize("bf16_logits", [False, True])
def test_forward_routing_is_its_parts(t, e, r, bf16_logits):
    h, i = 256, 256
    x, (wr, w1, w3, w2), logit_bias, bias, res, _ = _inputs(t, h, i, e, t)
    out = M.forward_routing(x, wr, w1, w3, w2, r, bias, residual=res, logit_bias=logit_bias, router_bf16_logits=bf16_logits)
    logits = M.router_topk(x, wr, 1, logit_bias, True, router_bf16_logits=bf16_logits)[2]
    idx, w = M.route(logits, r, bias)
    ws = M.make_workspace(M.make_shape(t, h, i, e, r.k))
    perm = M.permute(idx, x, e, i, ws)
    y = M.grouped_swiglu(perm["x_perm"], perm["offsets"], w1, w3, w2, t, r.k, ws)
    want = M.combine(y, perm["row_of"], w, res, e, i)
    assert_layer_close(out.float().cpu().numpy(), want.float().cpu().numpy())


@pytest.mark.parametrize("t,e,k,n", [(1, 8, 2, 3), (64, 64, 8, 5), (2000, 8, 2, 4)])
@pytest.mark.parametrize("bf16_logits", [False, True])
def test_forward_lora_of_zero_adapters_is_the_layer(t, e, k, n, bf16_logits):
    h, i = 128, 256
    x, (wr, w1, w3, w2), logit_bias, bias, res, g = _inputs(t, h, i, e, t + e)
    a = lambda *s: (torch.randn(*s, device="cuda", generator=g) / s[-1] ** 0.5).bfloat16()
    ad = M.LoraExperts(a(n, e, 16, h), torch.zeros_like(a(n, e, i, 16)), a(n, e, 8, h), torch.zeros_like(a(n, e, i, 8)),
                       a(n, e, 16, i), torch.zeros_like(a(n, e, h, 16)))
    ids = torch.randint(-1, n, (t,), device="cuda", generator=g).int()
    for routing in (None, M.Routing(k, "sigmoid", scale=1.5)):
        got = M.forward_lora(x, wr, w1, w3, w2, k, ad, ids, res, logit_bias, router_bf16_logits=bf16_logits,
                             routing=routing, bias=None if routing is None else bias)
        want = (M.forward(x, wr, w1, w3, w2, k, residual=res, logit_bias=logit_bias, router_bf16_logits=bf16_logits)
                if routing is None else
                M.forward_routing(x, wr, w1, w3, w2, routing, bias, res, logit_bias, router_bf16_logits=bf16_logits))
        assert_layer_close(got.float().cpu().numpy(), want.float().cpu().numpy())
