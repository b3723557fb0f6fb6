"""The layer with general routing, with adapters, and a tuning step of a router beside frozen
experts: the operators as they are used together, against fp64."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from oracle import routing_oracle as R
from sparse_mixture_experts_09_b200 import moe as M
from tests._cases import assert_layer_close

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _weights(e, h, i, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    return ((n(e, h) / h ** 0.5).bfloat16(), (n(e, i, h) / h ** 0.5).bfloat16(),
            (n(e, i, h) / h ** 0.5).bfloat16(), (n(e, h, i) / i ** 0.5).bfloat16())


def _silu(v):
    return v / (1 + np.exp(-v))


def _experts(x, idx, w, w1, w3, w2, res=None, lora=None, adapter=None):
    """fp64 layer for given routing; h and the output rounded to bf16 as the layer stores them
    (the storage mode that assert_layer_close's tolerance is for)."""
    f = lambda t: t.double().numpy()
    x, out = f(x), np.zeros((x.shape[0], x.shape[1])) if res is None else f(res).copy()
    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            e = idx[t, j]
            a1, a3, a2 = f(w1[e]), f(w3[e]), f(w2[e])
            if lora is not None and 0 <= adapter[t] < lora["n"]:
                a = int(adapter[t])
                s = 1.0 if lora["scale"] is None else float(lora["scale"][a])
                add = lambda m, p: m if lora["b" + p] is None else m + s * f(lora["b" + p][a, e]) @ f(lora["a" + p][a, e])
                a1, a3, a2 = add(a1, "1"), add(a3, "3"), add(a2, "2")
            h = O.round_bf16(_silu(a1 @ x[t]) * (a3 @ x[t]))
            out[t] += w[t, j] * (a2 @ h)
    return O.round_bf16(out)


@pytest.mark.parametrize("t,e,r", [(1, 8, M.Routing(2, "sigmoid", scale=2.0)), (70, 16, M.Routing(4, "sigmoid", 4, 2, 2, True, 2.5)),
                                   (300, 64, M.Routing(8, "softmax", 8, 4, 2, False)), (33, 8, M.Routing(2))])
@pytest.mark.parametrize("layout", [M.ROW_MAJOR, M.BLOCKED])
def test_forward_routing(t, e, r, layout):
    h, i = 128, 128
    wr, w1, w3, w2 = _weights(e, h, i, e)
    g = torch.Generator().manual_seed(t)
    x, res = torch.randn(t, h, generator=g).bfloat16(), torch.randn(t, h, generator=g).bfloat16()
    bias = 0.05 * torch.randn(e, generator=g)
    dev = [v.cuda() for v in (w1, w3, w2)]
    packed = M.pack_weights(*dev) if layout == M.BLOCKED else dev
    for b in (None, bias):
        bc = None if b is None else b.cuda()
        out = M.forward_routing(x.cuda(), wr.cuda(), *packed, r, bc, residual=res.cuda(), weight_layout=layout)
        # the layer's own logits decide; their values are the router tests' matter
        logits = M.router_topk(x.cuda(), wr.cuda(), 1, return_logits=True)[2].cpu()
        idx, w = R.route(logits.double().numpy(), r.k, r.scoring, r.num_groups, r.topk_groups, r.group_top,
                         r.renormalize, r.scale, None if b is None else b.double().numpy())
        pick = np.arange(0, t, max(1, t // 40))
        want = _experts(x[pick], idx[pick], w[pick], w1, w3, w2, res[pick])
        assert_layer_close(out.cpu().float().numpy()[pick], want)


def test_default_routing_is_the_layer():
    wr, w1, w3, w2 = [v.cuda() for v in _weights(8, 256, 256, 1)]
    x = torch.randn(200, 256, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    a, b = M.forward(x, wr, w1, w3, w2, 2), M.forward_routing(x, wr, w1, w3, w2, M.Routing(2))
    # the weights differ in their last places (fp32 against double), the sum is rounded to bf16
    assert_layer_close(b.float().cpu().numpy(), a.float().cpu().numpy())
    assert (a == b).float().mean() > 0.99


def test_forward_routing_in_a_graph_shares_no_state():
    wr, w1, w3, w2 = [v.cuda() for v in _weights(16, 128, 128, 2)]
    r, bias = M.Routing(4, "sigmoid", 4, 2, 2), 0.05 * torch.randn(16, device="cuda")
    x = torch.randn(40, 128, device="cuda").bfloat16()
    ws = M.make_workspace(M.make_shape(40, 128, 128, 16, 4))
    out = torch.empty_like(x)
    run = lambda: M.forward_routing(x, wr, w1, w3, w2, r, bias, ws=ws, out=out)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        run()
    x.copy_(torch.randn(40, 128, device="cuda").bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, M.forward_routing(x, wr, w1, w3, w2, r, bias))


def _adapters(n, e, h, i, rank, seed, which="123", scale=True):
    g = torch.Generator().manual_seed(seed)
    z = lambda *s: torch.randn(*s, generator=g)
    d = {"n": n, "scale": torch.rand(n, generator=g) + 0.5 if scale else None}
    for p, n_in, n_out, r in (("1", h, i, rank), ("3", h, i, rank), ("2", i, h, 2 * rank)):
        on = p in which
        d["a" + p] = (z(n, e, r, n_in) / n_in ** 0.5).bfloat16() if on else None
        d["b" + p] = (0.5 * z(n, e, n_out, r) / r ** 0.5).bfloat16() if on else None
    return d


def _cuda(d):
    return M.LoraExperts(*[None if d[k] is None else d[k].cuda() for k in ("a1", "b1", "a3", "b3", "a2", "b2", "scale")])


@pytest.mark.parametrize("t,which,scale", [(1, "123", True), (20, "123", True), (20, "2", False), (64, "13", True), (300, "123", True)])
@pytest.mark.parametrize("layout", [M.ROW_MAJOR, M.BLOCKED])
def test_forward_lora(t, which, scale, layout):
    h, i, e = 128, 256, 4
    wr, w1, w3, w2 = _weights(e, h, i, 3)
    g = torch.Generator().manual_seed(t)
    x, res = torch.randn(t, h, generator=g).bfloat16(), torch.randn(t, h, generator=g).bfloat16()
    adapter = torch.randint(-1, 3, (t,), generator=g).int()
    lora = _adapters(3, e, h, i, 8, 5, which, scale)
    dev = [v.cuda() for v in (w1, w3, w2)]
    packed = M.pack_weights(*dev) if layout == M.BLOCKED else dev
    out = M.forward_lora(x.cuda(), wr.cuda(), *packed, 2, _cuda(lora), adapter.cuda(), residual=res.cuda(), weight_layout=layout)
    idx, w = M.router_topk(x.cuda(), wr.cuda(), 2)
    pick = np.arange(0, t, max(1, t // 40))
    idx, w = idx.cpu().numpy()[pick], w.cpu().double().numpy()[pick]
    want = _experts(x[pick], idx, w, w1, w3, w2, res[pick], lora, adapter.numpy()[pick])
    assert_layer_close(out.float().cpu().numpy()[pick], want)
    plain = _experts(x[pick], idx, w, w1, w3, w2, res[pick])
    has = adapter.numpy()[pick] >= 0
    if has.any():                                    # the adapters move their own tokens
        assert np.abs(want - plain)[has].max() > 0.1
    if (~has).any():
        assert_layer_close(out.float().cpu().numpy()[pick][~has], plain[~has])


def test_forward_lora_with_general_routing():
    t, h, i, e = 50, 128, 128, 16
    wr, w1, w3, w2 = _weights(e, h, i, 7)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(t, h, generator=g).bfloat16()
    adapter = torch.randint(0, 2, (t,), generator=g).int()
    lora = _adapters(2, e, h, i, 8, 6)
    r, bias = M.Routing(3, "sigmoid", 4, 2, 1, True, 1.5), 0.05 * torch.randn(e, generator=g)
    out = M.forward_lora(x.cuda(), wr.cuda(), w1.cuda(), w3.cuda(), w2.cuda(), 3, _cuda(lora), adapter.cuda(),
                         routing=r, bias=bias.cuda())
    logits = M.router_topk(x.cuda(), wr.cuda(), 1, return_logits=True)[2].cpu().double().numpy()
    idx, w = R.route(logits, 3, "sigmoid", 4, 2, 1, True, 1.5, bias.double().numpy())
    assert_layer_close(out.float().cpu().numpy(), _experts(x, idx, w, w1, w3, w2, None, lora, adapter.numpy()))


def test_lora_rows_and_swiglu_rows():
    g = torch.Generator().manual_seed(3)
    t, e, k = 333, 5, 2
    idx = torch.rand(t, e, generator=g).topk(k, dim=1).indices.int()
    perm = M.permute(idx.cuda(), torch.zeros(t, 128, dtype=torch.bfloat16, device="cuda"), e, 128,
                     M.make_workspace(M.make_shape(t, 128, 128, e, k)))
    adapter = torch.randint(-2, 9, (t,), generator=g).int()
    ids = M.lora_rows(perm["token_of_row"], perm["offsets"], adapter.cuda(), 7).cpu()
    want = torch.full_like(ids, -1)
    row_of = perm["row_of"].cpu()
    for tok in range(t):
        for j in range(k):
            if 0 <= adapter[tok] < 7:
                want[row_of[tok, j]] = adapter[tok] * e + idx[tok, j]
    assert torch.equal(ids, want)
    rows, i = perm["token_of_row"].numel(), 72
    gate, up = 4 * torch.randn(rows, i, generator=g), torch.randn(rows, i, generator=g)
    h = torch.full((rows, i), 7.0, dtype=torch.bfloat16, device="cuda")
    M.swiglu_rows(gate.cuda(), up.cuda(), perm["offsets"], h)
    used = int(perm["offsets"][-1])
    ref = _silu(gate[:used].double().numpy()) * up[:used].double().numpy()
    # fp32: exponential 4u, its argument exact, addition, division, product 3u, then bf16
    assert np.all(np.abs(h[:used].cpu().double().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref) + 2.0 ** -133)
    assert (h[used:] == 7.0).all()


@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_a_tuning_step_of_the_router(scoring, renorm):
    """Router weights' gradient of  <v, layer(x)> + balance and z loss  with frozen experts: the
    step a user runs, against fp64 differentiation of the same function of the logits and
    against central differences of it."""
    t, h, i, e, k = 96, 128, 128, 8, 2
    wr, w1, w3, w2 = [v.cuda() for v in _weights(e, h, i, 11)]
    g = torch.Generator().manual_seed(4)
    x = torch.randn(t, h, generator=g).bfloat16().cuda()
    v = torch.randn(t, h, generator=g).bfloat16().cuda()
    mask = (torch.rand(t, generator=g) > 0.2).cuda()
    coef = torch.tensor([0.02, 0.001], device="cuda")
    r = M.Routing(k, scoring, renormalize=renorm, scale=1.25)
    ws = M.make_workspace(M.make_shape(t, h, i, e, k))
    # forward
    logits = M.router_topk(x, wr, 1, return_logits=True)[2]
    idx, w = M.route(logits, r)
    perm = M.permute(idx, x, e, i, ws)
    y = M.grouped_swiglu(perm["x_perm"], perm["offsets"], w1, w3, w2, t, k, ws)
    out = M.combine(y, perm["row_of"], w, None, e, i)
    los = M.router_losses(logits, idx, r, mask)
    # backward
    dy, d_w = M.combine_backward(v, y, perm["row_of"], w, perm["counts"], perm["offsets"])
    d_logits = M.route_backward(logits, idx, r, d_w, los.counts, coef, mask)
    d_wr = d_logits.t() @ x.float()

    # the same function of the logits in fp64
    l64 = logits.double().clone().requires_grad_()
    y64, rows = y.double(), perm["row_of"].long()

    def value(l):
        s = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 1)
        sel = s.gather(1, idx.long())
        ww = 1.25 * (sel / sel.sum(1, keepdim=True) if renorm else sel)
        mixed = (ww[:, :, None] * y64[rows]).sum(1)
        p = s / s.sum(1, keepdim=True)
        n = mask.sum()
        balance = e * ((los.counts[:e].double() / n) * p[mask].sum(0) / n).sum()
        z = torch.logsumexp(l[mask], 1).square().sum() / n
        return (mixed * v.double()).sum() + coef[0].double() * balance + coef[1].double() * z

    total = value(l64)
    want, = torch.autograd.grad(total, l64)
    size = float(want.abs().max())
    # fp32 terms of H-long sums: (8 + 14 + 160) u of the products' magnitudes, themselves at most
    # sqrt(H) times the sums for random signs
    assert float((d_logits.double() - want).abs().max()) <= 200 * U * np.sqrt(h) * 4 * size
    d_wr64 = want.t() @ x.double()
    assert float((d_wr.double() - d_wr64).norm() / d_wr64.norm()) <= 1e-4
    # the forward's value: out is rounded to bf16 (2^-8 of each), losses are fp32
    got = (out.double() * v.double()).sum() + (coef.double() * los.losses.double()).sum()
    bound = 2.0 ** -8 * (out.double().abs() * v.double().abs()).sum() + 1e-3
    assert abs(float(got - total.detach())) <= float(bound)
    # central differences along the gradient: error h^2 |f'''| / 6 and 2^-52 |f| / h
    step = 1e-4 * want / want.norm()
    slope = (value(logits.double() + step) - value(logits.double() - step)) / 2e-4
    assert abs(float(slope / want.norm()) - 1) <= 1e-5
    assert dy.shape == y.shape


def test_forward_lora_on_another_stream_and_captured():
    t, h, i, e = 30, 128, 128, 8
    wr, w1, w3, w2 = [v.cuda() for v in _weights(e, h, i, 21)]
    x = torch.randn(t, h, device="cuda").bfloat16()
    adapter = torch.randint(-1, 3, (t,), device="cuda").int()
    lora = _cuda(_adapters(3, e, h, i, 16, 9))
    run = lambda **k: M.forward_lora(x, wr, w1, w3, w2, 2, lora, adapter, residual=x, **k)
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        got = run()
    x.copy_(torch.randn(t, h, device="cuda").bfloat16())
    adapter.copy_(adapter.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, run())


def test_calls_on_two_streams_at_once():
    """Each call's scratch is its own: two streams work on different batches side by side."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    r = M.Routing(6, "sigmoid", 8, 4, 2)
    sets = []
    for rows in (700, 1000):
        a, b = (n(5, 16, 512) / 32).bfloat16(), (n(5, 520, 16) / 4).bfloat16()
        ids = torch.randint(-1, 5, (rows,), device="cuda", generator=g).int()
        sets.append((n(20000, 64), n(rows, 520), n(rows, 512).bfloat16(), a, b, ids))

    def run(s, **k):
        logits, base, x, a, b, ids = s
        idx, w = M.route(logits, r, **k)
        los = M.router_losses(logits, idx, r, **k)
        return (idx, w, M.route_backward(logits, idx, r, w, los.counts, los.losses, **k),
                M.lora_add(base, x, a, b, ids, **k)) + tuple(los)

    want = [run(s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for j, s in enumerate(sets):
            got[j].append(run(s, stream=streams[j]))
    torch.cuda.synchronize()
    for j in range(2):
        for out in got[j]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[j]))
