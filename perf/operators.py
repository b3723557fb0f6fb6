"""Operators around the sparse-MoE layer: plain forms, inputs and sizes.

Five operators, each as elementary torch operations (``own = False``) and as the calls
that a user makes of this repository (``own = True``):

- ``route``: router logits -> experts and weights (softmax or sigmoid scores, a selection
  bias, expert groups, top-k, renormalised and scaled weights);
- ``losses``: load-balancing loss and z-loss of the router over unmasked tokens;
- ``route_backward``: gradient of the weights and of both losses in the logits;
- ``combine_backward``: gradient of the weighted combine in the expert rows and the
  routing weights;
- ``lora``: low-rank adapters of many requests beside a shared projection.

Selections (which expert, which group) are decided on values in 64 bits, so that they do
not hang on a rounding; equal values go to the lower index.
"""
from __future__ import annotations

import math

import torch

own = False

ROW_PAD = 128  # expert groups of routed rows are padded to this many rows


# ---- cases ----

def _route(op, name, t, e, k, **kw):
    case = {"op": op, "t": t, "e": e, "k": k, "scoring": "softmax", "groups": 1, "topk_groups": 1,
            "group_top": 1, "bias": False, "renormalize": True, "scale": 1.0, "dtype": "fp32",
            "masked": 0.0}
    case.update(kw)
    if name:
        case["name"] = name
    return case


def _combine(name, t, h, k, e):
    case = {"op": "combine_backward", "t": t, "h": h, "k": k, "e": e}
    if name:
        case["name"] = name
    return case


def _lora(name, rows, h, n, rank, adapters, dtype, order):
    case = {"op": "lora", "rows": rows, "h": h, "n": n, "rank": rank, "adapters": adapters,
            "dtype": dtype, "order": order}
    if name:
        case["name"] = name
    return case


_GROUPED = {"scoring": "sigmoid", "groups": 8, "topk_groups": 4, "group_top": 2, "bias": True,
            "scale": 2.5}


def listed():
    return [
        # one new token of one request: latency
        _route("route", "route 1 token", 1, 8, 2),
        # a serving batch under a sigmoid router with a balance bias and groups, bf16 logits
        _route("route", "route decode batch", 250, 64, 8, dtype="bf16", **_GROUPED),
        # a long prefill (or training batch) over many experts
        _route("route", "route prefill", 16384, 256, 8, **_GROUPED),
        # one layer of a padded training batch at the 8-expert configuration
        _route("losses", "losses 8 experts", 4096, 8, 2, masked=0.15),
        # the concatenated logits of several layers, many experts
        _route("losses", "losses 64 experts", 65521, 64, 6, masked=0.05),
        # the gradient that goes with the first of these: weights, balance and z terms
        _route("route_backward", "route backward 8 experts", 4096, 8, 2, masked=0.15),
        # and of the grouped sigmoid router
        _route("route_backward", "route backward 256 experts", 16384, 256, 8, **_GROUPED),
        # gradient of the combine for a small batch of a router that is being tuned
        _combine("combine backward 16 tokens", 16, 4096, 2, 8),
        # and for a training sequence
        _combine("combine backward 4096 tokens", 4096, 4096, 2, 8),
        # one token's two routed rows beside the down projection of the experts
        _lora("lora 2 rows", 2, 14336, 4096, 16, 64, "fp32", "mixed"),
        # a decode batch, a request per row, beside a bf16 projection
        _lora("lora 61 rows", 61, 4096, 14336, 16, 128, "bf16", "mixed"),
        # prefill of a few long requests beside the gate (or up) projection, fp32 sums
        _lora("lora 4096 rows", 4096, 4096, 14336, 64, 16, "fp32", "runs"),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "losses", "route_backward", "combine_backward", "lora", "lora"))
    if op == "combine_backward":
        h = 8 * _between(rng, 16, 768)
        k = rng.randint(1, 4)
        t = _between(rng, 1, max(2, min(8192, 33_000_000 // (h * k))))
        return _combine(None, t, h, k, rng.choice((8, 8, 16, 64)))
    if op == "lora":
        h, n = 8 * _between(rng, 64, 1792), 8 * _between(rng, 64, 1792)
        rows = _between(rng, 1, max(2, min(4096, 50_000_000 // (h + n))))
        return _lora(None, rows, h, n, rng.choice((8, 16, 24, 32, 64)), _between(rng, 1, 16 if rows > 256 else 100),
                     rng.choice(("bf16", "fp32")), rng.choice(("mixed", "runs")))
    kw = {"scoring": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5,
          "renormalize": rng.random() < 0.8, "scale": rng.choice((1.0, 1.0, 2.5)),
          "dtype": rng.choice(("fp32", "bf16")), "masked": rng.choice((0.0, 0.1, 0.4))}
    if rng.random() < 0.5:
        kw["groups"] = rng.choice((2, 4, 8))
        kw["topk_groups"] = rng.randint(1, kw["groups"])
        kw["group_top"] = rng.choice((1, 2))
        e = kw["groups"] * rng.randint(8, 32)
        room = kw["topk_groups"] * (e // kw["groups"])
    else:
        e = _between(rng, 4, 256)
        room = e
    k = rng.randint(1, min(8, room))
    t = _between(rng, 1, min(65536, 4_000_000 // e))
    return _route(op, None, t, e, k, **kw)


# ---- inputs ----

_DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _rand(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _prepare_routing(case, g):
    t, e, k = case["t"], case["e"], case["k"]
    # logits of unit-variance tokens under a router of unit rows, wider for some experts
    logits = (_rand(g, t, e) * (0.6 + torch.rand(e, device="cuda", generator=g))).to(_DTYPE[case["dtype"]])
    st = {"case": case, "logits": logits}
    # balance biases after some updates of a few hundredths
    st["bias"] = 0.05 * _rand(g, e) if case["bias"] else None
    if case["op"] == "route":
        return st
    # slots as a forward pass chose them: distinct experts of a token
    st["idx"] = torch.topk(logits.float() + 0.1 * _rand(g, t, e), k, dim=1).indices.to(torch.int32)
    st["mask"] = (torch.rand(t, device="cuda", generator=g) >= case["masked"]) if case["masked"] else None
    if case["op"] == "route_backward":
        st["d_w"] = 1e-2 * _rand(g, t, k)
        # what the losses' coefficients hand down: 0.01 and 0.001
        st["d_losses"] = torch.tensor([1e-2, 1e-3], device="cuda") * (1 + 0.1 * _rand(g, 2))
        keep = torch.ones(t, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"]
        counts = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
        counts.index_add_(0, st["idx"].reshape(-1).long(), keep[:, None].expand(t, k).reshape(-1).int())
        counts[e] = keep.sum()
        st["counts"] = counts
    return st


def _max_rows(case):
    """Rows of the routed-row buffers: whole padded groups, whatever the routing."""
    return (case["t"] * case["k"] + ROW_PAD - 1) // ROW_PAD * ROW_PAD + ROW_PAD * case["e"]


def _prepare_combine(case, g):
    t, h, k, e = case["t"], case["h"], case["k"], case["e"]
    idx = torch.topk(_rand(g, t, e), k, dim=1).indices.reshape(-1)
    counts = torch.bincount(idx, minlength=e)
    padded = (counts + ROW_PAD - 1) // ROW_PAD * ROW_PAD
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), padded.cumsum(0)])
    order = torch.argsort(idx, stable=True)
    first = counts.cumsum(0) - counts
    row_of = torch.empty(t * k, dtype=torch.int32, device="cuda")
    row_of[order] = (offsets[idx[order]] + torch.arange(t * k, device="cuda") - first[idx[order]]).int()
    w = torch.rand(t, k, device="cuda", generator=g) + 0.1
    return {"case": case, "dout": (1e-2 * _rand(g, t, h)).to(torch.bfloat16),
            "y": _rand(g, _max_rows(case), h), "row_of": row_of.view(t, k),
            "w": w / w.sum(1, keepdim=True), "counts": counts.int(), "offsets": offsets.int()}


def _prepare_lora(case, g):
    r, h, n, rank, ad = (case[x] for x in ("rows", "h", "n", "rank", "adapters"))
    if case["order"] == "runs":  # requests one after another, each with its adapter
        cuts = torch.sort(torch.randint(0, r + 1, (min(r, 24),), device="cuda", generator=g)).values
        of_run = torch.randint(0, ad, (min(r, 24) + 1,), device="cuda", generator=g)
        ids = of_run[torch.searchsorted(cuts, torch.arange(r, device="cuda"), right=True)]
    else:
        ids = torch.randint(0, ad, (r,), device="cuda", generator=g)
        ids[torch.rand(r, device="cuda", generator=g) < 0.1] = -1  # requests without an adapter
    return {"case": case, "x": _rand(g, r, h).to(torch.bfloat16),
            "base": _rand(g, r, n).to(_DTYPE[case["dtype"]]),
            "a": (_rand(g, ad, rank, h) / math.sqrt(h)).to(torch.bfloat16),
            "b": (_rand(g, ad, n, rank) / math.sqrt(rank)).to(torch.bfloat16),
            "scale": 0.5 + torch.rand(ad, device="cuda", generator=g), "ids": ids.to(torch.int32)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "combine_backward":
        return _prepare_combine(case, g)
    if case["op"] == "lora":
        return _prepare_lora(case, g)
    return _prepare_routing(case, g)


# ---- plain forms ----

def _scores(l, scoring):
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    p = torch.exp(l - l.max(1, keepdim=True).values)
    return p / p.sum(1, keepdim=True)


def _plain_route(st):
    c = st["case"]
    t, e, k, groups = c["t"], c["e"], c["k"], c["groups"]
    s = _scores(st["logits"].double(), c["scoring"])  # 64 bits: the choice is made on them
    key = s if st["bias"] is None else s + st["bias"].double()
    if groups > 1:
        per = key.view(t, groups, e // groups)
        value = per.sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        stay = value.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        out = torch.ones(t, groups, dtype=torch.bool, device=key.device).scatter(1, stay, False)
        key = per.masked_fill(out[:, :, None], -math.inf).view(t, e)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), (w * c["scale"]).float()


def _plain_losses(st):
    c = st["case"]
    e, l = c["e"], st["logits"].float()
    keep = torch.ones(c["t"], device=l.device) if st["mask"] is None else st["mask"].float()
    n = keep.double().sum()
    m = l.max(1, keepdim=True).values
    x = torch.exp(l - m)
    lse = m + torch.log(x.sum(1, keepdim=True))
    if c["scoring"] == "sigmoid":
        x = _scores(l, "sigmoid")
    p = x / x.sum(1, keepdim=True)
    chosen = (st["idx"][:, :, None] == torch.arange(e, device=l.device, dtype=torch.int32)).any(1)
    counts = (chosen * keep[:, None]).double().sum(0)
    prob = (p * keep[:, None]).double().sum(0) / n.clamp(min=1)
    balance = e * (counts / n.clamp(min=1) * prob).sum()
    z = (lse[:, 0].double().square() * keep).sum() / n.clamp(min=1)
    return torch.stack([balance, z]).float(), torch.cat([counts, n[None]]).int(), prob.float()


def _plain_route_backward(st):
    c = st["case"]
    e, l, idx = c["e"], st["logits"].float(), st["idx"].long()
    keep = torch.ones(c["t"], device=l.device) if st["mask"] is None else st["mask"].float()
    n = st["counts"][e].float().clamp(min=1)
    s, g = _scores(l, c["scoring"]), st["d_w"] * c["scale"]
    if c["renormalize"]:
        sel = s.gather(1, idx)
        total = sel.sum(1, keepdim=True)
        g = (g - (g * sel).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter(1, idx, g)
    # losses: d balance / dp and d z / dl, for the unmasked tokens
    db = st["d_losses"][0] * e * st["counts"][:e].float() / (n * n)
    m = l.max(1, keepdim=True).values
    x = torch.exp(l - m)
    lse, soft = m + torch.log(x.sum(1, keepdim=True)), x / x.sum(1, keepdim=True)
    dz = st["d_losses"][1] * 2 / n * lse * soft
    if c["scoring"] == "sigmoid":
        total = s.sum(1, keepdim=True)
        ds = ds + keep[:, None] * (db - (db * s).sum(1, keepdim=True) / total) / total
        dl = s * (1 - s) * ds
    else:
        ds = ds + keep[:, None] * db
        dl = s * (ds - (s * ds).sum(1, keepdim=True))
    return (dl + keep[:, None] * dz).to(st["logits"].dtype)


def _plain_combine_backward(st):
    g, rows = st["dout"].float(), st["row_of"].long()
    dw = (g[:, None] * st["y"][rows]).sum(2)
    dy = torch.zeros_like(st["y"])
    dy[rows.reshape(-1)] = (st["w"][:, :, None] * g[:, None]).reshape(-1, g.shape[1])
    return dy, dw


def _plain_lora(st):
    c, ids, x = st["case"], st["ids"].long(), st["x"].float()
    r, n, rank, ad = c["rows"], c["n"], c["rank"], c["adapters"]
    has = (ids >= 0).float()
    at = ids.clamp(min=0)
    s = st["scale"][at] * has
    if r * rank * (c["h"] + n) < 1 << 28:  # a copy of each row's adapter
        t = (st["a"][at].float() @ x[:, :, None])[:, :, 0]
        delta = (st["b"][at].float() @ (s[:, None] * t)[:, :, None])[:, :, 0]
    else:                                  # the products with all adapters, others' ranks zero
        t = x @ st["a"].float().view(ad * rank, -1).t()
        mine = (torch.arange(ad, device=x.device)[None] == at[:, None]) * s[:, None]
        t = (t.view(r, ad, rank) * mine[:, :, None]).view(r, ad * rank)
        delta = t @ st["b"].float().transpose(1, 2).reshape(ad * rank, n)
    return (st["base"].float() + delta).to(st["base"].dtype)


_PLAIN = {"route": _plain_route, "losses": _plain_losses, "route_backward": _plain_route_backward,
          "combine_backward": _plain_combine_backward, "lora": _plain_lora}


# ---- this repository's calls ----

def _own(st):
    from sparse_mixture_experts_09_b200 import moe
    c = st["case"]
    if c["op"] == "lora":
        return moe.lora_add(st["base"], st["x"], st["a"], st["b"], st["ids"], st["scale"])
    if c["op"] == "combine_backward":
        return moe.combine_backward(st["dout"], st["y"], st["row_of"], st["w"], st["counts"], st["offsets"])
    r = moe.Routing(c["k"], c["scoring"], c["groups"], c["topk_groups"], c["group_top"],
                    c["renormalize"], c["scale"])
    if c["op"] == "route":
        return moe.route(st["logits"], r, st["bias"])
    if c["op"] == "losses":
        return moe.router_losses(st["logits"], st["idx"], r, st["mask"])
    return moe.route_backward(st["logits"], st["idx"], r, st["d_w"], st["counts"], st["d_losses"], st["mask"])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----

def work(case):
    op = case["op"]
    if op == "lora":
        r, h, n, rank, ad = (case[x] for x in ("rows", "h", "n", "rank", "adapters"))
        size = 4 if case["dtype"] == "fp32" else 2
        used = ad * (1 - (1 - 1 / ad) ** (r if case["order"] == "mixed" else min(r, 25)))
        return {"bytes": 2 * r * h + 2 * size * r * n + 2 * used * rank * (h + n) + 4 * r,
                "flops": 2 * r * rank * (h + n)}
    t, k, e = case["t"], case["k"], case["e"]
    if op == "combine_backward":
        h = case["h"]
        return {"bytes": 2 * t * h + 4 * (t * k + _max_rows(case)) * h + 12 * t * k, "flops": 3 * t * k * h}
    size = 4 if case["dtype"] == "fp32" else 2
    b = size * t * e + (t if case["masked"] else 0)
    if op == "route":
        return {"bytes": b + 8 * t * k, "flops": (8 + k) * t * e}
    if op == "losses":
        return {"bytes": b + 4 * t * k + 8 * e, "flops": 8 * t * e}
    return {"bytes": b + size * t * e + 8 * t * k + 4 * e, "flops": 16 * t * e}


# ---- the definitions in 64 bits ----

def _exact_scores(l, scoring):
    return torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 1)


def _exact_route(case, st):
    l = st["logits"].double()
    s = _exact_scores(l, case["scoring"])
    key = s.clone() if st["bias"] is None else s + st["bias"].double()
    t, e, groups = case["t"], case["e"], case["groups"]
    rows = torch.arange(t, device=l.device)
    if groups > 1:
        left, value = key.clone().view(t, groups, -1), 0
        for _ in range(case["group_top"]):
            best = left.max(2)
            value = value + best.values
            left.scatter_(2, best.indices[:, :, None], -math.inf)
        stay = torch.zeros(t, groups, dtype=torch.bool, device=l.device)
        for _ in range(case["topk_groups"]):
            stay[rows, value.argmax(1)] = True
            value[stay] = -math.inf
        key[~stay.repeat_interleave(e // groups, 1)] = -math.inf
    idx = []
    for _ in range(case["k"]):
        top = key.max(1, keepdim=True).values
        idx.append((key == top).int().argmax(1))  # the first of equal ones
        key[rows, idx[-1]] = -math.inf
    idx = torch.stack(idx, 1)
    w = torch.gather(s, 1, idx)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), w * case["scale"]


def _exact_loss_terms(case, st, l, counts, n):
    """Balance and z loss as functions of the logits (64 bits)."""
    s = _exact_scores(l, case["scoring"])
    p = s / s.sum(1, keepdim=True)
    keep = slice(None) if st["mask"] is None else st["mask"]
    prob = p[keep].sum(0) / max(n, 1)
    balance = case["e"] / max(n, 1) * torch.dot(counts.double(), prob)
    return balance, torch.logsumexp(l[keep], 1).square().sum() / max(n, 1), prob


def _exact_losses(case, st):
    keep = slice(None) if st["mask"] is None else st["mask"]
    counts = torch.bincount(st["idx"][keep].reshape(-1).long(), minlength=case["e"])
    n = int(st["idx"][keep].shape[0])
    balance, z, prob = _exact_loss_terms(case, st, st["logits"].double(), counts, n)
    return (torch.stack([balance, z]),
            torch.cat([counts, torch.tensor([n], device=counts.device)]).int(), prob)


def _exact_route_backward(case, st):
    """By differentiating the definition in 64 bits."""
    with torch.enable_grad():
        l = st["logits"].double().requires_grad_()
        w = torch.gather(_exact_scores(l, case["scoring"]), 1, st["idx"].long())
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        e = case["e"]
        balance, z, _ = _exact_loss_terms(case, st, l, st["counts"][:e], int(st["counts"][e]))
        d = st["d_losses"].double()
        total = (w * case["scale"] * st["d_w"].double()).sum() + d[0] * balance + d[1] * z
        return torch.autograd.grad(total, l)[0]


def _exact_combine_backward(case, st):
    g, w = st["dout"].double(), st["w"].double()
    dy = torch.zeros(st["y"].shape, dtype=torch.float64, device=g.device)
    dw = torch.zeros_like(w)
    for j in range(case["k"]):
        rows = st["row_of"][:, j].long()
        dy[rows] = w[:, j:j + 1] * g
        dw[:, j] = torch.linalg.vecdot(g, st["y"][rows].double())
    return dy, dw


def _exact_lora(case, st):
    out = st["base"].double()
    for i in torch.unique(st["ids"]).tolist():
        if i >= 0:
            rows = (st["ids"] == i).nonzero()[:, 0]
            t = st["x"][rows].double() @ st["a"][i].double().t()
            out[rows] += float(st["scale"][i]) * (t @ st["b"][i].double().t())
    return out


def exact(case, seed):
    st = prepare(case, seed)
    fn = {"route": _exact_route, "losses": _exact_losses, "route_backward": _exact_route_backward,
          "combine_backward": _exact_combine_backward, "lora": _exact_lora}[case["op"]]
    return fn(case, st)
