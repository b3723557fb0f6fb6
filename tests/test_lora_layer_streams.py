"""The layer with adapters queues nothing before its own stream is current: adapters that are
copied on the way (a shard's experts) are copied on the stream that reads them."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from sparse_mixture_experts_09_b200 import moe as M


class _Ops(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.append(func.overloadpacket._qualified_op_name)
        return func(*args, **(kwargs or {}))


class _Reached(Exception):
    pass


def test_nothing_is_copied_before_the_stream(monkeypatch):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    e, shard = 8, slice(2, 6)
    a, b = bf(3, e, 16, 128)[:, shard], bf(3, e, 256, 16)[:, shard]
    a2, b2 = bf(3, e, 8, 256)[:, shard], bf(3, e, 128, 8)[:, shard]
    ad = M.LoraExperts(a1=a, b1=b, a3=a, b3=b, a2=a2, b2=b2, scale=torch.ones(3))
    x, wr, w1, w2 = bf(4, 128), bf(4, 128), bf(4, 256, 128), bf(4, 128, 256)
    ids = torch.zeros(4, dtype=torch.int32)

    def on(device, stream, call):
        raise _Reached

    monkeypatch.setattr(M, "_on", on)
    with _Ops() as ops, pytest.raises(_Reached):
        M.forward_lora(x, wr, w1, w1, w2, 2, ad, ids)
    views = {"aten::view", "aten::_unsafe_view", "aten::alias", "aten::detach"}
    assert set(ops.seen) <= views, ops.seen


@pytest.mark.gpu
def test_a_shards_adapters_on_another_stream():
    """The caller's stream is busy while the call runs on its own."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)
    t, h, i, e, lo = 40, 128, 256, 4, 2
    wr, w1, w3, w2 = (n(e, h) / 11).bfloat16(), (n(e, i, h) / 11).bfloat16(), (n(e, i, h) / 11).bfloat16(), (n(e, h, i) / 16).bfloat16()
    x, ids = n(t, h).bfloat16(), torch.randint(-1, 3, (t,), device="cuda", generator=g).int()
    part = lambda *s: (n(*s) / s[-1] ** 0.5).bfloat16()[:, lo:lo + e]
    pairs = [part(3, 8, 16, h), part(3, 8, i, 16), part(3, 8, 16, h), part(3, 8, i, 16), part(3, 8, 8, i), part(3, 8, h, 8)]
    want = M.forward_lora(x, wr, w1, w3, w2, 2, M.LoraExperts(*[p.contiguous() for p in pairs]), ids)
    assert torch.equal(M.forward_lora(x, wr, w1, w3, w2, 2, M.LoraExperts(*pairs), ids), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)                 # some 10 ms on the caller's stream
        got = M.forward_lora(x, wr, w1, w3, w2, 2, M.LoraExperts(*pairs), ids, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        torch.cuda.synchronize()
