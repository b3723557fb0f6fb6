"""Adapter calls of several host threads at once, with different numbers of adapters."""
import threading

import pytest
import torch

from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu


def test_threads_with_different_numbers_of_adapters():
    """The sort's shared memory grows with the adapters loaded; what one call asks for does not
    take from another's."""
    rows, h, calls = 640, 8, 4000
    g = torch.Generator(device="cuda").manual_seed(1)
    sets = []
    for ad in (16384, 12100, 14000, 16384, 12100):
        a = torch.randn(ad, 8, h, device="cuda", generator=g).bfloat16()
        ids = torch.randint(0, ad, (rows,), device="cuda", generator=g).int()
        base = torch.randn(rows, h, device="cuda", generator=g)
        sets.append((base, torch.randn(rows, h, device="cuda", generator=g).bfloat16(), a, a, ids))
    want = [M.lora_add(*s) for s in sets]
    outs = [torch.empty_like(w) for w in want]
    args = [M._LoraArgs(rows, h, h, h, h, h, 8, s[2].shape[0], 1) for s in sets]
    scratch = [torch.empty(M.lib().moe_lora_workspace(p), dtype=torch.uint8, device="cuda") for p in args]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    refused = []

    def work(j):
        base, x, a, b, ids = (t.data_ptr() for t in sets[j])
        out, ws, n, st = outs[j].data_ptr(), scratch[j].data_ptr(), scratch[j].numel(), streams[j].cuda_stream
        call, p = M.lib().moe_lora_add, args[j]
        for _ in range(calls):
            if call(p, base, x, a, b, ids, None, out, ws, n, st) != 0:
                refused.append((j, M.lib().moe_last_error()))
                return

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, refused
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
