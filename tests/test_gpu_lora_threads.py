"""Adapter calls of several host threads at once, with different numbers of adapters."""
import threading

import pytest
import torch

from sparse_mixture_experts_09_b200 import moe as M

pytestmark = pytest.mark.gpu


def test_threads_with_different_numbers_of_adapters():
    """The sort's shared memory grows with the adapters loaded; what one call asks for does not
    take from another's."""
    rows, h = 640, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    sets = []
    for ad in (16384, 12100, 14000):
        a = torch.randn(ad, 8, h, device="cuda", generator=g).bfloat16()
        ids = torch.randint(0, ad, (rows,), device="cuda", generator=g).int()
        base = torch.randn(rows, h, device="cuda", generator=g)
        sets.append((base, torch.randn(rows, h, device="cuda", generator=g).bfloat16(), a, a, ids))
    want = [M.lora_add(*s) for s in sets]
    torch.cuda.synchronize()
    errors = []

    def work(j):
        stream = torch.cuda.Stream()
        try:
            for _ in range(600):
                got = M.lora_add(*sets[j], stream=stream)
            stream.synchronize()
            assert torch.equal(got, want[j])
        except Exception as e:      # a thread's error ends the test, not the thread alone
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
