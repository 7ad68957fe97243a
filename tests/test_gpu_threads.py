"""Host threads that call the library at once: ctypes lets go of the interpreter's
lock, so the calls really overlap on the host."""
import threading

import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu

pytestmark = pytest.mark.gpu


def test_dense_rounds_from_four_threads(cuda_device):
    """Attention and top-K of other sizes in each thread, on a stream each, against the
    same calls one after another: bit for bit."""
    def inputs(i):
        gen = torch.Generator(device="cuda").manual_seed(i)
        rn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
        B, N, Hkv, G, D, cap = (1, 1, 2, 20)[i], 20 + 31 * i, 2 + i % 2, 4, (64, 128)[i % 2], 700 + 900 * i
        mask, n = pu.tree(torch.Generator().manual_seed(i), B, N, [N] * B)
        plen = torch.full((B,), cap - 3, dtype=torch.int32, device="cuda")
        attn = (rn(B, N + 1, Hkv * G, D), rn(B, Hkv, cap, D), rn(B, Hkv, cap, D), rn(B, N + 1, Hkv, D),
                rn(B, N + 1, Hkv, D), plen, n.cuda(), mask.cuda())
        return attn, torch.randn(4 + i, 5000 + 977 * i, generator=gen, device="cuda")

    def calls(x, stream=None):
        return [*ops.tree_attn(*x[0], stream=stream), *ops.topk(x[1], 5 + x[1].shape[0], stream=stream)]

    cases = [inputs(i) for i in range(4)]
    torch.cuda.synchronize()
    got, torn = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    got[i] = calls(cases[i], s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            torn.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not torn, torn
    ops.ddtree_device_check()
    for x, g in zip(cases, got):
        for a, b in zip(calls(x), g):
            assert torch.equal(a, b)
