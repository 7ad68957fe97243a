"""Calls of the paged-cache operators that their documentation allows and that no
other test makes."""
import os
import subprocess
import sys

import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("stride", [4 * 128 + 4, 3, 0, 1 << 40])
def test_the_stride_between_tokens_of_a_single_token_says_nothing(cuda_device, stride):
    """One sequence, one token, out of a buffer whose rows are on no grid."""
    gen = torch.Generator().manual_seed(2)
    k, v, table = pu.pool(gen, [40], 1, 128, 16, BF16, device="cuda")
    cache = ops.PagedCache(k, v, table)
    q, kt, vt = (torch.randn(1, 1, h, 128, generator=gen).to(BF16).cuda() for h in (4, 1, 1))
    odd = [torch.as_strided(t, t.shape, (stride, stride, 128, 1)) for t in (q, kt, vt)]
    plen, n, mask = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([40], [0], [[[1]]]))
    out, lse = ops.tree_attn_paged(*odd[:1], cache, *odd[1:], plen, n, mask)
    ref = pu.attention64(q, k, v, table, plen, kt, vt, n, mask, 128 ** -0.5)
    pu.check_attention(out, lse, ref, BF16, 128)
    r, pos = ops.Rotary(128), torch.tensor([[40]], dtype=torch.int32, device="cuda")
    got, _ = ops.rope(odd[0], None, pos, r)
    assert torch.equal(got, ops.rope(q, None, pos, r)[0])
    ops.ddtree_device_check()


FIRST = r"""
import torch
from diffusion_draft_tree_gb300 import ops
bf = torch.bfloat16
d = "cuda"
k, v = (torch.randn(40, 2, 16, 64, device=d).to(bf) for _ in range(2))
cache = ops.PagedCache(k, v, torch.randperm(40, device=d).int().view(2, 20))
rot = ops.Rotary(64)
q, kt, vt = (torch.randn(2, N + 1, h, 64, device=d).to(bf) for h in (8, 2, 2))
q0 = q.clone()
pos = torch.arange(2 * (N + 1), device=d).int().view(2, N + 1)
plen, n = torch.tensor([200, 33], device=d).int(), torch.full((2,), N, device=d).int()
mask = torch.full((2, N + 1, (N + 32) // 32), -1, device=d).int()
alen, nodes, new = torch.zeros(2, device=d).int(), torch.full((2, 3), -1, device=d).int(), torch.zeros(2, device=d).int()
seq, at = torch.tensor([0, 1], device=d).int(), torch.tensor([300, 301], device=d).int()
out, lse, qr = torch.empty_like(q), torch.empty(2, N + 1, 8, device=d), torch.empty_like(q)
ws = ops.paged_attn_workspace(q, cache)

def calls():
    ops.ddtree_rope(q, None, pos, rot, qr)
    ops.ddtree_append_paged(kt[:, 0], vt[:, 0], seq, at, cache, rot)
    ops.ddtree_tree_attn_paged(qr, cache, kt, vt, plen, n, mask, out, lse, workspace=ws)
    ops.ddtree_commit_paged(cache, kt, vt, alen, nodes, plen, new)

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
ops.ddtree_device_check()
a = out.clone()
out.zero_()
k2, v2 = k.clone(), v.clone()
calls()
ops.ddtree_device_check()
# (the append and the commit wrote the same rows again, behind every prefix but the root's)
assert torch.equal(k, k2) and torch.equal(v, v2) and new.tolist() == [201, 34]
assert torch.equal(out, a), (out.float() - a.float()).abs().max()
print("same")
"""


@pytest.mark.parametrize("N", [0, 64])
def test_the_first_calls_of_a_process_are_captured(cuda_device, N):
    """Nothing that a first call looks up or prepares breaks a capture."""
    r = subprocess.run([sys.executable, "-c", f"N = {N}\n" + FIRST], capture_output=True, text=True,
                       cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
