"""The paged-cache calls write tensors behind autograd's back: it has to notice."""
import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _setup():
    gen = torch.Generator().manual_seed(1)
    r = ops.Rotary(64)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    k, v, table = pu.pool(gen, [32], 2, 64, 16, BF16, device="cuda")
    rows = [torch.randn(4, 2, 64, generator=gen).to(BF16).cuda() for _ in range(3)]
    return r, pos, ops.PagedCache(k, v, table), rows


def test_a_saved_tensor_that_is_rotated_in_place_is_noticed(cuda_device):
    r, pos, _, (x, y, _) = _setup()
    w = torch.ones_like(x).requires_grad_()
    loss = (w * x).sum()                      # saves x for w's gradient
    ops.ddtree_rope(x, y, pos, r)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_versions_of_what_is_written(cuda_device):
    r, pos, cache, (q, k, v) = _setup()
    seq = torch.zeros_like(pos)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)

    def moved(call, *tensors):
        before = [t._version for t in tensors]
        call()
        return [t._version - b for t, b in zip(tensors, before)]

    assert moved(lambda: ops.ddtree_rope(q, k, pos, r, q_out, k_out), q, k, q_out, k_out) == [0, 0, 1, 1]
    assert moved(lambda: ops.ddtree_rope(q, None, pos, r), q, k) == [1, 0]
    assert moved(lambda: ops.ddtree_append_paged(k, v, seq, pos, cache, r, q), q, k, v) == [1, 0, 0]
    assert moved(lambda: ops.ddtree_append_paged(k, v, seq, pos, cache, r, q, q_out), q, q_out) == [0, 1]
    assert moved(lambda: ops.ddtree_append_paged(k, v, seq, pos, cache), cache.k_pages, cache.v_pages) == [1, 1]
    one = torch.ones(1, 1, 1, dtype=torch.int32, device="cuda")
    t = [x[None, :1] for x in (q, k, v)]
    out, lse = torch.empty_like(t[0]), torch.empty(1, 1, 2, device="cuda")
    args = (t[0], cache, t[1], t[2], one[0, 0] * 4, one[0, 0] * 0, one, out, lse)
    ws = ops.paged_attn_workspace(t[0], cache)
    assert moved(lambda: ops.ddtree_tree_attn_paged(*args, workspace=ws), out, lse, t[0]) == [1, 1, 0]
    zero, new = one[0, 0] * 0, one[0, 0] * 0
    assert moved(lambda: ops.ddtree_commit_paged(cache, t[1], t[2], zero, one[0] * 0, one[0, 0] * 4, new),
                 cache.k_pages, cache.v_pages, new, t[1]) == [1, 1, 1, 0]
    with torch.inference_mode():              # (such tensors have no version)
        ops.ddtree_rope(q.clone(), None, pos, r)
    ops.ddtree_device_check()


def test_written_tensors_that_require_grad_are_refused(cuda_device):
    r, pos, cache, (q, k, v) = _setup()
    seq = torch.zeros_like(pos)
    leaf = q.clone().requires_grad_()
    for call in (lambda: ops.ddtree_rope(leaf, None, pos, r),
                 lambda: ops.ddtree_rope(q, None, pos, r, q_out=leaf),
                 lambda: ops.ddtree_rope(q, leaf * 1, pos, r),
                 lambda: ops.ddtree_append_paged(k, v, seq, pos, cache, r, leaf)):
        with pytest.raises(ValueError, match="requires grad"):
            call()
    with torch.no_grad():
        ops.ddtree_rope(leaf, None, pos, r)
    got, _ = ops.rope(leaf, None, pos, r)     # read only: a new tensor, without a graph
    assert not got.requires_grad
    ops.ddtree_device_check()
