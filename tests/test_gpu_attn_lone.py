"""A lone query tile (both softmax groups on one tile, 64 keys of a key tile
each) after a call that left large scores behind in the tensor memory: a group
must not see columns that are not its own."""
import numpy as np
import pytest
import torch

import oracle
from diffusion_draft_tree_gb300 import ops
from diffusion_draft_tree_gb300.workloads import bf16_to_f32
from tests.gpu_util import dev_bf16, dev_i32, tree_to_dev
from tests.test_gpu_attn import LSE_TOL, _random_case, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,P", [(100, (0,)), (120, (90,)), (70, (200,))])
def test_lone_tile_after_large_scores(cuda_device, N, P):
    big = [dev_bf16(x, cuda_device) if x.dtype == np.uint16 else dev_i32(x, cuda_device)
           for x in _random_case(5, 20, 255, 8, 8, 128, (300,) * 20, 300, 8, 4)[:6]]
    t = _random_case(5, 20, 255, 8, 8, 128, (300,) * 20, 300, 8, 4)[6]
    dt = tree_to_dev(t, cuda_device)
    q, kc, vc, kt, vt, plen, tree = _random_case(N, 1, N, 8, 8, 128, P, max(1, max(P)), 16, 16)
    for sign in (1.0, -1.0):
        # two query tiles a unit on every SM, scores of +-10^4 and beyond
        ops.tree_attn(torch.full_like(big[0], 30.0), torch.full_like(big[1], 30.0 * sign),
                      torch.ones_like(big[2]), torch.full_like(big[3], 30.0 * sign),
                      torch.ones_like(big[4]), big[5], dt["n_nodes"], dt["anc_mask"])
        out, lse = _run(q, kc, vc, kt, vt, plen, tree, cuda_device)
        ref, ref_lse = oracle.tree_attn(q, kc, vc, kt, vt, plen, tree["n_nodes"], tree["anc_mask"])
        # A row may see one or two keys only: its weights, partial output and output
        # are each rounded to bf16 (2^-8 of at most the largest |v|).
        n = int(tree["n_nodes"][0])
        v = np.concatenate([bf16_to_f32(vc[0, :, :P[0]]).ravel(), bf16_to_f32(vt[0, :n + 1]).ravel()])
        assert np.abs(out - ref).max() <= 3 * 2.0 ** -8 * np.abs(v).max()
        assert np.abs(lse - ref_lse)[:, :n + 1].max() <= LSE_TOL
