"""fp16 weights of a softmax with one key far above very many others: each of those
lies below fp16's numbers when the largest weight is 1, all together they are what
the output is made of."""
import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
FP16 = torch.float16


@pytest.mark.parametrize("B,P,N,G,Hkv,D", [
    (1, 60000, 0, 4, 2, 128),     # few rows, runs of one list joined
    (3, 9000, 7, 4, 2, 64),       # two blocks of rows
    (1, 60000, 40, 4, 2, 128),    # a cluster's splits
    (2, 20000, 31, 4, 1, 64),
    (20, 9000, 63, 4, 8, 128),    # whole tiles of a full GPU
    (20, 9000, 64, 4, 8, 128),    # ... and the rows left over
    (20, 9000, 70, 4, 8, 64),     # ... and a lone tile
])
@pytest.mark.parametrize("bits", [20.0, 26.0, 29.0])
def test_many_small_weights_beside_a_large_one(cuda_device, bits, B, P, N, G, Hkv, D):
    """The first key's score is `bits` powers of two above the others', its value 0,
    theirs 1: the output is P 2^-bits and less."""
    gen = torch.Generator(device="cuda").manual_seed(P + N)
    page, R = 64, N + 1
    per = -(-P // page)
    k = torch.zeros(B * per, Hkv, page, D, dtype=FP16, device="cuda")
    v = torch.rand(k.shape, generator=gen, device="cuda").mul(0.5).add(0.75).to(FP16)
    table = torch.randperm(B * per, generator=gen, device="cuda").int().view(B, per)
    q = torch.ones(B, R, Hkv * G, D, device="cuda").to(FP16)
    # q . k = D x = bits ln 2 sqrt(D), in halves of the first key's elements
    k[table[:, 0].long(), :, 0] = bits * 0.6931471805599453 / D ** 0.5
    v[table[:, 0].long(), :, 0] = 0
    kt = torch.zeros(B, R, Hkv, D, dtype=FP16, device="cuda")
    vt = torch.rand(kt.shape, generator=gen, device="cuda").to(FP16)
    mask, n = pu.tree(torch.Generator().manual_seed(1), B, N, [N] * B)
    cache, mask, n = ops.PagedCache(k, v, table), mask.cuda(), n.cuda()
    plen = torch.full((B,), P, dtype=torch.int32, device="cuda")
    out, lse = ops.tree_attn_paged(q, cache, kt, vt, plen, n, mask)
    ops.ddtree_device_check()
    r_out, r_lse, weight, score, mass = pu.attention64(q, k, v, table, plen, kt, vt, n, mask, D ** -0.5)
    assert float(r_out.max()) < 0.1
    # pu.check_attention's bound, its term for weights below fp16's normal numbers
    # (2^-25 of the unit of weights each) at the unit that the largest weight has:
    # at least 2^7 of it
    ds = score * D * 2.0 ** -24 + 2.0 ** -20 * (1 + score)
    u = 2.0 ** -11
    bound = weight * (u + 2 * ds[..., None] + 2.0 ** -18) * (1 + u) + r_out.abs() * u + 2.0 ** -24
    pu.assert_within(out, r_out, bound + 2.0 ** -32 * mass, "out")
    lim = ds + 2.0 ** -17 + r_lse.abs() * 2.0 ** -22
    assert bool(((lse.double() - r_lse).abs() <= lim).all())
