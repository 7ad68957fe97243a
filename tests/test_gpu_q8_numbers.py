"""What the calls over an 8-bit cache make of elements, codes and scale bytes at and past the
ends of the numbers."""
import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import q8_util as qu

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def raw(x):
    return x.view(torch.uint8) if x.dtype == qu.E4M3 else x


def snap(cache):
    return [(raw(c).cpu().view(qu.E4M3), s.cpu()) for c, s in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales))]


@pytest.mark.parametrize("dtype,size", [(BF16, 2.0 ** -60), (FP16, 2.0 ** -24)])
@pytest.mark.parametrize("eps", [1e-6, 1e-20, 1e-30, 1e-38])
@pytest.mark.parametrize("rows", [1, 40])
def test_append_under_a_norm_of_any_eps(cuda_device, dtype, size, eps, rows):
    """Zeros and nearly zeros: the norm's factor times the codes' unit passes the 32-bit range."""
    cache = ops.QuantCache.empty(3, 2, 32, 64, ints([[2, 0, 1]]), block=32, dtype=dtype)
    k = torch.zeros(rows, 2, 64)
    k[1::2, 1] = size * torch.randint(-4, 5, k[1::2, 1].shape, generator=torch.Generator().manual_seed(rows))
    k = k.to(dtype).cuda()
    q = k.clone()
    before = snap(cache)
    ops.ddtree_append_q8(k, k, ints([0, rows]), ints([0]), cache, norm=ops.HeadNorm(eps=eps), q=q)
    ops.ddtree_device_check()
    after = snap(cache)
    assert not bool(((raw(cache.k_pages) & 0x7F) == 0x7F).any())
    ref = qu.norm64(k, None, float(torch.tensor(eps)))
    off = ref.abs() * qu.norm_off(64)
    qu.check_16(q, ref, off, dtype, "queries")
    qu.check_written(before[0], after[0], None, cache.page_table.cpu(), 32, 32, dtype, [(0, 0, ref.cpu(), off.cpu())])
