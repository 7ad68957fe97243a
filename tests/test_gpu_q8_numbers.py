"""What the calls over an 8-bit cache make of elements, codes and scale bytes at and past the
ends of the numbers."""
import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import q8_util as qu
from tests.test_gpu_q8 import attn_case, check

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


def _with_nan_codes(args, share):
    """Some of the live codes 0x7F and 0xFF."""
    cache, plen = args[1], args[4]
    gen = torch.Generator(device="cuda").manual_seed(17)
    page, live = cache.page_size, torch.zeros(cache.num_pages, cache.page_size, dtype=torch.bool, device="cuda")
    for b, P in enumerate(plen.tolist()):
        pos = torch.arange(P, device="cuda")
        live[cache.page_table[b].long()[pos // page], pos % page] = True
    for codes in (raw(cache.k_pages), raw(cache.v_pages)):
        hit = (torch.rand(codes.shape, generator=gen, device="cuda") < share) & live[:, None, :, None]
        sign = torch.randint(0, 2, codes.shape, generator=gen, device="cuda", dtype=torch.uint8)
        codes.copy_(torch.where(hit, 0x7F + 0x80 * sign, codes))
    assert bool((raw(cache.k_pages)[live[:, None].expand(-1, cache.Hkv, -1)] == 0xFF).any())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("lens,N,Hq,Hkv,D,page,block", [
    ([300, 45], 0, 4, 1, 128, 16, 16), ([500, 7], 3, 8, 2, 64, 64, 32), ([300, 1000], 40, 4, 2, 128, 32, 8),
    ([700], 64, 8, 2, 64, 16, 16), ([260] * 20, 64, 32, 8, 128, 64, 64), ([200] * 24, 70, 32, 8, 64, 128, 32)])
def test_the_codes_of_no_number_are_480_in_every_form(cuda_device, dtype, lens, N, Hq, Hkv, D, page, block):
    args = attn_case(torch.Generator().manual_seed(N + D), lens, N, Hq, Hkv, D, page, block, dtype, spread=0.5)
    _with_nan_codes(args, 0.02)
    cache = args[1]
    check(args, scale=0.03)
    starts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    k, v = (torch.empty(starts[-1], Hkv, D, dtype=dtype, device="cuda") for _ in range(2))
    ops.ddtree_read_q8(cache, ints(starts), ints([0] * len(lens)), k, v)
    ops.ddtree_device_check()
    for got, codes, scales in ((k, cache.k_pages, cache.k_scales), (v, cache.v_pages, cache.v_scales)):
        val = qu.values64(codes, scales, dtype)
        for b, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            assert torch.equal(got[starts[b]:starts[b + 1]].double(), val[cache.page_table[b].long()[pos // page], :, pos % page])


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_the_codes_of_no_number_move_with_their_block(cuda_device, dtype):
    cache = ops.QuantCache.empty(1, 1, 16, 64, ints([[0]]), block=16, dtype=dtype)
    for c, s in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)):
        raw(c)[0, 0, 0], raw(c)[0, 0, 1] = 0x7F, 0xFF
        s.fill_(127)
    k = torch.full((1, 1, 64), 448.0 * 4, dtype=dtype, device="cuda")
    ops.ddtree_append_q8(k, k.clone(), ints([0, 1]), ints([2]), cache)
    ops.ddtree_device_check()
    for c, s in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)):
        assert s.item() == 129
        assert bool((c[0, 0, 0].float() == 120).all()) and bool((c[0, 0, 1].float() == -120).all())


def _recorded():
    with pytest.raises(ops.DDTreeError) as e:
        ops.ddtree_device_check()
    return e.value.detail


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("at,n,block,D", [(0, 1, 16, 64), (5, 3, 16, 128), (0, 40, 32, 64), (3, 130, 64, 128)])
@pytest.mark.parametrize("half", [0, 1])
def test_a_nan_among_keys_or_values_is_recorded(cuda_device, dtype, at, n, block, D, half):
    """... and everything but its own code is what it is with a zero there."""
    gen = torch.Generator().manual_seed(n)
    new = lambda: ops.QuantCache.empty(4, 2, 64, D, ints([[3, 1, 2]]), block=block, dtype=dtype)  # noqa: E731
    kv = [torch.randn(n, 2, D, generator=gen).to(dtype).cuda() for _ in range(2)]
    hit = (n - 1, 1, 7)
    kv[half][hit] = 0
    clean, dirty = new(), new()
    ops.ddtree_append_q8(*kv, ints([0, n]), ints([at]), clean)
    ops.ddtree_device_check()
    for bad in (float("nan"), -float("nan")):
        kv[half][hit] = bad
        ops.ddtree_append_q8(*kv, ints([0, n]), ints([at]), dirty)
        assert _recorded() == 0x06000005
    pos = at + n - 1
    for i, (a, b) in enumerate(zip(snap(clean), snap(dirty))):
        got, want = raw(b[0]).clone(), raw(a[0])
        if i == half:
            one = (int(clean.page_table[0, pos // 64]), 1, pos % 64, 7)
            assert int(got[one]) & 0x7F == 0x7F
            got[one] = want[one]
        assert torch.equal(got, want) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_norm_that_makes_no_number_is_recorded(cuda_device, dtype):
    k = torch.randn(3, 1, 64).to(dtype).cuda()
    cache = ops.QuantCache.empty(1, 1, 16, 64, ints([[0]]), block=16, dtype=dtype)
    ops.ddtree_append_q8(k, k, ints([0, 3]), ints([0]), cache, norm=ops.HeadNorm())
    ops.ddtree_device_check()
    k[1, 0, 0] = float("inf")
    ops.ddtree_append_q8(k, torch.zeros_like(k), ints([0, 3]), ints([0]), cache, norm=ops.HeadNorm())
    assert _recorded() == 0x06000005


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_nan_on_an_accepted_path_is_recorded(cuda_device, dtype):
    kt, vt = (torch.randn(2, 5, 2, 64).to(dtype).cuda() for _ in range(2))
    args = (ints([2, 1]), ints([[1, 3], [2, -1]]), ints([4, 15]))
    cache = ops.QuantCache.empty(4, 2, 16, 64, ints([[0, 1], [2, 3]]), block=8, dtype=dtype)
    kt[0, 2], vt[1, 4] = float("nan"), float("nan")  # not accepted
    ops.ddtree_commit_q8(cache, kt, vt, *args)
    ops.ddtree_device_check()
    vt[1, 2, 1, 5] = float("nan")
    ops.ddtree_commit_q8(cache, kt, vt, *args)
    assert _recorded() == 0x05000005


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_infinities_are_the_largest_code_of_the_largest_scale(cuda_device, dtype):
    cache = ops.QuantCache.empty(1, 1, 16, 64, ints([[0]]), block=16, dtype=dtype)
    k = torch.ones(2, 1, 64).to(dtype).cuda()
    k[1, 0, :2] = torch.tensor([float("inf"), -float("inf")])
    ops.ddtree_append_q8(k, k.clone(), ints([0, 2]), ints([0]), cache)
    ops.ddtree_device_check()
    out, _ = (torch.empty_like(k) for _ in range(2))
    ops.ddtree_read_q8(cache, ints([0, 2]), ints([0]), out, _)
    assert out[1, 0, :2].tolist() == [57344.0, -57344.0]


@pytest.mark.parametrize("first", [[0, 100, 50, 150], [0, 90, 20, 150, 150], [100, 40, 120, 10, 150], [0, 150, 0, 150, 3, 140],
                                   [0, 20, 120, 60, 61, 62, 63, 150], [140, 100, 60, 20, 150]])
@pytest.mark.parametrize("at0", [0, 13])
def test_where_first_descends_a_run_is_carried_out_as_a_whole_or_not_at_all(cuda_device, first, at0):
    B, T, S, D = len(first) - 1, 150, 16, 64
    table = torch.randperm(B * 3, generator=torch.Generator().manual_seed(B)).view(B, 3).tolist()
    cache = ops.QuantCache.empty(3 * B, 1, 64, D, ints(table), block=S)
    k = torch.ones(T, 1, D, dtype=BF16, device="cuda")
    q = torch.full((T, 2, D), 2.0, dtype=BF16, device="cuda")
    at = [at0 + b for b in range(B)]
    calls = []
    for b in range(B):  # (queries of a run show in rows that runs may share: one sequence's q at a time)
        f = [first[b], first[b + 1]]
        calls.append(f[0] <= f[1])
    q_out = torch.zeros_like(q)
    ops.ddtree_append_q8(k, k.clone(), ints(first), ints(at), cache, q=q, q_out=q_out)
    assert _recorded() == 0x06000005
    carried = []
    for b, good in enumerate(calls):
        n = first[b + 1] - first[b]
        pos = torch.arange(192, device="cuda")
        codes = raw(cache.k_pages)[ints(table)[b].long()[pos // 64], 0, pos % 64]
        wrote = (codes != 0).any(-1)
        if good and bool(wrote.any()):
            assert wrote.nonzero().flatten().tolist() == list(range(at[b], at[b] + n))
            assert bool((q_out[first[b]:first[b + 1]] == 2).all())
            carried.append(b)
        else:
            assert not bool(wrote.any())
    rows = set()
    for b in carried:
        rows |= set(range(first[b], first[b + 1]))
    assert (q_out == 2).all(-1).all(-1).nonzero().flatten().tolist() == sorted(rows)
    out = [torch.zeros_like(k) for _ in range(2)]
    for c in (cache.k_pages, cache.v_pages):
        raw(c).fill_(0x38)
    ops.ddtree_read_q8(cache, ints(first), ints(at), *out)
    assert _recorded() == 0x07000005
    assert (out[0] != 0).all(-1).all(-1).nonzero().flatten().tolist() == sorted(rows)
