"""Tree attention over 8-bit pages in the plans that the shapes of test_gpu_q8.py do not
reach: rows left over whose parts several pairs of query tiles or several pieces of a list
join, pieces of whole tiles merged through the workspace, and batches of as many sequences
as the kernel for few rows takes, and one more.  The size of the workspace says which plan a
case runs."""
import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu
from tests import q8_util as qu

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def _case(seed, lens, N, G, Hkv, D, page, block, dtype, width=None, live=None):
    """Inputs made on the GPU; 0x7F and NaN where a kernel must not read."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    B, R = len(lens), N + 1
    need = torch.tensor([-(-n // page) for n in lens], device="cuda")
    total = int(need.sum()) + 2
    width = max(1, int(need.max())) if width is None else width
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    there = torch.arange(width, device="cuda")[None] < need[:, None]
    order = torch.randperm(total, generator=gen, device="cuda").int()
    table[there] = order[:int(need.sum())]
    spare = order[int(need.sum()):].long()
    halves = []
    for _ in range(2):
        e = torch.randint(-3, 3, (total, Hkv, page // block), generator=gen, device="cuda")
        c = (rn(total, Hkv, page, D) * torch.exp2(-e.float()).repeat_interleave(block, 2)[..., None]).clamp(-448, 448)
        c = c.to(qu.E4M3).view(torch.uint8)
        for b, n in enumerate(lens):
            if n % page:
                c[table[b, n // page].long(), :, n % page:] = 0x7F
        c[spare] = 0x7F
        s = (e + 127).to(torch.uint8)
        s[spare] = 255
        halves.append((c.view(qu.E4M3), s))
    cache = ops.QuantCache(halves[0][0], halves[1][0], halves[0][1], halves[1][1], table, dtype)
    live = [(N, N // 2, max(0, N - 1), N, 0)[b % 5] for b in range(B)] if live is None else live
    mask, n = pu.tree(torch.Generator().manual_seed(seed), B, N, live)
    q, kt, vt = (rn(B, R, h, D).to(dtype) for h in (Hkv * G, Hkv, Hkv))
    for b in range(B):
        for x in (q, kt, vt):
            x[b, live[b] + 1:] = float("nan")
    return q, cache, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), n.cuda(), mask.cuda()


def _size(args):
    q, cache = args[:2]
    B, R, Hq, D = q.shape
    return ops.workspace_size(ops.OP_TREE_ATTN_Q8, B=B, N=R - 1, Hq=Hq, Hkv=cache.Hkv, D=D,
                              cache_cap=cache.max_pages * cache.page_size)


def _check(args, out, lse):
    q, cache, kt, vt, plen, n, mask = args
    k, v = (qu.values64(p, s, cache.dtype) for p, s in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)))
    ref = pu.attention64(q, k, v, cache.page_table, plen, kt, vt, n, mask, cache.D ** -0.5)
    pu.check_attention(out, lse, ref, q.dtype, cache.D)


def _runs(args, times=3):
    """A call's results, the same bits each time over one workspace."""
    ws = ops.q8_attn_workspace(args[0], args[1])
    first = ops.tree_attn_q8(*args, workspace=ws)
    ops.ddtree_device_check()
    for _ in range(times - 1):
        again = ops.tree_attn_q8(*args, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ops.ddtree_device_check()
    return first


def _lens(B, hi):
    return [hi if b % 3 == 1 else (hi - 97 * b) % (hi + 1) if b % 4 else 5 * b for b in range(B)]


@pytest.mark.parametrize("B,N,G,Hkv,D,page,block,dtype,hi,pairs,pieces", [
    (8, 128, 4, 8, 128, 64, 32, BF16, 2000, 2, 1),     # two pairs join
    (8, 128, 4, 8, 64, 16, 8, FP16, 1500, 2, 1),
    (8, 128, 4, 8, 128, 64, 32, BF16, 9000, 2, 2),     # ... and the pieces of their lists
    (8, 128, 4, 8, 128, 32, 8, FP16, 9000, 2, 2),
    (8, 128, 4, 8, 64, 128, 64, BF16, 9000, 2, 2),
    (8, 128, 4, 8, 64, 16, 16, FP16, 9000, 2, 2),
    (4, 256, 8, 8, 128, 128, 32, BF16, 8500, 8, 2),    # eight pairs, eight rows left over
    (4, 256, 8, 8, 64, 64, 32, FP16, 8500, 8, 2),
    (20, 64, 4, 8, 128, 64, 16, BF16, 9000, 1, 2),     # one pair: pieces alone
    (20, 64, 4, 8, 64, 32, 32, BF16, 9000, 1, 2),
    (100, 64, 4, 2, 64, 64, 32, BF16, 8500, 1, 2),     # too many sequences to rank
    (10, 64, 4, 8, 128, 64, 32, BF16, 900, 1, 1),      # few units and short lists: one part
    (10, 32, 8, 8, 64, 16, 8, FP16, 3000, 1, 1),
    (12, 128, 2, 8, 128, 32, 32, BF16, 8300, 1, 2),
    (40, 32, 4, 8, 128, 16, 16, BF16, 700, None, 1),   # (two tiles: none is left over)
])
def test_rows_left_over_join(cuda_device, B, N, G, Hkv, D, page, block, dtype, hi, pairs, pieces):
    args = _case(hi + N + D, _lens(B, hi), N, G, Hkv, D, page, block, dtype)
    if pairs is None:
        assert _size(args) == 0
    else:
        per = 128 // G
        assert (N + 1) % per * G <= 8 and (N + 1) // per == 2 * pairs
        left = B * Hkv * pieces * pairs * 8 * (D + 4) * 4 if pieces * pairs > 1 else 0
        assert _size(args) >= left + (B * Hkv * 2 * pairs * 2 * 128 * D * 4 if pieces > 1 else 0)
    _check(args, *_runs(args))


@pytest.mark.parametrize("B,N,G,Hkv,D,page,block,dtype,hi,width", [
    (10, 127, 4, 8, 128, 64, 32, BF16, 9500, None),    # two pairs
    (20, 63, 4, 8, 64, 16, 8, FP16, 9000, None),       # one
    (20, 63, 4, 8, 128, 16, 16, BF16, 9000, 4096),     # a table seven times too wide
    (5, 511, 4, 8, 128, 64, 64, FP16, 8500, None),     # eight pairs
    (20, 70, 4, 8, 128, 64, 32, BF16, 9500, None),     # lone tiles
    (22, 70, 4, 8, 64, 64, 32, FP16, 300, None),       # ... whole
])
def test_pieces_of_whole_tiles_merge_through_the_workspace(cuda_device, B, N, G, Hkv, D, page, block, dtype, hi,
                                                           width):
    args = _case(hi + N, _lens(B, hi), N, G, Hkv, D, page, block, dtype, width)
    tiles = -(-(N + 1) * G // 128)
    assert _size(args) >= B * Hkv * tiles * 3 * 128 * D * 4 if hi > 8192 else _size(args) == 0
    _check(args, *_runs(args))


@pytest.mark.parametrize("B", [1024, 1025])
@pytest.mark.parametrize("N,G,D,dtype", [(0, 2, 128, BF16), (3, 4, 64, FP16)])
def test_as_many_sequences_as_few_rows_take_and_one_more(cuda_device, B, N, G, D, dtype):
    lens = [(0, 128, 1, 256, 127, 129, 300, 64)[b % 8] if b % 3 else b % 260 for b in range(B)]
    args = _case(B + N, lens, N, G, 1, D, 16, 8, dtype)
    _check(args, *_runs(args, 2))


@pytest.mark.parametrize("N,G", [(3, 5), (3, 8), (6, 4), (7, 4)])
def test_more_rows_than_few_in_a_large_batch(cuda_device, N, G):
    """17 to 32 rows of a KV head."""
    args = _case(N, _lens(64, 900), N, G, 8, 128, 16, 16, BF16)
    _check(args, *_runs(args, 2))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("N,G,D", [(15, 1, 128), (15, 1, 64), (7, 2, 128), (4, 3, 64), (0, 16, 64), (8, 1, 128), (1, 4, 64)])
def test_as_many_rows_as_few_rows_take(cuda_device, dtype, N, G, D):
    """8, 9, 15 and 16 rows of a KV head, whole trees and roots alone."""
    args = _case(N + G, [0, 1, 127, 128, 129, 700, 2500], N, G, 3, D, 16, 8, dtype)
    _check(args, *_runs(args, 2))


@pytest.mark.parametrize("N", [0, 40])
def test_keys_and_values_in_one_tensor(cuda_device, N):
    """Pages of keys and values side by side: written, read and attended like pages apart."""
    B, Hkv, G, D, page, block, P = 3, 2, 4, 128, 32, 16, 150
    table = torch.randperm(20, generator=torch.Generator().manual_seed(3))[:15].view(B, 5).int().cuda()
    apart = ops.QuantCache.empty(20, Hkv, page, D, table, block=block)
    both = torch.zeros(20, 2, Hkv, page, D, dtype=torch.uint8, device="cuda").view(qu.E4M3)
    scales = [x.clone() for x in (apart.k_scales, apart.v_scales)]
    side = ops.QuantCache(both[:, 0], both[:, 1], *scales, table)
    k, v = (torch.randn(B * P, Hkv, D, device="cuda").to(BF16) for _ in range(2))
    runs, at = torch.arange(0, B * P + 1, P, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    q, kt, vt = (torch.randn(B, N + 1, h, D, device="cuda").to(BF16) for h in (Hkv * G, Hkv, Hkv))
    mask, n = pu.tree(torch.Generator().manual_seed(4), B, N, [N] * B)
    got = []
    for cache in (apart, side):
        ops.ddtree_append_q8(k, v, runs, at, cache)
        out, lse = ops.tree_attn_q8(q, cache, kt, vt, at + P, n.cuda(), mask.cuda())
        rows = [torch.empty_like(k) for _ in range(2)]
        ops.ddtree_read_q8(cache, runs, at, *rows)
        got.append((out, lse, *rows, cache.k_scales, cache.v_scales))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    ops.ddtree_device_check()
