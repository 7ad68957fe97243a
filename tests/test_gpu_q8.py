"""The round over an 8-bit paged cache on the GPU, against 64-bit references."""
import math

import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu
from tests import q8_util as qu

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def host(t):
    return t.contiguous().view(torch.uint8).cpu() if t.dtype == qu.E4M3 else t.cpu()


def snap(cache):
    return [(host(cache.k_pages.transpose(1, 2)).transpose(1, 2), host(cache.k_scales)),
            (host(cache.v_pages.transpose(1, 2)).transpose(1, 2), host(cache.v_scales))]


# ------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,inter,weights", [
    (1, 1, 1, 128, 128, BF16, False, True), (65, 32, 8, 128, 128, BF16, False, True),
    (7, 4, 2, 64, 64, FP16, True, True), (33, 3, 1, 80, 40, FP32, False, True),
    (19, 5, 1, 96, 96, BF16, True, False), (130, 2, 2, 256, 128, FP16, False, True),
    (9, 2, 1, 512, 512, FP32, True, True), (5, 2, 2, 17, 6, BF16, False, True),
    (11, 3, 2, 33, 32, FP32, True, True), (4, 2, 1, 2, 2, FP16, False, True),
    (3, 1, 1, 1, 0, FP32, False, True), (600, 7, 1, 128, 0, BF16, False, True),
    (4099, 32, 8, 128, 64, FP32, True, True), (21, 2, 1, 200, 72, FP16, False, False),
    (13, 2, 2, 510, 254, BF16, True, True)])
def test_norm_rope_matches_the_formula(cuda_device, T, Hq, Hkv, D, rot, dtype, inter, weights):
    gen = torch.Generator().manual_seed(T + D)
    q, k = (torch.randn(T, h, D, generator=gen).to(dtype).cuda() for h in (Hq, Hkv))
    q[0, 0] = 0  # eps alone under the root
    pos = torch.randint(0, 200000, (T,), generator=gen, dtype=I32).cuda()
    if T > 2:
        pos[1] = -1
    w = [(1 + 0.3 * torch.randn(D, generator=gen)).cuda() if weights else None for _ in range(2)]
    rotary = ops.Rotary(rot, base=1e5, interleaved=inter, scale=1.25) if rot else None
    norm = ops.HeadNorm(*w, eps=1e-5)
    got = ops.norm_rope(q, k, pos, norm, rotary)
    for x, y, wx in zip((q, k), got, w):
        ref, off = qu.turned64(x, wx, 1e-5, pos, rotary)
        qu.check_16(y, ref, off, dtype)
    ops.ddtree_norm_rope(q, k, pos, norm, rotary)  # in place
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])
    alone, none = ops.norm_rope(got[0], None, pos, norm, rotary)
    assert none is None
    again = got[0].clone()
    ops.ddtree_norm_rope(again, None, pos, norm, rotary)
    assert torch.equal(again, alone)


def test_norm_rope_takes_strides_and_any_alignment(cuda_device):
    gen = torch.Generator().manual_seed(3)
    T, Hq, Hkv, D = 37, 6, 2, 64
    pos = torch.randint(0, 5000, (T,), generator=gen, dtype=I32).cuda()
    norm = ops.HeadNorm((1 + torch.rand(D, generator=gen)).cuda(), None, offset=0.5)
    for dtype, pad, shift in ((BF16, 8, 8), (BF16, 4, 4), (FP16, 1, 1), (FP32, 1, 3), (FP32, 2, 2)):
        flat = torch.randn(shift + T * (Hq + Hkv) * (D + pad), generator=gen).to(dtype).cuda()
        x = flat[shift:].view(T, Hq + Hkv, D + pad)[..., :D]
        q, k = x[:, :Hq], x[:, Hq:]
        before = flat.clone()
        rotary = ops.Rotary(32)
        out = ops.norm_rope(q, k, pos, norm, rotary)
        for y, z, w in ((q, out[0], norm.q_weight), (k, out[1], None)):
            ref, off = qu.turned64(y, w, 1e-6, pos, rotary)
            qu.check_16(z, ref, off, dtype)
        ops.ddtree_norm_rope(q, k, pos, norm, rotary)
        assert torch.equal(q, out[0]) and torch.equal(k, out[1])
        gaps = torch.ones(T, Hq + Hkv, D + pad, dtype=torch.bool, device="cuda")
        gaps[..., :D] = False
        assert torch.equal(flat[shift:].view(T, Hq + Hkv, -1)[gaps], before[shift:].view(T, Hq + Hkv, -1)[gaps])


def test_norm_rope_is_the_rotation_after_the_norm_and_takes_nothing(cuda_device):
    q = torch.randn(4, 9, 8, 128, device="cuda")
    pos = torch.randint(0, 100, (4, 9), device="cuda", dtype=I32)
    rotary, norm = ops.Rotary(128, interleaved=True), ops.HeadNorm(eps=1e-6)
    a, _ = ops.norm_rope(q, None, pos, norm, rotary)
    normed, _ = ops.norm_rope(q, None, pos, norm)
    b, _ = ops.rope(normed, None, pos, rotary)
    assert (a - b).abs().max() <= 2.0 ** -20 * b.abs().max()
    e = torch.empty(0, 2, 128, device="cuda", dtype=BF16)
    ops.ddtree_norm_rope(e, None, ints([]), norm, rotary)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c, _ = ops.norm_rope(q, None, pos, norm, rotary, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, c)
    ops.ddtree_device_check()


def test_norm_rope_python_refusals(cuda_device):
    q, pos = torch.randn(3, 2, 64, device="cuda"), ints([0, 1, 2])
    norm, rot = ops.HeadNorm(torch.ones(64, device="cuda")), ops.Rotary(64)
    for call in (lambda: ops.ddtree_norm_rope(q, None, pos, ops.HeadNorm(torch.ones(32, device="cuda")), rot),
                 lambda: ops.ddtree_norm_rope(q, None, pos[:2], norm, rot),
                 lambda: ops.ddtree_norm_rope(q.double(), None, pos, norm, rot),
                 lambda: ops.ddtree_norm_rope(q, q[:2], pos, norm, rot),
                 lambda: ops.ddtree_norm_rope(q, None, pos, norm, rot, q[:2]),
                 lambda: ops.ddtree_norm_rope(q.cpu(), None, pos, norm, rot),
                 lambda: ops.ddtree_norm_rope(q.clone().requires_grad_(), None, pos, norm, rot),
                 lambda: ops.HeadNorm(torch.ones(64, device="cuda"), torch.ones(32, device="cuda")),
                 lambda: ops.HeadNorm(torch.ones(64)), lambda: ops.HeadNorm(eps=0.0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ops.DDTreeError):
        ops.ddtree_norm_rope(q, None, pos, norm, ops.Rotary(128))


# ------------------------------------------------------------------------ writers

APPENDS = [
    # runs [(at, n)], Hq, Hkv, D, page, block, dtype, rot, interleaved, norm, slots first, width
    ([(0, 1)], 4, 1, 128, 16, 16, BF16, 128, False, True, False, None),
    ([(0, 40), (17, 1), (5, 0), (33, 70)], 8, 2, 128, 16, 8, BF16, 128, True, True, False, None),
    ([(7, 9), (8, 8), (63, 2), (64, 64)], 3, 1, 64, 64, 32, FP16, 32, False, True, True, None),
    ([(1, 300)], 0, 5, 64, 128, 64, FP16, 64, True, False, False, 9),
    ([(100, 1)] * 7, 16, 8, 128, 32, 32, BF16, 64, False, True, True, 30),
    ([(0, 0), (0, 0)], 2, 2, 64, 8, 8, BF16, 16, False, True, False, None),
    ([(3, 517), (0, 33), (250, 6)], 7, 1, 128, 64, 16, BF16, 0, False, True, False, None),
    ([(15, 2), (16, 15), (31, 34), (2, 129)], 2, 1, 128, 256, 64, FP16, 128, False, False, False, None),
    ([(i, 1 + i % 19) for i in range(150)], 4, 2, 64, 16, 16, BF16, 64, False, True, False, 16),
]


@pytest.mark.parametrize("runs,Hq,Hkv,D,page,block,dtype,rot,inter,normed,first,width", APPENDS)
@pytest.mark.parametrize("lead,tail", [(0, 0), (3, 5)])
def test_append_matches_the_definition(cuda_device, runs, Hq, Hkv, D, page, block, dtype, rot, inter,
                                       normed, first, width, lead, tail):
    gen = torch.Generator().manual_seed(D + page + len(runs))
    p = qu.pool(gen, [a + n for a, n in runs], Hkv, D, page, block, dtype, width=width, slots_first=first)
    cache = ops.QuantCache(*p, dtype)
    n = [x for _, x in runs]
    T = lead + sum(n) + tail
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=gen)
    x *= torch.exp2(1.5 * torch.randn(T, 1, 1, generator=gen))
    x[:, :, 0] = 0
    x = x.to(dtype).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    starts = [lead + sum(n[:i]) for i in range(len(n) + 1)]
    w = [(1 + 0.2 * torch.randn(D, generator=gen)).cuda() for _ in range(2)]
    norm = ops.HeadNorm(*w) if normed else None
    rotary = ops.Rotary(rot, base=1e4, interleaved=inter) if rot else None
    q_out = torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda") if Hq else None
    before, x0 = snap(cache), x.clone()
    ops.ddtree_append_q8(k, v, ints(starts), ints([a for a, _ in runs]), cache, rotary, norm,
                         q=q if Hq else None, q_out=q_out)
    ops.ddtree_device_check()
    assert torch.equal(x, x0)
    after, table, eps = snap(cache), cache.page_table.cpu(), 1e-6 if normed else None
    lists = [[], []]
    for b, (at, m) in enumerate(runs):
        t = slice(starts[b], starts[b + 1])
        pos = torch.arange(at, at + m, device="cuda")
        if m:
            rk, ok = qu.turned64(k[t], w[1], eps, pos, rotary)
            lists[0].append((b, at, rk.cpu(), ok.cpu()))
            lists[1].append((b, at, v[t].double().cpu(), torch.zeros(m, Hkv, D, dtype=torch.float64)))
        if Hq and m:
            qu.check_16(q_out[t], *qu.turned64(q[t], w[0], eps, pos, rotary), dtype, "queries")
    if Hq:
        assert bool((q_out[:lead] == 7).all()) and bool((q_out[T - tail:] == 7).all())
    if not (rot or normed):
        lists[0] = [(b, at, x, torch.zeros_like(o)) for b, at, x, o in lists[0]]
    for half in range(2):
        qu.check_written(before[half], after[half], None, table, page, block, dtype, lists[half])
    if Hq:  # queries in place
        ops.ddtree_append_q8(k, v, ints(starts), ints([a for a, _ in runs]), cache, rotary, norm, q=q)
        assert torch.equal(q[lead:T - tail], q_out[lead:T - tail])
        assert torch.equal(q[T - tail:], x0[T - tail:, :Hq]) and torch.equal(q[:lead], x0[:lead, :Hq])


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_append_token_by_token_moves_the_scale(cuda_device, dtype):
    """Growing, shrinking, huge and zero elements, one position a call, across blocks."""
    cache = ops.QuantCache.empty(9, 2, 16, 64, ints([[4, 2, 7]]), block=16, dtype=dtype)
    gen = torch.Generator().manual_seed(1)
    sizes = [0.0, 1e-6, 1e-3, 1.0, 30.0, 500.0, 2.0, 60000.0, 1e-4, 3.0, 449.0, 448.0, 0.0, 5e4, 1.0, 2.0,
             2.0 ** -14, 2.0 ** -20, 1.0, 1e-2] + [4.0 ** i for i in range(-8, 8)]
    for i, size in enumerate(sizes):
        k, v = ((torch.rand(1, 2, 64, generator=gen) * 2 - 1) * size for _ in range(2))
        k, v = k.to(dtype).cuda(), v.to(dtype).cuda()
        before = snap(cache)
        ops.ddtree_append_q8(k, v, ints([0, 1]), ints([i]), cache)
        after = snap(cache)
        for half, x in enumerate((k, v)):
            x = x.double().cpu()
            qu.check_written(before[half], after[half], None, cache.page_table.cpu(), 16, 16, dtype,
                             [(0, i, x, torch.zeros_like(x))])
    ops.ddtree_device_check()


def test_append_extremes(cuda_device):
    """The largest and smallest elements of the types, signed zeros."""
    for dtype in (BF16, FP16):
        cache = ops.QuantCache.empty(1, 1, 8, 64, ints([[0]]), block=8, dtype=dtype)
        fi = torch.finfo(dtype)
        rows = [[fi.max], [-fi.max], [fi.tiny], [fi.smallest_normal * 0.5], [0.0], [-0.0], [57344.0], [57345.0]]
        for r in rows:
            k = torch.full((1, 1, 64), r[0], dtype=dtype, device="cuda")
            before = snap(cache)
            ops.ddtree_append_q8(k, -k, ints([0, 1]), ints([0]), cache)
            after = snap(cache)
            for half, x in enumerate((k, -k)):
                x = x.double().cpu()
                qu.check_written(before[half], after[half], None, cache.page_table.cpu(), 8, 8, dtype,
                                 [(0, 0, x, torch.zeros_like(x))])


def _bad(cache, first, at, T=8, q=True):
    k = torch.randn(T, 2, 64, device="cuda", dtype=BF16)
    qq = torch.randn(T, 4, 64, device="cuda", dtype=BF16)
    out = torch.full_like(qq, 3.0)
    ops.ddtree_append_q8(k, k.clone(), ints(first), ints(at), cache, q=qq, q_out=out)
    with pytest.raises(ops.DDTreeError) as e:
        ops.ddtree_device_check()
    return out, e.value.detail


def test_append_bad_runs_are_left_out_and_recorded(cuda_device):
    new = lambda table: ops.QuantCache.empty(6, 2, 16, 64, ints(table), block=8)  # noqa: E731
    for first, at, good in (([0, 4, 9], [0, 0], [0]), ([0, 4, 8], [29, 0], [1]), ([0, 4, 8], [-1, 3], [1]),
                            ([4, 2, 8], [0, 0], [1]), ([-3, 2, 8], [0, 0], [1]), ([0, 3, 2 ** 31 - 1], [0, 1], [0]),
                            ([0, 4, 8], [0, 2 ** 31 - 1], [0])):
        cache = new([[0, 1], [2, 3]])
        out, detail = _bad(cache, first, at)
        assert detail == 0x06000005
        for b in range(2):
            wrote = bool((cache.k_pages.view(torch.uint8)[2 * b:2 * b + 2] != 0).any())
            assert wrote == (b in good), (first, at, b)
        for b in good:
            assert bool((out[max(first[b], 0):first[b + 1]] != 3.0).any())
    # a page outside the pool: its block is left out, the rest of the run is written
    cache = new([[0, 6], [2, -1]])
    out, detail = _bad(cache, [0, 4, 8], [14, 14])
    assert detail == 0x06000007 and bool((out != 3.0).any(-1).all())
    assert bool((cache.k_pages.view(torch.uint8)[[0, 2], :, 14:] != 0).any())
    assert not bool((cache.k_pages.view(torch.uint8)[[1, 3, 4, 5]] != 0).any())


@pytest.mark.parametrize("lens,alens,N,L,Hkv,D,page,block,dtype,first", [
    ([0], [0], 1, 1, 1, 128, 16, 16, BF16, False), ([2048], [16], 64, 16, 8, 128, 16, 16, BF16, False),
    ([5, 16, 31, 100], [3, 0, 4, 2], 9, 4, 2, 64, 8, 8, FP16, True),
    ([63, 64, 65], [16, 15, 14], 512, 16, 5, 128, 64, 32, FP16, False),
    (list(range(0, 260, 2)), [i % 17 for i in range(130)], 128, 16, 1, 64, 128, 64, BF16, False)])
def test_commit_matches_the_definition(cuda_device, lens, alens, N, L, Hkv, D, page, block, dtype, first):
    gen = torch.Generator().manual_seed(N + D)
    B = len(lens)
    p = qu.pool(gen, [a + b + 1 for a, b in zip(lens, alens)], Hkv, D, page, block, dtype, slots_first=first)
    cache = ops.QuantCache(*p, dtype)
    kt, vt = (torch.randn(B, N + 1, Hkv, D, generator=gen).to(dtype).cuda() for _ in range(2))
    nodes = torch.full((B, L), -1, dtype=I32)
    for b, a in enumerate(alens):
        nodes[b, :a] = torch.randperm(N, generator=gen)[:a].sort().values + 1 if a <= N else 1
    new = torch.zeros(B, dtype=I32, device="cuda")
    before = snap(cache)
    ops.ddtree_commit_q8(cache, kt, vt, ints(alens), nodes.cuda(), ints(lens), new)
    ops.ddtree_device_check()
    assert new.tolist() == [a + b + 1 for a, b in zip(lens, alens)]
    after = snap(cache)
    for half, t in enumerate((kt, vt)):
        runs = []
        for b, (P, a) in enumerate(zip(lens, alens)):
            rows = t[b, [0] + nodes[b, :a].tolist()].double().cpu()
            runs.append((b, P, rows, torch.zeros_like(rows)))
        qu.check_written(before[half], after[half], None, cache.page_table.cpu(), page, block, dtype, runs)


def test_commit_bad_paths_leave_the_sequence(cuda_device):
    N, L = 6, 3
    kt = torch.randn(1, N + 1, 2, 64, device="cuda", dtype=BF16)
    for table, P, a, nodes, detail in (([[0, 1]], 30, 2, [1, 2, -1], 0x05000001), ([[0, 1]], -1, 0, [-1] * 3, 0x05000001),
                                       ([[0, 1]], 3, 4, [1, 2, 3], 0x05000001), ([[0, 1]], 3, 2, [1, 7, -1], 0x05000003),
                                       ([[0, 9]], 14, 2, [1, 2, -1], 0x05000007), ([[-1, 1]], 14, 2, [1, 2, -1], 0x05000007)):
        cache = ops.QuantCache.empty(4, 2, 16, 64, ints(table), block=8)
        new = ints([77])
        before = snap(cache)
        ops.ddtree_commit_q8(cache, kt, kt.clone(), ints([a]), ints([nodes]), ints([P]), new)
        with pytest.raises(ops.DDTreeError) as e:
            ops.ddtree_device_check()
        assert e.value.detail == detail and new.item() == P
        for x, y in zip(before, snap(cache)):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("runs,Hkv,D,page,block,dtype,first", [
    ([(0, 1)], 1, 128, 16, 16, BF16, False), ([(3, 100), (0, 0), (64, 64), (63, 2)], 3, 64, 32, 8, FP16, True),
    ([(0, 2000), (1, 777)], 8, 128, 64, 32, BF16, True), ([(i, 3) for i in range(200)], 2, 64, 8, 8, BF16, False),
    ([(5, 300)], 5, 128, 512, 64, FP16, False)])
def test_read_gives_the_values_back(cuda_device, runs, Hkv, D, page, block, dtype, first):
    gen = torch.Generator().manual_seed(D)
    p = qu.pool(gen, [a + n for a, n in runs], Hkv, D, page, block, dtype, slots_first=first, spread=6.0)
    p[2].view(-1)[:3] = torch.tensor([0, 1, 254], dtype=torch.uint8, device="cuda")  # scales past the ends
    cache = ops.QuantCache(*p, dtype)
    starts = [2 + sum(n for _, n in runs[:i]) for i in range(len(runs) + 1)]
    T = starts[-1] + 3
    out = torch.full((T, 2, Hkv, D), 9.0, dtype=dtype, device="cuda")
    k, v = out[:, 0], out[:, 1]
    ops.ddtree_read_q8(cache, ints(starts), ints([a for a, _ in runs]), k, v)
    ops.ddtree_device_check()
    for got, pages, scales in ((k, p[0], p[2]), (v, p[1], p[3])):
        val = qu.values64(pages, scales, dtype)
        for b, (at, n) in enumerate(runs):
            pos = torch.arange(at, at + n, device="cuda")
            ref = val[cache.page_table[b].long()[pos // page], :, pos % page]
            assert torch.equal(got[starts[b]:starts[b + 1]].double(), ref)
        assert bool((got[:2] == 9).all()) and bool((got[starts[-1]:] == 9).all())


def test_read_bad_runs_are_left_out_and_recorded(cuda_device):
    cache = ops.QuantCache.empty(3, 1, 16, 64, ints([[0, 1], [2, 5]]), block=16)
    for first, at, detail, good in (([0, 3, 9], [0, 0], 0x07000005, [0, 1, 2]), ([0, 3, 8], [30, 0], 0x07000005, [3, 4, 5, 6, 7]),
                                    ([0, 3, 8], [0, 14], 0x07000007, [0, 1, 2, 3, 4])):
        k, v = (torch.full((8, 1, 64), 5.0, device="cuda", dtype=BF16) for _ in range(2))
        ops.ddtree_read_q8(cache, ints(first), ints(at), k, v)
        with pytest.raises(ops.DDTreeError) as e:
            ops.ddtree_device_check()
        assert e.value.detail == detail
        want = torch.full((8,), 5.0, device="cuda")
        want[good] = 0
        assert torch.equal(k[:, 0, 0].float(), want) and torch.equal(v[:, 0, 63].float(), want)


# ---------------------------------------------------------------------- attention

def attn_case(gen, lens, N, Hq, Hkv, D, page, block, dtype, first=False, width=None, live=None, spread=1.0,
              chain=None):
    B = len(lens)
    p = qu.pool(gen, lens, Hkv, D, page, block, dtype, slots_first=first, width=width, spread=spread)
    cache = ops.QuantCache(*p, dtype)
    live = [N - (i % 3 if N > 3 else 0) for i in range(B)] if live is None else live
    mask, n = pu.tree(gen, B, N, live, chain)
    x = torch.randn(B, N + 1, Hq + 2 * Hkv, D, generator=gen).to(dtype)
    for b in range(B):
        x[b, live[b] + 1:] = float("nan")
    x = x.cuda()
    q, kt, vt = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    return q, cache, kt, vt, ints(lens), n.cuda(), mask.cuda()


def reference(q, cache, kt, vt, plen, n, mask, scale=None):
    k = qu.values64(cache.k_pages, cache.k_scales, cache.dtype)
    v = qu.values64(cache.v_pages, cache.v_scales, cache.dtype)
    return pu.attention64(q, k, v, cache.page_table, plen, kt, vt, n, mask,
                          q.shape[-1] ** -0.5 if scale is None else scale)


def check(args, scale=None):
    out, lse = ops.tree_attn_q8(*args, scale=scale)
    ops.ddtree_device_check()
    pu.check_attention(out, lse, reference(*args, scale=scale), args[0].dtype, args[0].shape[-1])
    return out, lse


ATTN = [
    # lens, N, Hq, Hkv, D, page, block, dtype, slots first, width
    ([0], 0, 1, 1, 64, 8, 8, BF16, False, None), ([1], 0, 1, 1, 128, 8, 8, FP16, False, None),
    ([64], 16, 2, 1, 64, 16, 16, BF16, False, None), ([127, 128, 129], 5, 4, 2, 128, 32, 8, BF16, True, None),
    ([2048], 64, 32, 8, 128, 16, 16, BF16, False, None), ([300, 0, 1000, 63], 21, 28, 4, 64, 32, 8, FP16, True, None),
    ([515, 77], 130, 8, 1, 128, 64, 64, BF16, False, 40), ([1500], 31, 12, 4, 128, 128, 64, FP16, False, None),
    ([700, 5, 260], 255, 16, 2, 64, 256, 32, BF16, True, 5), ([40], 7, 128, 1, 128, 16, 8, BF16, False, None),
    ([90, 3], 12, 127, 1, 64, 16, 16, FP16, False, None), ([33, 2000, 512], 0, 32, 8, 128, 16, 16, BF16, False, None),
    ([4097, 100], 0, 8, 1, 128, 64, 32, FP16, True, 100), ([777] * 3, 0, 7, 1, 64, 8, 8, BF16, False, None),
    ([1000, 20], 0, 40, 2, 128, 32, 32, BF16, False, None), ([250] * 5, 1, 16, 4, 64, 16, 8, FP16, False, None),
    ([3000], 1, 2, 2, 128, 128, 8, BF16, False, None), ([600, 601], 3, 5, 5, 128, 16, 16, BF16, False, None),
    ([10, 20], 1024, 2, 1, 64, 16, 16, BF16, False, None),
]


@pytest.mark.parametrize("lens,N,Hq,Hkv,D,page,block,dtype,first,width", ATTN)
def test_attention_matches_the_formula(cuda_device, lens, N, Hq, Hkv, D, page, block, dtype, first, width):
    gen = torch.Generator().manual_seed(sum(lens) + N)
    check(attn_case(gen, lens, N, Hq, Hkv, D, page, block, dtype, first, width))


@pytest.mark.parametrize("B,hi,N,Hq,Hkv,D,page,block,dtype", [
    (20, 700, 0, 32, 8, 128, 16, 16, BF16), (40, 900, 33, 16, 8, 128, 64, 32, BF16),
    (24, 1300, 64, 32, 8, 128, 32, 8, FP16), (30, 500, 20, 8, 8, 64, 16, 16, BF16),
    (16, 3000, 128, 8, 4, 64, 128, 64, FP16), (100, 200, 63, 8, 2, 128, 16, 16, BF16),
    (25, 9000, 31, 32, 8, 128, 64, 32, BF16), (200, 150, 2, 4, 1, 64, 8, 8, BF16)])
def test_attention_of_large_batches(cuda_device, B, hi, N, Hq, Hkv, D, page, block, dtype):
    gen = torch.Generator().manual_seed(B)
    lens = [hi * i // (B - 1) for i in range(B)]
    check(attn_case(gen, lens, N, Hq, Hkv, D, page, block, dtype))


@pytest.mark.parametrize("seed", range(24))
def test_attention_random_shapes(cuda_device, seed):
    r = torch.Generator().manual_seed(1000 + seed)
    pick = lambda xs: xs[int(torch.randint(len(xs), (1,), generator=r))]  # noqa: E731
    B, hi, N = pick([1, 2, 3, 9]), pick([5, 100, 600, 2500]), pick([0, 0, 1, 6, 30, 65, 200])
    Hkv, G, page = pick([1, 2, 4]), pick([1, 2, 3, 4, 5, 8, 11, 16]), pick([8, 16, 32, 64, 128, 256])
    block = pick([b for b in (8, 16, 32, 64) if b <= page])
    lens = torch.randint(0, hi + 1, (B,), generator=r).tolist()
    check(attn_case(r, lens, N, Hkv * G, Hkv, pick([64, 128]), page, block, pick([BF16, FP16]), pick([False, True]),
                    -(-hi // page) + pick([0, 3, 200]), [int(torch.randint(N + 1, (1,), generator=r)) for _ in range(B)]))


@pytest.mark.parametrize("N,Hq,lens", [(0, 8, [900]), (0, 64, [500, 60]), (40, 4, [1200])])
@pytest.mark.parametrize("spread", [0.0, 8.0])
def test_attention_scales_far_apart(cuda_device, N, Hq, lens, spread):
    gen = torch.Generator().manual_seed(5)
    check(attn_case(gen, lens, N, Hq, 2, 128, 64, 16, BF16, spread=spread), scale=0.02)


@pytest.mark.parametrize("N,Hq", [(0, 4), (3, 4), (70, 4)])
def test_attention_rows_without_a_key(cuda_device, N, Hq):
    gen = torch.Generator().manual_seed(6)
    args = list(attn_case(gen, [0, 50, 0], N, Hq, 1, 64, 16, 16, BF16, live=[N] * 3))
    args[6][0] = 0
    args[6][2, 0] = 0
    out, lse = check(args)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())


@pytest.mark.parametrize("N,lens,scale", [(0, [3000], 4.0), (40, [2500, 9], 4.0), (0, [3000] * 30, 1e-4), (65, [700], 1e-4)])
def test_attention_peaked_and_flat_softmax(cuda_device, N, lens, scale):
    gen = torch.Generator().manual_seed(7)
    check(attn_case(gen, lens, N, 8, 2, 128, 16, 16, FP16), scale=scale)


@pytest.mark.parametrize("N", [0, 40])
def test_attention_a_sink_and_a_far_tail(cuda_device, N):
    """One key takes nearly all of the weight and its value is small: the tail's weights, 2^-14
    and less of the largest, make the output."""
    gen = torch.Generator().manual_seed(8)
    for dtype in (BF16, FP16):
        q, cache, kt, vt, plen, n, mask = attn_case(gen, [6000], N, 4, 1, 128, 64, 16, dtype, spread=0.0)
        q = torch.ones_like(q)
        q[:, int(n[0]) + 1:] = float("nan")
        at = int(cache.page_table[0, 0])
        raw = cache.k_pages.view(torch.uint8)
        raw[cache.page_table[0].long()] = (0.25 * torch.randn(raw[cache.page_table[0].long()].shape, generator=gen)).to(qu.E4M3).view(torch.uint8).cuda()
        cache.k_scales.fill_(127)
        raw[at, :, 3] = torch.full((1, 128), 1.25).to(qu.E4M3).view(torch.uint8).cuda()
        cache.v_pages.view(torch.uint8)[at, :, 3] = 0
        check((q, cache, kt, vt, plen, n, mask))


@pytest.mark.parametrize("N", [0, 40])
def test_attention_bad_pages_count_as_zeros(cuda_device, N):
    gen = torch.Generator().manual_seed(9)
    args = attn_case(gen, [400, 90], N, 8, 2, 128, 16, 16, BF16)
    cache = args[1]
    good = cache.page_table.clone()
    spare = [i for i in range(cache.num_pages) if i not in good.flatten().tolist()][0]
    for x in (cache.k_pages, cache.v_pages):
        x.view(torch.uint8)[spare] = 0
    cache.page_table[0, 7] = spare
    ref = reference(*args)
    for bad in (-1, cache.num_pages, 2 ** 31 - 1):
        cache.page_table[0, 7] = bad
        out, lse = ops.tree_attn_q8(*args)
        with pytest.raises(ops.DDTreeError) as e:
            ops.ddtree_device_check()
        assert e.value.detail == 0x03000007
        pu.check_attention(out, lse, ref, BF16, 128)


@pytest.mark.parametrize("what,value,detail", [("P", -1, 1), ("P", 10 ** 6, 1), ("n", -1, 2), ("n", 10 ** 6, 2)])
@pytest.mark.parametrize("N", [0, 40])
def test_attention_bad_lengths_leave_the_sequence(cuda_device, what, value, detail, N):
    gen = torch.Generator().manual_seed(10)
    args = list(attn_case(gen, [200, 90, 31], N, 4, 1, 64, 16, 8, FP16))
    ref, _ = ops.tree_attn_q8(*args)
    args[4 if what == "P" else 5][1] = value
    out, lse = torch.full_like(args[0], 4.0), torch.full(args[0].shape[:3], 4.0, device="cuda")
    out = torch.full(args[0].shape, 4.0, dtype=FP16, device="cuda")
    ops.ddtree_tree_attn_q8(*args, out, lse, workspace=ops.q8_attn_workspace(args[0], args[1]))
    with pytest.raises(ops.DDTreeError) as e:
        ops.ddtree_device_check()
    assert e.value.detail == 0x03000000 + detail
    assert torch.equal(out[[0, 2]], ref[[0, 2]]) and bool((out[1] == 4).all()) and bool((lse[1] == 4).all())


@pytest.mark.parametrize("N,lens", [(0, [500, 3000]), (40, [700]), (64, [300] * 24)])
def test_attention_captured_replayed_and_repeatable(cuda_device, N, lens):
    gen = torch.Generator().manual_seed(11)
    args = attn_case(gen, lens, N, 16, 8, 128, 16, 16, BF16)
    ref, rlse = check(args)
    out, lse, ws = torch.empty_like(ref), torch.empty_like(rlse), ops.q8_attn_workspace(args[0], args[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ops.ddtree_tree_attn_q8(*args, out, lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.ddtree_tree_attn_q8(*args, out, lse, workspace=ws)
    for _ in range(3):
        out.fill_(1)
        g.replay()
        assert torch.equal(out, ref) and torch.equal(lse, rlse)
    ops.ddtree_device_check()


def test_attention_offsets_past_32_bits(cuda_device):
    """Codes more than 2^31 bytes into the pool."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 10 GB")
    pages, page, Hkv, D = 20000, 128, 8, 128
    raw = [torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, Hkv, 2), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = ops.QuantCache(*(x.view(qu.E4M3) for x in raw), *scales, ints([[19999, 3, 18000]]))
    x = torch.randn(300, 3 * Hkv, D, device="cuda", dtype=BF16)
    ops.ddtree_append_q8(x[:, :Hkv], x[:, Hkv:2 * Hkv], ints([0, 300]), ints([0]), cache)
    k, v = torch.empty(300, Hkv, D, device="cuda", dtype=BF16), torch.empty(300, Hkv, D, device="cuda", dtype=BF16)
    ops.ddtree_read_q8(cache, ints([0, 300]), ints([0]), k, v)
    assert float((k - x[:, :Hkv]).abs().max()) < 0.3 and float((v - x[:, Hkv:2 * Hkv]).abs().max()) < 0.3
    q, kt, vt = (torch.randn(1, 1, h, D, device="cuda", dtype=BF16) for h in (32, Hkv, Hkv))
    small = ops.QuantCache(*(t[[19999, 3, 18000]].contiguous().view(qu.E4M3) for t in raw),
                           *(t[[19999, 3, 18000]].contiguous() for t in scales), ints([[0, 1, 2]]))
    args = (kt, vt, ints([300]), ints([0]), ints([[[1]]]))
    a, _ = ops.tree_attn_q8(q, cache, *args)
    b, _ = ops.tree_attn_q8(q, small, *args)
    assert torch.equal(a, b)
    ops.ddtree_device_check()


# ------------------------------------------------------------------- used together

def test_rounds_over_an_8_bit_cache(cuda_device):
    """A prompt, drafted trees, their attention, commits, and decoding over what they left: each
    step against the 16-bit calls over the same cache read back."""
    gen = torch.Generator().manual_seed(12)
    B, Hq, Hkv, D, N, page = 3, 8, 2, 128, 20, 16
    table = torch.randperm(60, generator=gen)[:48].view(B, 16).to(I32).cuda()
    cache = ops.QuantCache.empty(60, Hkv, page, D, table, block=16)
    norm = ops.HeadNorm(torch.rand(D, generator=gen).cuda() + 0.5, torch.rand(D, generator=gen).cuda() + 0.5)
    rot = ops.Rotary(D, base=1e6)
    new = lambda *s: torch.randn(*s, generator=gen).to(BF16).cuda()  # noqa: E731
    lens = [37, 100, 5]
    starts = [0, 37, 137, 142]
    q, k, v = new(142, Hq, D), new(142, Hkv, D), new(142, Hkv, D)
    ops.ddtree_append_q8(k, v, ints(starts), ints([0] * B), cache, rot, norm, q=q)
    plen = ints(lens)
    for step in range(4):
        mask, n = pu.tree(gen, B, N, [N, N - 3, 7])
        mask, n = mask.cuda(), n.cuda()
        qt, kt, vt = new(B, N + 1, Hq, D), new(B, N + 1, Hkv, D), new(B, N + 1, Hkv, D)
        pos = (plen[:, None] + torch.arange(N + 1, device="cuda", dtype=I32)[None] % 5).contiguous()
        ops.ddtree_norm_rope(qt, kt, pos, norm, rot)
        out, lse = ops.tree_attn_q8(qt, cache, kt, vt, plen, n, mask)
        now = plen.tolist()
        at = [sum(now[:i]) for i in range(B + 1)]
        kk, vv = (torch.empty(at[-1], Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
        ops.ddtree_read_q8(cache, ints(at), ints([0] * B), kk, vv)
        kp, vp = (torch.zeros(60, Hkv, page, D, dtype=BF16, device="cuda") for _ in range(2))
        wide = ops.PagedCache(kp, vp, table)
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(now)).to(I32).cuda()
        where = torch.cat([torch.arange(m) for m in now]).to(I32).cuda()
        ops.ddtree_append_paged(kk, vv, seq, where, wide)
        o16, l16 = ops.tree_attn_paged(qt, wide, kt, vt, plen, n, mask)
        pu.check_attention(out, lse, reference(qt, cache, kt, vt, plen, n, mask), BF16, D)
        assert float((lse - l16)[torch.isfinite(l16)].abs().max()) < 1e-4
        assert float((out.float() - o16.float()).abs().max()) < 0.04
        alen = ints([3, 0, 1 + step])
        nodes = torch.full((B, 8), -1, dtype=I32)
        for b, a in enumerate(alen.tolist()):
            nodes[b, :a] = torch.arange(1, a + 1)
        nxt = torch.empty_like(plen)
        ops.ddtree_commit_q8(cache, kt, vt, alen, nodes.cuda(), plen, nxt)
        plen = nxt
        # plain decoding steps behind it
        q1, k1, v1 = new(B, Hq, D), new(B, Hkv, D), new(B, Hkv, D)
        ops.ddtree_append_q8(k1, v1, torch.arange(B + 1, dtype=I32, device="cuda"), plen, cache, rot, norm, q=q1)
        plen = plen + 1
    ops.ddtree_device_check()


def test_calls_on_a_stream_ahead_of_the_current_one(cuda_device):
    gen = torch.Generator().manual_seed(13)
    args = attn_case(gen, [900, 33], 20, 16, 4, 128, 32, 16, BF16)
    ref, rlse = ops.tree_attn_q8(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = ops.tree_attn_q8(*args, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, ref) and torch.equal(lse, rlse)
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1):
            out, _ = ops.tree_attn_q8(*args)
        assert torch.equal(out, ref)


def test_versions_and_gradients(cuda_device):
    cache = ops.QuantCache.empty(4, 1, 16, 64, ints([[0, 1]]), block=16)
    k = torch.randn(2, 1, 64, device="cuda", dtype=BF16)
    was = [t._version for t in (cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales)]
    ops.ddtree_append_q8(k.clone().requires_grad_(), k, ints([0, 2]), ints([0]), cache)
    assert all(t._version > w for t, w in zip((cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales), was))
    q = torch.randn(2, 2, 64, device="cuda", dtype=BF16).requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        ops.ddtree_append_q8(k, k, ints([0, 2]), ints([0]), cache, q=q)
    out = torch.empty(2, 1, 64, device="cuda", dtype=BF16)
    was = out._version
    ops.ddtree_read_q8(cache, ints([0, 2]), ints([0]), out, torch.empty_like(out))
    assert out._version > was


def test_python_refusals(cuda_device):
    c = ops.QuantCache.empty(4, 2, 16, 64, ints([[0, 1]]), block=8)
    k = torch.randn(3, 2, 64, device="cuda", dtype=BF16)
    f, at = ints([0, 3]), ints([0])
    qc = lambda **kw: ops.QuantCache(*[kw.get(n, getattr(c, n)) for n in (  # noqa: E731
        "k_pages", "v_pages", "k_scales", "v_scales", "page_table")], kw.get("dtype", BF16))
    for call in (lambda: qc(k_pages=c.k_pages.view(torch.uint8)), lambda: qc(v_pages=c.v_pages[:3]),
                 lambda: qc(k_scales=c.k_scales[..., :1]), lambda: qc(v_scales=c.v_scales.int()),
                 lambda: qc(page_table=c.page_table.long()), lambda: qc(dtype=FP32), lambda: qc(k_scales=c.k_scales[0]),
                 lambda: ops.QuantCache.empty(4, 2, 16, 64, ints([[0]]), block=5),
                 lambda: ops.ddtree_append_q8(k, k[:2], f, at, c), lambda: ops.ddtree_append_q8(k.half(), k.half(), f, at, c),
                 lambda: ops.ddtree_append_q8(k, k, f[:1], at, c), lambda: ops.ddtree_append_q8(k, k, f, ints([0, 0]), c),
                 lambda: ops.ddtree_append_q8(k, k, f.long(), at, c), lambda: ops.ddtree_append_q8(k, k, f, at, c, q_out=k),
                 lambda: ops.ddtree_append_q8(k, k, f, at, c, q=k[:2]),
                 lambda: ops.ddtree_append_q8(k, k, f, at, c, norm=ops.HeadNorm(torch.ones(32, device="cuda"))),
                 lambda: ops.ddtree_read_q8(c, f, at, k, k[:2]), lambda: ops.ddtree_read_q8(c, f, at, k.float(), k)):
        with pytest.raises(ValueError):
            call()
    odd = torch.randn(3 * 2 * 64 + 4, device="cuda").to(BF16)[4:].view(3, 2, 64)
    for call in (lambda: ops.ddtree_append_q8(odd, k, f, at, c), lambda: ops.ddtree_read_q8(c, f, at, k, k),
                 lambda: ops.ddtree_append_q8(k, k, f, at, c, ops.Rotary(24)),
                 lambda: ops.ddtree_read_q8(c, f, at, odd, k), lambda: ops.ddtree_append_q8(k, k, f, at, c, q=odd)):
        with pytest.raises(ops.DDTreeError):
            call()
    args = attn_case(torch.Generator().manual_seed(1), [30], 3, 4, 2, 64, 16, 8, BF16)
    with pytest.raises(ops.DDTreeError):
        ops.tree_attn_q8(*args, scale=float("nan"))
    with pytest.raises(ValueError):
        ops.tree_attn_q8(args[0].half(), *args[1:])
    ops.ddtree_device_check()
