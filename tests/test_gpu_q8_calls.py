"""Calls over an 8-bit cache that their documentation allows and no other test makes: captured
and replayed, from two threads, in other pieces, far out, next to what they are made of."""
import threading

import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu
from tests import q8_util as qu

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def held(c):
    return [c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.k_scales, c.v_scales]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(held(a), held(b)))


def fresh(pages, Hkv, page, D, table, block, dtype=BF16):
    return ops.QuantCache.empty(pages, Hkv, page, D, ints(table), block=block, dtype=dtype)


@pytest.mark.parametrize("block,D", [(8, 64), (32, 128), (64, 128)])
def test_a_prompt_in_chunks_of_whole_blocks_is_the_prompt_at_once(cuda_device, block, D):
    gen = torch.Generator().manual_seed(block)
    n, page = 5 * 64 + 13, 64
    table = [[4, 0, 7, 2, 9, 1]]
    k, v = (torch.randn(n, 3, D, generator=gen).to(BF16).cuda() for _ in range(2))
    rot, norm = ops.Rotary(D, interleaved=True), ops.HeadNorm()
    whole, parts, steps = (fresh(10, 3, page, D, table, block) for _ in range(3))
    ops.ddtree_append_q8(k, v, ints([0, n]), ints([0]), whole, rot, norm)
    for lo in range(0, n, 2 * block):
        hi = min(n, lo + 2 * block)
        ops.ddtree_append_q8(k[lo:hi], v[lo:hi], ints([0, hi - lo]), ints([lo]), parts, rot, norm)
    assert same(whole, parts)
    for i in range(n):  # one token a call: the same scales, codes rounded again where they grew
        ops.ddtree_append_q8(k[i:i + 1], v[i:i + 1], ints([0, 1]), ints([i]), steps, rot, norm)
    assert torch.equal(whole.k_scales, steps.k_scales) and torch.equal(whole.v_scales, steps.v_scales)
    a, b = (qu.values64(c.v_pages, c.v_scales, BF16) for c in (whole, steps))
    unit = torch.exp2(whole.v_scales.double() - 127).repeat_interleave(block, 2)[..., None]
    assert bool(((a - b).abs() <= unit * 2.0 ** -9).all())  # a step of the smallest codes, at most
    ops.ddtree_device_check()


@pytest.mark.parametrize("dtype,D,page,block", [(BF16, 128, 16, 16), (FP16, 64, 32, 8)])
def test_a_commit_is_the_append_of_its_rows(cuda_device, dtype, D, page, block):
    gen = torch.Generator().manual_seed(1)
    lens, alens, N, L, Hkv = [3, 40, 15], [5, 0, 7], 30, 8, 2
    p = qu.pool(gen, [a + b + 1 for a, b in zip(lens, alens)], Hkv, D, page, block, dtype)
    one = ops.QuantCache(*p, dtype)
    two = ops.QuantCache(*(x.clone() for x in p), dtype)
    kt, vt = (torch.randn(3, N + 1, Hkv, D, generator=gen).to(dtype).cuda() for _ in range(2))
    nodes = torch.full((3, L), -1, dtype=I32)
    rows, starts = [], [0]
    for b, a in enumerate(alens):
        path = (torch.randperm(N, generator=gen)[:a].sort().values + 1).tolist()
        nodes[b, :a] = torch.tensor(path, dtype=I32)
        rows += [(b, u) for u in [0] + path]
        starts.append(len(rows))
    ops.ddtree_commit_q8(one, kt, vt, ints(alens), nodes.cuda(), ints(lens))
    b, u = (list(x) for x in zip(*rows))
    ops.ddtree_append_q8(kt[b, u], vt[b, u], ints(starts), ints(lens), two)
    assert same(one, two)
    ops.ddtree_device_check()


def test_norm_and_rotation_on_the_way_are_those_of_norm_rope(cuda_device):
    gen = torch.Generator().manual_seed(2)
    D, n, at = 128, 77, 21
    q, k, v = (torch.randn(n, h, D, generator=gen).to(BF16).cuda() for h in (6, 2, 2))
    rot = ops.Rotary(64, base=5e5, scaling="yarn", factor=4.0, orig_len=4096, low=1, high=32)
    norm = ops.HeadNorm((torch.rand(D, generator=gen) + 0.5).cuda(), (torch.rand(D, generator=gen) + 0.5).cuda())
    cache = fresh(8, 2, 16, D, [[3, 1, 7, 0, 2, 5, 6, 4]], 16)
    q_out = torch.empty_like(q)
    ops.ddtree_append_q8(k, v, ints([0, n]), ints([at]), cache, rot, norm, q=q, q_out=q_out)
    pos = torch.arange(at, at + n, dtype=I32, device="cuda")
    nq, nk = ops.norm_rope(q, k, pos, norm, rot)
    # (the factor of the norm comes before or behind the rotation: two 32-bit results, each
    # within q8_util's bound of 2^-17 of a pair's |a| + |b| < 16, and one 16-bit step, where a
    # rounding falls the other way)
    near = 2 * 2.0 ** -17 * 16
    assert bool(((nq - q_out).float().abs() <= 2.0 ** -7 * nq.float().abs() + near).all())
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    ops.ddtree_read_q8(cache, ints([0, n]), ints([at]), kk, vv)
    for got, ref in ((kk, nk), (vv, v)):
        top = ref.float().abs().amax()
        # half a step of a code, of the 16-bit value compared with, of the smallest codes
        bound = ref.float().abs() * (2.0 ** -4 + 2.0 ** -7) + top * 2.0 ** -17 + near
        assert bool(((got - ref).float().abs() <= bound).all())
    ops.ddtree_device_check()


def test_positions_of_a_million(cuda_device):
    page, at, n, D = 256, 1_000_003, 40, 128
    table = torch.zeros(1, (at + n) // page + 1, dtype=I32)
    table[0, at // page:] = 1
    cache = ops.QuantCache.empty(2, 1, page, D, table.cuda(), block=64)
    k = torch.randn(n, 1, D, device="cuda").to(BF16)
    rot = ops.Rotary(D, base=1e6)
    before = [x.clone().cpu() for x in held(cache)]
    ops.ddtree_append_q8(k, k.clone(), ints([0, n]), ints([at]), cache, rot)
    ref, off = qu.turned64(k, None, None, torch.arange(at, at + n, device="cuda"), rot)
    after = [x.clone().cpu() for x in held(cache)]
    v = k.double().cpu()
    for half, (rows, o) in enumerate(((ref.cpu(), off.cpu()), (v, torch.zeros_like(v)))):
        rows_off = torch.full_like(o, 0) if half else o + ref.cpu().abs() * 2.0 ** -20
        qu.check_written((before[half].view(qu.E4M3), before[2 + half]), (after[half].view(qu.E4M3), after[2 + half]),
                         None, table, page, 64, BF16, [(0, at, rows, rows_off)])
    ops.ddtree_device_check()


@pytest.mark.parametrize("N", [0, 24])
def test_a_step_captured_in_one_graph_and_replayed(cuda_device, N):
    gen = torch.Generator().manual_seed(3)
    B, Hq, Hkv, D, page = 4, 8, 2, 128, 16
    table = torch.randperm(40, generator=gen)[:32].view(B, 8).to(I32).cuda()
    cache = ops.QuantCache.empty(40, Hkv, page, D, table, block=16)
    rot, norm = ops.Rotary(D), ops.HeadNorm()
    R = N + 1
    new = lambda *s: torch.randn(*s, generator=gen).to(BF16).cuda()  # noqa: E731
    q, k, v = new(B, Hq, D), new(B, Hkv, D), new(B, Hkv, D)
    qt, kt, vt = new(B, R, Hq, D), new(B, R, Hkv, D), new(B, R, Hkv, D)
    first, plen, n = torch.arange(B + 1, dtype=I32, device="cuda"), ints([0, 5, 31, 47]), ints([N] * B)
    mask, _ = pu.tree(gen, B, N, [N] * B)
    mask, pos = mask.cuda(), torch.randint(0, 90, (B, R), generator=gen, dtype=I32).cuda()
    alen, nodes, nxt = ints([min(2, N)] * B), torch.full((B, 4), -1, dtype=I32, device="cuda"), torch.zeros_like(plen)
    if N:
        nodes[:, :2] = ints([1, 2])
    out, lse = torch.empty_like(qt), torch.empty(B, R, Hq, device="cuda")
    q_out, qr, kr = torch.empty_like(q), torch.empty_like(qt), torch.empty_like(kt)
    kk, vv = (torch.zeros(B * 3, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    runs, ws = ints([0, 3, 3, 6, 9]), ops.q8_attn_workspace(qt, cache)

    def step():
        ops.ddtree_append_q8(k, v, first, plen, cache, rot, norm, q=q, q_out=q_out)
        ops.ddtree_norm_rope(qt, kt, pos, norm, rot, qr, kr)
        ops.ddtree_tree_attn_q8(qr, cache, kr, vt, plen, n, mask, out, lse, workspace=ws)
        ops.ddtree_commit_q8(cache, kr, vt, alen, nodes, plen, nxt)
        ops.ddtree_read_q8(cache, runs, plen, kk, vv)
        plen.copy_(nxt)

    def run(times, how):
        plen.copy_(ints([0, 5, 31, 47]))
        for x in held(cache)[:2]:
            x.zero_()
        for x in held(cache)[2:]:
            x.fill_(127)
        got = []
        for _ in range(times):
            how()
            got += [x.clone() for x in (*held(cache), out, lse, q_out, kk, vv, plen)]
        return got

    want = run(3, step)
    ops.ddtree_device_check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for a, b in zip(want, run(3, g.replay)):
        assert torch.equal(a, b)
    ops.ddtree_device_check()


def test_two_threads_on_their_own_streams(cuda_device):
    gen = torch.Generator().manual_seed(4)
    jobs = []
    for lens, N, Hq in (([700, 90], 0, 8), ([300, 41], 30, 8)):
        p = qu.pool(gen, lens, 2, 128, 32, 16, BF16)
        x = torch.randn(2, N + 1, Hq + 4, 128, generator=gen).to(BF16).cuda()
        mask, n = pu.tree(gen, 2, N, [N, N])
        args = (x[:, :, :Hq], ops.QuantCache(*p, BF16), x[:, :, Hq:Hq + 2], x[:, :, Hq + 2:], ints(lens), n.cuda(), mask.cuda())
        jobs.append((args, ops.tree_attn_q8(*args)))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        args, (ref, rlse) = jobs[i]
        with torch.cuda.stream(s):
            for _ in range(40):
                out, lse = ops.tree_attn_q8(*args)
                if not (torch.equal(out, ref) and torch.equal(lse, rlse)):
                    bad.append(i)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    ops.ddtree_device_check()


def test_handles_of_another_cache_are_refused(cuda_device):
    c8 = fresh(4, 2, 16, 64, [[0, 1]], 8)
    k16 = torch.zeros(4, 2, 16, 64, dtype=BF16, device="cuda")
    c16 = ops.PagedCache(k16, k16.clone(), ints([[0, 1]]))
    k = torch.randn(2, 2, 64, dtype=BF16, device="cuda")
    c8_as_16 = type("X", (), {n: getattr(c8, n) for n in ("_c", "_index", "B", "k_pages", "v_pages")})
    c16_as_8 = type("Y", (), {**{n: getattr(c16, n) for n in ("_c", "_index", "B", "k_pages", "v_pages")},
                              "k_scales": c8.k_scales, "v_scales": c8.v_scales})
    with pytest.raises(ValueError, match="handles"):
        ops.ddtree_append_paged(k, k, ints([0, 0]), ints([0, 1]), c8_as_16)
    with pytest.raises(ValueError, match="handles"):
        ops.ddtree_append_q8(k, k, ints([0, 2]), ints([0]), c16_as_8)


@pytest.mark.parametrize("T", [0, 3])
def test_batches_without_a_token_write_nothing(cuda_device, T):
    cache = fresh(4, 2, 16, 64, [[0, 1], [2, 3]], 16)
    k = torch.randn(T, 2, 64, dtype=BF16, device="cuda")
    q = torch.randn(T, 4, 64, dtype=BF16, device="cuda")
    was, q0 = [x.clone() for x in held(cache)], q.clone()
    ops.ddtree_append_q8(k, k.clone(), ints([T, T, T]), ints([0, 31]), cache, ops.Rotary(64), ops.HeadNorm(), q=q)
    out, out2 = torch.full_like(k, 2.0), torch.full_like(k, 2.0)
    ops.ddtree_read_q8(cache, ints([T, T, T]), ints([0, 31]), out, out2)
    assert all(torch.equal(a, b) for a, b in zip(was, held(cache))) and torch.equal(q, q0)
    assert bool((out == 2).all()) and bool((out2 == 2).all())
    ops.ddtree_device_check()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_an_empty_cache_has_the_least_scales(cuda_device, dtype):
    # (a run that enters a block in its middle keeps the larger of the old scale and its own)
    cache = fresh(3, 2, 16, 64, [[0]], 8, dtype)
    for s in (cache.k_scales, cache.v_scales):
        assert bool((s == 127 + qu.LEAST[dtype]).all())
