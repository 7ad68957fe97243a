"""Tree attention over pages in the plans that the shapes of test_gpu_paged.py do
not reach: there a few rows that whole pairs of query tiles leave over are mostly
taken along, so that the lone query tile of a full GPU, and with it the 32-bit merge
of the general kernel through the workspace, stood without a reference.  Each case
asserts by the size of its workspace which plan it runs."""
import threading

import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def _case(seed, lens, N, G, Hkv, D, page, dtype, width=None, live=None, chain=False):
    """Inputs made on the GPU; NaN where a kernel must not read."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    B, R = len(lens), N + 1
    need = torch.tensor([-(-n // page) for n in lens], device="cuda")
    total = int(need.sum()) + 2
    width = max(1, int(need.max())) if width is None else width
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    there = torch.arange(width, device="cuda")[None] < need[:, None]
    order = torch.randperm(total, generator=gen, device="cuda").int()
    table[there] = order[:int(need.sum())]
    k, v = rn(total, Hkv, page, D), rn(total, Hkv, page, D)
    for b, n in enumerate(lens):
        if n % page:
            for t in (k, v):
                t[table[b, n // page].long(), :, n % page:] = float("nan")
    for at in order[int(need.sum()):].long():
        k[at], v[at] = float("nan"), float("nan")
    live = [N if b % 3 != 2 else N // 2 for b in range(B)] if live is None else live
    mask, n = pu.tree(torch.Generator().manual_seed(seed), B, N, live, depth=1 if chain else None)
    q, kt, vt = rn(B, R, Hkv * G, D), rn(B, R, Hkv, D), rn(B, R, Hkv, D)
    for b in range(B):
        kt[b, live[b] + 1:], vt[b, live[b] + 1:] = float("nan"), float("nan")
    return dict(q=q, cache=ops.PagedCache(k, v, table), k_tree=kt, v_tree=vt,
                prefix_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                n_nodes=n.cuda(), anc_mask=mask.cuda())


def _size(c):
    B, R, Hq, D = c["q"].shape
    return ops.workspace_size(ops.OP_TREE_ATTN_PAGED, B=B, N=R - 1, Hq=Hq, Hkv=c["cache"].Hkv, D=D,
                              cache_cap=c["cache"].max_pages * c["cache"].page_size)


def _check(c, out, lse):
    D = c["cache"].D
    ref = pu.attention64(c["q"], c["cache"].k_pages, c["cache"].v_pages, c["cache"].page_table,
                         c["prefix_len"], c["k_tree"], c["v_tree"], c["n_nodes"], c["anc_mask"],
                         D ** -0.5)
    pu.check_attention(out, lse, ref, c["q"].dtype, D)


def _runs(c, times=3, merges=False):
    """A call's results, the same bits each time over one workspace; merges: it has to
    hold partial results after the first."""
    ws = ops.paged_attn_workspace(c["q"], c["cache"])
    first = ops.tree_attn_paged(**c, workspace=ws)
    ops.ddtree_device_check()
    assert not merges or bool(ws.any())
    for _ in range(times - 1):
        again = ops.tree_attn_paged(**c, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ops.ddtree_device_check()
    return first


def _lens(B, hi):
    return [hi if b % 3 == 1 else (hi - 97 * b) % (hi + 1) if b % 4 else 5 * b for b in range(B)]


# more than 8 rows left over: an odd number of query tiles, the last of them alone
LONE = [
    (22, 70, 4, 8, 128, 64, BF16),    # 28 rows of the third tile
    (22, 100, 3, 8, 64, 16, FP16),    # tiles of 126 rows, 51 of the third
    (24, 40, 7, 7, 128, 32, BF16),    # 18 nodes a tile, five of the third
    (40, 20, 5, 8, 128, 128, FP16),   # one tile in all, 105 rows
]


@pytest.mark.parametrize("B,N,G,Hkv,D,page,dtype", LONE)
@pytest.mark.parametrize("hi", [300, 3000, 9500])
def test_lone_query_tiles_of_a_full_gpu(cuda_device, hi, B, N, G, Hkv, D, page, dtype):
    """... whole lists, although those behind 9500 tokens could be cut."""
    c = _case(hi + N, _lens(B, hi), N, G, Hkv, D, page, dtype)
    per = 128 // G
    tiles = -(-(N + 1) // per)
    assert tiles % 2 and (N + 1 - (tiles - 1) * per) * G > 8 and B * Hkv * (tiles + 1) // 2 >= 152
    if hi > 8192:                             # every tile has parts of three pieces at least
        assert _size(c) >= B * Hkv * tiles * 3 * 128 * D * 4
    else:
        assert _size(c) == 0
    _check(c, *_runs(c))


@pytest.mark.parametrize("B,N,G,Hkv,D,page,dtype,hi,width", [
    (10, 127, 4, 8, 128, 64, BF16, 9500, None),     # two pairs
    (20, 63, 4, 8, 64, 16, FP16, 12000, None),      # one
    (20, 63, 4, 8, 128, 16, BF16, 9500, 4096),      # a table seven times too wide
    (12, 255, 2, 8, 64, 32, BF16, 8700, None),      # four tiles of 64 nodes
    (5, 511, 4, 8, 128, 64, FP16, 8500, None),      # eight pairs
    (20, 70, 4, 8, 128, 64, BF16, 9500, None),      # lone tiles
    (100, 70, 4, 2, 64, 64, BF16, 8500, None),      # too many sequences to rank; lone tiles
    (100, 63, 4, 2, 64, 64, FP16, 8500, 1024),      # ... and a table too wide
])
def test_pieces_of_whole_tiles_merge_through_the_workspace(cuda_device, B, N, G, Hkv, D, page, dtype,
                                                           hi, width):
    """Lists that the batch's lengths let the kernel cut: their parts are there."""
    c = _case(hi + N, _lens(B, hi), N, G, Hkv, D, page, dtype, width)
    tiles = -(-(N + 1) * G // 128)
    assert _size(c) >= B * Hkv * tiles * 3 * 128 * D * 4
    # (unranked lists are cut at the plan's share of the table: a quarter of 513 tiles,
    # under the wide one, is 129, more than the 68 of the longest list here)
    cut = B <= 96 or c["cache"].max_pages * page // 128 // 4 < hi // 128
    _check(c, *_runs(c, merges=cut))


@pytest.mark.parametrize("N,G", [(70, 4), (127, 4)])
def test_lone_and_whole_tiles_with_every_wait_a_real_one(cuda_device, N, G):
    """Long lists on a full GPU, run after run against the formula: a wait that takes
    one tile's end for another's shows here."""
    B, P = 16, 8000
    c = _case(N, [P] * B, N, G, 8, 128, 16, BF16, live=[N] * B)
    ws = ops.paged_attn_workspace(c["q"], c["cache"])
    want = None
    for _ in range(8):
        out, lse = ops.tree_attn_paged(**c, workspace=ws)
        ops.ddtree_device_check()
        if want is None:
            want = out, lse
            _check(c, out, lse)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("N", [512, 1023])
@pytest.mark.parametrize("P", [0, 2048, 32768])
def test_a_prompts_chunk(cuda_device, N, P):
    """A chain of nodes is a causal chunk of a prompt: to 1024 rows of it, behind
    nothing, behind pages, behind a long prefix."""
    c = _case(N + P, [P, max(0, P - 77)], N, 4, 2, 128, 64, BF16, live=[N, N - 200], chain=True)
    _check(c, *_runs(c, 2))


def test_the_workspaces_zeros_are_on_the_calls_stream(cuda_device):
    """A call that allocates its own workspace, with counters in it, on a stream far
    ahead of the current one: memory that held other bytes on both streams."""
    c = _case(3, _lens(20, 9500), 70, 4, 8, 128, 64, BF16)
    n = _size(c)
    assert n > 0
    want = _runs(c, 2, merges=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            dirty = torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda")
            del dirty
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)               # some 20 ms of the current stream
    out, lse = ops.tree_attn_paged(**c, stream=side)
    side.synchronize()
    ops.ddtree_device_check()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_two_threads_call_at_once(cuda_device):
    """Two host threads, a stream and a workspace each, first calls of a shape among
    them."""
    cases = [_case(11, [900], 50, 4, 2, 128, 16, BF16), _case(12, _lens(20, 9500), 70, 4, 8, 128, 64, BF16)]
    got, torn = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = ops.tree_attn_paged(**cases[i], stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            torn.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not torn, torn
    ops.ddtree_device_check()
    for c, g in zip(cases, got):
        _check(c, *g)
