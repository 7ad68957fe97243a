"""GPU tests of the paged-cache calls against 64-bit references (paged_util.py):
rotary positions, the append, tree attention over pages, the commit, and rounds
of them together.  NaN stands wherever a kernel must not read."""
import numpy as np
import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(gen, *shape, dtype=BF16):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


# ------------------------------------------------------------------ rotary

def _check_rope(x, got, pos, rot, inverse=False):
    ref = pu.rotate64(x, pos, rot.inv_freq, rot.scale, rot.interleaved, inverse)
    pu.assert_within(got, ref, pu.rotate_bound(x, ref, rot.inv_freq, rot.scale, rot.interleaved,
                                               x.dtype), "rope")
    assert torch.equal(got[..., rot.rot_dim:], x[..., rot.rot_dim:])
    assert torch.equal(got[pos < 0], x[pos < 0])


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,inter", [
    (1, 1, 1, 2, 2, FP32, False),         # the smallest
    (1, 32, 8, 128, 128, BF16, False),
    (65, 32, 8, 128, 128, BF16, False),
    (65, 32, 8, 128, 128, FP16, True),
    (37, 5, 0, 80, 40, BF16, False),      # half the head, 8-byte vectors, no keys
    (37, 5, 1, 80, 40, FP32, True),
    (19, 3, 3, 64, 2, FP16, False),       # one pair
    (19, 3, 3, 7, 6, FP16, True),         # odd rows: single elements
    (19, 3, 3, 7, 6, FP32, False),
    (9, 2, 1, 512, 512, FP32, False),     # the largest head
    (9, 2, 1, 511, 510, BF16, True),
    (1031, 7, 1, 96, 32, BF16, True),
])
def test_rope_matches_the_formula(cuda_device, T, Hq, Hkv, D, rot, dtype, inter):
    gen = _gen(T + D)
    r = ops.Rotary(rot, base=500000.0, interleaved=inter)
    q = _randn(gen, T, Hq, D, dtype=dtype)
    k = _randn(gen, T, Hkv, D, dtype=dtype) if Hkv else None
    pos = torch.randint(0, 200000, (T,), generator=gen).int().cuda()
    if T > 3:
        pos[1] = -1
        pos[3] = 0
    q2, k2 = ops.rope(q, k, pos, r)
    _check_rope(q, q2, pos, r)
    if k is not None:
        _check_rope(k, k2, pos, r)
    # in place: the same bits
    qi, ki = q.clone(), None if k is None else k.clone()
    ops.ddtree_rope(qi, ki, pos, r)
    assert torch.equal(qi, q2) and (k is None or torch.equal(ki, k2))


@pytest.mark.parametrize("scaling,kw", [
    ("linear", dict(factor=4.0)), ("ntk", dict(factor=3.0)),
    ("banded", dict(factor=8.0, orig_len=8192, low=1.0, high=4.0)),
    ("yarn", dict(factor=16.0, orig_len=4096, low=1.0, high=32.0))])
def test_rope_far_positions_and_scalings(cuda_device, scaling, kw):
    """Positions to the end of 32 bits: the angle has to keep its fraction."""
    gen = _gen(5)
    r = ops.Rotary(128, base=10000.0, scaling=scaling, **kw)
    x = _randn(gen, 8, 4, 128, dtype=FP32)
    pos = torch.tensor([0, 1, 4095, 131071, 1048575, 16777217, 2 ** 30 + 1, 2 ** 31 - 1],
                       dtype=torch.int32).cuda()
    got, _ = ops.rope(x, None, pos, r)
    ref = pu.rotate64(x, pos, r.inv_freq, r.scale, False)
    bound = pu.rotate_bound(x, ref, r.inv_freq, r.scale, False, FP32)
    # the reference's own angle, p f in 64 bits, is off by 2^-52 of it
    far = pos.double()[:, None, None] * 2.0 ** -51
    pu.assert_within(got, ref, bound + far * (x.double().abs().amax(-1, keepdim=True) * 2), scaling)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_transpose_and_the_gradient(cuda_device, inter):
    """<rope(x), g> = <x, inverse(g)>; inverse after forward is scale^2 x; and the
    gradient by central differences."""
    gen = _gen(9)
    r = ops.Rotary(48, base=10000.0, interleaved=inter, scaling="yarn", factor=4.0, orig_len=128,
                   low=1.0, high=8.0)
    x, g = (_randn(gen, 33, 3, 64, dtype=FP32) for _ in range(2))
    pos = torch.randint(0, 5000, (33,), generator=gen).int().cuda()
    y, _ = ops.rope(x, None, pos, r)
    gx, _ = ops.rope(g, None, pos, r, inverse=True)
    _check_rope(g, gx, pos, r, inverse=True)
    a, b = (y.double() * g.double()).sum(), (x.double() * gx.double()).sum()
    # 6336 products of values below 6, each factor within 2^-20 of its size
    assert abs(float(a - b)) <= 6336 * 36 * 2.0 ** -19
    back, _ = ops.rope(y, None, pos, r, inverse=True)
    want = x.double().clone()
    want[..., :48] *= r.scale ** 2
    pu.assert_within(back, want, torch.full_like(want, 2.0 ** -17), "inverse after forward")
    for at in ((0, 0, 0), (7, 1, 30), (32, 2, 63)):
        h = 0.5  # the map is linear: any step gives the derivative
        d = torch.zeros_like(x)
        d[at] = h
        up, _ = ops.rope(x + d, None, pos, r)
        dn, _ = ops.rope(x - d, None, pos, r)
        slope = ((up.double() - dn.double()) * g.double()).sum() / (2 * h)
        # 192 elements of one row's token, each difference off by 2^-20 of values below 8
        assert abs(float(slope - gx[at].double())) <= 192 * 6 * 2 * 8 * 2.0 ** -20


def test_rope_takes_strides_and_any_alignment(cuda_device):
    gen = _gen(11)
    r = ops.Rotary(64)
    pos = torch.arange(3 * 5).view(3, 5).int().cuda()
    buf = _randn(gen, 3, 5, 14, 64)                        # a fused projection: q, k, v
    q, k = buf[:, :, :8], buf[:, :, 8:10]
    before = buf.clone()
    q2, k2 = ops.rope(q, k, pos, r)
    _check_rope(q.reshape(15, 8, 64), q2.view(15, 8, 64), pos.view(-1), r)
    ops.ddtree_rope(q, k, pos, r)                          # in place, inside the buffer
    assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(buf[:, :, 10:], before[:, :, 10:])
    heads_first = _randn(gen, 4, 15, 64).transpose(0, 1)   # [heads][tokens][D]
    got, _ = ops.rope(heads_first, None, pos.view(-1), r)
    _check_rope(heads_first, got, pos.view(-1), r)
    one = _randn(gen, 15 * 2 * 64 + 1)[1:].view(15, 2, 64)  # two bytes off the grid
    got, _ = ops.rope(one, None, pos.view(-1), r)
    _check_rope(one, got, pos.view(-1), r)
    wide = _randn(gen, 15, 1, 64).expand(15, 3, 64)        # one head read three times
    got, _ = ops.rope(wide, None, pos.view(-1), r)
    _check_rope(wide, got, pos.view(-1), r)


def test_rope_custom_frequencies_streams_and_nothing(cuda_device):
    gen = _gen(13)
    r = ops.Rotary(8, inv_freq=[0.5, 7.0, 1e-6, -0.125], scale=1.5)
    x = _randn(gen, 20, 2, 16, dtype=FP32)
    pos = torch.arange(20).int().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = ops.rope(x, None, pos, r, stream=side)
    side.synchronize()
    _check_rope(x, got, pos, r)
    empty = x[:0]
    out, _ = ops.rope(empty, None, pos[:0], r)             # no tokens: nothing to do
    assert out.shape == (0, 2, 16)
    # padding rows may hold anything, and come back as they are
    x[5] = float("nan")
    x[6] = float("inf")
    pos[5:7] = -1
    got, _ = ops.rope(x, None, pos, r)
    assert torch.equal(torch.nan_to_num(got[5:7], 7.0), torch.nan_to_num(x[5:7], 7.0))


def test_rope_python_refusals(cuda_device):
    r = ops.Rotary(64)
    x, pos = torch.zeros(4, 2, 64, device="cuda", dtype=BF16), torch.zeros(4, device="cuda").int()
    for bad in (dict(q=x.double()), dict(pos=pos.long()), dict(pos=pos[:3]), dict(k=x[:3]),
                dict(k=x.half()), dict(q_out=x[:, :1]), dict(k_out=x), dict(q=x.cpu()),
                dict(q=x.transpose(1, 2)), dict(q=x[0])):
        args = dict(q=x, k=None, pos=pos, rotary=r) | bad
        with pytest.raises((ValueError, ops.DDTreeError)):
            ops.ddtree_rope(**args)
    with pytest.raises(ops.DDTreeError):                   # rot_dim above D
        ops.rope(x[..., :32], None, pos, r)
    with pytest.raises(ops.DDTreeError):                   # in place on overlapping rows
        ops.ddtree_rope(x[:, :1].expand(4, 2, 64), None, pos, r)


# ------------------------------------------------------------------ append

def _append_case(gen, B, new, at, Hkv, D, page, dtype, slots_first, pad=0):
    """A cache holding `at` positions, tokens that bring it to at + new."""
    k, v, table = pu.pool(gen, [a + n for a, n in zip(at, new)], Hkv, D, page, dtype,
                          slots_first=slots_first)
    seq = [b for b in range(B) for _ in range(new[b])] + [0] * pad
    pos = [at[b] + i for b in range(B) for i in range(new[b])] + [-1] * pad
    perm = torch.randperm(len(seq), generator=gen)         # tokens in any order
    seq, pos = torch.tensor(seq).int()[perm].cuda(), torch.tensor(pos).int()[perm].cuda()
    return ops.PagedCache(k, v, table), seq, pos


@pytest.mark.parametrize("B,new,at,Hq,Hkv,D,page,dtype,rot,inter,first,pad", [
    (1, [1], [0], 4, 1, 64, 16, BF16, 64, False, False, 0),
    (3, [1, 1, 1], [15, 16, 17], 32, 8, 128, 16, BF16, 128, False, False, 0),
    (3, [40, 0, 129], [3, 50, 0], 14, 2, 128, 64, FP16, 64, True, True, 3),
    (2, [70, 5], [0, 1], 0, 3, 80, 7, FP16, 40, False, False, 0),      # pages of 7, no queries
    (2, [9, 3], [2, 1], 3, 3, 33, 1, BF16, 0, False, True, 1),         # pages of 1, no rotation
    (2, [9, 3], [2, 1], 3, 1, 33, 128, BF16, 20, True, False, 0),
])
def test_append_matches_the_formula(cuda_device, B, new, at, Hq, Hkv, D, page, dtype, rot, inter,
                                    first, pad):
    gen = _gen(B + D + page)
    cache, seq, pos = _append_case(gen, B, new, at, Hkv, D, page, dtype, first, pad)
    T = seq.numel()
    buf = _randn(gen, T, Hq + 2 * Hkv, D, dtype=dtype)
    q, k, v = buf[:, :Hq], buf[:, Hq:Hq + Hkv], buf[:, Hq + Hkv:]
    r = ops.Rotary(rot, interleaved=inter, base=1e6) if rot else None
    k0, v0 = cache.k_pages.clone(), cache.v_pages.clone()
    q_out = torch.full_like(q, 7.0).contiguous() if Hq else None
    ops.ddtree_append_paged(k, v, seq, pos, cache, r, q if Hq else None, q_out)
    ops.ddtree_device_check()
    turn = lambda x: pu.rotate64(x, pos, r.inv_freq, r.scale, inter) if r else x.double()  # noqa: E731
    kk = turn(k)
    bound = (pu.rotate_bound(k, kk, r.inv_freq, r.scale, inter, dtype) if r
             else torch.zeros_like(kk))
    touched = torch.zeros(cache.num_pages, page, dtype=torch.bool)
    table = cache.page_table.cpu()
    for t in range(T):
        p, b = int(pos[t]), int(seq[t])
        if p < 0:
            continue
        pg = int(table[b, p // page])
        touched[pg, p % page] = True
        pu.assert_within(cache.k_pages[pg, :, p % page], kk[t], bound[t], f"key {t}")
        assert torch.equal(cache.v_pages[pg, :, p % page], v[t])
    rest = (~touched).cuda()
    for now, was in ((cache.k_pages, k0), (cache.v_pages, v0)):
        a, b = now.transpose(1, 2)[rest], was.transpose(1, 2)[rest]
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))  # bit for bit, NaN too
    if Hq:
        if r:
            _check_rope(q, q_out, pos, r)
        else:
            assert torch.equal(q_out, q)


def test_append_bad_tokens_are_skipped_and_recorded(cuda_device):
    gen = _gen(21)
    cache, seq, pos = _append_case(gen, 2, [4, 4], [0, 0], 2, 64, 4, BF16, False)
    k, v, q = (_randn(gen, 8, h, 64) for h in (2, 2, 4))
    r = ops.Rotary(64)
    good = (cache.k_pages.clone(), seq.clone(), pos.clone(), cache.page_table.clone())

    def expect(detail):
        with pytest.raises(ops.DDTreeError) as e:
            ops.ddtree_device_check()
        assert e.value.detail == detail
        assert torch.equal(torch.nan_to_num(cache.k_pages), torch.nan_to_num(good[0]))

    for bad_seq in (-1, 2, 2 ** 31 - 1):
        seq.fill_(bad_seq)
        q_out = torch.zeros_like(q)
        ops.ddtree_append_paged(k, v, seq, pos, cache, r, q, q_out)
        expect(0x06000005)
        _check_rope(q, q_out, pos, r)                      # queries are still rotated
    seq.copy_(good[1])
    pos.fill_(4 * cache.max_pages)
    ops.ddtree_append_paged(k, v, seq, pos, cache, r)
    expect(0x06000005)
    pos.copy_(good[2])
    for page in (-1, cache.num_pages, -2 ** 31):
        cache.page_table.fill_(page)
        ops.ddtree_append_paged(k, v, seq, pos, cache, r)
        expect(0x06000007)
    cache.page_table.copy_(good[3])
    ops.ddtree_append_paged(k, v, seq, pos, cache, r)
    ops.ddtree_device_check()


def test_append_offsets_past_32_bits(cuda_device):
    """A pool of more than 2^31 elements: its last page and one past the middle."""
    Hkv, D, page = 8, 128, 128
    pages = 2 ** 31 // (Hkv * D * page) + 5
    kp = torch.empty(pages, Hkv, page, D, dtype=BF16, device="cuda")
    vp = torch.empty_like(kp)
    table = torch.tensor([[pages - 1, 0, pages // 2 + 1]], dtype=torch.int32).cuda()
    for t in table[0].tolist():
        kp[t].zero_()
        vp[t].zero_()
    cache = ops.PagedCache(kp, vp, table)
    gen = _gen(2)
    k, v = _randn(gen, 3, Hkv, D), _randn(gen, 3, Hkv, D)
    pos = torch.tensor([127, 130, 300], dtype=torch.int32).cuda()
    ops.ddtree_append_paged(k, v, torch.zeros_like(pos), pos, cache)
    ops.ddtree_device_check()
    for i, p in enumerate(pos.tolist()):
        at = int(table[0, p // page])
        assert torch.equal(kp[at, :, p % page], k[i]) and torch.equal(vp[at, :, p % page], v[i])
    # and the attention reads them there
    q = _randn(gen, 1, 1, 16, D)
    plen, n, mask = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([384], [0], [[[1]]]))
    kt, vt = _randn(gen, 1, 1, Hkv, D), _randn(gen, 1, 1, Hkv, D)
    out, lse = ops.tree_attn_paged(q, cache, kt, vt, plen, n, mask)
    ops.ddtree_device_check()
    ref = pu.attention64(q, kp, vp, table, plen, kt, vt, n, mask, D ** -0.5)
    pu.check_attention(out, lse, ref, BF16, D)


# --------------------------------------------------------------- attention

def _attn_case(seed, lens, N, Hq, Hkv, D, page, dtype, slots_first=False, width=None, live=None,
               fused=False, chain=False):
    gen = _gen(seed)
    B, R = len(lens), N + 1
    live = [N if b % 3 != 2 else N // 2 for b in range(B)] if live is None else live
    k, v, table = pu.pool(gen, lens, Hkv, D, page, dtype, width=width, slots_first=slots_first,
                          device="cuda")
    mask, n = pu.tree(gen, B, N, live, depth=1 if chain else None)
    if fused:
        buf = _randn(gen, B, R, Hq + 2 * Hkv, D, dtype=dtype)
        q, kt, vt = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hkv], buf[:, :, Hq + Hkv:]
    else:
        q, kt, vt = (_randn(gen, B, R, h, D, dtype=dtype) for h in (Hq, Hkv, Hkv))
    for b in range(B):
        kt[b, live[b] + 1:] = float("nan")
        vt[b, live[b] + 1:] = float("nan")
    return dict(q=q, cache=ops.PagedCache(k, v, table), k_tree=kt, v_tree=vt,
                prefix_len=torch.tensor(lens, dtype=torch.int32).cuda(), n_nodes=n.cuda(),
                anc_mask=mask.cuda())


def _ref(c, scale=None):
    D = c["cache"].D
    return pu.attention64(c["q"], c["cache"].k_pages, c["cache"].v_pages, c["cache"].page_table,
                          c["prefix_len"], c["k_tree"], c["v_tree"], c["n_nodes"], c["anc_mask"],
                          D ** -0.5 if scale is None else scale)


CASES = [
    # lens, N, Hq, Hkv, D, page, dtype, slots_first, width, fused
    ([0], 0, 1, 1, 64, 16, BF16, False, None, False),        # one key: the token itself
    ([1], 0, 8, 2, 128, 16, BF16, False, None, False),
    ([127, 128, 129], 0, 32, 8, 128, 16, BF16, False, None, False),
    ([15, 16, 17, 0], 0, 3, 1, 128, 8, FP16, False, None, False),   # pages of 8, G = 3
    ([700, 3, 1500], 0, 14, 2, 64, 32, FP16, True, None, True),     # G = 7
    ([900], 0, 128, 1, 128, 64, BF16, False, None, False),          # G = 128
    ([1000, 20], 0, 16, 1, 128, 256, BF16, False, None, False),     # a page is two tiles
    ([3000], 0, 8, 8, 128, 16, BF16, False, 4096, False),           # a table far wider than used
    ([257, 64], 5, 4, 2, 128, 128, BF16, False, None, True),
    ([2048], 64, 32, 8, 128, 16, BF16, False, None, False),
    ([300, 0, 65], 21, 28, 4, 64, 32, FP16, True, None, True),
    ([129], 40, 5, 1, 128, 64, FP16, False, None, False),           # G = 5
    ([500, 10], 127, 8, 8, 128, 16, BF16, True, None, False),       # G = 1
    ([1000], 200, 32, 2, 64, 64, BF16, False, None, False),         # G = 16
    ([40], 130, 100, 1, 128, 16, FP16, False, None, False),         # G = 100: a node a tile
    ([129], 1024, 4, 2, 128, 32, BF16, False, None, False),         # the largest tree
    # few rows: 16, 32 and 64 of them, one over; two mask words; one long sequence
    ([64, 0, 63, 65, 200], 3, 8, 2, 128, 16, BF16, False, None, False),
    ([700, 5], 7, 8, 2, 64, 8, FP16, True, None, True),
    ([333, 64], 15, 16, 4, 128, 64, BF16, False, None, False),
    ([128, 1], 16, 16, 4, 128, 64, BF16, False, None, False),
    ([90, 700], 63, 3, 3, 128, 32, FP16, False, None, False),
    ([90, 700], 32, 1, 1, 64, 128, BF16, False, None, True),
    ([20011], 0, 4, 1, 128, 16, BF16, False, None, False),
    ([20011], 0, 40, 2, 64, 64, FP16, False, None, False),
    ([0, 0, 0, 9000, 0], 4, 8, 1, 128, 32, BF16, False, None, False),
]


@pytest.mark.parametrize("lens,N,Hq,Hkv,D,page,dtype,first,width,fused", CASES)
def test_attention_matches_the_formula(cuda_device, lens, N, Hq, Hkv, D, page, dtype, first, width,
                                       fused):
    c = _attn_case(N + D + Hq, lens, N, Hq, Hkv, D, page, dtype, first, width, None, fused)
    out, lse = ops.tree_attn_paged(**c)
    ops.ddtree_device_check()
    pu.check_attention(out, lse, _ref(c), dtype, D)


@pytest.mark.parametrize("B,hi,N,Hq,Hkv,D,page,dtype", [
    (20, 9500, 0, 8, 8, 64, 64, BF16),       # decoding, splits merged through the workspace
    (40, 300, 0, 16, 4, 128, 16, FP16),      # decoding, one tile or two each
    (20, 9000, 3, 16, 8, 128, 128, FP16),
    (24, 900, 70, 28, 4, 64, 32, BF16),      # many trees, a lone query tile
    (3, 9000, 300, 8, 8, 64, 64, FP16),      # two tile pairs a unit, splits merged
])
def test_attention_of_large_batches(cuda_device, B, hi, N, Hq, Hkv, D, page, dtype):
    lens = [(hi - 37 * b) % (hi + 1) if b % 4 else b for b in range(B)]
    c = _attn_case(B + N, lens, N, Hq, Hkv, D, page, dtype)
    ws = ops.paged_attn_workspace(c["q"], c["cache"])
    ref = _ref(c)
    for _ in range(2):                        # the workspace serves call after call
        out, lse = ops.tree_attn_paged(**c, workspace=ws)
        ops.ddtree_device_check()
        pu.check_attention(out, lse, ref, dtype, D)


@pytest.mark.parametrize("lens,width", [
    ([5000, 9, 4000, 700] * 5, 4096),        # ranked by length, splits of the longest list
    ([8300] * 8 + [0, 127, 128], 1 << 16),   # a table for a million positions
    ([300] * 12, 4096),                      # no list worth a split
    ([5000, 0, 60] * 40, 2048),              # too many to rank: thirds of the table
])
def test_attention_under_wide_tables(cuda_device, lens, width):
    """Tables far wider than the longest sequence, many query tiles; the workspace
    serves other lengths after that."""
    c = _attn_case(len(lens), lens, 64, 32, 8, 128, 16, BF16, width=width)
    ws = ops.paged_attn_workspace(c["q"], c["cache"])
    for shift in range(2):
        if shift:
            c["prefix_len"] = c["prefix_len"] - torch.clamp(c["prefix_len"] // 2, max=1500)
        out, lse = ops.tree_attn_paged(**c, workspace=ws)
        ops.ddtree_device_check()
        pu.check_attention(out, lse, _ref(c), BF16, 128)


@pytest.mark.parametrize("N,G,D,dtype,hi,width", [
    (64, 4, 128, BF16, 5000, None),    # one pair a unit and one node, lists cut
    (64, 4, 64, FP16, 900, None),      # ... whole
    (65, 4, 128, FP16, 700, 512),      # two nodes left over
    (128, 4, 128, BF16, 9000, None),   # two pairs share the key tiles
    (256, 8, 64, BF16, 300, None),     # eight pairs, lists shorter than that
    (32, 8, 128, BF16, 4000, 4096),    # 8 rows
    (84, 3, 128, FP16, 2000, None),    # tiles of 126 rows
    (263, 1, 128, BF16, 600, None),    # eight nodes of one row
    (128, 1, 64, FP16, 100, None),     # a single row; one list of a tile or two
])
def test_attention_rows_left_over(cuda_device, N, G, D, dtype, hi, width):
    """A few rows more than whole query tiles: prefixes of any length, last nodes that
    are there, that are not, and trees too small for a pair; a workspace for all."""
    B, Hkv = 22, 8
    lens = [(hi - 41 * b) % (hi + 1) if b % 4 else b // 4 for b in range(B)]
    lens[3] = hi
    live = [N if b % 3 else [N - 1, N // 2, 0, N][b // 3 % 4] for b in range(B)]
    c = _attn_case(N + G, lens, N, Hkv * G, Hkv, D, 16, dtype, live=live, width=width)
    c["anc_mask"][5, N] = 0                       # a last node that sees its prefix alone ...
    c["prefix_len"][5] = 0                        # ... and has none
    ws = ops.paged_attn_workspace(c["q"], c["cache"])
    first = None
    for _ in range(3):
        out, lse = ops.tree_attn_paged(**c, workspace=ws)
        ops.ddtree_device_check()
        if first is None:
            pu.check_attention(out, lse, _ref(c), dtype, D)
            assert bool((out[5, N] == 0).all()) and bool((lse[5, N] == -np.inf).all())
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])   # bit for bit
    # captured twice over one workspace, replayed in turn
    outs = [torch.full_like(out, 7.0) for _ in range(2)]
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.ddtree_tree_attn_paged(c["q"], c["cache"], c["k_tree"], c["v_tree"], c["prefix_len"],
                                       c["n_nodes"], c["anc_mask"], o, workspace=ws)
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    ops.ddtree_device_check()
    assert torch.equal(outs[0], first[0]) and torch.equal(outs[1], first[0])


def test_calls_on_a_stream_ahead_of_the_current_one(cuda_device):
    """What a call allocates itself -- the workspace's zeros above all -- is on its
    own stream: the current one may be far behind."""
    c = _attn_case(8, [5000] * 20, 64, 32, 8, 128, 16, BF16)
    rot = ops.Rotary(128)
    pos = torch.arange(20 * 65, device="cuda").int().view(20, 65)
    want = ops.tree_attn_paged(**c)
    want_q, want_k = ops.rope(c["q"], c["k_tree"], pos, rot)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)                # ~10 ms of the current stream
    out, lse = ops.tree_attn_paged(**c, stream=side)
    q, k = ops.rope(c["q"], c["k_tree"], pos, rot, stream=side)
    side.synchronize()
    ops.ddtree_device_check()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(q, want_q) and torch.equal(torch.nan_to_num(k), torch.nan_to_num(want_k))


@pytest.mark.parametrize("seed", range(24))
def test_attention_random_shapes(cuda_device, seed):
    """Seeded shapes over the whole range, rows kernel and general kernel, one CTA
    and many, with whatever lengths fall out."""
    rng = np.random.default_rng(1000 + seed)
    Hkv, G, D = int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 32])), int(rng.choice([64, 128]))
    B = int(min(rng.integers(1, 40), max(1, 300 // (Hkv * G))))
    N = int(rng.choice([0, 0, 1, 3, 7, 15, 16, 31, 63, 64, 127, 200]))
    hi = int(np.exp(rng.uniform(0, np.log(6000))))
    lens = [int(x) for x in rng.integers(0, hi + 1, size=B)]
    live = [int(x) for x in rng.integers(0, N + 1, size=B)]
    c = _attn_case(seed, lens, N, Hkv * G, Hkv, D, int(rng.choice([8, 16, 32, 64, 128, 256])),
                   BF16 if seed % 2 else FP16, bool(seed % 3 == 0), None, live, bool(seed % 4 == 0))
    out, lse = ops.tree_attn_paged(**c)
    ops.ddtree_device_check()
    pu.check_attention(out, lse, _ref(c), c["q"].dtype, D)


@pytest.mark.parametrize("B,Hkv,N", [(1024, 1, 0), (1025, 1, 0), (700, 2, 1)])
def test_attention_of_very_many_sequences(cuda_device, B, Hkv, N):
    """As many sequences as the rows kernel adds up, and one more (the general one)."""
    lens = [(37 * b) % 91 if b % 5 else 0 for b in range(B)]
    c = _attn_case(B, lens, N, 2 * Hkv, Hkv, 64, 16, BF16, live=[N * (b % 2) for b in range(B)])
    bad = B // 2
    ref = _ref(c)
    c["prefix_len"][bad] = -5                 # one sequence in the middle is skipped
    out, lse = torch.full_like(c["q"], 3.0), torch.full(c["q"].shape[:3], 3.0, device="cuda")
    ops.ddtree_tree_attn_paged(**c, out=out, lse=lse,
                               workspace=ops.paged_attn_workspace(c["q"], c["cache"]))
    with pytest.raises(ops.DDTreeError):
        ops.ddtree_device_check()
    assert bool((out[bad] == 3.0).all())
    keep = torch.arange(B, device="cuda") != bad
    pu.check_attention(out[keep], lse[keep], [x[keep] for x in ref], BF16, 64)


def test_attention_chain_mask_is_causal(cuda_device):
    """A chain of drafted tokens is a causal chunk: a plain lower triangle."""
    c = _attn_case(77, [100], 50, 8, 2, 128, 16, BF16, live=[50], chain=True)
    out, lse = ops.tree_attn_paged(**c)
    ops.ddtree_device_check()
    bits = c["anc_mask"].cpu().numpy().view(np.uint32)[0]
    for u in range(51):
        assert sum(int(w) << (32 * i) for i, w in enumerate(bits[u])) == (1 << (u + 1)) - 1
    pu.check_attention(out, lse, _ref(c), BF16, 128)


@pytest.mark.parametrize("N,Hq", [(0, 4), (40, 8)])
def test_attention_rows_without_a_key(cuda_device, N, Hq):
    """An empty prefix and an empty mask row: zeros and -inf, whatever v holds."""
    c = _attn_case(3, [0, 30], N, Hq, 2, 128, 16, BF16, live=[N, N])
    c["anc_mask"][0, 0] = 0
    if N:
        c["anc_mask"][0, 17] = 0
    out, lse = ops.tree_attn_paged(**c)
    ops.ddtree_device_check()
    assert bool((out[0, 0] == 0).all()) and bool((lse[0, 0] == -np.inf).all())
    pu.check_attention(out, lse, _ref(c), BF16, 128)


@pytest.mark.parametrize("N,lens,scale", [(0, [900, 5], 3.0), (30, [600, 257], 2.0)])
def test_attention_peaked_softmax(cuda_device, N, lens, scale):
    """Scores with a spread of hundreds, the largest key last: the running maximum
    climbs through the prefix, so every rescaling of the partial output counts."""
    c = _attn_case(8, lens, N, 8, 2, 128, 16, FP16)
    page = c["cache"].page_size
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            c["cache"].k_pages[int(c["cache"].page_table[b, i])] *= 0.02 + i * page / n
    out, lse = ops.tree_attn_paged(**c, scale=scale)
    ops.ddtree_device_check()
    pu.check_attention(out, lse, _ref(c, scale), FP16, 128)


def test_attention_shares_pages_between_sequences(cuda_device):
    """Two sequences with a common prefix name the same pages."""
    c = _attn_case(12, [200, 200], 9, 8, 2, 128, 16, BF16, live=[9, 9])
    c["cache"].page_table[1, :8] = c["cache"].page_table[0, :8]
    out, lse = ops.tree_attn_paged(**c)
    ops.ddtree_device_check()
    pu.check_attention(out, lse, _ref(c), BF16, 128)


@pytest.mark.parametrize("N", [0, 33])
def test_attention_bad_pages_count_as_zeros(cuda_device, N):
    c = _attn_case(14, [200, 90], N, 8, 2, 128, 16, BF16, live=[N, N])
    for bad in (-1, c["cache"].num_pages, 2 ** 31 - 1, -2 ** 31):
        table = c["cache"].page_table.clone()
        c["cache"].page_table[0, 3] = bad
        out, lse = ops.tree_attn_paged(**c)
        with pytest.raises(ops.DDTreeError) as e:
            ops.ddtree_device_check()
        assert e.value.detail == 0x03000007
        c["cache"].page_table.copy_(table)
        k, v = (torch.cat([t, torch.zeros_like(t[:1])]) for t in (c["cache"].k_pages,
                                                                  c["cache"].v_pages))
        table[0, 3] = c["cache"].num_pages
        ref = pu.attention64(c["q"], k, v, table, c["prefix_len"], c["k_tree"], c["v_tree"],
                             c["n_nodes"], c["anc_mask"], 128 ** -0.5)
        pu.check_attention(out, lse, ref, BF16, 128)


@pytest.mark.parametrize("what,value,detail", [
    ("prefix_len", -1, 0x03000001), ("prefix_len", 209, 0x03000001),
    ("n_nodes", -1, 0x03000002), ("n_nodes", 4, 0x03000002)])
@pytest.mark.parametrize("N", [0, 3])
def test_attention_bad_lengths_leave_the_sequence(cuda_device, what, value, detail, N):
    if what == "n_nodes" and value == 4:
        value = N + 1
    c = _attn_case(15, [200, 90], N, 8, 2, 128, 16, BF16, live=[N, N])
    ref = _ref(c)
    c[what][0] = value
    out, lse = torch.full_like(c["q"], 5.0), torch.full(c["q"].shape[:3], 5.0, device="cuda")
    ops.ddtree_tree_attn_paged(**c, out=out, lse=lse,
                               workspace=ops.paged_attn_workspace(c["q"], c["cache"]))
    with pytest.raises(ops.DDTreeError) as e:
        ops.ddtree_device_check()
    assert e.value.detail == detail
    assert bool((out[0] == 5.0).all()) and bool((lse[0] == 5.0).all())
    pu.check_attention(out[1:], lse[1:], [x[1:] for x in ref], BF16, 128)


@pytest.mark.parametrize("N,lens", [(0, [3000] * 3), (64, [2048])])
def test_attention_captured_and_replayed(cuda_device, N, lens):
    """A captured call follows what its tensors hold at each replay; two graphs
    on two streams with a workspace each."""
    c = _attn_case(16, lens, N, 32, 8, 128, 16, BF16, live=[N] * len(lens))
    out = [torch.empty_like(c["q"]) for _ in range(2)]
    lse = [torch.empty(c["q"].shape[:3], device="cuda") for _ in range(2)]
    ws = [ops.paged_attn_workspace(c["q"], c["cache"]) for _ in range(2)]
    ops.ddtree_tree_attn_paged(**c, out=out[0], lse=lse[0], workspace=ws[0])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.ddtree_tree_attn_paged(**c, out=out[i], lse=lse[i], workspace=ws[i])
        graphs.append(g)
    gen = _gen(99)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for n in (lens[0], 77, 0):
        c["prefix_len"].fill_(n)
        c["q"].copy_(_randn(gen, *c["q"].shape))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        ops.ddtree_device_check()
        ref = _ref(c)
        for o, z in zip(out, lse):
            pu.check_attention(o, z, ref, BF16, 128)


@pytest.mark.parametrize("B,P,page", [(16, 8000, 64), (16, 3001, 16)])
def test_attention_lone_tiles_of_a_full_gpu(cuda_device, B, P, page):
    """128 nodes and the root are four query tiles and four rows: the lone tile of
    every (sequence, KV head), with the GPU full and every wait a real one, run
    after run against the formula."""
    N, Hq, Hkv, D = 128, 32, 8, 128
    gen = torch.Generator(device="cuda").manual_seed(P)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    per = -(-P // page)
    k, v = rn(B * per, Hkv, page, D), rn(B * per, Hkv, page, D)
    table = torch.randperm(B * per, generator=gen, device="cuda").int().view(B, per)
    q, kt, vt = rn(B, N + 1, Hq, D), rn(B, N + 1, Hkv, D), rn(B, N + 1, Hkv, D)
    mask, n = pu.tree(_gen(P), B, N, [N] * B)
    cache, plen, n, mask = ops.PagedCache(k, v, table), torch.full((B,), P).int().cuda(), n.cuda(), mask.cuda()
    ws = ops.paged_attn_workspace(q, cache)
    u = N                                     # the node of the lone tile
    bits = ((mask[:, u, torch.arange(N + 1, device="cuda") // 32] >> (torch.arange(N + 1, device="cuda") % 32)) & 1).bool()
    ref = torch.empty(B, Hq, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        for g in range(Hkv):
            kk = torch.cat([k[table[b].long(), g].reshape(-1, D)[:P], kt[b, bits[b], g]]).double()
            vv = torch.cat([v[table[b].long(), g].reshape(-1, D)[:P], vt[b, bits[b], g]]).double()
            x = q[b, u, g * 4:g * 4 + 4].double() @ kk.T / D ** 0.5
            ref[b, g * 4:g * 4 + 4] = x.softmax(1) @ vv
    for _ in range(6):
        out, _ = ops.tree_attn_paged(q, cache, kt, vt, plen, n, mask, workspace=ws)
        ops.ddtree_device_check()
        # (averages of 3000 values and more: |out| stays below 0.5, sum w|v| below 1.5)
        assert float((out[:, u].double() - ref).abs().max()) <= 2 ** -8 * (0.5 + 1.5)


def test_attention_is_repeatable(cuda_device):
    """Run after run the same bits: merges do not depend on which split ends last."""
    for N, lens in ((0, [5000] * 20), (128, [3000, 2000]), (64, [9000] * 20)):
        c = _attn_case(18, lens, N, 16, 8, 128, 64, BF16)
        first = ops.tree_attn_paged(**c)
        for _ in range(5):
            again = ops.tree_attn_paged(**c)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_python_refusals(cuda_device):
    c = _attn_case(15, [20, 9], 3, 8, 2, 128, 16, BF16)
    out, lse = torch.empty_like(c["q"]), torch.empty(c["q"].shape[:3], device="cuda")
    ok = dict(c, out=out, lse=lse, workspace=ops.paged_attn_workspace(c["q"], c["cache"]))
    ops.ddtree_tree_attn_paged(**ok)
    for bad in (dict(q=c["q"].half()), dict(q=c["q"][:1]), dict(k_tree=c["k_tree"][:, :3]),
                dict(prefix_len=c["prefix_len"].long()), dict(n_nodes=c["n_nodes"][:1]),
                dict(anc_mask=c["anc_mask"][:, :3]), dict(out=out[:, :3]), dict(lse=lse.half()),
                dict(out=out.cpu()), dict(workspace=torch.zeros(64, device="cuda")),
                dict(workspace=None), dict(workspace=ok["workspace"][:256]),
                dict(q=c["q"].transpose(0, 1)), dict(scale=-1.0)):
        with pytest.raises((ValueError, ops.DDTreeError)):
            ops.ddtree_tree_attn_paged(**(ok | bad))
    with pytest.raises(ValueError):
        ops.PagedCache(c["cache"].k_pages, c["cache"].v_pages.half(), c["cache"].page_table)
    with pytest.raises(ValueError):
        ops.PagedCache(c["cache"].k_pages, c["cache"].v_pages, c["cache"].page_table.long())


# ------------------------------------------------------------------ commit

def _paths(gen, B, N, L, alens):
    nodes = torch.full((B, L), -1, dtype=torch.int32)
    for b, a in enumerate(alens):
        nodes[b, :a] = (torch.randperm(N, generator=gen)[:a] + 1).sort().values.int()
    return torch.tensor(alens, dtype=torch.int32).cuda(), nodes.cuda()


@pytest.mark.parametrize("lens,alens,N,L,Hkv,D,page,dtype,first", [
    ([0], [0], 0, 1, 1, 8, 16, BF16, False),
    ([5, 15, 16], [3, 1, 0], 8, 4, 2, 64, 16, FP16, True),
    ([100, 0, 63, 1], [16, 16, 0, 7], 64, 16, 8, 128, 4, BF16, False),   # five pages a path
    ([31], [16], 1024, 16, 3, 72, 1, BF16, False),                        # pages of one
])
def test_commit_matches_the_definition(cuda_device, lens, alens, N, L, Hkv, D, page, dtype, first):
    gen = _gen(N + L)
    B = len(lens)
    k, v, table = pu.pool(gen, [n + a + 1 for n, a in zip(lens, alens)], Hkv, D, page, dtype,
                          slots_first=first)
    cache = ops.PagedCache(k, v, table)
    buf = _randn(gen, B, N + 1, 2 * Hkv, D, dtype=dtype)
    kt, vt = buf[:, :, :Hkv], buf[:, :, Hkv:]
    alen, nodes = _paths(gen, B, N, L, alens)
    P = torch.tensor(lens, dtype=torch.int32).cuda()
    new = torch.full_like(P, -7)
    wk, wv = k.clone(), v.clone()
    for b in range(B):
        for i, u in enumerate([0] + nodes[b, :alens[b]].tolist()):
            at = lens[b] + i
            wk[table[b, at // page].long(), :, at % page] = kt[b, u]
            wv[table[b, at // page].long(), :, at % page] = vt[b, u]
    ops.ddtree_commit_paged(cache, kt, vt, alen, nodes, P, new)
    ops.ddtree_device_check()
    assert torch.equal(k.view(torch.int16), wk.view(torch.int16))
    assert torch.equal(v.view(torch.int16), wv.view(torch.int16))
    assert new.tolist() == [n + a + 1 for n, a in zip(lens, alens)] and P.tolist() == lens


def test_commit_bad_paths_leave_the_sequence(cuda_device):
    gen = _gen(31)
    lens, alens = [10, 20], [4, 5]
    k, v, table = pu.pool(gen, [16, 32], 2, 64, 8, BF16)
    cache = ops.PagedCache(k, v, table)
    kt, vt = _randn(gen, 2, 9, 2, 64), _randn(gen, 2, 9, 2, 64)
    alen, nodes = _paths(gen, 2, 8, 6, alens)
    P = torch.tensor(lens, dtype=torch.int32).cuda()
    new = torch.zeros_like(P)
    ok = [x.clone() for x in (alen, nodes, P, table, k, v)]

    def run(detail):
        k.copy_(ok[4])
        ops.ddtree_commit_paged(cache, kt, vt, alen, nodes, P, new)
        with pytest.raises(ops.DDTreeError) as e:
            ops.ddtree_device_check()
        assert e.value.detail == detail
        mine = torch.zeros(cache.num_pages, dtype=torch.bool, device="cuda")
        mine[ok[3][0, :2].long()] = True
        assert torch.equal(torch.nan_to_num(k[mine]), torch.nan_to_num(ok[4][mine]))
        assert new.tolist() == [int(P[0]), 26]             # the other sequence is committed
        for x, y in zip((alen, nodes, P, table), ok):
            x.copy_(y)

    for a in (-1, 7):
        alen[0] = a
        run(0x05000001)
    for p in (-1, 8 * cache.max_pages - 4):
        P[0] = p
        run(0x05000001)
    for u in (0, 9, -1):
        nodes[0, 2] = u
        run(0x05000003)
    for page in (-1, cache.num_pages):
        table[0, 1] = page
        run(0x05000007)


# ---------------------------------------------------------- whole rounds

def _rotate_rows(x, pos, r):
    return pu.rotate64(x, pos, r.inv_freq, r.scale, r.interleaved)


def test_rounds_over_a_paged_cache(cuda_device):
    """Prompts appended, then rounds of two layers: draft top-K, build, queries and
    tree keys rotated at pos_id, attention over the pages, walk, commit.  After
    each round the pages hold exactly the prompt and the accepted paths, and the
    attention equals the formula over them."""
    dev, gen = cuda_device, _gen(41)
    B, L, V, K, N, Hq, Hkv, D, page, layers = 3, 6, 500, 4, 24, 12, 4, 64, 16, 2
    prompts = [37, 1, 128]
    reach = 400
    width = reach // page
    order = torch.randperm(B * width, generator=gen).int().view(B, width).cuda()
    caches = [ops.PagedCache(torch.full((B * width, Hkv, page, D), float("nan"), dtype=BF16, device=dev),
                             torch.full((B * width, Hkv, page, D), float("nan"), dtype=BF16, device=dev),
                             order) for _ in range(layers)]
    r = ops.Rotary(D, base=1e6)
    kept = [[[] for _ in range(B)] for _ in range(layers)]  # (key, value) rows in order
    seq = torch.tensor([b for b in range(B) for _ in range(prompts[b])] + [0, 0]).int().cuda()
    pos = torch.tensor([i for b in range(B) for i in range(prompts[b])] + [-1, -1]).int().cuda()
    for c, rows in zip(caches, kept):
        k, v = _randn(gen, seq.numel(), Hkv, D), _randn(gen, seq.numel(), Hkv, D)
        q = _randn(gen, seq.numel(), Hq, D)
        ops.ddtree_append_paged(k, v, seq, pos, c, r, q)
        k2, _ = ops.rope(k, None, pos, r)                  # the same rotation, the same bits
        for t in range(sum(prompts)):
            rows[int(seq[t])].append((k2[t], v[t]))
    plen = torch.tensor(prompts, dtype=torch.int32, device=dev)
    bonus = torch.tensor([1, 2, 3], dtype=torch.int32, device=dev)
    accepted = 0
    for step in range(4):
        draft = torch.randn(B, L, V, generator=gen).mul(3).to(dev)
        idx, lp, _ = ops.topk(draft, K)
        tree = ops.build(lp, idx, bonus, plen, N)
        new_len = torch.empty_like(plen)
        depth = tree["depth"].clamp(0, L - 1).long()
        target = torch.gather(draft, 1, depth[..., None].expand(-1, -1, V)).contiguous()
        acc = ops.accept(target, tree, L)
        for c, rows in zip(caches, kept):
            buf = _randn(gen, B, N + 1, Hq + 2 * Hkv, D)
            q, kt, vt = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hkv], buf[:, :, Hq + Hkv:]
            raw = buf.clone()
            ops.ddtree_rope(q, kt, tree["pos_id"], r)
            flat = raw[:, :, :Hq].reshape(-1, Hq, D)
            _check_rope(flat, q.reshape(-1, Hq, D), tree["pos_id"].view(-1), r)
            out, lse = ops.tree_attn_paged(q, c, kt, vt, plen, tree["n_nodes"], tree["anc_mask"])
            ops.ddtree_device_check()
            ref = pu.attention64(q, c.k_pages, c.v_pages, c.page_table, plen, kt, vt,
                                 tree["n_nodes"], tree["anc_mask"], D ** -0.5)
            pu.check_attention(out, lse, ref, BF16, D)
            ops.ddtree_commit_paged(c, kt, vt, acc["accept_len"], acc["accepted_nodes"], plen,
                                    new_len)
            ops.ddtree_device_check()
            for b in range(B):
                a = int(acc["accept_len"][b])
                for u in [0] + acc["accepted_nodes"][b, :a].tolist():
                    rows[b].append((kt[b, u].clone(), vt[b, u].clone()))
                accepted += a
        plen, bonus = new_len, acc["next_bonus"]
        for c, rows in zip(caches, kept):
            for b in range(B):
                n = int(plen[b])
                assert n == len(rows[b])
                at = c.page_table[b, torch.arange(n, device=dev) // page].long()
                slot = torch.arange(n, device=dev) % page
                assert torch.equal(c.k_pages.transpose(1, 2)[at, slot], torch.stack([k for k, _ in rows[b]]))
                assert torch.equal(c.v_pages.transpose(1, 2)[at, slot], torch.stack([v for _, v in rows[b]]))
    assert accepted > 0


def test_decoding_steps_captured_in_one_graph(cuda_device):
    """Plain decoding, one token a sequence and step: append with rotation, then
    attention of the token over the pages before it; one captured graph replayed
    while positions advance."""
    gen, B, Hq, Hkv, D, page, width = _gen(43), 5, 14, 2, 128, 16, 8
    table = torch.randperm(B * width, generator=gen).int().view(B, width).cuda()
    pages = [torch.zeros(B * width, Hkv, page, D, dtype=FP16, device="cuda") for _ in range(2)]
    cache = ops.PagedCache(*pages, table)
    r = ops.Rotary(D, interleaved=True)
    q, k, v = (torch.zeros(B, 1, h, D, dtype=FP16, device="cuda") for h in (Hq, Hkv, Hkv))
    kr, qr = torch.zeros_like(k), torch.zeros_like(q)
    seq = torch.arange(B).int().cuda()
    pos = torch.tensor([0, 1, 14, 15, 60]).int().cuda()
    n = torch.zeros(B).int().cuda()
    mask = torch.ones(B, 1, 1).int().cuda()
    out, lse = torch.empty_like(q), torch.empty(B, 1, Hq, device="cuda")
    ws = ops.paged_attn_workspace(q, cache)

    def step():
        ops.ddtree_rope(q, k, pos, r, qr, kr)
        ops.ddtree_tree_attn_paged(qr, cache, kr, v, pos, n, mask, out, lse, workspace=ws)
        ops.ddtree_append_paged(k, v, seq, pos, cache, r)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(20):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen).half())
        qq = pu.rotate64(q[:, 0], pos, r.inv_freq, r.scale, True)
        g.replay()
        ops.ddtree_device_check()
        ref = pu.attention64(qr, *pages, table, pos, kr, v, n, mask, D ** -0.5)
        pu.check_attention(out, lse, ref, FP16, D)
        pu.assert_within(qr[:, 0], qq, pu.rotate_bound(q[:, 0], qq, r.inv_freq, r.scale, True, FP16))
        at, slot = table[torch.arange(B), (pos // page).long()].long(), (pos % page).long()
        assert torch.equal(pages[0].transpose(1, 2)[at, slot], kr[:, 0])
        pos += 1
