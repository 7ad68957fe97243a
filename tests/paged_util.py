"""Inputs and 64-bit references of the paged-cache calls: plain torch, from the
formulas.  Everything a kernel must not read is NaN: slots past a sequence's
last position, pages of no sequence, tree rows past the tree."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}  # half the last subnormal


def rotate64(x, pos, inv_freq, scale, interleaved, inverse=False):
    """x [tokens][heads][D] in 64 bits; tokens at negative positions unchanged."""
    rot = 2 * len(inv_freq)
    f = torch.tensor(list(inv_freq), dtype=torch.float64, device=x.device)
    a = pos.double()[:, None, None] * f * (-1.0 if inverse else 1.0)
    c, s = a.cos() * scale, a.sin() * scale
    y = x.double().clone()
    i = torch.arange(rot // 2, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., lo] = x.double()[..., lo] * c - x.double()[..., hi] * s
    y[..., hi] = x.double()[..., lo] * s + x.double()[..., hi] * c
    return torch.where((pos >= 0)[:, None, None], y, x.double())


def rotate_bound(x, ref, inv_freq, scale, interleaved, dtype):
    """Largest error of a rotated element: one rounding to the type, and in 32
    bits at most 2^-21 of |a| + |b| -- sine and cosine each within 2^-22 (their
    argument is rounded at 2^-25 of a turn's quarter, the function at 2 units),
    two products and a sum at 2^-24 each."""
    rot = 2 * len(inv_freq)
    i = torch.arange(rot // 2, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    pair = (x.double()[..., lo].abs() + x.double()[..., hi].abs()) * abs(scale)
    extra = torch.zeros_like(ref)
    extra[..., lo] = pair * 2.0 ** -21
    extra[..., hi] = pair * 2.0 ** -21
    return extra + ref.abs() * HALF_STEP[dtype] * (1 + 2.0 ** -7) + TINY[dtype]


def assert_within(got, ref, bound, what=""):
    bad = (got.double() - ref).abs() > bound
    bad |= torch.isnan(got.double()) != torch.isnan(ref)
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {at}: "
                             f"{float(got[at])} for {float(ref[at])} +- {float(bound[at])}")


def pool(gen, lens, Hkv, D, page, dtype, spare=2, width=None, slots_first=False, device="cuda"):
    """k_pages, v_pages [num_pages][Hkv][page][D] and table [B][width]: random rows
    below lens, NaN elsewhere; table entries past the last page are -1."""
    B = len(lens)
    need = [-(-n // page) for n in lens]
    width = max(1, max(need)) if width is None else width
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen).tolist()
    shape = (total, page, Hkv, D) if slots_first else (total, Hkv, page, D)
    k, v = (torch.full(shape, float("nan"), dtype=dtype) for _ in range(2))
    if slots_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(need[b]):
            at = order.pop()
            table[b, i] = at
            m = min(page, n - i * page)
            for t in (k, v):
                t[at, :, :m] = torch.randn(Hkv, m, D, generator=gen).to(dtype)
    if device == "cpu":
        return k, v, table
    dense = [torch.empty_strided(t.shape, t.stride(), dtype=dtype, device=device) for t in (k, v)]
    for d, t in zip(dense, (k, v)):
        d.copy_(t)
    return dense[0], dense[1], table.to(device)


def tree(gen, B, N, live, depth=None):
    """anc_mask int32 [B][N+1][W] of random trees, and n_nodes: node u's parent is
    any earlier node (depth=1: always the one before, a chain)."""
    R, W = N + 1, (N + 32) // 32
    seen = torch.zeros(B, R, R, dtype=torch.bool)
    for b in range(B):
        for u in range(live[b] + 1):
            if u:
                p = u - 1 if depth == 1 else int(torch.randint(0, u, (1,), generator=gen))
                seen[b, u] = seen[b, p]
            seen[b, u, u] = True
    bits = torch.zeros(B, R, W * 32, dtype=torch.int64)
    bits[..., :R] = seen
    words = (bits.view(B, R, W, 32) << torch.arange(32)).sum(-1)
    return words.to(torch.int32), torch.tensor(live, dtype=torch.int32)


def attention64(q, k_pages, v_pages, table, prefix, k_tree, v_tree, n_nodes, mask, scale):
    """(out, lse, weight, score, mass) in 64 bits: weight = sum_j w_j |v_j|, score =
    the largest sum_d |q_d k_jd| scale of a row, mass = sum_j |v_j| over the keys
    it sees (what the error bounds need)."""
    B, R, Hq, D = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, R, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, R, Hq), -math.inf, dtype=torch.float64, device=q.device)
    weight, score, mass = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(out)
    bit = torch.arange(R, device=q.device)
    for b in range(B):
        P, n = int(prefix[b]), int(n_nodes[b])
        pages = table[b, :-(-P // page)].long()
        see = ((mask[b, :n + 1][:, bit[:n + 1] // 32] >> (bit[:n + 1] % 32)) & 1).bool()
        for g in range(Hkv):
            k = torch.cat([k_pages[pages, g].reshape(-1, D)[:P], k_tree[b, :n + 1, g]]).double()
            v = torch.cat([v_pages[pages, g].reshape(-1, D)[:P], v_tree[b, :n + 1, g]]).double()
            for h in range(g * G, (g + 1) * G):
                x = (q[b, :n + 1, h].double() @ k.T) * scale
                x[:, P:] = x[:, P:].masked_fill(~see, -math.inf)
                z = torch.logsumexp(x, 1)
                w = (x - z.clamp(min=-1e300)[:, None]).exp()
                out[b, :n + 1, h], lse[b, :n + 1, h] = w @ v, z
                weight[b, :n + 1, h] = w @ v.abs()
                mass[b, :n + 1, h] = (x > -math.inf).double() @ v.abs()
                score[b, :n + 1, h] = (q[b, :n + 1, h].double().abs() @ k.abs().T).amax(1) * scale
    return out, lse, weight, score, mass


def check_attention(out, lse, ref, dtype, D):
    """The kernel's arithmetic: scores from exact products summed in 32 bits (D
    additions of at most 2^-24 of sum |q k|), scaled and exponentiated in 32 bits
    (2^-20 in all, arguments below 2^6), weights rounded to the type, output
    rounded once."""
    r_out, r_lse, weight, score, mass = ref
    u = HALF_STEP[dtype]
    ds = score * D * 2.0 ** -24 + 2.0 ** -20 * (1 + score)
    bound = weight * (u + 2 * ds[..., None] + 2.0 ** -18) * (1 + u) + r_out.abs() * u + 2 * TINY[dtype]
    if dtype == torch.float16:  # a weight below the normal numbers: half of 2^-24 off, and
        bound = bound + 2.0 ** -25 * mass  # the unit of weights is at most the row's sum
    assert_within(out, r_out, bound, "out")
    live = torch.isfinite(r_lse)
    assert torch.equal(live, torch.isfinite(lse)) and bool((lse[~live] == -math.inf).all())
    assert bool((out[~live] == 0).all())
    off = (lse.double() - r_lse).abs()
    lim = ds + 2.0 ** -17 + r_lse.abs() * 2.0 ** -22
    assert bool((off[live] <= lim[live]).all()), f"lse off by {float((off - lim)[live].max())}"
