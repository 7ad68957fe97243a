"""Inputs and 64-bit references of the 8-bit cache's calls: plain torch, from the
format's definition.  Slots that a call must not read hold the code 0x7F, pages of no
sequence the scale byte 255."""
import torch

from tests import paged_util as pu

E4M3 = torch.float8_e4m3fn
LEAST = {torch.bfloat16: -96, torch.float16: -15}
MOST = 7


def exponent64(amax, dtype):
    """The least e with amax <= 448 * 2^e, within the type's range."""
    e = torch.full(amax.shape, LEAST[dtype], dtype=torch.int64, device=amax.device)
    for _ in range(MOST - LEAST[dtype]):
        e += (amax > 448 * torch.exp2(e.double())) & (e < MOST)
    return e


def grid64(x):
    """The nearest e4m3 number, ties to even, at most 448 in size."""
    unit = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6) - 3)
    return (torch.round(x / unit) * unit).clamp(-448, 448)


def codes64(pages):
    """Codes as numbers (0x7F, which is none, as 480), in 64 bits."""
    c = pages.view(torch.uint8).int()
    e, m = (c >> 3) & 15, c & 7
    size = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    return torch.where(c >= 128, -size, size)


def values64(pages, scales, dtype):
    """What a pool's codes stand for."""
    S = pages.shape[2] // scales.shape[2]
    e = (scales.int() - 127).clamp(LEAST[dtype], MOST).double()
    return codes64(pages) * torch.exp2(e).repeat_interleave(S, 2)[..., None]


def pool(gen, lens, Hkv, D, page, block, dtype, spare=2, width=None, slots_first=False, device="cuda",
         spread=1.0):
    """k_pages, v_pages (codes), k_scales, v_scales and table of a pool whose sequences hold
    lens positions; magnitudes differ by block."""
    B, nb = len(lens), page // block
    need = [-(-n // page) for n in lens]
    width = max(1, max(need)) if width is None else width
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    live = torch.zeros(total, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(need[b]):
            table[b, i] = order.pop()
            live[table[b, i], :min(page, n - i * page)] = True
    owned = torch.zeros(total, dtype=torch.bool)
    owned[order] = True  # (what is left: nobody's)
    made = []
    for _ in range(2):
        x = torch.randn(total, Hkv, nb, block, D, generator=gen)
        x *= torch.exp2(spread * torch.randn(total, Hkv, nb, 1, 1, generator=gen))
        e = exponent64(x.abs().amax((3, 4)).double(), dtype)
        c = (x * torch.exp2(-e.float())[..., None, None]).clamp(-448, 448)  # (as the writers do)
        c = c.view(total, Hkv, page, D).to(E4M3).view(torch.uint8)
        c = torch.where(live[:, None, :, None], c, torch.full_like(c, 0x7F))
        s = torch.where(owned[:, None, None], torch.full_like(e, 255), e + 127).to(torch.uint8)
        if slots_first:
            c = c.transpose(1, 2).contiguous().to(device).transpose(1, 2)
        made += [c.to(device).view(E4M3), s.to(device)]
    return made[0], made[2], made[1], made[3], table.to(device)


def cache(ops, p, dtype):
    return ops.QuantCache(*p, dtype)


def norm64(x, w, eps):
    y = x.double()
    y = y / ((y ** 2).mean(-1, keepdim=True) + eps).sqrt()
    return y if w is None else y * w.double()


def norm_off(D):
    """Relative error of a normed element in 32 bits: a sum of D squares (D roundings of
    2^-24, halved by the root), its mean and eps (2), the root's two units, and two
    products."""
    return D * 2.0 ** -25 + 6 * 2.0 ** -24 + 2.0 ** -22


def turned64(x, w, eps, pos, rotary):
    """(normed and rotated in 64 bits, the 32-bit result's error).  Tokens at negative
    positions as they are."""
    y = x.double() if eps is None else norm64(x, w, eps)
    off = y.abs() * (0.0 if eps is None else norm_off(x.shape[-1]))
    z = y
    if rotary is not None:
        z = pu.rotate64(y, pos, rotary.inv_freq, rotary.scale, rotary.interleaved)
        rot = rotary.rot_dim
        i = torch.arange(rot // 2, device=x.device)
        lo, hi = (2 * i, 2 * i + 1) if rotary.interleaved else (i, i + rot // 2)
        pair = (y[..., lo].abs() + y[..., hi].abs()) * abs(rotary.scale)
        each = (0.0 if eps is None else norm_off(x.shape[-1])) + 2.0 ** -21
        off = off.clone()
        off[..., lo], off[..., hi] = pair * each, pair * each
    there = (pos >= 0)[:, None, None]
    return torch.where(there, z, x.double()), torch.where(there, off, torch.zeros_like(off))


def check_16(got, ref, off, dtype, what=""):
    """One rounding to the type of a 32-bit result that is `off` away at most."""
    bound = off + (ref.abs() + off) * pu.HALF_STEP[dtype] + pu.TINY[dtype]
    pu.assert_within(got, ref, bound, what)


def check_written(before, after, ks, table, page, S, dtype, runs):
    """One half of a cache after runs [(b, at, rows64 [n][H][D], off)]: `before` and `after`
    are (codes, scales) on the CPU.  Every byte that no run owns is as it was."""
    codes0, scales0 = before
    codes1, scales1 = after
    want_same = torch.ones(codes0.shape[:3], dtype=torch.bool)
    scale_same = torch.ones(scales0.shape, dtype=torch.bool)
    c1, least = codes64(codes1), LEAST[dtype]
    for b, at, rows, off in runs:
        n = len(rows)
        for p0 in range(at // S * S, at + n if n else 0, S):
            lo, hi = max(p0, at), min(p0 + S, at + n)
            g, slot = int(table[b, p0 // page]), p0 % page
            x, d = rows[lo - at:hi - at], off[lo - at:hi - at]
            e = scales1[g, :, slot // S].long() - 127
            amax, far = x.abs().amax((0, 2)), d.amax((0, 2))
            small, large = exponent64((amax - far).clamp(min=0), dtype), exponent64(amax + far, dtype)
            scale_same[g, :, slot // S] = False
            want_same[g, :, slot + lo - p0:slot + hi - p0] = False
            if lo > p0:
                old = (scales0[g, :, slot // S].long() - 127).clamp(least, MOST)
                small, large = torch.maximum(small, old), torch.maximum(large, old)
                kept = codes64(codes0[g, :, slot:slot + lo - p0]) * torch.exp2((old - e).double())[:, None, None]
                grown = e > old
                got = c1[g, :, slot:slot + lo - p0]
                assert torch.equal(got[grown], grid64(kept)[grown]), f"codes before a run of {b} at {p0}"
                want_same[g, grown, slot:slot + lo - p0] = False
            assert bool(((e >= small) & (e <= large)).all()), (b, p0, e.tolist(), small.tolist(), large.tolist())
            unit = torch.exp2(e.double())[None, :, None]
            got = c1[g, :, slot + lo - p0:slot + hi - p0].transpose(0, 1) * unit
            ref = x.clamp(-448 * unit, 448 * unit)
            # half a step: 2^-4 of the value, or half of 2^-9 below the normal numbers
            bound = d + (ref.abs() + d) * 2.0 ** -4 + unit * 2.0 ** -10
            nearest = grid64(x / unit) * unit
            bound = torch.where(d == 0, (nearest - ref).abs(), bound)  # (exact inputs: the nearest code)
            pu.assert_within(got, ref, bound * (1 + 2.0 ** -40), f"codes of {b} at {p0}")
    same = codes0.view(torch.uint8) == codes1.view(torch.uint8)
    assert bool(same.all(-1)[want_same].all()), "codes that no run owns changed"
    assert bool((scales0 == scales1)[scale_same].all()), "scales that no run owns changed"
