"""Rotary positions and the append with thousands of tokens.  A CTA of the rotary
kernel takes several tokens once there are enough to fill the GPU with such CTAs
(16 of them on each of 152 SMs: two tokens each from 4864 tokens on, 16 from 38912):
the step from token to token, the tables of several tokens, and a last CTA with
fewer tokens than the others run here only."""
import pytest
import torch

from diffusion_draft_tree_gb300 import ops
from tests import paged_util as pu
from tests.test_gpu_paged import _check_rope

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape, dtype=BF16):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,inter", [
    (5003, 5, 1, 128, 128, BF16, False),   # two tokens a CTA
    (5003, 5, 1, 128, 64, FP16, True),
    (5001, 3, 2, 80, 40, FP32, True),      # 16-byte vectors of four
    (5001, 3, 1, 33, 20, BF16, False),     # single elements
    (9999, 8, 1, 64, 64, BF16, True),      # four
    (20011, 2, 1, 128, 32, FP16, False),   # eight
    (38912, 1, 1, 64, 64, BF16, False),    # 16, none left over
    (40001, 5, 1, 128, 128, BF16, False),  # 16, one in the last CTA
    (40001, 1, 1, 128, 128, FP16, True),
    (80021, 1, 0, 64, 16, FP32, False),
    (80021, 2, 1, 96, 48, BF16, True),
])
def test_rope_of_many_tokens(cuda_device, T, Hq, Hkv, D, rot, dtype, inter):
    gen = _gen(T + D)
    r = ops.Rotary(rot, base=500000.0, interleaved=inter)
    q = _randn(gen, T, Hq, D, dtype=dtype)
    k = _randn(gen, T, Hkv, D, dtype=dtype) if Hkv else None
    pos = torch.randint(0, 200000, (T,), generator=gen, device="cuda").int()
    pos[torch.randint(0, T, (T // 7,), generator=gen, device="cuda")] = -1
    q2, k2 = ops.rope(q, k, pos, r)
    _check_rope(q, q2, pos, r)
    if k is not None:
        _check_rope(k, k2, pos, r)
    back, _ = ops.rope(q, None, pos, r, inverse=True)
    _check_rope(q, back, pos, r, inverse=True)
    ops.ddtree_rope(q, k, pos, r)          # in place: the same bits
    assert torch.equal(q, q2) and (k is None or torch.equal(k, k2))


@pytest.mark.parametrize("T,Hq,Hkv,D,page,rot,dtype,inter,first", [
    (5003, 5, 1, 128, 16, 128, BF16, False, False),
    (5003, 0, 2, 64, 64, 32, FP16, True, True),
    (5001, 4, 2, 33, 7, 20, BF16, False, False),
    (40001, 5, 1, 128, 64, 128, BF16, False, True),
    (40001, 0, 1, 64, 16, 64, FP16, True, False),
    (80021, 1, 1, 64, 128, 0, BF16, False, False),   # as they are
])
def test_append_of_many_tokens(cuda_device, T, Hq, Hkv, D, page, rot, dtype, inter, first):
    """Tokens in any order over seven sequences, one in nine of them padding, and
    some whose sequence does not exist."""
    gen, B = _gen(T + D + page), 7
    width = -(-T // (B * page)) + 1
    total = B * width + 2
    shape = (total, page, Hkv, D) if first else (total, Hkv, page, D)
    pages = [_randn(gen, *shape, dtype=dtype) for _ in range(2)]
    view = [p.transpose(1, 2) if first else p for p in pages]
    table = torch.randperm(total, generator=gen, device="cuda")[:B * width].int().view(B, width)
    cache = ops.PagedCache(*view, table)
    where = torch.randperm(B * width * page, generator=gen, device="cuda")[:T]  # all different
    seq, pos = (where // (width * page)).int(), (where % (width * page)).int()
    kind = torch.randint(0, 18, (T,), generator=gen, device="cuda")
    pos[kind < 2] = -1
    seq[kind == 2] = B
    put = kind > 2
    buf = _randn(gen, T, Hq + 2 * Hkv, D, dtype=dtype)
    q, k, v = buf[:, :Hq], buf[:, Hq:Hq + Hkv], buf[:, Hq + Hkv:]
    q_out = torch.empty(T, Hq, D, dtype=dtype, device="cuda") if Hq else None
    r = ops.Rotary(rot, interleaved=inter, base=1e6) if rot else None
    was = [x.clone() for x in view]
    ops.ddtree_append_paged(k, v, seq, pos, cache, r, q if Hq else None, q_out)
    with pytest.raises(ops.DDTreeError) as e:
        ops.ddtree_device_check()
    assert e.value.detail == 0x06000005
    at, slot = table[seq[put].long(), (pos[put] // page).long()].long(), (pos[put] % page).long()
    rows = [x.transpose(1, 2)[at, slot] for x in view]
    if r:
        _check_rope(k[put], rows[0], pos[put], r)
    else:
        assert torch.equal(rows[0], k[put])
    assert torch.equal(rows[1], v[put])
    touched = torch.zeros(total, page, dtype=torch.bool, device="cuda")
    touched[at, slot] = True
    for now, old in zip(view, was):        # and nothing else
        assert torch.equal(now.transpose(1, 2)[~touched], old.transpose(1, 2)[~touched])
    if Hq and r:
        _check_rope(q, q_out, pos, r)
    elif Hq:
        assert torch.equal(q_out, q)
