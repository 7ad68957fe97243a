"""Host side of the paged-cache calls, no GPU: rotary frequencies and turns
against their formulas, and every refusal of a bad argument before a launch."""
import ctypes
import math
import struct

import pytest

from diffusion_draft_tree_gb300 import ops

P = ctypes.c_void_p
L = ops.lib


def _freq(rot, base, scaling, factor=1.0, orig=8192.0, low=1.0, high=4.0):
    f, s = (ctypes.c_double * (rot // 2))(), ctypes.c_float()
    assert L.ddtree_rope_frequencies(rot, base, ops.ROPE_SCALINGS[scaling], factor, orig, low,
                                     high, f, ctypes.byref(s)) == 0
    return list(f), s.value


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 1e6), (510, 500000.0)])
def test_frequencies_follow_their_formulas(rot, base):
    plain = [base ** (-2 * j / rot) for j in range(rot // 2)]
    close = lambda a, b: all(math.isclose(x, y, rel_tol=1e-13) for x, y in zip(a, b))  # noqa: E731
    assert close(_freq(rot, base, "none")[0], plain)
    assert close(_freq(rot, base, "linear", 4.0)[0], [f / 4 for f in plain])
    if rot > 2:
        b2 = base * 3.0 ** (rot / (rot - 2))
        assert close(_freq(rot, base, "ntk", 3.0)[0], [b2 ** (-2 * j / rot) for j in range(rot // 2)])
    got, scale = _freq(rot, base, "banded", 8.0, 8192, 1, 4)
    assert scale == 1.0
    for g, f in zip(got, plain):
        wave = 2 * math.pi / f
        if wave < 8192 / 4:
            assert g == f
        elif wave > 8192:
            assert math.isclose(g, f / 8, rel_tol=1e-13)
        else:
            s = (8192 / wave - 1) / 3
            assert math.isclose(g, (1 - s) * f / 8 + s * f, rel_tol=1e-12)
    got, scale = _freq(rot, base, "yarn", 16.0, 4096, 1, 32)
    assert math.isclose(scale, 0.1 * math.log(16) + 1, rel_tol=1e-6)
    assert all(f / 16 * (1 - 1e-13) <= g <= f * (1 + 1e-13) for g, f in zip(got, plain))
    assert _freq(rot, base, "yarn", 1.0, 4096, 1, 32)[1] == 1.0
    if rot == 128:
        d = lambda t: rot * math.log(4096 / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(d(32))), min(rot - 1, math.ceil(d(1)))
        assert 0 < lo < hi < rot // 2
        assert got[lo] == plain[lo] and math.isclose(got[hi], plain[hi] / 16, rel_tol=1e-13)
        mid = (lo + hi) // 2
        s = (mid - lo) / (hi - lo)
        assert math.isclose(got[mid], (1 - s) * plain[mid] + s * plain[mid] / 16, rel_tol=1e-12)


def test_frequency_refusals():
    f, s = (ctypes.c_double * 512)(), ctypes.c_float()
    call = lambda *a: L.ddtree_rope_frequencies(*a, f, ctypes.byref(s))  # noqa: E731
    assert call(3, 1e4, 0, 1, 0, 0, 0) == 1       # odd
    assert call(0, 1e4, 0, 1, 0, 0, 0) == 1
    assert call(514, 1e4, 0, 1, 0, 0, 0) == 2
    assert call(64, 0.0, 0, 1, 0, 0, 0) == 1
    assert call(64, float("nan"), 0, 1, 0, 0, 0) == 1
    assert call(64, 1e4, 5, 1, 0, 0, 0) == 1
    assert call(64, 1e4, 1, 0.0, 0, 0, 0) == 1
    assert call(2, 1e4, 2, 2.0, 0, 0, 0) == 1     # NTK divides by rot - 2
    assert call(64, 1e4, 3, 2.0, 0, 1, 4) == 1    # no original length
    assert call(64, 1e4, 3, 2.0, 8192, 4, 4) == 1
    assert call(64, 1.0, 4, 2.0, 8192, 1, 32) == 1  # YARN divides by ln base
    assert L.ddtree_rope_frequencies(64, 1e4, 0, 1, 0, 0, 0, None, ctypes.byref(s)) == 1


def test_turns_are_fractions_of_a_turn():
    values = [1.0, 1e-7, 2 * math.pi * 3, -0.25, 0.0, 123456.789]
    f = (ctypes.c_double * len(values))(*values)
    out = (ctypes.c_uint64 * len(values))()
    assert L.ddtree_rope_turns(f, len(values), out) == 0
    for v, t in zip(values, out):
        want = (v / (2 * math.pi)) % 1.0
        d = abs(t / 2.0 ** 64 - want)
        assert min(d, 1 - d) <= 2.0 ** -52 * max(1.0, abs(v))
    assert out[4] == 0
    f[2] = float("inf")
    assert L.ddtree_rope_turns(f, len(values), out) == 1
    assert L.ddtree_rope_turns(f, 0, out) == 1


def _rows(data=0x10000, heads=2, ts=256, hs=128):
    return struct.pack("@Piqq", data, heads, ts, hs)  # ddtree_rows


def _cache(**kw):
    d = dict(k_pages=0x10000, v_pages=0x20000, dtype=0, num_pages=9, page_size=16, Hkv=2, D=128,
             page_stride=4096, head_stride=2048, slot_stride=128, page_table=0x30000, max_pages=4,
             table_stride=4)
    d.update(kw)
    return ops._pack_cache(*d.values())


def _rot(turns=0x40000, rot_dim=128, scale=1.0):
    return ops._pack_rotary(turns, rot_dim, 0, scale)


OK = P(0x50000)
ODD = P(0x50002)


def _rope(q=None, qo=None, k=None, ko=None, dtype=0, T=4, D=128, pos=OK, rot=None, inverse=0):
    q = _rows() if q is None else q
    return L.ddtree_rope(q, q if qo is None else qo, k, ko, dtype, T, D, pos,
                         _rot() if rot is None else rot, inverse, None)


def test_rope_refusals():
    assert L.ddtree_rope(None, _rows(), None, None, 0, 4, 128, OK, _rot(), 0, None) == 1
    assert L.ddtree_rope(_rows(), None, None, None, 0, 4, 128, OK, _rot(), 0, None) == 1
    assert L.ddtree_rope(_rows(), _rows(), None, None, 0, 4, 128, OK, None, 0, None) == 1
    assert _rope(pos=None) == 1
    assert _rope(pos=ODD) == 1
    assert _rope(dtype=3) == 1
    assert _rope(T=-1) == 1
    assert _rope(D=513) == 2
    assert _rope(inverse=2) == 1
    assert _rope(rot=_rot(rot_dim=130)) == 1      # more than D
    assert _rope(rot=_rot(rot_dim=7)) == 1
    assert _rope(rot=_rot(turns=0x40004)) == 1
    assert _rope(rot=_rot(scale=float("nan"))) == 1
    assert _rope(q=_rows(data=0x10001)) == 1
    assert _rope(q=_rows(heads=0)) == 1
    assert _rope(qo=_rows(heads=3, data=0x90000)) == 1
    assert _rope(qo=_rows(data=0x90000, hs=64)) == 1    # written rows overlap
    assert _rope(qo=_rows(ts=512)) == 1                 # in place, other strides
    assert _rope(q=_rows(heads=70000), qo=_rows(heads=70000)) == 2
    assert _rope(k=_rows()) == 1                        # k without k_out
    assert _rope(ko=_rows()) == 1
    assert _rope(dtype=1, q=_rows(data=0x10002)) == 1   # off the 4-byte grid
    far, other = _rows(data=0x90000), _rows(data=0xa0000)
    assert _rope(k=_rows(), ko=_rows()) == 1            # one tensor turned twice in place
    assert _rope(qo=far, k=far, ko=other) == 1          # q_out is k
    assert _rope(qo=other, k=far, ko=_rows()) == 1      # k_out is q
    assert _rope(qo=other, k=far, ko=other) == 1        # one output for both
    assert _rope(T=0, pos=None) == 0                    # nothing to do


def _append(k=None, v=None, T=4, seq=OK, pos=OK, B=2, cache=None, rot=None, q=None, qo=None):
    return L.ddtree_append_paged(_rows() if k is None else k, _rows() if v is None else v, T, seq,
                                 pos, B, _cache() if cache is None else cache, rot, q, qo, None)


def test_append_refusals():
    assert L.ddtree_append_paged(None, _rows(), 4, OK, OK, 2, _cache(), None, None, None, None) == 1
    assert L.ddtree_append_paged(_rows(), _rows(), 4, OK, OK, 2, None, None, None, None, None) == 1
    assert _append(seq=None) == 1
    assert _append(pos=ODD) == 1
    assert _append(B=0) == 1
    assert _append(T=-1) == 1
    assert _append(k=_rows(heads=3)) == 1               # not the cache's heads
    assert _append(v=_rows(heads=1)) == 1
    assert _append(q=_rows()) == 1                      # q without q_out
    assert _append(qo=_rows()) == 1
    assert _append(rot=_rot(rot_dim=256)) == 1
    assert _append(q=_rows(), qo=_rows()) == 1          # q is k: read while it is turned
    assert _append(v=_rows(data=0x90000), k=_rows(data=0xa0000), q=_rows(),
                   qo=_rows(data=0x90000)) == 1         # q_out is v
    assert _append(k=_rows(data=0x10000), cache=_cache(k_pages=0x10000)) == 1
    assert _append(cache=_cache(D=600, page_stride=60000, head_stride=30000, slot_stride=600)) == 2
    assert _append(T=0, seq=None, pos=None) == 0


@pytest.mark.parametrize("bad", [
    dict(k_pages=0), dict(v_pages=0), dict(page_table=0), dict(dtype=1), dict(dtype=3),
    dict(num_pages=0), dict(page_size=0), dict(Hkv=0), dict(D=0), dict(max_pages=0),
    dict(table_stride=3), dict(page_stride=64), dict(head_stride=-2048), dict(slot_stride=64),
    dict(k_pages=0x10001), dict(page_table=0x30002),
    dict(max_pages=1 << 20, table_stride=1 << 20, page_size=1 << 11),  # 2^31 positions
])
def test_cache_refusals(bad):
    c = _cache(**bad)
    assert _append(cache=c) == 1
    assert _attn(cache=c) == 1
    assert _commit(cache=c) == 1


def _attn(q=None, cache=None, kt=None, vt=None, pl=OK, nn=OK, mask=OK, B=1, N=4, scale=0.1,
          out=P(0x60000), lse=None, ws=P(0x100000), wsb=1 << 30):
    return L.ddtree_tree_attn_paged(
        _rows(heads=8, ts=1024) if q is None else q, _cache() if cache is None else cache,
        _rows() if kt is None else kt, _rows() if vt is None else vt, pl, nn, mask, B, N, scale,
        out, lse, ws, wsb, None)


def test_attention_refusals():
    for name in ("pl", "nn", "mask", "out"):
        assert _attn(**{name: None}) == 1
    for name in ("pl", "nn", "mask", "lse"):
        assert _attn(**{name: ODD}) == 1
    assert _attn(out=P(0x60008)) == 1
    assert _attn(out=P(0x10000)) == 1                      # an input
    assert _attn(q=_rows(heads=7, ts=1024)) == 1           # not a multiple of Hkv
    assert _attn(q=_rows(heads=258, ts=1 << 16)) == 2      # G = 129
    assert _attn(q=_rows(heads=8, ts=1024, data=0x10008)) == 1
    assert _attn(q=_rows(heads=8, ts=1028)) == 1           # strides in 16-byte steps
    assert _attn(kt=_rows(hs=64)) == 1                     # rows overlap
    assert _attn(vt=_rows(heads=1)) == 1
    assert _attn(B=0) == 1
    assert _attn(N=-1) == 1
    assert _attn(N=1025) == 2
    assert _attn(scale=0.0) == 1
    assert _attn(scale=float("inf")) == 1
    for size in (4, 12, 48):                               # not a power of two >= 8
        assert _attn(cache=_cache(page_size=size)) == 2
    c = dict(D=96, page_stride=4096, head_stride=2048, slot_stride=96)
    assert _attn(cache=_cache(**c)) == 2
    assert _attn(cache=_cache(k_pages=0x10008)) == 1
    assert _attn(cache=_cache(page_stride=4100)) == 1
    # a batch that merges through the workspace, and too small a one
    wide = _cache(max_pages=4096, table_stride=4096)
    need = ops.workspace_size(ops.OP_TREE_ATTN_PAGED, B=400, N=4, Hq=8, Hkv=2, D=128,
                              cache_cap=4096 * 16)
    assert need > 0
    assert _attn(cache=wide, B=400, wsb=need - 1) == 1
    assert _attn(cache=wide, B=400, ws=None) == 1
    assert _attn(cache=wide, B=400, ws=P(0x100010)) == 1
    assert ops.workspace_size(ops.OP_TREE_ATTN_PAGED, B=1, N=0, Hq=7, Hkv=2, D=128) == 0


def _commit(cache=None, kt=None, vt=None, al=OK, an=OK, pl=OK, nl=P(0x70000), B=1, Lp=4, N=8):
    return L.ddtree_commit_paged(_cache() if cache is None else cache,
                                 _rows() if kt is None else kt, _rows() if vt is None else vt, al,
                                 an, pl, nl, B, Lp, N, None)


def test_commit_refusals():
    for name in ("al", "an", "pl"):
        assert _commit(**{name: None}) == 1
        assert _commit(**{name: ODD}) == 1
    assert _commit(nl=ODD) == 1
    for name in ("al", "an", "pl"):                        # new_len is an input
        other = {n: P(0x50000 + 0x100 * i) for i, n in enumerate(("al", "an", "pl"))}
        assert _commit(**other, nl=other[name]) == 1
    assert _commit(B=0) == 1
    assert _commit(Lp=0) == 1
    assert _commit(Lp=17) == 2
    assert _commit(N=1025) == 2
    assert _commit(kt=_rows(heads=1)) == 1
    assert _commit(kt=_rows(data=0x10008)) == 1
    assert _commit(cache=_cache(D=100)) == 2
    assert _commit(cache=_cache(slot_stride=132)) == 1


def test_python_refusals_need_no_gpu():
    import torch
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.PagedCache(x[None], x[None], torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        ops.ddtree_rope(x, None, torch.zeros(4, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="scaling"):
        ops.Rotary(64, scaling="dynamic")
    with pytest.raises(ops.DDTreeError):
        ops.Rotary(63)
    with pytest.raises(ValueError, match="rot_dim / 2"):
        ops.Rotary(64, inv_freq=[1.0])
