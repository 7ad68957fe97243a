"""Host side of the 8-bit cache's calls and of norm with rotation, no GPU: every refusal of
a bad argument before a launch."""
import ctypes
import struct

import pytest
import torch

from diffusion_draft_tree_gb300 import ops

P = ctypes.c_void_p
L = ops.lib
OK, ODD = P(0x50000), P(0x50002)


def _rows(data=0x10000, heads=2, ts=256, hs=128):
    return struct.pack("@Piqq", data, heads, ts, hs)  # ddtree_rows


def _cache(**kw):
    d = dict(k_pages=0x1000000, v_pages=0x2000000, k_scales=0x3000000, v_scales=0x4000000, dtype=0, num_pages=9,
             page_size=16, block=16, Hkv=2, D=128, page_stride=4096, head_stride=2048, slot_stride=128,
             page_table=0x30000, max_pages=4, table_stride=4)
    d.update(kw)
    return ops._pack_q8(*d.values())


def _rot(turns=0x40000, rot_dim=128, scale=1.0):
    return ops._pack_rotary(turns, rot_dim, 0, scale)


def _norm(q=0x70000, k=0x80000, eps=1e-6):
    return ops._pack_norm(q, k, eps)


def test_the_packed_structs_have_the_sizes_of_the_header():
    assert len(_cache()) == 32 + 6 * 4 + 3 * 8 + 8 + 8 + 8 and len(_norm()) == 24


def _nr(q=None, qo=None, k=None, ko=None, dtype=0, T=4, D=128, pos=OK, norm=0, rot=0):
    q = _rows() if q is None else q
    return L.ddtree_norm_rope(q, q if qo is None else qo, k, ko, dtype, T, D, pos, _norm() if norm == 0 else norm,
                              _rot() if rot == 0 else rot, None)


def test_norm_rope_refusals():
    assert _nr(norm=None) == 1
    assert _nr(norm=_norm(eps=0.0)) == 1 and _nr(norm=_norm(eps=float("nan"))) == 1
    assert _nr(norm=_norm(eps=-1.0)) == 1 and _nr(norm=_norm(eps=float("inf"))) == 1
    assert _nr(norm=_norm(q=0x70002)) == 1 and _nr(norm=_norm(k=0x80001)) == 1
    assert _nr(pos=None) == 1 and _nr(pos=ODD) == 1
    assert _nr(dtype=3) == 1 and _nr(T=-1) == 1 and _nr(D=0) == 1 and _nr(D=513) == 2
    assert _nr(rot=_rot(rot_dim=130)) == 1 and _nr(rot=_rot(rot_dim=7)) == 1
    assert _nr(q=_rows(data=0x10001)) == 1 and _nr(q=_rows(heads=0)) == 1
    assert _nr(qo=_rows(heads=3, data=0x90000)) == 1 and _nr(qo=_rows(ts=512)) == 1
    assert _nr(q=_rows(heads=70000), qo=_rows(heads=70000)) == 2
    assert _nr(k=_rows()) == 1 and _nr(ko=_rows()) == 1
    far, other = _rows(data=0x90000), _rows(data=0xa0000)
    assert _nr(k=_rows(), ko=_rows()) == 1 and _nr(qo=far, k=far, ko=other) == 1
    assert _nr(qo=other, k=far, ko=_rows()) == 1 and _nr(qo=other, k=far, ko=other) == 1
    assert _nr(T=0, pos=None) == 0


def _append(k=None, v=None, T=4, first=OK, at=OK, B=2, cache=0, rot=None, norm=None, q=None, qo=None):
    return L.ddtree_append_q8(_rows() if k is None else k, _rows(data=0x20000) if v is None else v, T, first, at, B,
                              _cache() if cache == 0 else cache, rot, norm, q, qo, None)


def _commit(kt=None, vt=None, alen=OK, nodes=P(0x51000), pl=P(0x52000), new=None, B=1, L_=4, N=8, cache=0):
    return L.ddtree_commit_q8(_cache() if cache == 0 else cache, _rows() if kt is None else kt,
                              _rows() if vt is None else vt, alen, nodes, pl, new, B, L_, N, None)


def _read(first=OK, at=OK, B=2, ko=None, vo=None, T=4, cache=0):
    return L.ddtree_read_q8(_cache() if cache == 0 else cache, first, at, B, _rows() if ko is None else ko,
                            _rows(data=0x20000) if vo is None else vo, T, None)


def _attn(q=None, cache=0, kt=None, vt=None, pl=OK, nn=OK, mask=OK, B=1, N=4, scale=0.1, out=P(0x60000), lse=None,
          ws=P(0x100000), wsb=1 << 30):
    return L.ddtree_tree_attn_q8(_rows(heads=8, ts=1024) if q is None else q, _cache() if cache == 0 else cache,
                                 _rows() if kt is None else kt, _rows() if vt is None else vt, pl, nn, mask, B, N,
                                 scale, out, lse, ws, wsb, None)


@pytest.mark.parametrize("bad", [
    dict(k_pages=0), dict(v_pages=0), dict(k_scales=0), dict(v_scales=0), dict(page_table=0), dict(dtype=1),
    dict(dtype=3), dict(num_pages=0), dict(page_size=0), dict(block=0), dict(Hkv=0), dict(D=0), dict(max_pages=0),
    dict(table_stride=3), dict(page_stride=64), dict(head_stride=-2048), dict(slot_stride=64), dict(slot_stride=136),
    dict(k_pages=0x1000008), dict(v_scales=0x4000004), dict(page_table=0x30002), dict(v_pages=0x1000000),
    dict(v_scales=0x3000000), dict(max_pages=1 << 20, table_stride=1 << 20, page_size=1 << 11)])
def test_cache_refusals(bad):
    c = _cache(**bad)
    assert _append(cache=c) == 1 and _commit(cache=c) == 1 and _read(cache=c) == 1 and _attn(cache=c) == 1


@pytest.mark.parametrize("bad", [dict(D=96), dict(D=256, slot_stride=256), dict(page_size=24, block=8),
                                 dict(page_size=4, block=4), dict(block=4), dict(block=12), dict(block=32),
                                 dict(page_size=128, block=128)])
def test_cache_sizes_that_are_not_taken(bad):
    c = _cache(**bad)
    ts = dict(ts=1024, hs=512)
    assert _append(cache=c, k=_rows(**ts), v=_rows(data=0x20000, **ts)) == 2
    assert _commit(cache=c) == 2 and _read(cache=c) == 2 and _attn(cache=c) == 2


def test_null_caches():
    assert _append(cache=None) == 1 and _commit(cache=None) == 1 and _read(cache=None) == 1 and _attn(cache=None) == 1


def test_append_refusals():
    assert _append(first=None) == 1 and _append(at=None) == 1 and _append(first=ODD) == 1 and _append(at=ODD) == 1
    assert _append(B=0) == 1 and _append(T=-1) == 1
    assert _append(k=_rows(heads=3)) == 1 and _append(v=_rows(heads=1)) == 1
    assert _append(k=_rows(data=0x10008)) == 1 and _append(v=_rows(ts=260)) == 1 and _append(k=_rows(hs=132)) == 1
    assert _append(q=_rows()) == 1 and _append(qo=_rows()) == 1
    assert _append(rot=_rot(rot_dim=256)) == 1 and _append(rot=_rot(rot_dim=24)) == 2
    assert _append(norm=_norm(eps=0.0)) == 1
    assert _append(q=_rows(), qo=_rows()) == 1                            # q is k
    assert _append(q=_rows(data=0x90000), qo=_rows(data=0x20000)) == 1    # q_out is v
    assert _append(q=_rows(data=0x90008), qo=_rows(data=0xa0000)) == 1
    assert _append(T=0, first=None, at=None) == 0


def test_commit_refusals():
    for name in ("alen", "nodes", "pl"):
        assert _commit(**{name: None}) == 1 and _commit(**{name: ODD}) == 1
    assert _commit(new=ODD) == 1 and _commit(new=OK) == 1 and _commit(new=P(0x52000)) == 1
    assert _commit(B=0) == 1 and _commit(B=70000) == 1 and _commit(L_=0) == 1 and _commit(N=-1) == 1
    assert _commit(L_=17) == 2 and _commit(N=1025) == 2
    assert _commit(kt=_rows(heads=3)) == 1 and _commit(vt=_rows(data=0x10008)) == 1


def test_read_refusals():
    assert _read(first=None) == 1 and _read(at=ODD) == 1 and _read(B=0) == 1 and _read(T=-1) == 1
    assert _read(ko=_rows(heads=3)) == 1 and _read(vo=_rows(data=0x20008)) == 1 and _read(ko=_rows(hs=64)) == 1
    assert _read(vo=_rows()) == 1  # one tensor for both
    assert _read(T=0, first=None) == 0


def test_attention_refusals():
    for name in ("pl", "nn", "mask", "out"):
        assert _attn(**{name: None}) == 1
    for name in ("pl", "nn", "mask", "lse"):
        assert _attn(**{name: ODD}) == 1
    assert _attn(out=P(0x60008)) == 1 and _attn(out=P(0x10000)) == 1
    assert _attn(q=_rows(heads=7, ts=1024)) == 1 and _attn(kt=_rows(heads=3)) == 1 and _attn(vt=_rows(ts=64)) == 1
    assert _attn(q=_rows(heads=8, ts=1028)) == 1
    assert _attn(B=0) == 1 and _attn(N=-1) == 1 and _attn(scale=0.0) == 1 and _attn(scale=float("nan")) == 1
    assert _attn(N=1025) == 2 and _attn(q=_rows(heads=258, ts=40000)) == 2
    need = ops.workspace_size(ops.OP_TREE_ATTN_Q8, B=1, N=0, Hq=8, Hkv=2, D=128, cache_cap=64)
    assert need > 0  # (few rows: the pieces of cut units)
    assert _attn(N=0, ws=None) == 1 and _attn(N=0, wsb=need - 1) == 1 and _attn(N=0, ws=P(0x100080)) == 1
    assert ops.workspace_size(ops.OP_TREE_ATTN_Q8, B=0, N=4, Hq=8, Hkv=2, D=128, cache_cap=64) == 0
    assert ops.workspace_size(ops.OP_TREE_ATTN_Q8, B=1, N=4, Hq=7, Hkv=2, D=128, cache_cap=64) == 0


def test_the_kernel_for_few_rows_keeps_its_warps_whole_and_drains_its_copies():
    """The rules of the attention kernels' sources (test_kernel_sources_cpu.py) in the one over an
    8-bit cache."""
    import os
    import re
    at = os.path.join(os.path.dirname(ops.LIB_PATH), "csrc", "tree_attn_q8_rows.cu")
    with open(at) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert text.count("mbar_wait_warp(") >= 3
    for m in re.finditer(r"\bmbar_wait\(", text):
        assert text[:m.start()].rstrip().endswith((";", ")", "{", "}")), text[m.start() - 60:m.end() + 40]
    assert re.search(r"mbar_wait\(&bar_full\[it % NS\],[^;]*nullptr, 100000000ull\);", text)


def test_an_empty_cache_of_another_type_is_refused():
    with pytest.raises(ValueError, match="dtype"):
        ops.QuantCache.empty(3, 2, 16, 64, torch.zeros(1, 1, dtype=torch.int32), dtype=torch.float32)
