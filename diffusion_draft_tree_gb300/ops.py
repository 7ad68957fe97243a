"""Python binding of libddtree.so (include/ddtree.h): argument marshalling only.

Every function here takes torch CUDA tensors, checks dtypes/shapes/devices,
passes raw device pointers and the current CUDA stream to the C ABI, and turns
a non-OK status into an exception.  All arithmetic runs in the library's CUDA
kernels; there is no CPU path.  If the library has not been built, importing
this module raises instead of falling back.

Names and argument order follow the C ABI: ddtree_topk, ddtree_build,
ddtree_tree_attn, ddtree_accept (one DDTree round, "Accelerating Speculative
Decoding with Block Diffusion Draft Trees" §3-§4.3), plus helpers that allocate
the outputs with torch.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libddtree.so")

BF16, FP32, FP16 = 0, 1, 2
OP_TOPK, OP_TREE_ATTN, OP_ACCEPT, OP_TREE_ATTN_PAGED, OP_TREE_ATTN_Q8 = 0, 2, 3, 4, 5
MAX_K, MAX_L, MAX_N = 32, 16, 1024

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "CUDA error",
          4: "kernel recorded bad device data or a timeout"}


# Structs of include/ddtree.h, packed with the platform's own alignment.
_pack_cache = struct.Struct("@PPiiiiiqqqPiq").pack    # ddtree_paged_cache
_pack_rotary = struct.Struct("@Piif4x").pack          # ddtree_rotary
_pack_norm = struct.Struct("@PPf4x").pack             # ddtree_head_norm
_pack_q8 = struct.Struct("@PPPPiiiiiiqqqPi4xq").pack  # ddtree_q8_cache


class DDTreeError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: int = 0):
        msg = f"{fn}: {STATUS.get(status, status)}"
        if status == 3:
            msg += f" ({lib.ddtree_last_cuda_error().decode()})"
        if detail:
            msg += f" (detail 0x{detail:08x})"
        super().__init__(msg)
        self.status = status
        self.detail = detail


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                                 ctypes.c_float, ctypes.c_size_t)
    lib.ddtree_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, i64]
    lib.ddtree_workspace_size.restype = sz
    lib.ddtree_topk.argtypes = [P, i32, i32, i32, i64, i32, P, P, P, P, sz, P]
    lib.ddtree_build.argtypes = [P, P, P, P, i32, i32, i32, i32] + [P] * 9 + [P]
    lib.ddtree_build_heap.argtypes = lib.ddtree_build.argtypes
    lib.ddtree_tree_attn.argtypes = [P, P, P, i64, P, P, P, P, P, i32, i32, i32, i32, i32, f32,
                                     P, P, P, sz, P]
    lib.ddtree_accept.argtypes = [P, i32, i64, P, P, P, i32, i32, i32, i32, f32, u64, u64, P, P,
                                  P, P, P, P, sz, P]
    lib.ddtree_commit.argtypes = [P, P, i64, P, P, P, P, P, i32, i32, i32, i32, i32, P]
    lib.ddtree_accept_path.argtypes = [P, i32, i64, P, P, P, i32, i32, i32, i32, f32, u64, u64,
                                       P, P, P, P, P, P]
    lib.ddtree_topk_noalloc.argtypes = [P, i32, i32, i32, i64, i32, P, P, P, P]
    rows = cache = rotary = P  # packed bytes
    f64 = ctypes.c_double
    lib.ddtree_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64,
                                            ctypes.POINTER(f64), ctypes.POINTER(f32)]
    lib.ddtree_rope_turns.argtypes = [ctypes.POINTER(f64), i32, ctypes.POINTER(u64)]
    lib.ddtree_rope.argtypes = [rows, rows, rows, rows, i32, i32, i32, P, rotary, i32, P]
    lib.ddtree_append_paged.argtypes = [rows, rows, i32, P, P, i32, cache, rotary, rows, rows, P]
    lib.ddtree_tree_attn_paged.argtypes = [rows, cache, rows, rows, P, P, P, i32, i32, f32, P, P,
                                           P, sz, P]
    lib.ddtree_commit_paged.argtypes = [cache, rows, rows, P, P, P, P, i32, i32, i32, P]
    q8 = norm = P
    lib.ddtree_norm_rope.argtypes = [rows, rows, rows, rows, i32, i32, i32, P, norm, rotary, P]
    lib.ddtree_append_q8.argtypes = [rows, rows, i32, P, P, i32, q8, rotary, norm, rows, rows, P]
    lib.ddtree_commit_q8.argtypes = [q8, rows, rows, P, P, P, P, i32, i32, i32, P]
    lib.ddtree_read_q8.argtypes = [q8, P, P, i32, rows, rows, i32, P]
    lib.ddtree_tree_attn_q8.argtypes = lib.ddtree_tree_attn_paged.argtypes
    lib.ddtree_device_check.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    lib.ddtree_selftest_wait.argtypes = [ctypes.c_uint32, P]
    lib.ddtree_last_cuda_error.argtypes = []
    lib.ddtree_last_cuda_error.restype = ctypes.c_char_p
    lib.ddtree_status_str.argtypes = [i32]
    lib.ddtree_status_str.restype = ctypes.c_char_p
    for f in ("ddtree_topk", "ddtree_build", "ddtree_build_heap", "ddtree_tree_attn",
              "ddtree_accept", "ddtree_accept_path", "ddtree_commit", "ddtree_topk_noalloc",
              "ddtree_device_check", "ddtree_selftest_wait", "ddtree_rope_frequencies",
              "ddtree_rope_turns", "ddtree_rope", "ddtree_append_paged",
              "ddtree_tree_attn_paged", "ddtree_commit_paged", "ddtree_norm_rope",
              "ddtree_append_q8", "ddtree_commit_q8", "ddtree_read_q8", "ddtree_tree_attn_q8"):
        getattr(lib, f).restype = i32
    return lib


lib = _load()

from . import _build, _ddtree  # noqa: E402  (built beside libddtree.so, which it uses)

if getattr(_ddtree, "built_for", None) != _build.abi_key():
    # (it reads torch's tensors through their C++ layout)
    raise ImportError(f"{_ddtree.__file__} was built for another torch or interpreter than "
                      f"{_build.abi_key()}: build it again with "
                      "`python -c 'import __graft_entry__ as g; g.build()'`")

EXPORTED = ("ddtree_workspace_size", "ddtree_topk", "ddtree_build", "ddtree_build_heap",
            "ddtree_tree_attn", "ddtree_accept", "ddtree_device_check", "ddtree_last_cuda_error",
            "ddtree_status_str", "ddtree_rope", "ddtree_append_paged", "ddtree_tree_attn_paged",
            "ddtree_commit_paged", "ddtree_norm_rope", "ddtree_append_q8", "ddtree_commit_q8",
            "ddtree_read_q8", "ddtree_tree_attn_q8")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("ddtree kernels take CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("ddtree kernels take contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, status: int):
    if status != 0:
        raise DDTreeError(fn, status)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise ValueError(f"logits must be bfloat16 or float32, got {t.dtype}")


def workspace_size(op: int, B=0, L=0, N=0, V=0, K=0, dtype=BF16, Hq=0, Hkv=0, D=0,
                   cache_cap=0) -> int:
    return int(lib.ddtree_workspace_size(op, B, L, N, V, K, dtype, Hq, Hkv, D, cache_cap))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled, 256-byte aligned workspace (torch allocations are)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# --------------------------------------------------------------------------
# raw calls (caller-provided outputs), same names as the C ABI
# --------------------------------------------------------------------------

def ddtree_topk(draft_logits, K, topk_idx, topk_logp, lse=None, workspace=None, stream=None):
    """draft_logits [rows][V] (bf16/fp32) -> topk_idx int32 [rows][K], topk_logp fp32."""
    rows, V = draft_logits.shape[0], draft_logits.shape[-1]
    ws = workspace
    _check("ddtree_topk", lib.ddtree_topk(
        _ptr(draft_logits), _dtype_code(draft_logits), rows, V, V, K, _ptr(topk_idx),
        _ptr(topk_logp), _ptr(lse), _ptr(ws), ws.numel() if ws is not None else 0,
        _stream(stream)))


def ddtree_build(topk_logp, topk_idx, bonus, prefix_len, N, out: dict, stream=None,
                 heap=False):
    """heap=False: the level-synchronous build; heap=True: ddtree_build_heap."""
    B, L, K = topk_logp.shape
    fn = lib.ddtree_build_heap if heap else lib.ddtree_build
    _check("ddtree_build", fn(
        _ptr(topk_logp), _ptr(topk_idx), _ptr(bonus), _ptr(prefix_len), B, L, K, N,
        _ptr(out["parent"]), _ptr(out["depth"]), _ptr(out["rank"]), _ptr(out["token"]),
        _ptr(out["pos_id"]), _ptr(out["score"]), _ptr(out["child_count"]),
        _ptr(out["anc_mask"]), _ptr(out["n_nodes"]), _stream(stream)))


def ddtree_tree_attn(q, k_cache, v_cache, k_tree, v_tree, prefix_len, n_nodes, anc_mask, out,
                     lse=None, scale=None, workspace=None, stream=None):
    B, R, Hq, D = q.shape
    Hkv, cap = k_cache.shape[1], k_cache.shape[2]
    scale = float(scale) if scale is not None else D ** -0.5
    ws = workspace
    _check("ddtree_tree_attn", lib.ddtree_tree_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), cap, _ptr(k_tree), _ptr(v_tree), _ptr(prefix_len),
        _ptr(n_nodes), _ptr(anc_mask), B, R - 1, Hq, Hkv, D, scale, _ptr(out), _ptr(lse),
        _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))


def ddtree_accept(target_logits, parent, token, n_nodes, L, out: dict, temperature=0.0, seed=0,
                  step=0, workspace=None, stream=None):
    B, R, V = target_logits.shape
    ws = workspace
    _check("ddtree_accept", lib.ddtree_accept(
        _ptr(target_logits), _dtype_code(target_logits), V, _ptr(parent), _ptr(token),
        _ptr(n_nodes), B, L, R - 1, V, float(temperature), int(seed), int(step),
        _ptr(out.get("target_token")), _ptr(out["accept_len"]), _ptr(out["accepted_nodes"]),
        _ptr(out["out_tokens"]), _ptr(out["next_bonus"]), _ptr(ws),
        ws.numel() if ws is not None else 0, _stream(stream)))


def ddtree_accept_path(target_logits, parent, token, n_nodes, L, out: dict, temperature=0.0,
                       seed=0, step=0, stream=None):
    """The walk reading only the rows on the accepted path (same outputs as
    ddtree_accept; target_token on the path only)."""
    B, R, V = target_logits.shape
    _check("ddtree_accept_path", lib.ddtree_accept_path(
        _ptr(target_logits), _dtype_code(target_logits), V, _ptr(parent), _ptr(token),
        _ptr(n_nodes), B, L, R - 1, V, float(temperature), int(seed), int(step),
        _ptr(out.get("target_token")), _ptr(out["accept_len"]), _ptr(out["accepted_nodes"]),
        _ptr(out["out_tokens"]), _ptr(out["next_bonus"]), _stream(stream)))


def accept_path(target_logits, tree: dict, L: int, temperature=0.0, seed=0, step=0,
                stream=None) -> dict:
    B, R, V = target_logits.shape
    out = accept_buffers(B, L, R - 1, target_logits.device)
    ddtree_accept_path(target_logits, tree["parent"], tree["token"], tree["n_nodes"], L, out,
                       temperature, seed, step, stream)
    return out


def ddtree_commit(k_cache, v_cache, k_tree, v_tree, accept_len, accepted_nodes, prefix_len,
                  stream=None):
    """Commit the accepted path (root + accepted nodes) to the KV cache in place
    and advance prefix_len in place."""
    B, Hkv, cap, D = k_cache.shape
    R = k_tree.shape[1]
    L = accepted_nodes.shape[1]
    _check("ddtree_commit", lib.ddtree_commit(
        _ptr(k_cache), _ptr(v_cache), cap, _ptr(k_tree), _ptr(v_tree), _ptr(accept_len),
        _ptr(accepted_nodes), _ptr(prefix_len), B, L, R - 1, Hkv, D, _stream(stream)))


def ddtree_selftest_wait(limit_us: int, stream=None):
    """Enqueues a bounded wait that runs out (see include/ddtree.h)."""
    _check("ddtree_selftest_wait", lib.ddtree_selftest_wait(int(limit_us), _stream(stream)))


def ddtree_device_check(stream=None) -> int:
    """Synchronises the stream; raises DDTreeError if a kernel recorded an error."""
    detail = ctypes.c_uint32(0)
    st = lib.ddtree_device_check(_stream(stream), ctypes.byref(detail))
    if st != 0:
        raise DDTreeError("ddtree_device_check", st, detail.value)
    return 0


# --------------------------------------------------------------------------
# allocating helpers
# --------------------------------------------------------------------------

def topk(draft_logits: torch.Tensor, K: int, workspace=None, stream=None):
    """[..., V] logits -> (idx int32 [..., K], logp fp32 [..., K], lse fp32 [...])."""
    lead = draft_logits.shape[:-1]
    x = draft_logits.reshape(-1, draft_logits.shape[-1])
    dev = x.device
    idx = torch.empty((x.shape[0], K), dtype=torch.int32, device=dev)
    lp = torch.empty((x.shape[0], K), dtype=torch.float32, device=dev)
    lse = torch.empty((x.shape[0],), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(workspace_size(OP_TOPK, B=x.shape[0], L=1, V=x.shape[1],
                                                   K=K, dtype=_dtype_code(x)), dev)
    ddtree_topk(x, K, idx, lp, lse, workspace, stream)
    return idx.reshape(*lead, K), lp.reshape(*lead, K), lse.reshape(lead)


def tree_buffers(B: int, N: int, device) -> dict:
    R, W = N + 1, (N + 1 + 31) // 32
    t = {k: torch.empty((B, R), dtype=torch.int32, device=device)
         for k in ("parent", "depth", "rank", "token", "pos_id", "child_count")}
    t["score"] = torch.empty((B, R), dtype=torch.float32, device=device)
    t["anc_mask"] = torch.empty((B, R, W), dtype=torch.int32, device=device)
    t["n_nodes"] = torch.empty((B,), dtype=torch.int32, device=device)
    return t


def build(topk_logp, topk_idx, bonus, prefix_len, N: int, stream=None, heap=False) -> dict:
    B = topk_logp.shape[0]
    t = tree_buffers(B, N, topk_logp.device)
    ddtree_build(topk_logp, topk_idx, bonus, prefix_len, N, t, stream, heap)
    return t


def tree_attn(q, k_cache, v_cache, k_tree, v_tree, prefix_len, n_nodes, anc_mask, scale=None,
              want_lse=True, workspace=None, stream=None):
    B, R, Hq, D = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((B, R, Hq), dtype=torch.float32, device=q.device) if want_lse else None
    if workspace is None:
        workspace = alloc_workspace(workspace_size(OP_TREE_ATTN, B=B, N=R - 1, Hq=Hq,
                                                   Hkv=k_cache.shape[1], D=D,
                                                   cache_cap=k_cache.shape[2]), q.device)
    ddtree_tree_attn(q, k_cache, v_cache, k_tree, v_tree, prefix_len, n_nodes, anc_mask, out, lse,
                     scale, workspace, stream)
    return out, lse


def accept_buffers(B: int, L: int, N: int, device) -> dict:
    return {"target_token": torch.empty((B, N + 1), dtype=torch.int32, device=device),
            "accept_len": torch.empty((B,), dtype=torch.int32, device=device),
            "accepted_nodes": torch.empty((B, L), dtype=torch.int32, device=device),
            "out_tokens": torch.empty((B, L + 1), dtype=torch.int32, device=device),
            "next_bonus": torch.empty((B,), dtype=torch.int32, device=device)}


def accept(target_logits, tree: dict, L: int, temperature=0.0, seed=0, step=0, workspace=None,
           stream=None) -> dict:
    B, R, V = target_logits.shape
    out = accept_buffers(B, L, R - 1, target_logits.device)
    if workspace is None:
        workspace = alloc_workspace(workspace_size(OP_ACCEPT, B=B, N=R - 1, V=V,
                                                   dtype=_dtype_code(target_logits)),
                                    target_logits.device)
    ddtree_accept(target_logits, tree["parent"], tree["token"], tree["n_nodes"], L, out,
                  temperature, seed, step, workspace, stream)
    return out


# --------------------------------------------------------------------------
# the round over a paged cache
# --------------------------------------------------------------------------
# These calls take strided views: slices of a fused projection, either page
# layout, a pool that interleaves keys and values.  Only the last dimension of a
# tensor has to be contiguous.  Everything a call is given has to be on one
# device, which need not be the current one; without `stream` it is enqueued on
# that device's current stream.  No call records a gradient graph: a tensor that
# is written may not require grad (outside torch.no_grad()), and its version goes up;
# the gradient of a rotation is the call with inverse=True.  The module _ddtree
# (csrc/binding.cpp) checks and passes on the tensors.

_CODES = {torch.bfloat16: BF16, torch.float32: FP32, torch.float16: FP16}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "banded": 3, "yarn": 4}


def _raw(name: str, stream: Optional[torch.cuda.Stream], index: int):
    """The stream's handle for _ddtree: None for the device's current stream."""
    if stream is None:
        return None
    if stream.device.index != index:
        raise ValueError(f"{name}: the stream belongs to {stream.device}, the tensors to "
                         f"cuda:{index}")
    return stream.cuda_stream


def _empty(stream: Optional[torch.cuda.Stream], *specs):
    """New tensors (shape, dtype, device) for a call on `stream` whose results the
    caller's current stream reads.  Memory comes back from the allocator in the
    order of the stream that it was taken on: that is the call's."""
    if stream is None:
        return [torch.empty(n, dtype=t, device=d) for n, t, d in specs]
    with torch.cuda.stream(stream):
        new = [torch.empty(n, dtype=t, device=d) for n, t, d in specs]
    for x in new:
        x.record_stream(torch.cuda.current_stream(x.device))
    return new


def _index(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("ddtree kernels take CUDA tensors")
    return t.get_device()


class Rotary:
    """A rotation: which elements are paired, by how much a position turns each
    pair (include/ddtree.h, ddtree_rotary).  Made once, used by every call.

    rot_dim elements of a head are rotated; `interleaved` pairs (2j, 2j+1),
    otherwise (j, j + rot_dim/2).  scaling is "none", "linear", "ntk", "banded" or
    "yarn", with factor, orig_len, low and high as ddtree_rope_frequencies has
    them.  Frequencies of another kind can be given as inv_freq (radians per
    position, rot_dim/2 of them), with their scale on cosine and sine."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, orig_len: float = 0.0,
                 low: float = 1.0, high: float = 4.0, inv_freq=None,
                 scale: Optional[float] = None, device="cuda"):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
        n = max(rot_dim // 2, 1)
        freq, own_scale = (ctypes.c_double * n)(), ctypes.c_float(1.0)
        if inv_freq is None:
            _check("ddtree_rope_frequencies", lib.ddtree_rope_frequencies(
                rot_dim, base, ROPE_SCALINGS[scaling], factor, orig_len, low, high, freq,
                ctypes.byref(own_scale)))
        else:
            values = [float(x) for x in inv_freq]
            if rot_dim < 2 or rot_dim % 2 or len(values) != n:
                raise ValueError(f"inv_freq must hold rot_dim / 2 values, rot_dim even; got "
                                 f"{len(values)} for {rot_dim}")
            freq = (ctypes.c_double * n)(*values)
        turns = (ctypes.c_uint64 * n)()
        _check("ddtree_rope_turns", lib.ddtree_rope_turns(freq, n, turns))
        self.rot_dim, self.interleaved = rot_dim, bool(interleaved)
        self.inv_freq = list(freq)
        self.scale = own_scale.value if scale is None else float(scale)
        signed = [x - (1 << 64) if x >> 63 else x for x in turns]
        self.turns = torch.tensor(signed, dtype=torch.int64).to(device)
        self._index = _index(self.turns)
        self._c = _pack_rotary(self.turns.data_ptr(), rot_dim, int(self.interleaved), self.scale)


class PagedCache:
    """A paged KV cache: k_pages and v_pages [num_pages][Hkv][page_size][D] (bf16 or
    fp16; views with equal strides, e.g. of a [num_pages][page_size][Hkv][D] pool
    transposed) and page_table int32 [B][max_pages].  Holds the tensors, copies
    nothing: pages and table may be changed in place between calls."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor):
        index = _index(k_pages)
        if k_pages.dim() != 4 or k_pages.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("k_pages must be a bf16 or fp16 [num_pages][Hkv][page_size][D] tensor")
        if v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype or \
                v_pages.stride() != k_pages.stride() or v_pages.get_device() != index:
            raise ValueError("v_pages must match k_pages in shape, type, strides and device")
        if k_pages.stride(3) != 1 and k_pages.shape[3] > 1:
            raise ValueError("a page's rows must be contiguous")
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or \
                page_table.get_device() != index or \
                (page_table.stride(1) != 1 and page_table.shape[1] > 1):
            raise ValueError("page_table must be int32 [B][max_pages] with contiguous rows, on the "
                             "pages' device")
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        self.num_pages, self.Hkv, self.page_size, self.D = k_pages.shape
        self.B, self.max_pages = page_table.shape
        self.dtype, self.device, self._index = k_pages.dtype, k_pages.device, index
        if 0 in k_pages.shape or 0 in page_table.shape:
            raise ValueError("a paged cache needs at least one page, head, slot and table entry")
        st = [s if n > 1 else k_pages.shape[3] for n, s in zip(k_pages.shape, k_pages.stride())]
        self._c = _pack_cache(k_pages.data_ptr(), v_pages.data_ptr(), _CODES[self.dtype],
                              self.num_pages, self.page_size, self.Hkv, self.D, *st[:3],
                              page_table.data_ptr(), self.max_pages,
                              page_table.stride(0) if self.B > 1 else self.max_pages)


def ddtree_rope(q, k, pos, rotary: Rotary, q_out=None, k_out=None, inverse=False, stream=None):
    """Rotates q and, unless it is None, k ([tokens][heads][D] or
    [B][nodes][heads][D], bf16 / fp16 / fp32) for pos int32 [tokens] or
    [B][nodes]; in place where no output is given."""
    if not q.is_cuda:
        raise ValueError("ddtree kernels take CUDA tensors")
    st = _ddtree.rope(q, k, pos, rotary._c, rotary._index, q_out, k_out, inverse,
                      _raw("ddtree_rope", stream, rotary._index))
    if st:
        raise DDTreeError("ddtree_rope", st)


def rope(q, k, pos, rotary: Rotary, inverse=False, stream=None):
    """ddtree_rope into new tensors: (q, k) rotated; k may be None."""
    made = _empty(stream, *[(x.shape, x.dtype, x.device) for x in (q, k) if x is not None])
    q_out, k_out = made[0], made[1] if len(made) > 1 else None
    ddtree_rope(q, k, pos, rotary, q_out, k_out, inverse, stream)
    return q_out, k_out


def ddtree_append_paged(k, v, seq, pos, cache: PagedCache, rotary: Optional[Rotary] = None,
                        q=None, q_out=None, stream=None):
    """Writes tokens' k (rotated for pos if a rotary is given) and v to positions
    pos of sequences seq of the cache (int32 [tokens]; a negative pos: not
    written), and rotates their queries q, in place unless q_out is given."""
    turns, where = (None, None) if rotary is None else (rotary._c, rotary._index)
    st = _ddtree.append_paged(cache._c, cache._index, cache.B, k, v, seq, pos, turns, where, q,
                              q_out, _raw("ddtree_append_paged", stream, cache._index), cache.k_pages,
                              cache.v_pages)
    if st:
        raise DDTreeError("ddtree_append_paged", st)


def paged_attn_workspace(q, cache: PagedCache) -> torch.Tensor:
    """A workspace for ddtree_tree_attn_paged of q's sizes over the cache."""
    B, R, Hq, D = q.shape
    with torch.cuda.device(cache._index):
        n = workspace_size(OP_TREE_ATTN_PAGED, B=B, N=R - 1, Hq=Hq, Hkv=cache.Hkv, D=D,
                           cache_cap=cache.max_pages * cache.page_size)
    return alloc_workspace(n, cache.device)


def ddtree_tree_attn_paged(q, cache: PagedCache, k_tree, v_tree, prefix_len, n_nodes, anc_mask,
                           out, lse=None, scale=None, workspace=None, stream=None):
    """q [B][N+1][Hq][D], k_tree / v_tree [B][N+1][Hkv][D], prefix_len and n_nodes
    [B], anc_mask int32 [B][N+1][W] -> out like q (contiguous), lse fp32
    [B][N+1][Hq]."""
    st = _ddtree.tree_attn_paged(cache._c, cache._index, cache.B, q, k_tree, v_tree, prefix_len,
                                 n_nodes, anc_mask, out, lse, scale, workspace,
                                 _raw("ddtree_tree_attn_paged", stream, cache._index))
    if st:
        raise DDTreeError("ddtree_tree_attn_paged", st)


def tree_attn_paged(q, cache: PagedCache, k_tree, v_tree, prefix_len, n_nodes, anc_mask,
                    scale=None, want_lse=True, workspace=None, stream=None):
    B, R, Hq, _ = q.shape
    specs = [(q.shape, q.dtype, q.device), ((B, R, Hq), torch.float32, q.device)]
    made = _empty(stream, *specs[:2 if want_lse else 1])
    out, lse = made[0], made[1] if want_lse else None
    if workspace is None:  # (its zeros have to be on the call's stream)
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            workspace = paged_attn_workspace(q, cache)
    ddtree_tree_attn_paged(q, cache, k_tree, v_tree, prefix_len, n_nodes, anc_mask, out, lse,
                           scale, workspace, stream)
    return out, lse


def ddtree_commit_paged(cache: PagedCache, k_tree, v_tree, accept_len, accepted_nodes, prefix_len,
                        new_len=None, stream=None):
    """Writes the accepted path (root + accepted nodes, as ddtree_accept gives them)
    of k_tree / v_tree [B][N+1][Hkv][D] to positions prefix_len.. of the cache;
    prefix_len stays, new_len [B] receives prefix_len + accept_len + 1."""
    st = _ddtree.commit_paged(cache._c, cache._index, cache.B, k_tree, v_tree, accept_len,
                              accepted_nodes, prefix_len, new_len,
                              _raw("ddtree_commit_paged", stream, cache._index), cache.k_pages,
                              cache.v_pages)
    if st:
        raise DDTreeError("ddtree_commit_paged", st)


# --------------------------------------------------------------------------
# the round over an 8-bit paged cache, and the norm of queries and keys
# --------------------------------------------------------------------------

class HeadNorm:
    """The norm of every head before its rotation, x / sqrt(mean x^2 + eps) * weight:
    the weights of queries and keys, [D] of any floating type (None: ones), taken
    once, in 32 bits.  `offset` is added to them (models that keep weight - 1)."""

    def __init__(self, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, offset: float = 0.0):
        if not eps > 0:
            raise ValueError(f"eps must be positive, got {eps}")
        self.eps, self._index, self.D = float(eps), -1, -1
        held = []
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is None:
                held.append(None)
                continue
            if w.dim() != 1 or not w.is_floating_point():
                raise ValueError(f"{name} must be a floating [D] tensor")
            at = _index(w)
            if self._index not in (-1, at) or self.D not in (-1, w.shape[0]):
                raise ValueError("q_weight and k_weight must agree in size and device")
            self._index, self.D = at, w.shape[0]
            held.append((w.detach().float() + offset).contiguous())
        self.q_weight, self.k_weight = held
        self._c = (_pack_norm(*(0 if w is None else w.data_ptr() for w in held), self.eps),
                   self._index, self.D)


class QuantCache:
    """A paged KV cache in 8 bits: k_pages and v_pages float8_e4m3fn codes
    [num_pages][Hkv][page_size][D] (views with equal strides), k_scales and v_scales
    uint8 [num_pages][Hkv][page_size // block], a byte x for each block of positions:
    a code c stands for c * 2^(x - 127) (include/ddtree.h, ddtree_q8_cache), and
    page_table int32 [B][max_pages].  dtype (bfloat16 or float16) is that of the tokens.
    Holds the tensors, copies nothing."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor, page_table: torch.Tensor, dtype: torch.dtype = torch.bfloat16):
        index = _index(k_pages)
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        if k_pages.dim() != 4 or k_pages.dtype != torch.float8_e4m3fn:
            raise ValueError("k_pages must be a float8_e4m3fn [num_pages][Hkv][page_size][D] tensor")
        if v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype or \
                v_pages.stride() != k_pages.stride() or v_pages.get_device() != index:
            raise ValueError("v_pages must match k_pages in shape, type, strides and device")
        if k_pages.stride(3) != 1 and k_pages.shape[3] > 1:
            raise ValueError("a page's rows must be contiguous")
        if 0 in k_pages.shape or 0 in page_table.shape:
            raise ValueError("a paged cache needs at least one page, head, slot and table entry")
        self.num_pages, self.Hkv, self.page_size, self.D = k_pages.shape
        blocks = k_scales.shape[-1] if k_scales.dim() == 3 else 0
        if blocks == 0 or self.page_size % blocks:
            raise ValueError("k_scales must be [num_pages][Hkv][page_size // block]")
        for name, s in (("k_scales", k_scales), ("v_scales", v_scales)):
            if s.dtype != torch.uint8 or s.shape != (self.num_pages, self.Hkv, blocks) or \
                    not s.is_contiguous() or s.get_device() != index:
                raise ValueError(f"{name} must be a contiguous uint8 tensor "
                                 f"{[self.num_pages, self.Hkv, blocks]} on the pages' device")
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or \
                page_table.get_device() != index or \
                (page_table.stride(1) != 1 and page_table.shape[1] > 1):
            raise ValueError("page_table must be int32 [B][max_pages] with contiguous rows, on the "
                             "pages' device")
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        self.k_scales, self.v_scales, self.block = k_scales, v_scales, self.page_size // blocks
        self.B, self.max_pages = page_table.shape
        self.dtype, self.device, self._index = dtype, k_pages.device, index
        st = [s if n > 1 else self.D for n, s in zip(k_pages.shape, k_pages.stride())]
        self._c = _pack_q8(k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
                           v_scales.data_ptr(), _CODES[dtype], self.num_pages, self.page_size,
                           self.block, self.Hkv, self.D, *st[:3], page_table.data_ptr(),
                           self.max_pages, page_table.stride(0) if self.B > 1 else self.max_pages)

    @classmethod
    def empty(cls, num_pages: int, Hkv: int, page_size: int, D: int, page_table: torch.Tensor,
              block: int = 32, dtype: torch.dtype = torch.bfloat16) -> "QuantCache":
        """New pages of zeros on the table's device, under the type's least scale: a block that
        a run enters in its middle keeps the larger of its old scale and the one it needs."""
        if dtype not in _LEAST_SCALE:
            raise ValueError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        if block < 1 or page_size % block:
            raise ValueError(f"block must divide page_size, got {block} and {page_size}")
        dev = page_table.device
        pages = [torch.zeros(num_pages, Hkv, page_size, D, dtype=torch.uint8, device=dev)
                 .view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.full((num_pages, Hkv, page_size // block), _LEAST_SCALE[dtype],
                             dtype=torch.uint8, device=dev) for _ in range(2)]
        return cls(*pages, *scales, page_table, dtype)


_NO_NORM = (None, -1, -1)
_LEAST_SCALE = {torch.bfloat16: 127 - 96, torch.float16: 127 - 15}


def ddtree_norm_rope(q, k, pos, norm: HeadNorm, rotary: Optional[Rotary] = None, q_out=None,
                     k_out=None, stream=None):
    """Norms every head of q and, unless it is None, k and rotates them for pos, as
    ddtree_rope takes them; in place where no output is given.  A token at a negative
    position is copied as it is."""
    turns, where = (None, None) if rotary is None else (rotary._c, rotary._index)
    st = _ddtree.norm_rope(q, k, pos, *norm._c, turns, where, q_out, k_out,
                           _raw("ddtree_norm_rope", stream, _index(q)))
    if st:
        raise DDTreeError("ddtree_norm_rope", st)


def norm_rope(q, k, pos, norm: HeadNorm, rotary: Optional[Rotary] = None, stream=None):
    """ddtree_norm_rope into new tensors: (q, k); k may be None."""
    made = _empty(stream, *[(x.shape, x.dtype, x.device) for x in (q, k) if x is not None])
    q_out, k_out = made[0], made[1] if len(made) > 1 else None
    ddtree_norm_rope(q, k, pos, norm, rotary, q_out, k_out, stream)
    return q_out, k_out


def ddtree_append_q8(k, v, first, at, cache: QuantCache, rotary: Optional[Rotary] = None,
                     norm: Optional[HeadNorm] = None, q=None, q_out=None, stream=None):
    """Quantises runs of tokens into the cache: tokens first[b] .. first[b + 1] - 1 (first int32
    [B + 1]) become positions at[b].. (int32 [B]) of sequence b, k normed and rotated on the
    way if a norm and a rotary are given, and their queries q likewise, in place unless
    q_out is given.  A NaN among keys or values is recorded for ddtree_device_check."""
    turns, where = (None, None) if rotary is None else (rotary._c, rotary._index)
    st = _ddtree.append_q8(cache._c, cache._index, cache.B, k, v, first, at, turns, where,
                           *(_NO_NORM if norm is None else norm._c), q, q_out,
                           _raw("ddtree_append_q8", stream, cache._index), cache.k_pages,
                           cache.v_pages, cache.k_scales, cache.v_scales)
    if st:
        raise DDTreeError("ddtree_append_q8", st)


def ddtree_commit_q8(cache: QuantCache, k_tree, v_tree, accept_len, accepted_nodes, prefix_len,
                     new_len=None, stream=None):
    """ddtree_commit_paged into an 8-bit cache."""
    st = _ddtree.commit_q8(cache._c, cache._index, cache.B, k_tree, v_tree, accept_len,
                           accepted_nodes, prefix_len, new_len,
                           _raw("ddtree_commit_q8", stream, cache._index), cache.k_pages,
                           cache.v_pages, cache.k_scales, cache.v_scales)
    if st:
        raise DDTreeError("ddtree_commit_q8", st)


def ddtree_read_q8(cache: QuantCache, first, at, k_out, v_out, stream=None):
    """Reads runs of positions back in the tokens' type: position at[b] + i of sequence b
    becomes row first[b] + i of k_out and v_out ([tokens][Hkv][D])."""
    st = _ddtree.read_q8(cache._c, cache._index, cache.B, first, at, k_out, v_out,
                         _raw("ddtree_read_q8", stream, cache._index))
    if st:
        raise DDTreeError("ddtree_read_q8", st)


def q8_attn_workspace(q, cache: QuantCache) -> torch.Tensor:
    """A workspace for ddtree_tree_attn_q8 of q's sizes over the cache."""
    B, R, Hq, D = q.shape
    with torch.cuda.device(cache._index):
        n = workspace_size(OP_TREE_ATTN_Q8, B=B, N=R - 1, Hq=Hq, Hkv=cache.Hkv, D=D,
                           cache_cap=cache.max_pages * cache.page_size)
    return alloc_workspace(n, cache.device)


def ddtree_tree_attn_q8(q, cache: QuantCache, k_tree, v_tree, prefix_len, n_nodes, anc_mask, out,
                        lse=None, scale=None, workspace=None, stream=None):
    """ddtree_tree_attn_paged over an 8-bit cache; q, k_tree, v_tree and out of its dtype."""
    st = _ddtree.tree_attn_q8(cache._c, cache._index, cache.B, q, k_tree, v_tree, prefix_len,
                              n_nodes, anc_mask, out, lse, scale, workspace,
                              _raw("ddtree_tree_attn_q8", stream, cache._index))
    if st:
        raise DDTreeError("ddtree_tree_attn_q8", st)


def tree_attn_q8(q, cache: QuantCache, k_tree, v_tree, prefix_len, n_nodes, anc_mask, scale=None,
                 want_lse=True, workspace=None, stream=None):
    B, R, Hq, _ = q.shape
    specs = [(q.shape, q.dtype, q.device), ((B, R, Hq), torch.float32, q.device)]
    made = _empty(stream, *specs[:2 if want_lse else 1])
    out, lse = made[0], made[1] if want_lse else None
    if workspace is None:  # (its zeros have to be on the call's stream)
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            workspace = q8_attn_workspace(q, cache)
    ddtree_tree_attn_q8(q, cache, k_tree, v_tree, prefix_len, n_nodes, anc_mask, out, lse, scale,
                        workspace, stream)
    return out, lse
