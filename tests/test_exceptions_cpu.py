"""No C++ exception leaves a C entry: the host's memory runs out inside a call (an
operator new that throws while it is told to), and the call returns a status."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NEW = r"""
#include <cstdlib>
#include <new>
extern "C" { int ddt_no_memory = 0; }
void* operator new(std::size_t n) {
    if (ddt_no_memory) throw std::bad_alloc();
    if (void* p = std::malloc(n ? n : 1)) return p;
    throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
"""

CALLS = r"""
import ctypes, os, struct
P = ctypes.c_void_p
new = ctypes.CDLL(os.environ["LD_PRELOAD"])
flag = ctypes.c_int.in_dll(new, "ddt_no_memory")
lib = ctypes.CDLL(os.environ["DDT_LIB"])
lib.ddtree_workspace_size.restype = ctypes.c_size_t
lib.ddtree_workspace_size.argtypes = [ctypes.c_int] * 10 + [ctypes.c_int64]
lib.ddtree_last_cuda_error.restype = ctypes.c_char_p
lib.ddtree_tree_attn_paged.argtypes = [P] * 7 + [ctypes.c_int] * 2 + [ctypes.c_float] + [P] * 3 + [ctypes.c_size_t, P]
lib.ddtree_tree_attn.argtypes = [P] * 3 + [ctypes.c_int64] + [P] * 5 + [ctypes.c_int] * 5 + [ctypes.c_float] + [P] * 3 + [ctypes.c_size_t, P]
size = lambda op: lib.ddtree_workspace_size(op, 40, 0, 64, 0, 0, 0, 32, 8, 128, 30000)
x = lambda i: P(0x100000 * (i + 1))
rows = lambda at, heads: struct.pack("@Piqq", at, heads, heads * 128, 128)
cache = struct.pack("@PPiiiiiqqqPiq", 0x10000, 0x20000, 0, 9, 16, 8, 128, 16384, 2048, 128, 0x30000, 1875, 1875)
paged = lambda: lib.ddtree_tree_attn_paged(rows(0x40000, 32), cache, rows(0x50000, 8), rows(0x60000, 8), x(1), x(2),
                                           x(3), 40, 64, 0.1, x(4), None, None, 0, None)
dense = lambda: lib.ddtree_tree_attn(x(0), x(1), x(2), 30000, x(3), x(4), x(5), x(6), x(7), 40, 64, 32, 8, 128, 0.1,
                                     x(8), None, None, 0, None)
flag.value = 1
got = [size(2), size(4), paged(), lib.ddtree_last_cuda_error(), dense()]
flag.value = 0
after = [size(2) > 0, size(4) > 0, paged(), dense()]
print(got, after)
"""


def test_running_out_of_memory_is_a_status(tmp_path):
    import __graft_entry__
    lib = __graft_entry__.build_library()
    (tmp_path / "new.cpp").write_text(NEW)
    so = str(tmp_path / "new.so")
    r = subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-o", so, str(tmp_path / "new.cpp")],
                       capture_output=True, text=True)
    if r.returncode:
        pytest.skip("no C++ compiler: " + r.stderr[:200])
    env = dict(os.environ, LD_PRELOAD=so, DDT_LIB=lib)
    r = subprocess.run([sys.executable, "-c", CALLS], capture_output=True, text=True, env=env, cwd=ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    # without memory: no size, a CUDA error that says so; with it again: sizes, and
    # the refusal of a call without a workspace
    assert r.stdout.strip() == "[0, 0, 3, b'cudaErrorMemoryAllocation', 3] [True, True, 1, 1]"
