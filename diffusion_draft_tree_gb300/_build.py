"""Builds libddtree.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_ddtree.so, the module that hands torch tensors to its paged-cache calls.

Each .cu file compiles to an object in parallel; the objects link into one
shared library with the CUDA runtime linked statically, so the library loads
(and its symbols can be inspected) on a machine without a GPU driver.  The
module (csrc/binding.cpp) compiles beside them against the installed torch.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libddtree.so")
BINDING = os.path.join(PKG, "_ddtree.so")
SOURCES = ["api.cu", "topk.cu", "build.cu", "build_level.cu", "tree_attn.cu", "accept.cu",
           "accept_path.cu", "commit.cu", "rotary.cu", "tree_attn_paged.cu", "tree_attn_left.cu",
           "tree_attn_rows.cu", "norm_rope.cu", "quant.cu", "tree_attn_q8.cu",
           "tree_attn_q8_rows.cu", "tree_attn_q8_left.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libddtree.so")
    return cand


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def abi_key() -> str:
    """What the module's object code depends on besides its sources: it reads torch's
    tensors through inline C++ and is a module of this interpreter."""
    import torch
    return f"{torch.__version__}.{sysconfig.get_config_var('SOABI')}"


def _linked_key() -> str:
    try:
        with open(os.path.join(OUT_DIR, "binding.linked")) as f:
            return f.read()
    except OSError:
        return ""


def _binding_cmd(obj: str, key: str):
    from torch.utils import cpp_extension
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-w", f'-DDDTREE_BUILT_FOR="{key}"', *(f"-I{i}" for i in dict.fromkeys(inc)),
            "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]


def _link_binding(obj: str, key: str):
    from torch.utils import cpp_extension
    mark = os.path.join(OUT_DIR, "binding.linked")
    if os.path.exists(mark):
        os.remove(mark)
    tmp = BINDING + f".{os.getpid()}.tmp"
    dirs = cpp_extension.library_paths()
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-lddtree", "-Wl,-rpath,$ORIGIN",
                        *(f"-L{d}" for d in dirs), "-ltorch_python", "-ltorch_cpu", "-lc10",
                        "-lc10_cuda"], capture_output=True, text=True)
    if r.returncode:
        print(r.stdout + r.stderr)
        raise RuntimeError("link of _ddtree.so failed")
    os.replace(tmp, BINDING)
    with open(mark, "w") as f:
        f.write(key)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(os.path.dirname(PKG), "include", "ddtree.h"))
    nvcc = _nvcc()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o]
            jobs.append(cmd)
    # The module: again where its source, the header, or the torch or interpreter it
    # was built against changed.  There is one module, so the key that it was linked
    # for stands beside it: an older torch's object may be older than the module too.
    key = abi_key()
    bind_obj = os.path.join(OUT_DIR, f"binding.{key}.o")
    bind_src = [os.path.join(CSRC, "binding.cpp"), headers[-1]]
    new_binding = force or _stale(bind_obj, bind_src)
    if new_binding:
        jobs.insert(0, _binding_cmd(bind_obj, key))
    cuda_jobs = len(jobs) - int(new_binding)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode:
                print(" ".join(cmd))
                print(r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {cmd[-3]}")
    if force or cuda_jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            print(r.stdout + r.stderr)
            raise RuntimeError("link of libddtree.so failed")
        os.replace(tmp, LIB)
    if force or _linked_key() != key or _stale(BINDING, [bind_obj]):
        _link_binding(bind_obj, key)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
