"""Rules that the attention kernels' sources keep so that no warp is divided and no
memory is read too early -- mistakes that show on a GPU as a hang or as wrong
values now and then, and so are looked for in the text."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "diffusion_draft_tree_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_that_decide_a_branch_are_the_whole_warps():
    """mbar_wait answers a lane; where its answer decides what a warp does next the
    warp has to vote (mbar_wait_warp), or lanes that saw the abort flag leave
    lanes that saw the barrier alone at the next warp-wide instruction."""
    for name in ("tree_attn.cuh", "tree_attn_rows.cu"):
        text = _source(name)
        assert text.count("mbar_wait_warp(") >= 4
        for m in re.finditer(r"\bmbar_wait\(", text):
            before = text[:m.start()].rstrip()
            # a drain at a role's end: the answer is not used
            assert before.endswith((";", ")", "{", "}")), (name, text[m.start() - 60:m.end() + 40])


def test_copies_and_products_in_flight_are_drained():
    """Every barrier that a copy or a product may still signal when a wait gives up
    is waited for before its role ends."""
    tree, rows = _source("tree_attn.cuh"), _source("tree_attn_rows.cu")
    for bar in ("bar_q", "bar_drain", "v ? &bar_vfull[j % NS] : &bar_kfull[j % NS]"):
        bar = bar if bar.startswith("v ?") else "&" + bar
        assert re.search(r"[;){}]\s*mbar_wait\(" + re.escape(bar) + r",[^;]*nullptr, 100000000ull\);", tree), bar
    for bar in ("&bar_qfull", "&bar_full[it % NS]"):
        assert re.search(r"[;){}]\s*mbar_wait\(" + re.escape(bar) + r",[^;]*nullptr, 100000000ull\);", rows), bar


def test_scratch_under_the_tiles_is_fenced_before_copies():
    """Shared memory that ordinary stores filled and copies fill next: the copies are
    another proxy's, which a CTA barrier alone does not put behind the stores."""
    text = _source("tree_attn.cuh")
    ranked = text[text.index("int3 ranked_item("):text.index("struct LeftArgs")]
    dense = text[text.index("int* s_perm"):text.index("if constexpr (PAGED)", text.index("int* s_perm"))]
    for part in (ranked, dense):
        barriers = [m.start() for m in re.finditer(r"__syncthreads\(\)", part)]
        last_store = max(m.start() for m in re.finditer(r"s_(cost|whole|w|perm)\[[^\]]*\] = ", part))
        fence = part.rindex("fence_proxy_async_smem()")
        assert last_store < fence < barriers[-1]


def test_tensor_memory_loads_are_waited_for_by_name():
    """A load from tensor memory writes its registers asynchronously: between it and
    the wait that names them, nothing but other loads and stores uses them."""
    text = _source("tree_attn.cuh")
    waits = list(re.finditer(r"tmem_ld_wait\(([^)]*)\)", text))
    assert len(waits) > 10 and all(m.group(1).strip() for m in waits)
    loads = list(re.finditer(r"tmem_ld32\([^;]*, (\w+)\);", text))
    assert loads
    for m in loads:
        name = m.group(1)
        behind = next(w for w in waits if w.start() > m.end()
                      and name in [x.strip() for x in w.group(1).split(",")])
        between = text[m.end():behind.start()]
        assert not re.search(r"\b%s\b" % name, between), (name, between)


def test_tables_that_calls_fill_are_safe_for_threads():
    """Function-local tables on the host, filled by the first call that needs an
    entry: two host threads may be that call, and Arm may show one thread the flag
    before the value."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh", ".h")):
            continue
        for m in re.finditer(r"^ +static (?!constexpr|_)([^;=(]*)[;=]", _source(name), re.M):
            kind = m.group(1)
            locked = kind.startswith(("std::once_flag", "std::atomic<", "std::mutex", "std::map<"))
            # (filled inside a call_once)
            assert locked or kind.startswith(("cudaError_t attr_err", "PFN_")), (name, kind)
