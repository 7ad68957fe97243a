"""Cases of the paged-cache operators: rotary positions, the append to a paged
KV cache, the commit of an accepted path, and tree attention over the pages.

A serving round over a paged cache uses them in this order, per layer: the
projections' queries and keys are rotated (`rope`, or on the way into the cache
with `append`), every drafted node attends to the pages of its sequence and to
its own root path (`attn`), and after the walk the accepted path joins the
pages (`commit`).  A cache is a pool of pages [page][KV head][slot][D] (or
[page][slot][KV head][D], seen through strides) and a table of page numbers per
sequence; entries behind a sequence's last page are -1.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BASE = 1e6  # base of the rotary frequencies


# ------------------------------------------------------------------- cases

def _rope(name, T, pad, hq, hkv, d, rot, pairs, scaling, factor, dtype, top, inverse=False,
          fused=False):
    return {"name": name, "op": "rope", "T": T, "pad": pad, "hq": hq, "hkv": hkv, "d": d,
            "rot": rot, "pairs": pairs, "scaling": scaling, "factor": factor, "dtype": dtype,
            "top": top, "inverse": inverse, "fused": fused}


def _append(name, B, new_lo, new_hi, at_lo, at_hi, pad, hq, hkv, d, rot, pairs, scaling, factor,
            dtype, page, fused=False, slots_first=False):
    return {"name": name, "op": "append", "B": B, "lo": new_lo, "hi": new_hi, "at_lo": at_lo,
            "at_hi": at_hi, "pad": pad, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "pairs": pairs,
            "scaling": scaling, "factor": factor, "dtype": dtype, "page": page, "fused": fused,
            "slots_first": slots_first}


def _commit(name, B, N, L, at_lo, at_hi, hkv, d, dtype, page, slots_first=False):
    return {"name": name, "op": "commit", "B": B, "N": N, "L": L, "lo": at_lo, "hi": at_hi,
            "hkv": hkv, "d": d, "dtype": dtype, "page": page, "slots_first": slots_first}


def _attn(name, B, N, lo, hi, hq, hkv, d, dtype, page, slots_first=False, fused=False):
    return {"name": name, "op": "attn", "B": B, "N": N, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "dtype": dtype, "page": page, "slots_first": slots_first, "fused": fused}


def listed():
    return [
        # the 65 rows of an 8B-class draft tree behind a 2K prefix: the smallest step, latency
        _rope("rope_tree_8b", 65, 0, 32, 8, 128, 128, "half", "none", 1.0, "bf16", 2112),
        # a long prompt's chunk, 70B-class heads, taken out of one fused projection
        _rope("rope_prompt_yarn", 8192, 17, 64, 8, 128, 128, "half", "yarn", 4.0, "fp16", 131072,
              fused=True),
        # the gradient of a rotation of half the head, in 32 bits, an odd number of tokens
        _rope("rope_grad_partial", 4099, 0, 32, 8, 128, 64, "interleaved", "banded", 8.0, "fp32",
              65536, inverse=True),
        # one token each of a serving batch, queries rotated in the same call
        _append("append_step", 16, 1, 1, 256, 4096, 0, 32, 8, 128, 128, "half", "none", 1.0,
                "bf16", 16),
        # ragged prompts of a batch, behind shared-prefix lengths, padded to a fixed shape
        _append("append_prompts", 8, 517, 4001, 0, 4096, 129, 32, 8, 128, 128, "interleaved",
                "linear", 4.0, "fp16", 64, fused=True, slots_first=True),
        # the accepted path of one 8B-class tree
        _commit("commit_8b_single", 1, 64, 16, 2048, 2048, 8, 128, "bf16", 16),
        # accepted paths of a large serving batch
        _commit("commit_serving", 128, 128, 16, 100, 1000, 8, 128, "bf16", 64),
        # one layer of the 8B-class single stream's verification
        _attn("tree_8b_single", 1, 64, 2048, 2048, 32, 8, 128, "bf16", 16),
        # ragged serving: 16 sequences of 1K to 32K, 128 drafted nodes each
        _attn("tree_ragged_serving", 16, 128, 1024, 32768, 32, 8, 128, "bf16", 64),
        # 70B-class long context, 256 drafted nodes: the largest
        _attn("tree_long_context_70b", 4, 256, 131072, 131072, 64, 8, 128, "bf16", 128),
        # plain decoding of a batch: the bonus token alone, one row a sequence
        _attn("decode_batch", 64, 0, 512, 16384, 32, 8, 128, "bf16", 16),
        # small trees, seven queries a KV head, an empty prefix among them, the other layout
        _attn("tree_small_odd", 7, 21, 0, 5003, 28, 4, 64, "fp16", 32, slots_first=True,
              fused=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "commit", "attn", "attn", "attn"])
    hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    first = rng.random() < 0.4
    fused = rng.random() < 0.4
    dtype = rng.choice(["bf16", "fp16"])
    pairs = rng.choice(["half", "interleaved"])
    scaling, factor = rng.choice([("none", 1.0), ("linear", 4.0), ("ntk", 3.0), ("banded", 8.0),
                                  ("yarn", 16.0)])
    rot = rng.choice([d, d, d // 2, d // 4])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2])
        c = _rope("", _spread(rng, 1, 8192), rng.choice([0, 0, 3]), hkv * g, hkv, d, rot, pairs,
                  scaling, factor, rng.choice(["bf16", "fp16", "fp32"]), _spread(rng, 16, 1000000),
                  rng.random() < 0.3, fused)
    elif op == "append":
        hi = _spread(rng, 1, 2048)
        at = _spread(rng, 1, 16384)
        c = _append("", _spread(rng, 1, 32), rng.randint(0, hi), hi, rng.randint(0, at), at,
                    rng.choice([0, 0, 5]), hkv * g, hkv, d, rot, pairs, scaling, factor, dtype,
                    page, fused, first)
    elif op == "commit":
        N = _spread(rng, 1, 512)
        hi = _spread(rng, 1, 8192)
        c = _commit("", _spread(rng, 1, 128), N, rng.randint(1, 16), rng.randint(0, hi), hi, hkv,
                    d, dtype, page, first)
    else:
        N = 0 if rng.random() < 0.35 else _spread(rng, 1, 512)
        hi = _spread(rng, 1, 65536)
        B = max(1, min(_spread(rng, 1, 96), 300000 // hi))
        N = min(N, int(1e12 / (4 * B * (hi + N) * hkv * g * d)))
        c = _attn("", B, N, rng.randint(0, hi), hi, hkv * g, hkv, d, dtype, page, first, fused)
    del c["name"]
    return c


def _lens(lo, hi, B):
    """Lengths of a ragged batch, evenly from lo to hi."""
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _live(case):
    """Nodes of each sequence's tree: one in five falls short of the budget."""
    return [case["N"] // 2 if i % 5 == 3 else case["N"] for i in range(case["B"])]


def work(case):
    op, es, d = case["op"], SIZE[case["dtype"]], case["d"]
    if op == "rope":
        T = case["T"] + case["pad"]
        heads = case["hq"] + case["hkv"]
        return {"bytes": 2 * T * heads * d * es + 4 * T + 4 * case["rot"],
                "flops": 3 * case["T"] * heads * case["rot"]}
    if op == "append":
        live = sum(_lens(case["lo"], case["hi"], case["B"]))
        T = live + case["pad"]
        row = d * es
        return {"bytes": 2 * row * (T * case["hq"] + 2 * live * case["hkv"]) + 8 * T,
                "flops": 3 * live * (case["hq"] + case["hkv"]) * case["rot"]}
    if op == "commit":
        rows = sum(1 + min(a, case["N"]) for a in _lens(0, case["L"], case["B"]))
        return {"bytes": 4 * rows * case["hkv"] * d * es + 12 * case["B"] + 4 * rows, "flops": 0}
    P, n = _lens(case["lo"], case["hi"], case["B"]), _live(case)
    R, hq, hkv = case["N"] + 1, case["hq"], case["hkv"]
    rows = sum(x + 1 for x in n)
    return {"bytes": (2 * hkv * d * es) * (sum(P) + rows) + 2 * rows * hq * d * es
            + (case["B"] * R - rows) * hq * d * es + case["B"] * R * (hq * 4 + (R + 31) // 32 * 4),
            "flops": 4 * hq * d * sum((x + 1) * (p + 1) for x, p in zip(n, P))}


# ------------------------------------------------------------------ inputs

def _frequencies(case):
    """Angles per position of each pair, and the factor on cosine and sine, in 64 bits."""
    rot, factor, kind = case["rot"], case["factor"], case["scaling"]
    orig, low, high = 8192.0, 1.0, 32.0 if kind == "yarn" else 4.0
    base = BASE * factor ** (rot / (rot - 2)) if kind == "ntk" else BASE
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if kind == "linear":
        f = f / factor
    elif kind == "banded":
        turns = orig * f / (2 * math.pi)
        s = ((turns - low) / (high - low)).clamp(0, 1)
        f = (1 - s) * f / factor + s * f
    elif kind == "yarn":
        def dim(beta):
            return rot * math.log(orig / (2 * math.pi * beta)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
        s = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = (1 - s) * f + s * f / factor
    return f, 0.1 * math.log(factor) + 1.0 if kind == "yarn" and factor > 1 else 1.0


def _rotary(case):
    """The framework's handle for the same rotation."""
    from diffusion_draft_tree_gb300 import ops
    return ops.Rotary(case["rot"], base=BASE, interleaved=case["pairs"] == "interleaved",
                      scaling=case["scaling"], factor=case["factor"], orig_len=8192, low=1.0,
                      high=32.0 if case["scaling"] == "yarn" else 4.0, device="cuda")


def _randn(gen, *shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _heads(case, gen, T):
    """Queries, keys and values of T tokens: slices of one projection, or three tensors."""
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], DT[case["dtype"]]
    if case["fused"]:
        x = _randn(gen, T, hq + 2 * hkv, d, dtype=dt)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return (_randn(gen, T, hq, d, dtype=dt), _randn(gen, T, hkv, d, dtype=dt),
            _randn(gen, T, hkv, d, dtype=dt))


def _shuffled(gen, values):
    x = torch.tensor(values, dtype=torch.int32, device="cuda")
    return x[torch.randperm(len(values), generator=gen, device="cuda")]


def _pool(case, gen, longest, B):
    """A pool with every sequence's pages in random places, and their table."""
    page, hkv, d, dt = case["page"], case["hkv"], case["d"], DT[case["dtype"]]
    need = (longest.long() + page - 1) // page
    width = max(1, -(-case_reach(case) // page))
    total = B * width + 3
    where = torch.randperm(total, generator=gen, device="cuda")[:B * width].int().view(B, width)
    live = torch.arange(width, device="cuda")[None] < need[:, None]
    table = torch.where(live, where, torch.full_like(where, -1))
    if case["slots_first"]:
        k = _randn(gen, total, page, hkv, d, dtype=dt).transpose(1, 2)
        v = _randn(gen, total, page, hkv, d, dtype=dt).transpose(1, 2)
    else:
        k = _randn(gen, total, hkv, page, d, dtype=dt)
        v = _randn(gen, total, hkv, page, d, dtype=dt)
    return k, v, table


def case_reach(case):
    """Positions that a case's longest sequence may come to hold."""
    if case["op"] == "append":
        return case["at_hi"] + case["hi"]
    return case["hi"] + (case["L"] + 1 if case["op"] == "commit" else 0)


def _tree(case, gen, n):
    """Ancestor masks (bit a of row u: a is u or above it) of random trees of n nodes."""
    B, R = case["B"], case["N"] + 1
    W = (R + 31) // 32
    u = torch.arange(R, device="cuda")
    parent = (torch.rand(B, R, generator=gen, device="cuda") * u).long().clamp_(min=0)
    up = torch.zeros(B, R, R, device="cuda", dtype=torch.float64)
    up.scatter_(2, parent[..., None], 1.0)
    up[:, 0] = 0
    up += torch.eye(R, device="cuda", dtype=torch.float64)
    above = torch.linalg.matrix_power(up, 64) > 0  # no path here is longer than 64
    above &= (u[None] <= n[:, None])[..., None]
    bits = torch.zeros(B, R, W * 32, device="cuda", dtype=torch.int64)
    bits[..., :R] = above
    words = (bits.view(B, R, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    return words.to(torch.int32)  # (the low 32 bits)


def _paths(case, gen):
    """Accepted paths: ascending nodes, -1 behind the last; the lengths of a batch."""
    B, N, L = case["B"], case["N"], case["L"]
    alen = _shuffled(gen, [min(a, N) for a in _lens(0, L, B)])
    order = torch.rand(B, max(N, L), generator=gen, device="cuda")
    order[:, N:] = 2.0
    pick = order.argsort(1)[:, :L].int() + 1
    keep = torch.arange(L, device="cuda")[None] < alen[:, None]
    big = torch.full_like(pick, N + 2)
    nodes = torch.where(keep, pick, big).sort(1).values
    return alen, torch.where(keep, nodes, torch.full_like(nodes, -1))


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "rope":
        T, pad = case["T"], case["pad"]
        s["q"], s["k"], _ = _heads(case, gen, T + pad)
        at = torch.randint(0, case["top"], (T + pad,), generator=gen, device="cuda").int()
        at[T:] = -1
        s["pos"] = at
        s["q_out"], s["k_out"] = (torch.zeros(x.shape, dtype=x.dtype, device="cuda")
                                  for x in (s["q"], s["k"]))
        return s
    B = case["B"]
    if op == "append":
        new = _shuffled(gen, _lens(case["lo"], case["hi"], B)).long()
        at = _shuffled(gen, _lens(case["at_lo"], case["at_hi"], B)).long()
        live = sum(_lens(case["lo"], case["hi"], B))
        T = live + case["pad"]
        s["q"], s["k"], s["v"] = _heads(case, gen, T)
        s["k_pages"], s["v_pages"], s["table"] = _pool(case, gen, at + new, B)
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), new, output_size=live)
        first = new.cumsum(0) - new
        pos = torch.arange(live, device="cuda") - first[seq] + at[seq]
        s["seq"] = torch.zeros(T, dtype=torch.int32, device="cuda")
        s["pos"] = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        s["seq"][:live], s["pos"][:live] = seq.int(), pos.int()
        s["live"] = live
        s["q_out"] = torch.zeros(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        return s
    P = _shuffled(gen, _lens(case["lo"], case["hi"], B))
    hkv, d, dt = case["hkv"], case["d"], DT[case["dtype"]]
    s["prefix"] = P
    if op == "commit":
        s["alen"], s["nodes"] = _paths(case, gen)
        s["k_pages"], s["v_pages"], s["table"] = _pool(case, gen, P + s["alen"] + 1, B)
        s["k_tree"] = _randn(gen, B, case["N"] + 1, hkv, d, dtype=dt)
        s["v_tree"] = _randn(gen, B, case["N"] + 1, hkv, d, dtype=dt)
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    R, hq = case["N"] + 1, case["hq"]
    s["k_pages"], s["v_pages"], s["table"] = _pool(case, gen, P, B)
    q, k, v = _heads(case, gen, B * R)
    s["q"], s["k_tree"], s["v_tree"] = (x.unflatten(0, (B, R)) for x in (q, k, v))
    s["n"] = _shuffled(gen, _live(case))
    s["mask"] = _tree(case, gen, s["n"])
    s["out"] = torch.zeros(B, R, hq, d, dtype=dt, device="cuda")
    s["lse"] = torch.zeros(B, R, hq, dtype=torch.float32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("rope", "append"):
        f, s["scale"] = _frequencies(case)
        s["freq"] = f.cuda()
    if own:  # the handles that a program makes once: the rotation, the cache, a workspace
        from diffusion_draft_tree_gb300 import ops
        if case["op"] in ("rope", "append"):
            s["rotary"] = _rotary(case)
        if case["op"] != "rope":
            s["cache"] = ops.PagedCache(s["k_pages"], s["v_pages"], s["table"])
        if case["op"] == "attn":
            s["ws"] = ops.paged_attn_workspace(s["q"], s["cache"])
    return s


# --------------------------------------------------------------- one pass

def _rotated(x, s, live):
    """x with its first `live` tokens rotated: products in 32 bits, angles in 64."""
    case = s["case"]
    rot, sign = case["rot"], -1.0 if case.get("inverse") else 1.0
    a = s["pos"][:live].double()[:, None, None] * s["freq"]
    c, n = (a.cos() * s["scale"]).float(), (a.sin() * (s["scale"] * sign)).float()
    y = x[:live, :, :rot].float()
    if case["pairs"] == "half":
        lo, hi = y[..., :rot // 2], y[..., rot // 2:]
        z = torch.cat([lo * c - hi * n, lo * n + hi * c], -1)
    else:
        lo, hi = y[..., 0::2], y[..., 1::2]
        z = torch.stack([lo * c - hi * n, lo * n + hi * c], -1).flatten(-2)
    z = torch.cat([z.to(x.dtype), x[:live, :, rot:]], -1)
    return torch.cat([z, x[live:]], 0)


def _plain_attn(s):
    case, table, page = s["case"], s["table"].long().clamp(min=0), s["case"]["page"]
    B, R, hkv, d = case["B"], case["N"] + 1, case["hkv"], case["d"]
    G, W = case["hq"] // hkv, table.shape[1]
    k = s["k_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, hkv, W * page, d)
    v = s["v_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, hkv, W * page, d)
    k = torch.cat([k, s["k_tree"].permute(0, 2, 1, 3)], 2).float()
    v = torch.cat([v, s["v_tree"].permute(0, 2, 1, 3)], 2).float()
    there = torch.arange(W * page, device="cuda")[None] < s["prefix"][:, None]
    bits = (s["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    seen = torch.cat([there[:, None].expand(B, R, W * page), bits.flatten(-2)[..., :R].bool()], -1)
    rows = torch.arange(R, device="cuda")[None] <= s["n"][:, None]
    seen = seen & rows[..., None]
    v.masked_fill_(~seen.any(1)[:, None, :, None], 0.0)
    q = s["q"].unflatten(2, (hkv, G)).permute(0, 2, 1, 3, 4).float() * d ** -0.5
    x = (q.reshape(B, hkv, R * G, d) @ k.transpose(2, 3)).view(B, hkv, R, G, -1)
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(B, hkv, R * G, -1) @ v).view(B, hkv, R, G, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).flatten(2, 3))
    lse = torch.where(total > 0, m + total.log(), torch.full_like(m, -math.inf))
    s["lse"].copy_(lse.squeeze(-1).permute(0, 2, 1, 3).flatten(2))


def run(s):
    op = s["case"]["op"]
    if own:
        from diffusion_draft_tree_gb300 import ops
        if op == "rope":
            ops.ddtree_rope(s["q"], s["k"], s["pos"], s["rotary"], q_out=s["q_out"],
                            k_out=s["k_out"], inverse=s["case"]["inverse"])
            return [s["q_out"], s["k_out"]]
        if op == "append":
            ops.ddtree_append_paged(s["k"], s["v"], s["seq"], s["pos"], s["cache"], s["rotary"],
                                    q=s["q"], q_out=s["q_out"])
            return [s["k_pages"], s["v_pages"], s["q_out"]]
        if op == "commit":
            ops.ddtree_commit_paged(s["cache"], s["k_tree"], s["v_tree"], s["alen"], s["nodes"],
                                    s["prefix"], s["new_len"])
            return [s["k_pages"], s["v_pages"], s["new_len"]]
        ops.ddtree_tree_attn_paged(s["q"], s["cache"], s["k_tree"], s["v_tree"], s["prefix"],
                                   s["n"], s["mask"], s["out"], s["lse"], workspace=s["ws"])
        return [s["out"], s["lse"]]
    if op == "rope":
        s["q_out"].copy_(_rotated(s["q"], s, s["case"]["T"]))
        s["k_out"].copy_(_rotated(s["k"], s, s["case"]["T"]))
        return [s["q_out"], s["k_out"]]
    if op == "append":
        n, page = s["live"], s["case"]["page"]
        s["q_out"].copy_(_rotated(s["q"], s, n))
        pos = s["pos"][:n].long()
        at = s["table"].long()[s["seq"][:n].long(), pos // page]
        s["k_pages"].transpose(1, 2)[at, pos % page] = _rotated(s["k"], s, n)[:n]
        s["v_pages"].transpose(1, 2)[at, pos % page] = s["v"][:n]
        return [s["k_pages"], s["v_pages"], s["q_out"]]
    if op == "commit":
        B, L, page = s["case"]["B"], s["case"]["L"], s["case"]["page"]
        step = torch.arange(L + 1, device="cuda")[None]
        node = torch.cat([torch.zeros_like(s["nodes"][:, :1]), s["nodes"]], 1).long()
        # a row behind the path repeats the path's root: the same values to the same slot
        keep = step <= s["alen"][:, None]
        node, step = torch.where(keep, node, 0), torch.where(keep, step, 0)
        pos = s["prefix"].long()[:, None] + step
        b = torch.arange(B, device="cuda")[:, None].expand(B, L + 1)
        at = s["table"].long()[b, pos // page]
        s["k_pages"].transpose(1, 2)[at, pos % page] = s["k_tree"][b, node]
        s["v_pages"].transpose(1, 2)[at, pos % page] = s["v_tree"][b, node]
        s["new_len"].copy_(s["prefix"] + s["alen"] + 1)
        return [s["k_pages"], s["v_pages"], s["new_len"]]
    _plain_attn(s)
    return [s["out"], s["lse"]]


# ------------------------------------------------------------- in 64 bits

def _turned(x, pos, case):
    """Rotation by complex numbers, in 64 bits; tokens at a negative position as they are."""
    f, scale = _frequencies(case)
    rot = case["rot"]
    angle = pos.double()[:, None] * f.to(x.device)[None]
    if case.get("inverse"):
        angle = -angle
    w = torch.polar(torch.full_like(angle, scale), angle)[:, None]
    y = x.double()
    if case["pairs"] == "half":
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * w
        head = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * w
        head = torch.view_as_real(z).flatten(-2)
    out = torch.cat([head, y[..., rot:]], -1)
    return torch.where((pos >= 0)[:, None, None], out, y)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        return [_turned(s["q"], s["pos"], case), _turned(s["k"], s["pos"], case)]
    page = case["page"]
    if op == "append":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        turned, n = _turned(s["k"], s["pos"], case), s["live"]
        pos, seq = s["pos"][:n].long(), s["seq"][:n].long()
        at, slot = s["table"][seq, pos // page].long(), pos % page
        for h in range(case["hkv"]):
            k[:, h].index_put_((at, slot), turned[:n, h])
            v[:, h].index_put_((at, slot), s["v"][:n, h].double())
        return [k, v, _turned(s["q"], s["pos"], case)]
    if op == "commit":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        table, P, alen, nodes = (s[x].tolist() for x in ("table", "prefix", "alen", "nodes"))
        for b in range(case["B"]):
            for i, u in enumerate([0] + nodes[b][:alen[b]]):
                at = P[b] + i
                k[table[b][at // page], :, at % page] = s["k_tree"][b, u].double()
                v[table[b][at // page], :, at % page] = s["v_tree"][b, u].double()
        new = torch.tensor([p + a + 1 for p, a in zip(P, alen)], dtype=torch.int32, device="cuda")
        return [k, v, new]
    B, R, hq, hkv, d = case["B"], case["N"] + 1, case["hq"], case["hkv"], case["d"]
    G = hq // hkv
    out = torch.zeros(B, R, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, R, hq), -math.inf, dtype=torch.float64, device="cuda")
    bit = torch.arange(R, device="cuda")
    for b, (P, n) in enumerate(zip(s["prefix"].tolist(), s["n"].tolist())):
        pages = s["table"][b, :-(-P // page)].long()
        sees = (s["mask"][b, :n + 1][:, bit // 32] >> (bit % 32)) & 1  # [n + 1][R]
        hide = (sees == 0)[:, None, :n + 1].expand(n + 1, G, n + 1).reshape((n + 1) * G, n + 1)
        for g in range(hkv):
            k = torch.cat([s["k_pages"][pages, g].reshape(-1, d)[:P], s["k_tree"][b, :n + 1, g]])
            v = torch.cat([s["v_pages"][pages, g].reshape(-1, d)[:P], s["v_tree"][b, :n + 1, g]])
            q = s["q"][b, :n + 1, g * G:(g + 1) * G].reshape(-1, d).double()
            x = (q @ k.double().T) / math.sqrt(d)
            x[:, P:] = x[:, P:].masked_fill(hide, -math.inf)
            z = torch.logsumexp(x, 1)
            o = (x - z[:, None]).exp_() @ v.double()
            out[b, :n + 1, g * G:(g + 1) * G] = o.view(n + 1, G, d)
            lse[b, :n + 1, g * G:(g + 1) * G] = z.view(n + 1, G)
    return [out, lse]
