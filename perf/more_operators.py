"""Cases of the round over an 8-bit paged cache: the norm and rotation of queries
and keys, the writers that quantise, the reader, and tree attention over it.

A serving round over a quantised cache uses them in this order, per layer: the
projections' queries and keys are normed per head and rotated (`norm`, or on the
way into the cache with `append`), every drafted node attends to the pages of
its sequence and to its own root path (`attn`), and after the walk the accepted
path joins the pages (`commit`).  `read` gives a prefix back in 16 bits, for a cache
of another layout.

The cache holds e4m3 codes, [page][KV head][slot][D] (or [page][slot][KV head][D], seen
through strides), and one byte x for each block of positions of a page and head:
a code c stands for c * 2^(x - 127).  The exponent of a block is the least one at
which its largest element is at most 448; a block that a sequence enters in its
middle keeps at least its old one, and its earlier codes move to the new one.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
LEAST = {"bf16": -96, "fp16": -15}  # exponents of a block, by the type of its tokens
MOST = 7
BASE = 1e6   # base of the rotary frequencies
EPS = 1e-6   # of the norms
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def _norm(name, T, pad, hq, hkv, d, rot, pairs, scaling, factor, dtype, top, fused=False):
    return {"name": name, "op": "norm", "T": T, "pad": pad, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "pairs": pairs, "scaling": scaling, "factor": factor, "dtype": dtype, "top": top,
            "fused": fused}


def _append(name, B, new_lo, new_hi, at_lo, at_hi, pad, hq, hkv, d, rot, pairs, scaling, factor,
            dtype, page, block, normed=True, fused=False, slots_first=False):
    return {"name": name, "op": "append", "B": B, "lo": new_lo, "hi": new_hi, "at_lo": at_lo,
            "at_hi": at_hi, "pad": pad, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "pairs": pairs,
            "scaling": scaling, "factor": factor, "dtype": dtype, "page": page, "block": block,
            "normed": normed, "fused": fused, "slots_first": slots_first}


def _commit(name, B, N, L, at_lo, at_hi, hkv, d, dtype, page, block, slots_first=False):
    return {"name": name, "op": "commit", "B": B, "N": N, "L": L, "at_lo": at_lo, "at_hi": at_hi,
            "hkv": hkv, "d": d, "dtype": dtype, "page": page, "block": block,
            "slots_first": slots_first}


def _read(name, B, lo, hi, at_lo, at_hi, hkv, d, dtype, page, block, slots_first=False):
    return {"name": name, "op": "read", "B": B, "lo": lo, "hi": hi, "at_lo": at_lo, "at_hi": at_hi,
            "hkv": hkv, "d": d, "dtype": dtype, "page": page, "block": block,
            "slots_first": slots_first}


def _attn(name, B, N, lo, hi, hq, hkv, d, dtype, page, block, slots_first=False, fused=False):
    return {"name": name, "op": "attn", "B": B, "N": N, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "dtype": dtype, "page": page, "block": block, "slots_first": slots_first,
            "fused": fused}


def listed():
    return [
        # the 65 rows of an 8B-class draft tree behind a 2K prefix: the smallest step, latency
        _norm("norm_tree_8b", 65, 0, 32, 8, 128, 128, "half", "none", 1.0, "bf16", 2112),
        # a long prompt's chunk, 70B-class heads, taken out of one fused projection
        _norm("norm_prompt_yarn", 8192, 17, 64, 8, 128, 128, "half", "yarn", 4.0, "fp16", 131072,
              fused=True),
        # one token each of a serving batch, queries normed and rotated in the same call
        _append("append_step", 16, 1, 1, 256, 4096, 0, 32, 8, 128, 128, "half", "none", 1.0,
                "bf16", 16, 16),
        # ragged prompts of a batch, behind shared-prefix lengths, padded to a fixed shape
        _append("append_prompts", 8, 517, 4001, 0, 4096, 129, 32, 8, 128, 128, "interleaved",
                "linear", 4.0, "fp16", 64, 32, fused=True, slots_first=True),
        # accepted paths of a large serving batch
        _commit("commit_serving", 128, 128, 16, 100, 1000, 8, 128, "bf16", 64, 16),
        # the prefix of one sequence back in 16 bits
        _read("read_single", 1, 2048, 2048, 0, 0, 8, 128, "bf16", 16, 16),
        # ... of a serving batch, ragged, from where a shared part ends
        _read("read_serving", 16, 1024, 32768, 0, 4096, 8, 128, "bf16", 64, 32, slots_first=True),
        # one layer of the 8B-class single stream's verification
        _attn("tree_8b_single", 1, 64, 2048, 2048, 32, 8, 128, "bf16", 16, 16),
        # ragged serving: 16 sequences of 1K to 32K, 128 drafted nodes each
        _attn("tree_ragged_serving", 16, 128, 1024, 32768, 32, 8, 128, "bf16", 64, 32),
        # 70B-class long context, 256 drafted nodes: the largest
        _attn("tree_long_context_70b", 4, 256, 131072, 131072, 64, 8, 128, "bf16", 128, 64),
        # plain decoding of a batch: the bonus token alone, one row a sequence
        _attn("decode_batch", 64, 0, 512, 16384, 32, 8, 128, "bf16", 16, 16),
        # small trees, seven queries a KV head, an empty prefix among them, the other layout
        _attn("tree_small_odd", 7, 21, 0, 5003, 28, 4, 64, "fp16", 32, 8, slots_first=True,
              fused=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "append", "commit", "read", "attn", "attn", "attn", "attn"])
    hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([x for x in (8, 16, 32, 64) if x <= page])
    first = rng.random() < 0.4
    fused = rng.random() < 0.4
    dtype = rng.choice(["bf16", "fp16"])
    pairs = rng.choice(["half", "interleaved"])
    scaling, factor = rng.choice([("none", 1.0), ("linear", 4.0), ("ntk", 3.0), ("banded", 8.0),
                                  ("yarn", 16.0)])
    rot = rng.choice([d, d, d // 2, d // 4])
    if op == "norm":
        d = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2])
        c = _norm("", _spread(rng, 1, 8192), rng.choice([0, 0, 3]), hkv * g, hkv, d, rot, pairs,
                  scaling, factor, rng.choice(["bf16", "fp16", "fp32"]), _spread(rng, 16, 1000000),
                  fused)
    elif op == "append":
        hi = _spread(rng, 1, 2048)
        at = _spread(rng, 1, 16384)
        c = _append("", _spread(rng, 1, 32), rng.randint(0, hi), hi, rng.randint(0, at), at,
                    rng.choice([0, 0, 5]), hkv * g, hkv, d, rot, pairs, scaling, factor, dtype,
                    page, block, rng.random() < 0.6, fused, first)
    elif op == "commit":
        hi = _spread(rng, 1, 8192)
        c = _commit("", _spread(rng, 1, 128), _spread(rng, 1, 512), rng.randint(1, 16),
                    rng.randint(0, hi), hi, hkv, d, dtype, page, block, first)
    elif op == "read":
        hi = _spread(rng, 1, 16384)
        at = _spread(rng, 1, 4096)
        c = _read("", max(1, min(_spread(rng, 1, 64), 200000 // hi)), rng.randint(0, hi), hi,
                  rng.randint(0, at), at, hkv, d, dtype, page, block, first)
    else:
        N = 0 if rng.random() < 0.35 else _spread(rng, 1, 512)
        hi = _spread(rng, 1, 65536)
        B = max(1, min(_spread(rng, 1, 96), 300000 // hi))
        N = min(N, int(1e12 / (4 * B * (hi + N) * hkv * g * d)))
        c = _attn("", B, N, rng.randint(0, hi), hi, hkv * g, hkv, d, dtype, page, block, first,
                  fused)
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
    if op == "norm":
        T, heads = case["T"] + case["pad"], case["hq"] + case["hkv"]
        return {"bytes": 2 * T * heads * d * es + 4 * T + 4 * case["rot"] + 8 * d,
                "flops": case["T"] * heads * (4 * d + 3 * case["rot"])}
    if op == "append":
        live = sum(_lens(case["lo"], case["hi"], case["B"]))
        row, heads = d * es, case["hq"] + case["hkv"]
        # (the codes of a block that is entered in its middle are touched only where its scale grows)
        return {"bytes": live * (2 * case["hq"] * row + 2 * case["hkv"] * (row + d)) + 8 * case["B"]
                + 2 * case["hkv"] * (-(-live // case["block"]) + case["B"]),
                "flops": live * heads * (4 * d + 3 * case["rot"]) + 4 * live * case["hkv"] * d}
    if op == "commit":
        rows = sum(1 + min(a, case["N"]) for a in _lens(0, case["L"], case["B"]))
        return {"bytes": rows * 2 * case["hkv"] * d * (es + 1) + 12 * case["B"] + 4 * rows
                + 4 * case["hkv"] * case["B"], "flops": 4 * rows * case["hkv"] * d}
    if op == "read":
        T = sum(_lens(case["lo"], case["hi"], case["B"]))
        return {"bytes": T * 2 * case["hkv"] * d * (1 + es) + 2 * case["hkv"] * -(-T // case["block"])
                + 8 * case["B"] + 4, "flops": 2 * T * case["hkv"] * d}
    P, n = _lens(case["lo"], case["hi"], case["B"]), _live(case)
    R, hq, hkv = case["N"] + 1, case["hq"], case["hkv"]
    rows = sum(x + 1 for x in n)
    return {"bytes": 2 * hkv * (d * sum(P) + sum(-(-p // case["block"]) for p in P))
            + 2 * hkv * d * es * rows + 2 * rows * hq * d * es
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
        s = ((orig * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = (1 - s) * f / factor + s * f
    elif kind == "yarn":
        def dim(beta):
            return rot * math.log(orig / (2 * math.pi * beta)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
        s = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = (1 - s) * f + s * f / factor
    return f, 0.1 * math.log(factor) + 1.0 if kind == "yarn" and factor > 1 else 1.0


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


def _exponent(amax, dtype):
    """The least e with amax <= 448 * 2^e, within the type's range, of 32-bit values."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [0.5, 1): 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, LEAST[dtype])).clamp(LEAST[dtype], MOST)


def _two(e):
    """2^e in 32 bits, e a whole number in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(case, gen, total):
    """A pool's codes and scales: random rows, magnitudes that differ by block and head."""
    page, hkv, d, S = case["page"], case["hkv"], case["d"], case["block"]
    codes = torch.empty(total, hkv, page, d, dtype=E4M3, device="cuda")
    scales = torch.empty(total, hkv, page // S, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (hkv * page * d))
    for i in range(0, total, step):
        n = min(step, total - i)
        x = _randn(gen, n, hkv, page // S, S, d, dtype=torch.float32)
        x *= torch.exp2(0.5 * _randn(gen, n, hkv, page // S, 1, 1, dtype=torch.float32))
        e = _exponent(x.abs().amax((-1, -2)), case["dtype"])
        scales[i:i + n] = (e + 127).to(torch.uint8)
        codes[i:i + n] = (x * _two(-e)[..., None, None]).to(E4M3).view(n, hkv, page, d)
    if case["slots_first"]:
        codes = codes.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(E4M3)
    return codes, scales


def _pool(case, gen, longest, B):
    """A pool with every sequence's pages in random places, and their table; the last of
    the pages that no sequence has."""
    page = case["page"]
    need = (longest.long() + page - 1) // page
    reach = case["hi"] if case["op"] == "attn" else case["at_hi"] + case.get("hi", case.get("L", 0) + 1)
    width = max(1, -(-reach // page))
    total = B * width + 3
    order = torch.randperm(total, generator=gen, device="cuda").int()
    where = order[:B * width].view(B, width)
    live = torch.arange(width, device="cuda")[None] < need[:, None]
    table = torch.where(live, where, torch.full_like(where, -1))
    k, ks = _codes(case, gen, total)
    v, vs = _codes(case, gen, total)
    return {"k_pages": k, "v_pages": v, "k_scales": ks, "v_scales": vs, "table": table,
            "spare": order[B * width].long()}


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
    nodes = torch.where(keep, pick, torch.full_like(pick, N + 2)).sort(1).values
    return alen, torch.where(keep, nodes, torch.full_like(nodes, -1))


def _weights(case, gen):
    """Norm weights of queries and keys, near one."""
    return (1 + 0.2 * _randn(gen, case["d"], dtype=torch.float32),
            1 + 0.2 * _randn(gen, case["d"], dtype=torch.float32))


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "norm":
        T, pad = case["T"], case["pad"]
        s["q"], s["k"], _ = _heads(case, gen, T + pad)
        s["wq"], s["wk"] = _weights(case, gen)
        s["pos"] = torch.randint(0, case["top"], (T + pad,), generator=gen, device="cuda").int()
        s["pos"][T:] = -1
        s["q_out"], s["k_out"] = (torch.zeros(x.shape, dtype=x.dtype, device="cuda")
                                  for x in (s["q"], s["k"]))
        return s
    B, hkv, d, dt = case["B"], case["hkv"], case["d"], DT[case["dtype"]]
    if op in ("append", "read"):
        lens = _lens(case["lo"], case["hi"], B)
        s["n"] = _shuffled(gen, lens)
        s["at"] = _shuffled(gen, _lens(case["at_lo"], case["at_hi"], B))
        s["first"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        s["first"][1:] = s["n"].cumsum(0)
        s["live"] = sum(lens)
        s |= _pool(case, gen, s["at"] + s["n"], B)
        T = s["live"] + case.get("pad", 0)
        if op == "read":
            s["k_out"], s["v_out"] = (torch.zeros(T, hkv, d, dtype=dt, device="cuda") for _ in "kv")
            return s
        s["q"], s["k"], s["v"] = _heads(case, gen, T)
        s["wq"], s["wk"] = _weights(case, gen)
        s["q_out"] = torch.zeros(s["q"].shape, dtype=dt, device="cuda")
        return s
    if op == "commit":
        s["prefix"] = _shuffled(gen, _lens(case["at_lo"], case["at_hi"], B))
        s["alen"], s["nodes"] = _paths(case, gen)
        s |= _pool(case, gen, s["prefix"] + s["alen"] + 1, B)
        s["k_tree"] = _randn(gen, B, case["N"] + 1, hkv, d, dtype=dt)
        s["v_tree"] = _randn(gen, B, case["N"] + 1, hkv, d, dtype=dt)
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    R, hq = case["N"] + 1, case["hq"]
    s["prefix"] = _shuffled(gen, _lens(case["lo"], case["hi"], B))
    s |= _pool(case, gen, s["prefix"], B)
    q, k, v = _heads(case, gen, B * R)
    s["q"], s["k_tree"], s["v_tree"] = (x.unflatten(0, (B, R)) for x in (q, k, v))
    s["n"] = _shuffled(gen, _live(case))
    s["mask"] = _tree(case, gen, s["n"])
    s["out"] = torch.zeros(B, R, hq, d, dtype=dt, device="cuda")
    s["lse"] = torch.zeros(B, R, hq, dtype=torch.float32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("norm", "append"):
        f, s["scale"] = _frequencies(case)
        s["freq"] = f.cuda()
    if own:  # the handles that a program makes once: rotation, norms, the cache, a workspace
        from diffusion_draft_tree_gb300 import ops
        if op in ("norm", "append"):
            s["rotary"] = ops.Rotary(case["rot"], base=BASE, interleaved=case["pairs"] == "interleaved",
                                     scaling=case["scaling"], factor=case["factor"], orig_len=8192,
                                     low=1.0, high=32.0 if case["scaling"] == "yarn" else 4.0,
                                     device="cuda")
            s["norm"] = ops.HeadNorm(s["wq"], s["wk"], eps=EPS) if case.get("normed", True) else None
        if op != "norm":
            s["cache"] = ops.QuantCache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                                        s["table"], DT[case["dtype"]])
        if op == "attn":
            s["ws"] = ops.q8_attn_workspace(s["q"], s["cache"])
    return s


# --------------------------------------------------------------- one pass

def _held(s):
    """The pool's codes and scales as the values that they are."""
    e8m0 = torch.float8_e8m0fnu
    return [s["k_pages"], s["v_pages"], s["k_scales"].view(e8m0), s["v_scales"].view(e8m0)]


def _turned32(x, w, s, pos):
    """x [T][heads][d] normed (w not None) and rotated for pos: products in 32 bits, angles in 64."""
    case = s["case"]
    rot = case["rot"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    a = pos.double()[:, None, None] * s["freq"]
    c, n = (a.cos() * s["scale"]).float(), (a.sin() * s["scale"]).float()
    if case["pairs"] == "half":
        lo, hi = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([lo * c - hi * n, lo * n + hi * c], -1)
    else:
        lo, hi = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([lo * c - hi * n, lo * n + hi * c], -1).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1)


def _places(s, seq, pos):
    page = s["case"]["page"]
    return s["table"].long()[seq, pos // page], pos % page


def _write32(s, pages, scales, x, seq, pos, at, n):
    """Rows x [T][hkv][d], in 32 bits, to positions pos of sequences seq of one half of the
    cache; at and n [B]: each sequence's first position, and how many follow."""
    case = s["case"]
    page, S, hkv = case["page"], case["block"], case["hkv"]
    nb = page // S
    where, slot = _places(s, seq, pos)
    blk = where * nb + slot // S
    raw = pages.view(torch.uint8).transpose(1, 2)  # [page][slot][head][d]
    flat = scales.transpose(1, 2).reshape(-1, hkv)  # (a copy) [page * blocks][head]
    old = flat.int() - 127
    amax = torch.zeros(flat.shape, dtype=torch.float32, device="cuda")
    amax.index_reduce_(0, blk, x.abs().amax(-1), "amax")
    need = _exponent(amax, case["dtype"])
    hit = torch.zeros(len(flat), dtype=torch.bool, device="cuda")
    hit[blk] = True
    # each sequence's first block, if it is entered in its middle; else a page of nobody
    mid = (n > 0) & (at % S > 0)
    b = torch.arange(len(at), device="cuda")
    p0 = torch.where(mid, at, 0).long()
    w0, s0 = _places(s, b, p0)
    w0 = torch.where(mid, w0, s["spare"])
    kept = torch.zeros(len(flat), dtype=torch.bool, device="cuda")
    kept[w0 * nb + s0 // S] = True
    new = torch.where(hit[:, None], torch.where(kept[:, None], torch.maximum(old, need), need), old)
    live = torch.arange(S, device="cuda")[None] < torch.where(mid, at % S, 0)[:, None]
    at_w, at_s = w0[:, None].expand(-1, S), (s0 // S * S)[:, None] + torch.arange(S, device="cuda")
    codes = raw[at_w, at_s]  # [B][S][head][d]
    g = w0 * nb + s0 // S
    moved = (codes.view(E4M3).float() * _two(old[g] - new[g])[:, None, :, None]).to(E4M3)
    raw[at_w, at_s] = torch.where(live[..., None, None], moved.view(torch.uint8), codes)
    fresh = (x * _two(-new[blk])[..., None]).clamp(-448, 448).to(E4M3)
    raw[where, slot] = fresh.view(torch.uint8)
    scales.copy_((new + 127).to(torch.uint8).view(-1, nb, hkv).transpose(1, 2))


def _values32(pages, scales, table, block):
    """Pages listed in a table, as the values that they stand for: [..][head][page][d], 32 bits."""
    c = pages.view(torch.uint8)[table].view(E4M3).float()
    return c * _two(scales[table].int() - 127).repeat_interleave(block, -1)[..., None]


def _plain_attn(s):
    case, table, page = s["case"], s["table"].long().clamp(min=0), s["case"]["page"]
    B, R, hkv, d = case["B"], case["N"] + 1, case["hkv"], case["d"]
    G, W = case["hq"] // hkv, table.shape[1]
    k = _values32(s["k_pages"], s["k_scales"], table, case["block"])
    k = k.permute(0, 2, 1, 3, 4).reshape(B, hkv, W * page, d)
    v = _values32(s["v_pages"], s["v_scales"], table, case["block"])
    v = v.permute(0, 2, 1, 3, 4).reshape(B, hkv, W * page, d)
    k = torch.cat([k, s["k_tree"].permute(0, 2, 1, 3).float()], 2)
    v = torch.cat([v, s["v_tree"].permute(0, 2, 1, 3).float()], 2)
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


def _runs(s):
    """Sequence and position of each token of a batch of runs."""
    n, live = s["n"].long(), s["live"]
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=live)
    pos = torch.arange(live, device="cuda") - s["first"].long()[seq] + s["at"].long()[seq]
    return seq, pos


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from diffusion_draft_tree_gb300 import ops
        if op == "norm":
            ops.ddtree_norm_rope(s["q"], s["k"], s["pos"], s["norm"], s["rotary"], q_out=s["q_out"],
                                 k_out=s["k_out"])
            return [s["q_out"], s["k_out"]]
        if op == "append":
            ops.ddtree_append_q8(s["k"], s["v"], s["first"], s["at"], s["cache"], s["rotary"],
                                 s["norm"], q=s["q"], q_out=s["q_out"])
            return [*_held(s), s["q_out"]]
        if op == "commit":
            ops.ddtree_commit_q8(s["cache"], s["k_tree"], s["v_tree"], s["alen"], s["nodes"],
                                 s["prefix"], s["new_len"])
            return [*_held(s), s["new_len"]]
        if op == "read":
            ops.ddtree_read_q8(s["cache"], s["first"], s["at"], s["k_out"], s["v_out"])
            return [s["k_out"], s["v_out"]]
        ops.ddtree_tree_attn_q8(s["q"], s["cache"], s["k_tree"], s["v_tree"], s["prefix"], s["n"],
                                s["mask"], s["out"], s["lse"], workspace=s["ws"])
        return [s["out"], s["lse"]]
    if op == "norm":
        T = case["T"]
        for x, w, to in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
            to[:T] = _turned32(x[:T], w, s, s["pos"][:T]).to(to.dtype)
            to[T:] = x[T:]
        return [s["q_out"], s["k_out"]]
    if op == "append":
        T = s["live"]
        seq, pos = _runs(s)
        wq, wk = (s["wq"], s["wk"]) if case["normed"] else (None, None)
        s["q_out"][:T] = _turned32(s["q"][:T], wq, s, pos).to(s["q_out"].dtype)
        k = _turned32(s["k"][:T], wk, s, pos)
        _write32(s, s["k_pages"], s["k_scales"], k, seq, pos, s["at"], s["n"])
        _write32(s, s["v_pages"], s["v_scales"], s["v"][:T].float(), seq, pos, s["at"], s["n"])
        return [*_held(s), s["q_out"]]
    if op == "commit":
        B, L = case["B"], case["L"]
        step = torch.arange(L + 1, device="cuda")[None]
        node = torch.cat([torch.zeros_like(s["nodes"][:, :1]), s["nodes"]], 1).long()
        # a row behind the path repeats the path's root: the same values to the same slot
        keep = step <= s["alen"][:, None]
        node, step = torch.where(keep, node, 0), torch.where(keep, step, 0)
        pos = (s["prefix"].long()[:, None] + step).flatten()
        b = torch.arange(B, device="cuda")[:, None].expand(B, L + 1)
        for half, x in (("k", s["k_tree"]), ("v", s["v_tree"])):
            _write32(s, s[half + "_pages"], s[half + "_scales"], x[b, node].flatten(0, 1).float(),
                     b.flatten(), pos, s["prefix"], s["alen"] + 1)
        s["new_len"].copy_(s["prefix"] + s["alen"] + 1)
        return [*_held(s), s["new_len"]]
    if op == "read":
        seq, pos = _runs(s)
        where, slot = _places(s, seq, pos)
        for half in "kv":
            c = s[half + "_pages"].view(torch.uint8)[where, :, slot].view(E4M3).float()
            e = s[half + "_scales"][where, :, slot // case["block"]].int() - 127
            s[half + "_out"].copy_(c * _two(e)[..., None])
        return [s["k_out"], s["v_out"]]
    _plain_attn(s)
    return [s["out"], s["lse"]]


# ------------------------------------------------------------- in 64 bits

def _turned64(x, w, pos, case):
    """Norm, and rotation by complex numbers, in 64 bits."""
    f, scale = _frequencies(case)
    rot, y = case["rot"], x.double()
    if w is not None:
        y = y / ((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * w.double()
    angle = pos.double()[:, None] * f.to(x.device)[None]
    turn = torch.polar(torch.full_like(angle, scale), angle)[:, None]
    if case["pairs"] == "half":
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    return torch.cat([head, y[..., rot:]], -1)


def _grid64(x):
    """The nearest e4m3 numbers to 64-bit values, ties to even."""
    top = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    unit = torch.exp2(top - 3)
    return (torch.round(x / unit) * unit).clamp(-448, 448)


def _write64(s, pages, scales, rows, b, at):
    """Rows [n][hkv][d] to positions at.. of sequence b: pages and scales hold values in 64 bits."""
    case = s["case"]
    page, S = case["page"], case["block"]
    n = len(rows)
    for p0 in range(at - at % S, at + n, S):
        lo, hi = max(p0, at), min(p0 + S, at + n)
        where, slot = s["rows"][b][p0 // page], p0 % page
        x = rows[lo - at:hi - at].double()
        amax = x.abs().amax((0, 2))
        e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448))
        e = e + (448 * torch.exp2(e) < amax).double() - (448 * torch.exp2(e - 1) >= amax).double()
        e = e.clamp(LEAST[case["dtype"]], MOST)
        if lo > p0:
            old = torch.log2(scales[where, :, slot // S])
            e = torch.maximum(e, old)
            part = pages[where, :, slot:slot + lo - p0]
            part.copy_(_grid64(part * torch.exp2(old - e)[:, None, None]))
        pages[where, :, slot + lo - p0:slot + hi - p0] = _grid64(x / torch.exp2(e)[:, None]).transpose(0, 1)
        scales[where, :, slot // S] = torch.exp2(e)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "norm":
        T = case["T"]
        return [torch.cat([_turned64(x[:T], w, s["pos"][:T], case), x[T:].double()])
                for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"]))]
    S = case["block"]
    if op in ("append", "commit", "read"):
        k, v = s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64)
        ks, vs = (torch.exp2(s[x].double() - 127) for x in ("k_scales", "v_scales"))
        s["rows"] = s["table"].tolist()
    if op == "append":
        q, at, first = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), s["at"].tolist(), s["first"].tolist()
        wq, wk = (s["wq"], s["wk"]) if case["normed"] else (None, None)
        for b, p in enumerate(at):
            t = slice(first[b], first[b + 1])
            pos = torch.arange(p, p + first[b + 1] - first[b], device="cuda")
            q[t] = _turned64(s["q"][t], wq, pos, case)
            _write64(s, k, ks, _turned64(s["k"][t], wk, pos, case), b, p)
            _write64(s, v, vs, s["v"][t], b, p)
        return [k, v, ks, vs, q]
    if op == "commit":
        P, alen, nodes = (s[x].tolist() for x in ("prefix", "alen", "nodes"))
        for b in range(case["B"]):
            path = [0] + nodes[b][:alen[b]]
            _write64(s, k, ks, s["k_tree"][b, path], b, P[b])
            _write64(s, v, vs, s["v_tree"][b, path], b, P[b])
        new = torch.tensor([p + a + 1 for p, a in zip(P, alen)], dtype=torch.int32, device="cuda")
        return [k, v, ks, vs, new]
    if op == "read":
        page, out = case["page"], []
        for x, e in ((k, ks), (v, vs)):
            got = []
            for b, (p, n) in enumerate(zip(s["at"].tolist(), s["n"].tolist())):
                pages = s["table"][b, p // page:-(-(p + n) // page)].long()
                y = x[pages].unflatten(2, (-1, S)) * e[pages][..., None, None]  # [page][head][block][slot][d]
                got.append(y.flatten(2, 3).transpose(1, 2).flatten(0, 1)[p % page:p % page + n])
            out.append(torch.cat(got))
        return out
    B, R, hq, hkv, d, page = case["B"], case["N"] + 1, case["hq"], case["hkv"], case["d"], case["page"]
    G = hq // hkv
    out = torch.zeros(B, R, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, R, hq), -math.inf, dtype=torch.float64, device="cuda")
    bit = torch.arange(R, device="cuda")
    for b, (P, n) in enumerate(zip(s["prefix"].tolist(), s["n"].tolist())):
        pages = s["table"][b, :-(-P // page)].long()
        sees = (s["mask"][b, :n + 1][:, bit // 32] >> (bit % 32)) & 1  # [n + 1][R]
        hide = (sees == 0)[:, None, :n + 1].expand(n + 1, G, n + 1).reshape((n + 1) * G, n + 1)
        for g in range(hkv):
            def column(x, e, tree):
                c = x.view(torch.uint8)[pages, g].view(E4M3).to(torch.float64).unflatten(1, (-1, S))
                c = c * torch.exp2(e[pages, g].double() - 127)[..., None, None]
                return torch.cat([c.reshape(-1, d)[:P], tree[b, :n + 1, g].double()])
            k, v = column(s["k_pages"], s["k_scales"], s["k_tree"]), column(s["v_pages"], s["v_scales"], s["v_tree"])
            q = s["q"][b, :n + 1, g * G:(g + 1) * G].reshape(-1, d).double()
            x = (q @ k.T) / math.sqrt(d)
            x[:, P:] = x[:, P:].masked_fill(hide, -math.inf)
            z = torch.logsumexp(x, 1)
            o = (x - z[:, None]).exp_() @ v
            out[b, :n + 1, g * G:(g + 1) * G] = o.view(n + 1, G, d)
            lse[b, :n + 1, g * G:(g + 1) * G] = z.view(n + 1, G)
    return [out, lse]
