"""Timed cases of the operators of a serving step over a paged cache: norms of the heads with the
rotation in the same pass (positions with several axes among them), block tables and slot maps made
on the device, attention with a sliding window and first tokens that stay visible, and attention of
a batch whose sequences begin with the same cells.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, angles in 64) or,
with ``own`` set, through the library's entry points; ``exact`` says what the definition gives in 64
bits.  A case is a dict of plain values; lengths are texts such as "8192,20480".

    norm    q, k half [T][heads][D]: each head over its root mean square, times a weight, then rotated
            to its position; without the norm, the rotation by positions of several axes alone
    maps    from lengths and new tokens: blocks taken from the free list, offsets, lengths, positions,
            slots and the cell plan
    window  causal attention in which a token sees its last `window` cells and the first `sinks`:
            of packed prompts, or of new tokens over a cache
    shared  causal attention of new tokens over caches whose first `prefix` cells are the same
"""
import math

import torch

own = False

SCALE_GROUP = 32  # elements that share one scale in a quantised cache row
RECORD = 128      # cells of a record of a cell plan
BITS = {"f16": (16, 16), "q8_0": (8, 8), "q8_0_q4_0": (8, 4), "q4_0": (4, 4)}
KINDS = tuple(BITS)
# One pass of the largest listed cases costs about this much; no drawn case costs more.
MOST_FLOPS = 4.0e10
MOST_SCORES = 2.2e9
MOST_CELLS = 6.0e8   # elements of a cache plane
MOST_ENTRIES = 8000000   # of a cell plan


# --------------------------------------- cases ---------------------------------------

def listed():
    return [
        # a decode step's new tokens of 64 sequences, far along in their contexts, both sides normed
        {"name": "norm step", "op": "norm", "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128, "n_rot": 128, "norm": "both",
         "layout": "half", "sections": "64", "order": "blocks", "restart": False, "base": 1000000.0, "far": 131072},
        # a long prompt of a wide-headed model, a quarter of each head rotated
        {"name": "norm prompt", "op": "norm", "tokens": 16384, "heads": 16, "kv_heads": 8, "dim": 256, "n_rot": 64,
         "norm": "both", "layout": "interleaved", "sections": "32", "order": "blocks", "restart": False, "base": 10000.0,
         "far": 32768},
        # images and video in a prompt: time, height and width turn pairs of their own, no norm
        {"name": "axes video", "op": "norm", "tokens": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "n_rot": 128,
         "norm": "none", "layout": "half", "sections": "16,24,24", "order": "cycle", "restart": False, "base": 1000000.0,
         "far": 16384},
        # one decode step: a token for each of 64 sequences, the plan kept from the step before
        {"name": "maps step", "op": "maps", "seqs": 64, "most": 131072, "new": 1, "block": 128, "whole": False},
        # a batch put together anew: the whole plan of 64 long sequences over small blocks
        {"name": "maps batch", "op": "maps", "seqs": 64, "most": 131072, "new": 512, "block": 16, "whole": True},
        # a decode step of 64 sequences in a layer with a window
        {"name": "window step", "op": "window", "form": "chunk", "kind": "f16", "tokens": ",".join(["1"] * 64),
         "lens": ",".join(str(40 + 127 * i) for i in range(64)), "heads": 32, "kv_heads": 8, "dim": 128, "window": 1024,
         "sinks": 4, "plan": False, "holes": 0.0},
        # one long prompt through the same layer
        {"name": "window prompt", "op": "window", "form": "prompt", "lens": "8192", "heads": 32, "kv_heads": 8, "dim": 128,
         "window": 1024, "sinks": 4},
        # ragged prompts of the 256-wide heads, a short window
        {"name": "window ragged d256", "op": "window", "form": "prompt", "lens": "2049,513,3000,77,1023", "heads": 16,
         "kv_heads": 8, "dim": 256, "window": 500, "sinks": 130},
        # chunks of prompts and a single token over an 8-bit unified cache with holes
        {"name": "window chunk q8", "op": "window", "form": "chunk", "kind": "q8_0", "tokens": "256,128,1,64",
         "lens": "8192,20480,40960,65536", "heads": 48, "kv_heads": 8, "dim": 128, "window": 4096, "sinks": 64, "plan": True,
         "holes": 0.1},
        # 64 requests behind one system prompt, a token each
        {"name": "shared step", "op": "shared", "kind": "f16", "tokens": ",".join(["1"] * 64), "prefix": 8192,
         "lens": ",".join(str(30 + 16 * i) for i in range(64)), "heads": 32, "kv_heads": 8, "dim": 128, "plan": True,
         "holes": 0.0},
        # sixteen questions about one very long document in an 8-bit cache
        {"name": "shared q8 long", "op": "shared", "kind": "q8_0", "tokens": ",".join(["1"] * 16), "prefix": 131072,
         "lens": ",".join(str(20 + 30 * i) for i in range(16)), "heads": 32, "kv_heads": 8, "dim": 128, "plan": True,
         "holes": 0.0},
        # eight samples from one prompt, each verifying four drafted tokens, caches of their own
        {"name": "shared verify d256", "op": "shared", "kind": "f16", "tokens": "4,4,4,4,4,4,4,4", "prefix": 4096,
         "lens": "5,90,61,200,33,128,77,150", "heads": 16, "kv_heads": 8, "dim": 256, "plan": False, "holes": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 3, 4, 6, 8]), kv


def _draw_sections(rng, pairs):
    """One to four axes; every pair has one."""
    axes = min(rng.choice([1, 1, 2, 3, 3, 4]), pairs)
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [pairs])]


def draw(rng):
    op = rng.choice(["norm", "norm", "maps", "window", "window", "window", "shared", "shared"])
    dim = rng.choice([128, 256])
    if op == "norm":
        heads, kv = _draw_heads(rng)
        n_rot = 16 * rng.randint(1, dim // 16)
        sections = _draw_sections(rng, n_rot // 2)
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "heads": heads, "kv_heads": kv, "dim": dim, "n_rot": n_rot,
                "norm": rng.choice(["both", "both", "q", "k", "none"]), "layout": rng.choice(["half", "interleaved"]),
                "sections": ",".join(map(str, sections)), "order": rng.choice(["blocks", "cycle"]),
                "restart": len(sections) > 1 and rng.random() < 0.3, "base": rng.choice([10000.0, 500000.0, 1000000.0]),
                "far": _log_int(rng, 16, 262144)}
    if op == "maps":
        seqs = _log_int(rng, 1, 300)
        return {"op": op, "seqs": seqs, "most": _log_int(rng, 16, min(131072, MOST_ENTRIES // seqs)), "new": _log_int(rng, 1, 512),
                "block": rng.choice([16, 32, 64, 128, 256]), "whole": rng.random() < 0.5}
    while True:
        heads, kv = _draw_heads(rng)
        c = {"op": op, "heads": heads, "kv_heads": kv, "dim": dim}
        if op == "window":
            c |= {"form": rng.choice(["prompt", "chunk", "chunk"]), "window": _log_int(rng, 1, 8192),
                  "sinks": rng.choice([0, 0, 1, 4, 17, 64, 128, 200])}
        step = rng.random() < 0.4   # a token for each sequence
        n_seq = _log_int(rng, 2 if op == "shared" else 1, 64 if step else 12)
        plan = rng.random() < 0.5
        if op == "window" and c["form"] == "prompt":
            top = _log_int(rng, 16, 8192)
            c["lens"] = ",".join(str(_log_int(rng, 1, top)) for _ in range(n_seq))
            scores = n_seq * max(_ints(c["lens"])) ** 2 * heads
            cells = 0
        else:
            most = 16 if op == "shared" else 512
            new = [1 if step else _log_int(rng, 1, most) for _ in range(n_seq)]
            top = _log_int(rng, 16, 1024 if op == "shared" else 65536)
            lens = [n + _log_int(rng, 1, top) - 1 for n in new]
            c |= {"kind": rng.choice(KINDS), "tokens": ",".join(map(str, new)), "lens": ",".join(map(str, lens)), "plan": plan,
                  "holes": rng.choice([0.0, 0.1]) if plan else 0.0}
            if op == "shared":
                c["prefix"] = _log_int(rng, 64, 65536)
                scores = (c["prefix"] * sum(new) + n_seq * max(new) * max(lens)) * heads
                cells = (c["prefix"] * (1 if plan else n_seq) + n_seq * max(lens)) * kv * dim
            else:
                scores = n_seq * max(new) * min(max(lens), c["sinks"] + c["window"] + max(new)) * heads
                cells = n_seq * max(lens) * kv * dim
        if work(c)["flops"] <= MOST_FLOPS and scores <= MOST_SCORES and cells <= MOST_CELLS:
            return c


def _ints(text):
    return [int(x) for x in text.split(",")]


# ------------------------------- inputs, made on the device -------------------------------

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).half()


def _planes(g, kind, cells, kv_heads, dim):
    """A cache as a serving program holds it: (k, v, k_scales, v_scales)."""
    def side(bits):
        if bits == 16:
            return torch.randn((cells, kv_heads, dim), generator=g, device="cuda", dtype=torch.float16), None
        shape = (cells, kv_heads, dim // SCALE_GROUP)
        if bits == 8:
            rows = torch.randint(-127, 128, (cells, kv_heads, dim), generator=g, device="cuda", dtype=torch.int8)
            top = 0.02
        else:
            rows = torch.randint(0, 256, (cells, kv_heads, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
            top = 0.3
        return rows, (torch.rand(shape, generator=g, device="cuda") * (top - 0.001) + 0.001).half()
    k, ks = side(BITS[kind][0])
    v, vs = side(BITS[kind][1])
    return k, v, ks, vs


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def _device_ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_norm(case, s, g):
    T, H, Hk, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    s["q"], s["k"] = _normal(g, T, H, D), _normal(g, T, Hk, D)
    s["sections"] = _ints(case["sections"])
    axes = len(s["sections"])
    pos = torch.randint(0, case["far"], (axes, T), generator=g, device="cuda", dtype=torch.int32)
    s["pos"] = pos if axes > 1 else pos[0]
    s["q_weight"] = (1.0 + 0.2 * _normal(g, D).float()).half() if case["norm"] in ("both", "q") else None
    s["k_weight"] = (1.0 + 0.2 * _normal(g, D).float()).half() if case["norm"] in ("both", "k") else None
    s["eps"] = 1e-6
    half = {"dtype": torch.float16, "device": "cuda"}
    s["q_out"], s["k_out"] = torch.empty((T, H, D), **half), torch.empty((T, Hk, D), **half)
    if own:  # the angle table that a program makes once for its model
        from kv_cache_decode_02_gb300 import kvattn
        s["table"] = kvattn.rope_table(case["n_rot"], base=case["base"], sections=s["sections"] if axes > 1 else None,
                                       order=case["order"], restart=case["restart"])


def _prepare_maps(case, s, g):
    """Sequences of random lengths hold random blocks of a pool; the free list names the others, with
    a few to spare."""
    S, block, top = case["seqs"], case["block"], case["most"]
    def lengths(lo, hi):
        x = torch.rand((S,), generator=g, device="cuda", dtype=torch.float64)
        return (lo * (hi / lo) ** x).round().clamp(lo, hi)
    lens = lengths(1, top) - 1.0
    new = lengths(1, case["new"])
    s["lens"], s["new"] = lens.to(torch.int32), new.to(torch.int32)
    stride = -(-(top + case["new"]) // block)
    pool = S * stride + 16
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = torch.arange(S, device="cuda")[:, None] * stride + torch.arange(stride, device="cuda")
    held = torch.arange(stride, device="cuda") * block < s["lens"][:, None]
    s["tables"] = torch.where(held, perm[first], -1)
    free = torch.ones(pool, dtype=torch.bool, device="cuda")
    free[first[held]] = False
    s["free"] = perm[free]
    s["n_free"] = free.sum(dtype=torch.int32).reshape(1)
    s["n_cells"] = pool * block
    s["n_tok"] = S * case["new"]   # rows of the step's buffers; the ones behind the last token stay empty
    s["plan"] = torch.full((S, stride * block), -1, dtype=torch.int32, device="cuda")
    if not case["whole"]:
        s["plan"].copy_(_plan_of(s["tables"], s["lens"].long(), block))
    if own:
        from kv_cache_decode_02_gb300 import kvattn
        s["out"] = kvattn.step_maps_buffers(S, s["n_tok"])


def _records(s, g, counts, shared):
    """Scattered ascending records of a pool for every sequence: `shared` of them the same for all,
    in front.  Returns the plan's records [S][most] (-1 past a sequence's) and the pool's size."""
    most = shared + max(counts)
    pool = shared + sum(counts) + 8
    perm = torch.randperm(pool, generator=g, device="cuda")
    front = perm[:shared].sort().values
    at = torch.arange(max(counts), device="cuda")
    first = _device_ints(_offsets(counts)[:-1]).long() + shared
    count = _device_ints(counts).long()
    tail = torch.where(at[None, :] < count[:, None], perm[(first[:, None] + at).clamp(max=pool - 1)], pool).sort(dim=1).values
    records = torch.cat((front.expand(len(counts), -1), tail), 1)
    return torch.where(records < pool, records, -1).view(len(counts), most), pool


def _prepare_attention(case, s, g):
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    half = {"dtype": torch.float16, "device": "cuda"}
    if case.get("form") == "prompt":
        lens = _ints(case["lens"])
        T = sum(lens)
        s["lens"] = s["new"] = lens
        s["q"], s["k"], s["v"] = _normal(g, T, H, D), _normal(g, T, Hk, D), _normal(g, T, Hk, D)
        s["offsets"] = _device_ints(_offsets(lens))
        s["out"] = torch.empty((T, H, D), **half)
        s["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
        if own:  # the workspace that a program allocates once
            from kv_cache_decode_02_gb300 import kvattn
            s["ws"] = kvattn.prefill_workspace(T, len(lens), H, Hk, D)
        return
    prefix = case.get("prefix", 0)
    new, lens = _ints(case["tokens"]), [prefix + n for n in _ints(case["lens"])]
    T, S, top = sum(new), len(new), max(lens)
    s["new"], s["lens"] = new, lens
    s["q"] = _normal(g, T, H, D)
    s["offsets"], s["seq_lens"] = _device_ints(_offsets(new)), _device_ints(lens)
    s["plan"] = None
    if case["plan"]:
        shared = prefix // RECORD   # (a record that the prefix ends in is each sequence's own)
        records, pool = _records(s, g, [-(-n // RECORD) - shared for n in lens], shared)
        at = torch.arange(RECORD * records.shape[1], device="cuda")
        n, t = s["seq_lens"].long()[:, None], _device_ints(new).long()[:, None]
        hole = torch.rand((S, at.numel()), generator=g, device="cuda") < case["holes"]
        hole[:, :prefix] = hole[0, :prefix].clone()
        keep = (at < n) & (~hole | (at >= n - t))
        s["plan"] = torch.where(keep, records.repeat_interleave(RECORD, dim=1) * RECORD + at % RECORD, -1).to(torch.int32)
        s["n_cells"] = pool * RECORD
        s["cache"] = _planes(g, case["kind"], s["n_cells"], Hk, D)
        if prefix % RECORD:   # its last cells, each sequence's copy
            rest = s["plan"][:, shared * RECORD:prefix].long()
            rest = rest[:, rest[0] >= 0]
            for x in s["cache"]:
                if x is not None:
                    x[rest] = x[rest[0]].expand(S, *(-1 for _ in range(x.dim())))
    else:
        s["n_cells"] = top   # one cache of this many cells for each sequence
        s["cache"] = _planes(g, case["kind"], S * top, Hk, D)
        for x in s["cache"]:
            if x is not None and prefix:
                x.view(S, top, *x.shape[1:])[1:, :prefix] = x[:prefix].clone()
    s["out"] = torch.empty((T, H, D), **half)
    # the log-sum-exp goes to programs that merge this cache's result with another part's; the ones
    # that hold a whole context in a quantised cache take the output alone
    s["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda") if case["kind"] == "f16" else None
    if own:
        from kv_cache_decode_02_gb300 import kvattn
        s["ws"] = kvattn.prefill_chunk_workspace(T, S, H, Hk, D, top, shared=prefix)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    {"norm": _prepare_norm, "maps": _prepare_maps}.get(case["op"], _prepare_attention)(case, s, g)
    return s


# ------------------------------------- plain forms -------------------------------------

def _axes_of(case):
    """Of each pair: its axis, and the exponent's numerator and denominator of its frequency."""
    sections, n = _ints(case["sections"]), case["n_rot"]
    axis = []
    if case["order"] == "blocks":
        for a, count in enumerate(sections):
            axis += [a] * count
    else:   # dealt out in turn, an axis that has its pairs left out
        left = list(sections)
        while sum(left):
            for a in range(len(left)):
                if left[a]:
                    axis.append(a)
                    left[a] -= 1
    if not case["restart"]:
        return axis, [(2 * i, n) for i in range(n // 2)]
    seen, power = [0] * len(sections), []
    for a in axis:   # every axis has the frequencies of a head of its own pairs alone
        power.append((2 * seen[a], 2 * sections[a]))
        seen[a] += 1
    return axis, power


def _plain_norm(s):
    case = s["case"]
    n = case["n_rot"]
    axis, power = _axes_of(case)
    theta = torch.tensor([case["base"] ** (-a / b) for a, b in power], dtype=torch.float64, device="cuda")
    pos = s["pos"].reshape(-1, case["tokens"])[torch.tensor(axis, device="cuda")]
    angle = pos.T.double() * theta
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def side(x, weight):
        f = x.float()
        if weight is not None:
            f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + s["eps"]) * weight.float()
        a, b = (f[..., :n // 2], f[..., n // 2:n]) if case["layout"] == "half" else (f[..., 0:n:2], f[..., 1:n:2])
        u, w = a * cos - b * sin, a * sin + b * cos
        y = torch.cat((u, w), -1) if case["layout"] == "half" else torch.stack((u, w), -1).flatten(-2)
        return torch.cat((y, f[..., n:]), -1).half()

    return {"q": side(s["q"], s["q_weight"]), "k": side(s["k"], s["k_weight"])}


def _plan_of(tables, lens, block):
    at = torch.arange(tables.shape[1] * block, device="cuda")
    cells = tables.repeat_interleave(block, dim=1) * block + (at % block).to(torch.int32)
    return torch.where(at < lens[:, None], cells, -1)


def _plain_maps(s):
    case = s["case"]
    block, tables = case["block"], s["tables"]
    lens, new = s["lens"].long(), s["new"].long()
    held = (lens + block - 1) // block
    need = (lens + new + block - 1) // block - held
    taken = need.cumsum(0)
    served = (need == 0) | (taken <= s["n_free"])
    e = torch.arange(tables.shape[1], device="cuda")
    fresh = served[:, None] & (e >= held[:, None]) & (e < (held + need)[:, None])
    number = torch.where(fresh, (taken - need)[:, None] + e - held[:, None], 0)
    tables = torch.where(fresh, s["free"][s["n_free"] - 1 - number], tables)
    s["tables"].copy_(tables)
    after = torch.where(served, lens + new, lens)
    offsets = torch.cat((torch.zeros_like(lens[:1]), new.cumsum(0)))
    t = torch.arange(s["n_tok"], device="cuda")
    seq = torch.searchsorted(offsets[1:], t, right=True).clamp(max=case["seqs"] - 1)
    token = t < offsets[-1]
    pos = torch.where(token, lens[seq] + t - offsets[seq], 0)
    slots = torch.where(token & served[seq], tables[seq, pos // block].long() * block + pos % block, -1)
    plan = _plan_of(tables, after, block)
    if not case["whole"]:
        at = torch.arange(plan.shape[1], device="cuda")
        fresh = (at >= lens[:, None]) & (at < after[:, None])
        plan = torch.where(fresh, plan, s["plan"])
    s["plan"].copy_(plan)
    return {"tables": s["tables"], "n_free": (s["n_free"][0] - torch.where(served, taken, 0).max()).to(torch.int32),
            "offsets": offsets.to(torch.int32), "seq_lens": after.to(torch.int32), "positions": pos.to(torch.int32),
            "slots": slots.to(torch.int32), "plan": s["plan"]}


def _values(rows, scales, bits):
    """Stored rows as the 32-bit values they stand for."""
    if bits == 16:
        return rows.float()
    if bits == 8:
        codes = rows.float().unflatten(-1, (-1, SCALE_GROUP))
    else:
        b = rows.unflatten(-1, (-1, SCALE_GROUP // 2))
        codes = torch.cat((b & 15, b >> 4), -1).float() - 8.0
    return (codes * scales.float()[..., None]).flatten(-2)


def _cells_at(s, at, valid):
    """K and V in 32 bits at the logical places at [S][n], and which of them are cells."""
    kb, vb = BITS[s["case"]["kind"]]
    k, v, ks, vs = s["cache"]
    if s["plan"] is None:
        cells = torch.arange(len(s["lens"]), device="cuda")[:, None] * s["n_cells"] + at
    else:
        cells = s["plan"].long().gather(1, at.clamp(max=s["plan"].shape[1] - 1))
        valid = valid & (cells >= 0)
    cells = torch.where(valid, cells, 0)
    return (_values(k[cells], None if ks is None else ks[cells], kb),
            _values(v[cells], None if vs is None else vs[cells], vb), valid)


def _scores(q, k, heads, kv_heads):
    """q [S][T][H][D], k [S][L][Hk][D] -> [S][Hk][G][T][L]."""
    S, T, _, D = q.shape
    G = heads // kv_heads
    rows = q.view(S, T, kv_heads, G, D).permute(0, 2, 3, 1, 4).reshape(S, kv_heads, G * T, D)
    x = torch.matmul(rows, k.permute(0, 2, 3, 1)).view(S, kv_heads, G, T, k.shape[1])
    x *= 1.0 / math.sqrt(D)
    return x


def _weighted(p, v):
    """p [S][Hk][G][T][L], v [S][L][Hk][D] -> [S][Hk][G][T][D]."""
    S, Hk, G, T, L = p.shape
    return torch.matmul(p.view(S, Hk, G * T, L), v.transpose(1, 2)).view(S, Hk, G, T, -1)


def _by_token(x):
    """[S][Hk][G][T][..] -> [S][T][H][..]"""
    return x.permute(0, 3, 1, 2, 4).flatten(2, 3)


def _pack_index(offsets, lens, top):
    """Padded places of packed rows: (sequence, place) of every token, and every place's token."""
    t = torch.arange(sum(lens), device="cuda")
    seq = torch.searchsorted(offsets[1:].long(), t, right=True)
    place = t - offsets.long()[seq]
    pad = (offsets.long()[:-1, None] + torch.arange(top, device="cuda")[None, :]).clamp(max=max(sum(lens) - 1, 0))
    return seq, place, pad


def _attend(q, k, v, seen, heads, kv_heads):
    """seen [S][T][L].  Returns out [S][T][H][D] and lse [S][T][H]."""
    x = _scores(q, k, heads, kv_heads)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    some = top > -math.inf
    x -= torch.where(some, top, 0.0)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    lse = torch.where(some, top + total.log(), -math.inf)
    return _by_token(_weighted(x, v) / torch.where(some, total, 1.0)), _by_token(lse)[..., 0]


def _plain_window(s):
    case, new = s["case"], s["new"]
    W, K, H, Hk = case["window"], case["sinks"], case["heads"], case["kv_heads"]
    most = max(new)
    seq, place, pad = _pack_index(s["offsets"], new, most)
    t = torch.arange(most, device="cuda")
    if case["form"] == "prompt":
        n = (s["offsets"][1:] - s["offsets"][:-1]).long()[:, None, None]
        lim = (t + 1)[None, :, None]
        at = t[None, None, :]
        seen = (at < lim) & ((at < K) | (at >= lim - W)) & (at < n)
        k, v = s["k"].float()[pad], s["v"].float()[pad]
    else:
        # the cells that any of a sequence's tokens sees: the first ones and a stretch at the end
        n, n_new = s["seq_lens"].long()[:, None], _device_ints(new).long()[:, None]
        front = torch.arange(min(K, max(s["lens"])), device="cuda")[None, :].expand(len(new), -1)
        low = (n - n_new + 1 - W).clamp(min=K)
        back = low + torch.arange(min(W + most - 1, max(s["lens"])), device="cuda")[None, :]
        at = torch.cat((front, back), 1)
        k, v, valid = _cells_at(s, at, at < n)
        lim = (n - n_new + 1 + t)[:, :, None]
        at = at[:, None, :]
        seen = (at < lim) & ((at < K) | (at >= lim - W)) & valid[:, None, :]
    out, lse = _attend(s["q"].float()[pad], k, v, seen, H, Hk)
    out, lse = out[seq, place].half(), lse[seq, place]
    return {"out": out} if s["lse"] is None else {"out": out, "lse": lse}


def _plain_shared(s):
    """The prefix once for all rows, each sequence's rest for its own, joined by their maxima and sums."""
    case, new = s["case"], s["new"]
    P, H, Hk = case["prefix"], case["heads"], case["kv_heads"]
    most = max(new)
    seq, place, pad = _pack_index(s["offsets"], new, most)
    kp, vp, there = _prefix_cells(s, P)
    xp = _scores(s["q"].float()[None], kp, H, Hk)
    xp.masked_fill_(~there[:, None, None, None, :], -math.inf)
    n, n_new = s["seq_lens"].long()[:, None], _device_ints(new).long()[:, None]
    at = P + torch.arange(max(s["lens"]) - P, device="cuda")[None, :].expand(len(new), -1)
    ko, vo, valid = _cells_at(s, at, at < n)
    lim = (n - n_new + 1 + torch.arange(most, device="cuda"))[:, :, None]
    xo = _scores(s["q"].float()[pad], ko, H, Hk)
    xo.masked_fill_(~((at[:, None, :] < lim) & valid[:, None, :])[:, None, None], -math.inf)
    pack = lambda x: _by_token(x)[seq, place]   # of padded rows
    top_p = _by_token(xp.amax(-1, keepdim=True))[0]
    top = torch.maximum(top_p, pack(xo.amax(-1, keepdim=True)))
    some = top > -math.inf
    top = torch.where(some, top, 0.0)
    G = H // Hk
    xp -= top.view(-1, Hk, G).permute(1, 2, 0)[None, ..., None]
    xp.exp_()
    xo -= top[pad].view(len(new), most, Hk, G).permute(0, 2, 3, 1)[..., None]
    xo.exp_()
    total = _by_token(xp.sum(-1, keepdim=True))[0] + pack(xo.sum(-1, keepdim=True))
    out = _by_token(_weighted(xp, vp))[0] + pack(_weighted(xo, vo))
    out = (out / torch.where(some, total, 1.0)).half()
    lse = torch.where(some, top + total.log(), -math.inf)[..., 0]
    return {"out": out} if s["lse"] is None else {"out": out, "lse": lse}


def _prefix_cells(s, P):
    """K and V of the first sequence's first P places, [1][P], and which of them are cells."""
    kb, vb = BITS[s["case"]["kind"]]
    k, v, ks, vs = s["cache"]
    cells = torch.arange(P, device="cuda")[None, :] if s["plan"] is None else s["plan"][:1, :P].long()
    at = cells.clamp(min=0)
    return (_values(k[at], None if ks is None else ks[at], kb), _values(v[at], None if vs is None else vs[at], vb),
            cells >= 0)


PLAIN = {"norm": _plain_norm, "maps": _plain_maps, "window": _plain_window, "shared": _plain_shared}


# ------------------------------- the library's own operators -------------------------------

def _own(s):
    from kv_cache_decode_02_gb300 import kvattn
    case = s["case"]
    op = case["op"]
    if op == "norm":
        if case["norm"] == "none":
            q, k = kvattn.rope(s["q"], s["k"], s["pos"], s["table"], layout=case["layout"], q_out=s["q_out"], k_out=s["k_out"])
        else:
            q, k = kvattn.norm_rope(s["q"], s["k"], s["pos"], s["table"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                    eps=s["eps"], layout=case["layout"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    if op == "maps":
        m = kvattn.step_maps(s["lens"], s["new"], s["tables"], s["free"], s["n_free"], block_cells=case["block"],
                             n_cells=s["n_cells"], plan=s["plan"], whole_plan=case["whole"], out=s["out"])
        return {"tables": s["tables"], "n_free": m.n_free[0], "offsets": m.offsets, "seq_lens": m.seq_lens,
                "positions": m.positions, "slots": m.slots, "plan": s["plan"]}
    if case.get("form") == "prompt":
        out, lse = kvattn.prefill(s["q"], s["k"], s["v"], s["offsets"], window=case["window"], sinks=case["sinks"],
                                  out=s["out"], lse=s["lse"], ws=s["ws"])
    else:
        k, v, ks, vs = s["cache"]
        how = {"shared": case["prefix"]} if op == "shared" else {"window": case["window"], "sinks": case["sinks"]}
        out, lse = kvattn.prefill_chunk(s["q"], s["offsets"], k, v, s["seq_lens"], max_len=max(s["lens"]),
                                        n_cells=s["n_cells"], cell_plan=s["plan"], k_scales=ks, v_scales=vs, out=s["out"],
                                        lse=s["lse"], ws=s["ws"], **how)
    return {"out": out} if lse is None else {"out": out, "lse": lse}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------- what a pass has to do ----------------------------------

def _row_bytes(bits, heads, dim):
    return heads * dim * bits // 8 + (0 if bits == 16 else heads * dim // SCALE_GROUP * 2)


def _seen(lim, window, sinks):
    """Cells that a token sees, of lim in front of its end."""
    return min(lim, window) + max(min(sinks, lim - window), 0)


def work(case):
    op = case["op"]
    if op == "maps":
        # (lengths are spread evenly over their logarithm)
        mean = lambda hi: 1.0 if hi == 1 else (hi - 1) / math.log(hi)
        S, new, held = case["seqs"], mean(case["new"]), mean(case["most"])
        plan = S * (-(-(case["most"] + case["new"]) // case["block"])) * case["block"] if case["whole"] else S * new
        blocks = S * held / case["block"] if case["whole"] else S
        return {"bytes": int(4 * (plan + blocks + 2 * S * case["new"] + 5 * S)), "flops": int(S * new + plan)}
    D, H, Hk = case["dim"], case["heads"], case["kv_heads"]
    if op == "norm":
        T = case["tokens"]
        axes = len(_ints(case["sections"]))
        normed = {"both": H + Hk, "q": H, "k": Hk, "none": 0}[case["norm"]]
        return {"bytes": T * ((H + Hk) * D * 2 * 2 + 4 * axes), "flops": T * ((H + Hk) * case["n_rot"] * 3 + normed * D * 4)}
    lens = _ints(case["lens"])
    if case.get("form") == "prompt":
        pairs = sum(_seen(i + 1, case["window"], case["sinks"]) for n in lens for i in range(n))
        return {"bytes": sum(lens) * ((2 * H + 2 * Hk) * D * 2 + H * 4), "flops": 4 * D * H * pairs}
    new, full = _ints(case["tokens"]), 1.0 - case["holes"]
    if op == "shared":
        P = case["prefix"]
        pairs = sum(t * (P + n - t) * full + t * (t + 1) // 2 for t, n in zip(new, lens))
        cells = P * full + sum(t + (n - t) * full for t, n in zip(new, lens))
        listed_cells = P + sum(lens)
    else:
        W, K = case["window"], case["sinks"]
        pairs = sum(_seen(n - t + 1 + i, W, K) * full for t, n in zip(new, lens) for i in range(t))
        each = [min(n, W + t - 1 + max(min(K, n - W - t + 1), 0)) for t, n in zip(new, lens)]
        cells, listed_cells = sum(each) * full, sum(each)
    kb, vb = BITS[case["kind"]]
    rows = _row_bytes(kb, Hk, D) + _row_bytes(vb, Hk, D)
    plan = 4 * listed_cells if case["plan"] else 0
    row = 2 * H * D * 2 + (H * 4 if case["kind"] == "f16" else 0)
    return {"bytes": int(cells * rows + plan + sum(new) * row), "flops": int(4 * D * H * pairs)}


# ------------------------------ the definitions in 64 bits ------------------------------

def _exact_norm(s):
    case = s["case"]
    n, T = case["n_rot"], case["tokens"]
    sections = _ints(case["sections"])
    # pairs in the order in which axes get them: blocks, or (round, axis) of a deal
    owner = sorted((((0, a, i) if case["order"] == "blocks" else (i, a, 0)), a, i)
                   for a, count in enumerate(sections) for i in range(count))
    pos = s["pos"].view(len(sections), T).double()
    turn = torch.empty((T, n // 2), dtype=torch.complex128, device="cuda")
    for pair, (_, a, i) in enumerate(owner):
        share = i / sections[a] if case["restart"] else 2.0 * pair / n
        angle = pos[a] * math.exp(-share * math.log(case["base"]))
        turn[:, pair] = torch.complex(torch.cos(angle), torch.sin(angle))
    pair = torch.arange(n // 2, device="cuda")
    first, second = (pair, pair + n // 2) if case["layout"] == "half" else (2 * pair, 2 * pair + 1)
    out = {}
    for name in ("q", "k"):
        y = s[name].double()
        weight = s[name + "_weight"]
        if weight is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + s["eps"]) * weight.double()
        else:
            y = y.clone()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _exact_maps(s):
    """Sequence by sequence on the host."""
    case = s["case"]
    block = case["block"]
    tables, plan = s["tables"].tolist(), s["plan"].cpu()
    free = s["free"].tolist()
    have = asked = int(s["n_free"])
    offsets, after, positions, slots = [0], [], [], []
    for i, (n, t) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        need = -(-(n + t) // block) - -(-n // block)
        asked -= need
        good = need == 0 or asked >= 0
        if good:
            for e in range(need):
                tables[i][-(-n // block) + e] = free[asked + need - 1 - e]
            have = min(have, asked) if need else have
        cell = lambda c: tables[i][c // block] * block + c % block
        offsets.append(offsets[-1] + t)
        after.append(n + t if good else n)
        positions += range(n, n + t)
        slots += [cell(c) if good else -1 for c in range(n, n + t)]
        if case["whole"]:
            plan[i] = -1
            row = torch.tensor(tables[i])[:, None] * block + torch.arange(block)
            plan[i, :after[-1]] = row.flatten()[:after[-1]].to(torch.int32)
        else:
            plan[i, n:after[-1]] = torch.tensor([cell(c) for c in range(n, after[-1])], dtype=torch.int32)
    behind = s["n_tok"] - offsets[-1]
    positions += [0] * behind
    slots += [-1] * behind
    return {"tables": _device_ints(tables), "n_free": torch.tensor(have, dtype=torch.int32, device="cuda"),
            "offsets": _device_ints(offsets), "seq_lens": _device_ints(after), "positions": _device_ints(positions),
            "slots": _device_ints(slots), "plan": plan.to("cuda")}


def _exact_values(rows, scales, bits, index):
    """Stored rows at `index` in 64 bits, element by element from the format."""
    if bits == 16:
        return rows[index].double()
    d = scales[index].double().repeat_interleave(SCALE_GROUP, dim=-1)
    if bits == 8:
        return rows[index].double() * d
    e = torch.arange(rows.shape[-1] * 2, device=rows.device)
    byte = (e // SCALE_GROUP) * 16 + e % 16
    nibble = (rows[index][..., byte].int() >> ((e % SCALE_GROUP) // 16 * 4).int()) & 15
    return (nibble - 8).double() * d


def _exact_rows(q, k, v, ok):
    """q [R][D], k and v [L][D], ok [R][L]."""
    x = torch.where(ok, (q @ k.T) / math.sqrt(q.shape[1]), -math.inf)
    lse = torch.logsumexp(x, 1)
    p = torch.where(ok, torch.exp(x - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[:, None]), 0.0)
    return p @ v, lse


def _exact_attention(s):
    case = s["case"]
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G, T = H // Hk, sum(s["new"])
    window = case.get("window", 1 << 40)
    sinks = case.get("sinks", 0)
    out = torch.empty((T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((T, H), dtype=torch.float64, device="cuda")
    start = 0
    for i, (t, n) in enumerate(zip(s["new"], s["lens"])):
        for t0 in range(0, t, 1024):   # (so that long prompts need not hold all scores at once)
            t1 = min(t0 + 1024, t)
            lo, hi = max(n - t + t0 + 1 - window, 0), n - t + t1
            at = torch.arange(lo, hi, device="cuda")
            if lo > 0 and sinks > 0:
                at = torch.cat((torch.arange(min(sinks, lo), device="cuda"), at))
            seen = torch.ones_like(at, dtype=torch.bool)
            cells = at
            if case.get("form") == "prompt":
                cells = at + start
            elif s["plan"] is None:
                cells = at + i * s["n_cells"]
            else:
                cells = s["plan"][i].long()[at]
                seen, cells = cells >= 0, cells.clamp(min=0)
            end = (torch.arange(t0, t1, device="cuda") + n - t).repeat_interleave(G)[:, None]   # its own cell
            ok = seen & (at <= end) & ((at > end - window) | (at < sinks))
            for h in range(Hk):
                if case.get("form") == "prompt":
                    k, v = s["k"][cells, h].double(), s["v"][cells, h].double()
                else:
                    kb, vb = BITS[case["kind"]]
                    ck, cv, ks, vs = s["cache"]
                    k = _exact_values(ck[:, h], None if ks is None else ks[:, h], kb, cells)
                    v = _exact_values(cv[:, h], None if vs is None else vs[:, h], vb, cells)
                rows = slice(start + t0, start + t1)
                q = s["q"][rows, h * G:(h + 1) * G].double().reshape(-1, D)
                o, l = _exact_rows(q, k, v, ok)
                out[rows, h * G:(h + 1) * G] = o.view(t1 - t0, G, D)
                lse[rows, h * G:(h + 1) * G] = l.view(t1 - t0, G)
        start += t
    return {"out": out} if s["lse"] is None else {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "maps": _exact_maps}.get(case["op"], _exact_attention)(s)
