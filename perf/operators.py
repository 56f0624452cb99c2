"""Timed cases of the prompt-side operators: rotary positions, the cache written in its stored type
and read back, attention over whole packed prompts, and attention of chunks of new tokens over a
cache that already holds them.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, angles in 64) or,
with ``own`` set, through the library's entry points; ``exact`` says what the definition gives in 64
bits.  A case is a dict of plain values; lengths are texts such as "8192,20480".

    rope     q, k half [T][heads][D] rotated to their positions
    store    k, v half [T][Hk][D] written to cache cells in the stored type, then read back
    load     cache cells read back as half rows (holes give zero rows)
    prefill  causal attention of packed sequences over their own keys and values
    chunk    causal attention of each sequence's new tokens over its cache (their own cells are in it)
"""
import math

import torch

own = False

SCALE_GROUP = 32  # elements that share one scale in a quantised cache row
BITS = {"f16": (16, 16), "q8_0": (8, 8), "q8_0_q4_0": (8, 4), "q4_0": (4, 4)}
KINDS = tuple(BITS)
# One pass of the largest listed case costs about this much; no drawn case costs more.
MOST_FLOPS = 5.0e11
MOST_SCORES = 2.5e9


# --------------------------------------- cases ---------------------------------------

def listed():
    return [
        # a decode step's new tokens of 64 sequences, far along in their contexts
        {"name": "rope step", "op": "rope", "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128, "n_rot": 128,
         "layout": "half", "scaling": "none", "factor": 1.0, "base": 1000000.0, "original": 32768, "far": 131072},
        # a prompt of a wide-headed model, a quarter of each head rotated, context stretched eight times
        {"name": "rope prompt", "op": "rope", "tokens": 16384, "heads": 16, "kv_heads": 8, "dim": 256, "n_rot": 64,
         "layout": "interleaved", "scaling": "yarn", "factor": 8.0, "base": 10000.0, "original": 4096, "far": 32768},
        # the same decode step's keys and values entering an 8-bit cache
        {"name": "store step q8", "op": "store", "kind": "q8_0", "tokens": 64, "cells": 65536, "kv_heads": 8, "dim": 128},
        # a long prompt entering a cache of 8-bit keys and 4-bit values
        {"name": "store prompt q8q4", "op": "store", "kind": "q8_0_q4_0", "tokens": 16384, "cells": 65536, "kv_heads": 8,
         "dim": 128},
        # one slot's cells through its plan, a tenth of them holes
        {"name": "load slot q4", "op": "load", "kind": "q4_0", "tokens": 8192, "cells": 147456, "kv_heads": 8, "dim": 128,
         "holes": 0.1},
        # a whole 8-bit long-context cache of the wide heads turned back into half rows
        {"name": "load cache q8", "op": "load", "kind": "q8_0", "tokens": 131072, "cells": 131072, "kv_heads": 8, "dim": 256,
         "holes": 0.0},
        # a few short questions, packed
        {"name": "prefill short", "op": "prefill", "lens": "37,128,1,260,95", "heads": 32, "kv_heads": 8, "dim": 128},
        # one long prompt of the 32 / 8 head layer
        {"name": "prefill long", "op": "prefill", "lens": "8192", "heads": 32, "kv_heads": 8, "dim": 128},
        # ragged prompts of the 256-wide heads
        {"name": "prefill ragged d256", "op": "prefill", "lens": "2049,513,3000,77,1023", "heads": 16, "kv_heads": 8, "dim": 256},
        # a chunk of a prompt after 16384 cells of it, one sequence in its own cache
        {"name": "chunk f16", "op": "chunk", "kind": "f16", "tokens": "512", "lens": "16384", "heads": 32, "kv_heads": 8,
         "dim": 128, "plan": False, "holes": 0.0},
        # four slots of a unified cache at once: chunks of different sizes, one of them a single token
        {"name": "chunk plan gqa6", "op": "chunk", "kind": "f16", "tokens": "256,128,1,64", "lens": "8192,20480,40960,65536",
         "heads": 48, "kv_heads": 8, "dim": 128, "plan": True, "holes": 0.1},
        # a short turn after a very long 8-bit context
        {"name": "chunk q8 long", "op": "chunk", "kind": "q8_0", "tokens": "100", "lens": "131072", "heads": 32, "kv_heads": 8,
         "dim": 128, "plan": False, "holes": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 3, 4, 6, 8]), kv


def draw(rng):
    op = rng.choice(["rope", "store", "load", "prefill", "prefill", "chunk", "chunk", "chunk"])
    dim = rng.choice([128, 256])
    if op == "rope":
        heads, kv = _draw_heads(rng)
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "heads": heads, "kv_heads": kv, "dim": dim,
                "n_rot": 16 * rng.randint(1, dim // 16), "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "yarn"]), "factor": rng.choice([2.0, 4.0, 8.0]),
                "base": rng.choice([10000.0, 500000.0, 1000000.0]), "original": rng.choice([4096, 32768]),
                "far": _log_int(rng, 16, 262144)}
    if op == "store":
        tokens = _log_int(rng, 1, 16384)
        return {"op": op, "kind": rng.choice(KINDS), "tokens": tokens, "cells": _log_int(rng, tokens, 65536),
                "kv_heads": rng.choice([1, 2, 3, 4, 8]), "dim": dim}
    if op == "load":
        tokens = _log_int(rng, 1, 65536)
        return {"op": op, "kind": rng.choice(KINDS), "tokens": tokens, "cells": _log_int(rng, 65536, 131072),
                "kv_heads": rng.choice([1, 2, 3, 4, 8]), "dim": dim, "holes": rng.choice([0.0, 0.1, 0.5])}
    while True:
        heads, kv = _draw_heads(rng)
        n_seq = _log_int(rng, 1, 12)
        c = {"op": op, "heads": heads, "kv_heads": kv, "dim": dim}
        if op == "prefill":
            top = _log_int(rng, 1, 8192)
            c["lens"] = ",".join(str(_log_int(rng, 1, top)) for _ in range(n_seq))
            if sum(_ints(c["lens"])) < 16:
                continue
            scores = n_seq * max(_ints(c["lens"])) ** 2 * heads
        else:
            plan = rng.random() < 0.5
            new = [_log_int(rng, 1, 512) for _ in range(n_seq)]
            top = _log_int(rng, 512, 131072)
            lens = [n + _log_int(rng, 1, top) - 1 for n in new]
            c |= {"kind": rng.choice(KINDS), "tokens": ",".join(map(str, new)), "lens": ",".join(map(str, lens)),
                  "plan": plan, "holes": rng.choice([0.0, 0.1]) if plan else 0.0}
            scores = n_seq * max(new) * max(lens) * heads
            if n_seq * max(lens) * kv * dim > 3e8:
                continue
        if work(c)["flops"] <= MOST_FLOPS and scores <= MOST_SCORES:
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
            return _normal(g, cells, kv_heads, dim), None
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


def _empty_planes(kind, cells, kv_heads, dim):
    def side(bits):
        if bits == 16:
            return torch.zeros((cells, kv_heads, dim), device="cuda", dtype=torch.float16), None
        rows = torch.zeros((cells, kv_heads, dim * bits // 8), device="cuda", dtype=torch.int8 if bits == 8 else torch.uint8)
        return rows, torch.zeros((cells, kv_heads, dim // SCALE_GROUP), device="cuda", dtype=torch.float16)
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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    D, Hk = case["dim"], case["kv_heads"]
    op = case["op"]
    half = {"dtype": torch.float16, "device": "cuda"}
    if op == "rope":
        T, H = case["tokens"], case["heads"]
        s["q"], s["k"] = _normal(g, T, H, D), _normal(g, T, Hk, D)
        s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"], s["k_out"] = torch.empty((T, H, D), **half), torch.empty((T, Hk, D), **half)
        if own:  # the angle table that a program makes once for its model
            from kv_cache_decode_02_gb300 import kvattn
            s["table"] = kvattn.rope_table(case["n_rot"], base=case["base"], scaling=case["scaling"],
                                           factor=case["factor"], original=case["original"])
    elif op == "store":
        T, cells = case["tokens"], case["cells"]
        s["k"], s["v"] = _normal(g, T, Hk, D), _normal(g, T, Hk, D)
        s["slots"] = torch.randperm(cells, generator=g, device="cuda")[:T].to(torch.int32)
        s["cache"] = _empty_planes(case["kind"], cells, Hk, D)
        s["k_out"], s["v_out"] = torch.empty((T, Hk, D), **half), torch.empty((T, Hk, D), **half)
    elif op == "load":
        T, cells = case["tokens"], case["cells"]
        s["cache"] = _planes(g, case["kind"], cells, Hk, D)
        slots = torch.randperm(cells, generator=g, device="cuda")[:T].sort().values.to(torch.int32)
        hole = torch.rand((T,), generator=g, device="cuda") < case["holes"]
        s["slots"] = torch.where(hole, torch.full_like(slots, -1), slots)
        s["k_out"], s["v_out"] = torch.empty((T, Hk, D), **half), torch.empty((T, Hk, D), **half)
    elif op == "prefill":
        lens, H = _ints(case["lens"]), case["heads"]
        T = sum(lens)
        s["lens"] = lens
        s["q"], s["k"], s["v"] = _normal(g, T, H, D), _normal(g, T, Hk, D), _normal(g, T, Hk, D)
        s["offsets"] = _device_ints(_offsets(lens))
        s["out"] = torch.empty((T, H, D), **half)
        s["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
        if own:  # the workspace that a program allocates once
            from kv_cache_decode_02_gb300 import kvattn
            s["ws"] = kvattn.prefill_workspace(T, len(lens), H, Hk, D)
    else:
        new, lens, H = _ints(case["tokens"]), _ints(case["lens"]), case["heads"]
        T, S, top = sum(new), len(new), max(lens)
        s["new"], s["lens"] = new, lens
        s["q"] = _normal(g, T, H, D)
        s["offsets"], s["seq_lens"] = _device_ints(_offsets(new)), _device_ints(lens)
        s["plan"] = None
        if case["plan"]:
            # every sequence owns records of 128 cells scattered over the pool, ascending, with
            # holes where cells were dropped; the new tokens' own cells are all there
            records = [-(-n // 128) for n in lens]
            pool = sum(records) + 8
            stride = 128 * max(records)
            perm = torch.randperm(pool, generator=g, device="cuda")
            at = torch.arange(stride, device="cuda")
            first = _device_ints(_offsets(records)[:-1]).long()
            count = _device_ints(records).long()
            rec = (at[None, :] // 128).expand(S, -1)
            ids = torch.where(rec < count[:, None], perm[(first[:, None] + rec).clamp(max=pool - 1)], pool)
            ids = ids.view(S, -1, 128)[:, :, 0].sort(dim=1).values.repeat_interleave(128, dim=1)
            n, t = s["seq_lens"].long()[:, None], _device_ints(new).long()[:, None]
            hole = torch.rand((S, stride), generator=g, device="cuda") < case["holes"]
            keep = (at < n) & (~hole | (at >= n - t))
            s["plan"] = torch.where(keep, ids * 128 + at % 128, -1).to(torch.int32)
            cells = pool * 128
            s["cache"] = _planes(g, case["kind"], cells, Hk, D)
        else:
            cells = top  # one cache of this many cells for each sequence
            s["cache"] = _planes(g, case["kind"], S * cells, Hk, D)
        s["n_cells"] = cells
        s["out"] = torch.empty((T, H, D), **half)
        # the log-sum-exp goes to programs that merge this cache's result with another part's;
        # the ones that hold a whole context in a quantised cache take the output alone
        s["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda") if case["kind"] == "f16" else None
        if own:  # the workspace that a program allocates once
            from kv_cache_decode_02_gb300 import kvattn
            s["ws"] = kvattn.prefill_chunk_workspace(T, S, H, Hk, D, top)
    return s


# ------------------------------------- plain forms -------------------------------------

def _angles(case, pos):
    """Angles of each token and pair in 64 bits, and what cosine and sine are multiplied by."""
    i = torch.arange(case["n_rot"] // 2, device=pos.device, dtype=torch.float64)
    theta = case["base"] ** (-2.0 * i / case["n_rot"])
    scale = 1.0
    if case["scaling"] == "linear":
        theta = theta / case["factor"]
    elif case["scaling"] == "yarn":
        turns = case["original"] * theta / (2.0 * math.pi)
        ramp = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        theta = theta / case["factor"] * (1.0 - ramp) + theta * ramp
        scale = 0.1 * math.log(case["factor"]) + 1.0
    return pos.double()[:, None] * theta[None, :], scale


def _rotate(case, x, cos, sin):
    n, f = case["n_rot"], x.float()
    a, b = (f[..., : n // 2], f[..., n // 2: n]) if case["layout"] == "half" else (f[..., 0:n:2], f[..., 1:n:2])
    u, w = a * cos - b * sin, a * sin + b * cos
    y = torch.cat((u, w), -1) if case["layout"] == "half" else torch.stack((u, w), -1).flatten(-2)
    return torch.cat((y, f[..., n:]), -1).half()


def _plain_rope(s):
    case = s["case"]
    angle, scale = _angles(case, s["pos"])
    cos, sin = (angle.cos() * scale).float()[:, None, :], (angle.sin() * scale).float()[:, None, :]
    return {"q": _rotate(case, s["q"], cos, sin), "k": _rotate(case, s["k"], cos, sin)}


def _half_up(x):
    """The magnitude rounded to half precision away from zero (x in 32 bits, sign kept)."""
    h = x.half()
    short = h.float().abs() < x.abs()
    return torch.where(short, h.view(torch.int16) + 1, h.view(torch.int16)).view(torch.float16)


def _quantise(x, bits):
    """Half rows -> (codes as whole 32-bit floats, scales): the stored scale is rounded away from
    zero, so no code leaves its range but the 4-bit +8, which becomes 7."""
    b = x.float().unflatten(-1, (-1, SCALE_GROUP))
    top = b.abs().amax(-1)
    if bits == 8:
        d = _half_up(top / 127.0)
    else:
        at = (b.abs() == top[..., None]).to(torch.int8).argmax(-1, keepdim=True)  # the lowest index
        d = _half_up(b.gather(-1, at)[..., 0] / -8.0)
    f = d.float()[..., None]
    codes = torch.where(f == 0.0, torch.zeros_like(b), torch.round(b / torch.where(f == 0.0, torch.ones_like(f), f)))
    return codes.clamp(max=7.0) if bits == 4 else codes, d


def _store_side(x, bits, rows, scales, slots):
    if bits == 16:
        rows[slots] = x
        return
    codes, d = _quantise(x, bits)
    scales[slots] = d
    if bits == 8:
        rows[slots] = codes.flatten(-2).to(torch.int8)
    else:
        u = (codes + 8.0).to(torch.uint8)
        rows[slots] = (u[..., :16] | (u[..., 16:] << 4)).flatten(-2)


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


def _plain_load(s):
    kb, vb = BITS[s["case"]["kind"]]
    k, v, ks, vs = s["cache"]
    slots = s["slots"].long()
    hole, at = (slots < 0)[:, None, None], slots.clamp(min=0)
    k = _values(k[at], None if ks is None else ks[at], kb).masked_fill(hole, 0.0)
    v = _values(v[at], None if vs is None else vs[at], vb).masked_fill(hole, 0.0)
    return {"k": k.clamp(-65504.0, 65504.0).half(), "v": v.clamp(-65504.0, 65504.0).half()}


def _plain_store(s):
    kb, vb = BITS[s["case"]["kind"]]
    k, v, ks, vs = s["cache"]
    slots = s["slots"].long()
    _store_side(s["k"], kb, k, ks, slots)
    _store_side(s["v"], vb, v, vs, slots)
    return _plain_load(s)


def _attend(q, k, v, visible, valid, heads, kv_heads):
    """q [S][T][H][D], k and v [S][L][Hk][D] in 32 bits; token t of sequence s sees the valid cells
    below visible[s][t].  Returns out [S][T][H][D] and lse [S][T][H]."""
    S, T, _, D = q.shape
    L, G = k.shape[1], heads // kv_heads
    rows = q.view(S, T, kv_heads, G, D).permute(0, 2, 3, 1, 4).reshape(S, kv_heads, G * T, D)
    x = torch.matmul(rows, k.permute(0, 2, 3, 1)).view(S, kv_heads, G, T, L)
    x *= 1.0 / math.sqrt(D)
    seen = (torch.arange(L, device=q.device) < visible[:, :, None]) & valid[:, None, :]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    some = top > -math.inf
    x -= torch.where(some, top, 0.0)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    lse = torch.where(some, top + total.log(), -math.inf)
    o = torch.matmul(x.view(S, kv_heads, G * T, L), v.transpose(1, 2)).view(S, kv_heads, G, T, D)
    o = o / torch.where(some, total, 1.0)
    return o.permute(0, 3, 1, 2, 4).reshape(S, T, heads, D), lse[..., 0].permute(0, 3, 1, 2).reshape(S, T, heads)


def _pack_index(offsets, lens, top):
    """Padded places of packed rows: (sequence, place) of every token, and every place's token."""
    t = torch.arange(sum(lens), device="cuda")
    seq = torch.searchsorted(offsets[1:].long(), t, right=True)
    place = t - offsets.long()[seq]
    pad = (offsets.long()[:-1, None] + torch.arange(top, device="cuda")[None, :]).clamp(max=max(sum(lens) - 1, 0))
    return seq, place, pad


def _plain_prefill(s):
    case, lens = s["case"], s["lens"]
    top = max(lens)
    seq, place, pad = _pack_index(s["offsets"], lens, top)
    at = torch.arange(top, device="cuda")
    valid = at[None, :] < (s["offsets"][1:] - s["offsets"][:-1])[:, None]
    out, lse = _attend(s["q"].float()[pad], s["k"].float()[pad], s["v"].float()[pad], (at + 1).expand(len(lens), -1), valid,
                       case["heads"], case["kv_heads"])
    return {"out": out[seq, place].half(), "lse": lse[seq, place]}


def _plain_chunk(s):
    case, new, lens = s["case"], s["new"], s["lens"]
    kb, vb = BITS[case["kind"]]
    k, v, ks, vs = s["cache"]
    S, most, top = len(new), max(new), max(lens)
    n, n_new = s["seq_lens"].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    at = torch.arange(top, device="cuda")
    if s["plan"] is None:
        cells = torch.arange(S, device="cuda")[:, None] * s["n_cells"] + at
        valid = at < n[:, None]
    else:
        cells = s["plan"][:, :top].long()
        valid = (cells >= 0) & (at < n[:, None])
    cells = torch.where(valid, cells, 0)
    kf = _values(k[cells], None if ks is None else ks[cells], kb)
    vf = _values(v[cells], None if vs is None else vs[cells], vb)
    seq, place, pad = _pack_index(s["offsets"], new, most)
    visible = (n - n_new + 1)[:, None] + torch.arange(most, device="cuda")
    out, lse = _attend(s["q"].float()[pad], kf, vf, visible, valid, case["heads"], case["kv_heads"])
    out, lse = out[seq, place].half(), lse[seq, place]
    return {"out": out} if s["lse"] is None else {"out": out, "lse": lse}


PLAIN = {"rope": _plain_rope, "store": _plain_store, "load": _plain_load, "prefill": _plain_prefill, "chunk": _plain_chunk}


# ------------------------------- the library's own operators -------------------------------

def _own(s):
    from kv_cache_decode_02_gb300 import kvattn
    case = s["case"]
    op = case["op"]
    if op == "rope":
        q, k = kvattn.rope(s["q"], s["k"], s["pos"], s["table"], layout=case["layout"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    if op in ("store", "load"):
        k, v, ks, vs = s["cache"]
        if op == "store":
            kvattn.cache_write(s["k"], s["v"], s["slots"], k, v, k_scales=ks, v_scales=vs)
        k, v = kvattn.cache_read(k, v, s["slots"], head_dim=case["dim"], k_scales=ks, v_scales=vs, k_out=s["k_out"],
                                 v_out=s["v_out"])
        return {"k": k, "v": v}
    if op == "prefill":
        out, lse = kvattn.prefill(s["q"], s["k"], s["v"], s["offsets"], out=s["out"], lse=s["lse"], ws=s["ws"])
    else:
        k, v, ks, vs = s["cache"]
        out, lse = kvattn.prefill_chunk(s["q"], s["offsets"], k, v, s["seq_lens"], max_len=max(s["lens"]),
                                        n_cells=s["n_cells"], cell_plan=s["plan"], k_scales=ks, v_scales=vs, out=s["out"],
                                        lse=s["lse"], ws=s["ws"])
    return {"out": out} if lse is None else {"out": out, "lse": lse}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------- what a pass has to do ----------------------------------

def _row_bytes(bits, heads, dim):
    return heads * dim * bits // 8 + (0 if bits == 16 else heads * dim // SCALE_GROUP * 2)


def work(case):
    op, D, Hk = case["op"], case["dim"], case["kv_heads"]
    if op == "rope":
        T, H = case["tokens"], case["heads"]
        return {"bytes": T * ((H + Hk) * D * 2 * 2 + 4), "flops": T * (H + Hk) * case["n_rot"] * 3}
    if op in ("store", "load"):
        T = case["tokens"]
        kb, vb = BITS[case["kind"]]
        rows, half = _row_bytes(kb, Hk, D) + _row_bytes(vb, Hk, D), 2 * Hk * D * 2
        if op == "load":
            full = T * (1.0 - case["holes"])
            return {"bytes": int(full * rows) + T * (half + 4), "flops": int(full * 2 * Hk * D)}
        return {"bytes": T * (2 * half + 2 * rows + 4), "flops": T * Hk * D * 2 * 4}
    H = case["heads"]
    if op == "prefill":
        lens = _ints(case["lens"])
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * ((2 * H + 2 * Hk) * D * 2 + H * 4), "flops": 4 * D * H * pairs}
    new, lens = _ints(case["tokens"]), _ints(case["lens"])
    full = 1.0 - case["holes"]
    pairs = sum(t * (n - t) * full + t * (t + 1) // 2 for t, n in zip(new, lens))
    kb, vb = BITS[case["kind"]]
    rows = _row_bytes(kb, Hk, D) + _row_bytes(vb, Hk, D)
    cells = sum(t + (n - t) * full for t, n in zip(new, lens))
    plan = 4 * sum(lens) if case["plan"] else 0
    row = 2 * H * D * 2 + (H * 4 if case["kind"] == "f16" else 0)
    return {"bytes": int(cells * rows + plan + sum(new) * row), "flops": int(4 * D * H * pairs)}


# ------------------------------ the definitions in 64 bits ------------------------------

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


def _exact_scale(x):
    """The half-precision number next to x in 64 bits, away from zero."""
    mag = x.abs()
    step = torch.exp2(torch.floor(torch.log2(torch.where(mag > 0, mag, torch.ones_like(mag)))).clamp(min=-14) - 10)
    return torch.sign(x) * torch.ceil(mag / step) * step


def _exact_stored(x, bits):
    """What a row of halves reads back as after it was stored, before the last rounding."""
    if bits == 16:
        return x.double()
    b = x.double().reshape(*x.shape[:-1], -1, SCALE_GROUP)
    if bits == 8:
        d = _exact_scale(b.abs().max(-1).values / 127.0)
        low, high = -127, 127
    else:
        mag = b.abs()
        first = torch.where(mag == mag.max(-1, keepdim=True).values, torch.arange(SCALE_GROUP, device=x.device),
                            SCALE_GROUP).min(-1, keepdim=True).values
        d = _exact_scale(torch.take_along_dim(b, first, -1).squeeze(-1) / -8.0)
        low, high = -8, 7
    d = d[..., None]
    code = torch.where(d != 0, (b / torch.where(d != 0, d, torch.ones_like(d))).round(), torch.zeros_like(b))
    return (code.clamp(low, high) * d).reshape(x.shape)


def _exact_rope(s):
    case = s["case"]
    n = case["n_rot"]
    out = {}
    pair = torch.arange(n // 2, device="cuda")
    first, second = (pair, pair + n // 2) if case["layout"] == "half" else (2 * pair, 2 * pair + 1)
    freq = torch.pow(torch.tensor(case["base"], dtype=torch.float64, device="cuda"), -(2.0 * pair.double()) / n)
    gain = 1.0
    if case["scaling"] == "linear":
        freq = freq / case["factor"]
    if case["scaling"] == "yarn":
        rounds = case["original"] / (2.0 * math.pi / freq)
        keep = torch.clamp((rounds - 1.0) / 31.0, 0.0, 1.0)
        freq = keep * freq + (1.0 - keep) * (freq / case["factor"])
        gain = 1.0 + 0.1 * math.log(case["factor"])
    for name in ("q", "k"):
        y = s[name].double().clone()
        turn = torch.polar(torch.full((y.shape[0], n // 2), gain, dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * freq)
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _exact_attention(q, k, v, limits, seen):
    """One sequence and KV head: q [R][D], k and v [L][D], row r sees the cells below limits[r] that are seen."""
    x = (q @ k.T) / math.sqrt(q.shape[1])
    ok = (torch.arange(k.shape[0], device=q.device)[None, :] < limits[:, None]) & seen[None, :]
    x = torch.where(ok, x, -math.inf)
    lse = torch.logsumexp(x, 1)
    p = torch.where(ok, torch.exp(x - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[:, None]), 0.0)
    return p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op, D, Hk = case["op"], case["dim"], case["kv_heads"]
    if op == "rope":
        return _exact_rope(s)
    if op == "store":
        kb, vb = BITS[case["kind"]]
        return {"k": _exact_stored(s["k"], kb), "v": _exact_stored(s["v"], vb)}
    if op == "load":
        got = {}
        at = s["slots"].long()
        for name, bits, rows, scales in zip("kv", BITS[case["kind"]], s["cache"][:2], s["cache"][2:]):
            x = _exact_values(rows, scales, bits, at.clamp(min=0))
            x[at < 0] = 0.0
            got[name] = x
        return got
    H = case["heads"]
    G = H // Hk
    new = s["lens"] if op == "prefill" else s["new"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((sum(new), H), dtype=torch.float64, device="cuda")
    start = 0
    for i, (t, n) in enumerate(zip(new, s["lens"])):
        if op == "prefill":
            cells = start + torch.arange(n, device="cuda")
            seen = torch.ones(n, dtype=torch.bool, device="cuda")
        elif s["plan"] is None:
            cells = i * s["n_cells"] + torch.arange(n, device="cuda")
            seen = torch.ones(n, dtype=torch.bool, device="cuda")
        else:
            cells = s["plan"][i, :n].long()
            seen, cells = cells >= 0, cells.clamp(min=0)
        limits = (torch.arange(t, device="cuda") + n - t + 1).repeat_interleave(G)
        for h in range(Hk):
            if op == "prefill":
                k, v = s["k"][cells, h].double(), s["v"][cells, h].double()
            else:
                kb, vb = BITS[case["kind"]]
                ck, cv, ks, vs = s["cache"]
                k = _exact_values(ck[:, h], None if ks is None else ks[:, h], kb, cells)
                v = _exact_values(cv[:, h], None if vs is None else vs[:, h], vb, cells)
            q = s["q"][start:start + t, h * G:(h + 1) * G].double().reshape(t * G, D)
            o, l = _exact_attention(q, k, v, limits, seen)
            out[start:start + t, h * G:(h + 1) * G] = o.view(t, G, D)
            lse[start:start + t, h * G:(h + 1) * G] = l.view(t, G)
        start += t
    return {"out": out} if s["lse"] is None else {"out": out, "lse": lse}
