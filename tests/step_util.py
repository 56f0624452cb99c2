"""Plain 64-bit forms of a serving step's operators for the tests, with the tolerances that the kernels'
roundings allow.  Nothing here calls the library."""
import math

import torch

from tests import prompt_util as U


def attend(q, k, v, ok, scale, rounded=False):
    """prompt_util.attend with any mask: row t of ok [n][cells] says what token t sees."""
    n, H, D = q.shape
    G = H // k.shape[1]
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    some = ok.any(1)
    for h in range(H):
        kk, vv = k[:, h // G], v[:, h // G]
        x = torch.where(ok, scale * (q[:, h].double() @ kk.T), -math.inf)
        l = torch.logsumexp(x, 1)
        p = torch.where(ok, torch.exp(x - torch.where(some, l, 0.0)[:, None]), 0.0)
        wild = ~torch.isfinite(vv)     # these reach the rows that see them, and no others
        pure = torch.where(wild, 0.0, vv)
        o = p @ pure
        for c in wild.any(1).nonzero().flatten().tolist():
            o = torch.where(ok[:, c, None] & wild[c], o + vv[c], o)
        # as there: a score's products and sums of D terms in fp32, K of a quantised cache rounded to
        # half; p, V of a quantised cache and the result rounded to half
        mag = abs(scale) * (q[:, h].double().abs() @ torch.where(torch.isfinite(kk), kk, 0.0).abs().T)
        es = torch.where(ok, mag, 0.0) * ((U.HALF if rounded else 0.0) + 2.0 ** -18) + 2.0 ** -20
        worst = es.max(1).values if es.shape[1] else torch.zeros(n, dtype=torch.float64, device=q.device)
        a = p @ pure.abs()
        tol_o[:, h] = a * (U.HALF * (2 if rounded else 1) + 2.0 ** -18) + 2 * worst[:, None] * a + o.abs() * U.HALF + U.HALF_MIN
        tol_l[:, h] = worst + 2.0 ** -20 * (1 + torch.where(some, l, 0.0).abs())
        out[:, h], lse[:, h] = torch.where(some[:, None], o, 0.0), torch.where(some, l, -math.inf)
    return out, lse, tol_o, tol_l


def window_mask(lim, cells, window, sinks):
    """[tokens][cells]: what tokens of limits `lim` see of the logical places 0 .. cells - 1."""
    at = torch.arange(cells, device=lim.device)[None, :]
    return (at < lim[:, None]) & ((at < sinks) | (at >= lim[:, None] - window))


def rows_of(c, s):
    """Of sequence s of a chunk (test_gpu_prefill.make_chunk): K and V of its logical places in 64 bits,
    and which of those are cells."""
    L, D = c["L"][s], c["D"]
    if c["plan"] is None:
        cells, there = s * c["n_cells"] + torch.arange(L, device="cuda"), torch.ones(L, dtype=torch.bool, device="cuda")
    else:
        row = c["plan"][s, :L].long()
        there, cells = row >= 0, row.clamp(min=0)
    k = U.dequant(c["k"][cells], None if c["ks"] is None else c["ks"][cells], D)
    v = U.dequant(c["v"][cells], None if c["vs"] is None else c["vs"][cells], D)
    return torch.where(there[:, None, None], k, 0.0), torch.where(there[:, None, None], v, 0.0), there


def check_chunk(c, out, lse, window=None, sinks=0, scale=None):
    """Every sequence of a chunk's result against the definition."""
    a = 0
    for s, (n, L) in enumerate(zip(c["new"], c["L"])):
        if n:
            k, v, there = rows_of(c, s)
            lim = torch.arange(n, device="cuda") + L - n + 1
            ok = window_mask(lim, L, L + n + 1 if window is None else window, sinks) & there
            o, l, to, tl = attend(c["q"][a:a + n], k, v, ok, 1.0 / math.sqrt(c["D"]) if scale is None else scale, c["ks"] is not None)
            U.check(out[a:a + n], o, to, f"out of sequence {s}")
            if lse is not None:
                U.check(lse[a:a + n], l, tl, f"lse of sequence {s}")
        a += n


def maps(lens, new, tables, free, n_free, block, n_cells, n_tok, plan=None, whole=True):
    """step_maps on the host, one sequence after the other.  Returns a dict of lists (tables and plan:
    the rows after the step) and the status bits."""
    B, stride = block, len(tables[0]) if tables else 0
    most = min(stride * B, 2 ** 31 - 1 if plan is None else (len(plan[0]) if plan else 0))
    most = min(most, (2 ** 31 - 1) // B * B)
    tables, plan = [list(r) for r in tables], None if plan is None else [list(r) for r in plan]
    count = 0 if free is None else min(max(n_free, 0), len(free))
    asked, left, rows, status = 0, count, 0, 0
    offsets, after, positions, slots = [0], [], [0] * n_tok, [-1] * n_tok
    for s, (n, t) in enumerate(zip(lens, new)):
        n, t = min(max(n, 0), most), max(t, 0)
        fits = t == 0 or (n + t <= most and rows + t <= n_tok)
        need = -(-(n + t) // B) - -(-n // B) if fits and free is not None else 0
        asked += need
        served = fits and (need == 0 or asked <= count)
        if served:
            for j in range(need):
                tables[s][-(-n // B) + j] = free[count - 1 - (asked - need + j)]
            if need:
                left = count - asked
        else:
            status |= 4
        end = n + t if served else n

        def cell(i, s=s):
            nonlocal status
            b = tables[s][i // B]
            if b < 0 or (b + 1) * B > n_cells:
                status |= 2
                return -1
            return b * B + i % B
        for i in range(min(t, max(n_tok - rows, 0))):   # (the others have no rows)
            positions[rows + i] = min(n + i, 2 ** 31 - 1)
            slots[rows + i] = cell(n + i) if served else -1
        if plan is not None:
            if whole:
                plan[s] = [cell(i) if i < end else -1 for i in range(len(plan[s]))]
            elif served:
                for i in range(n, end):
                    plan[s][i] = cell(i)
        rows += t
        offsets.append(min(rows, n_tok))
        after.append(end)
    return {"tables": tables, "plan": plan, "offsets": offsets, "seq_lens": after, "positions": positions, "slots": slots,
            "n_free": left}, status
