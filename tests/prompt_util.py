"""Plain 64-bit torch forms of the prompt-side operators for the tests, and the tolerances that the
kernels' roundings allow.  Nothing here calls the library."""
import math

import torch

HALF = 2.0 ** -11   # a rounding to f16 is off by at most half a step, 2^-11 of the value
# f16 values below 2^-14 are spaced 2^-24
HALF_MIN = 2.0 ** -25


def dequant(rows, scales, head_dim):
    """Stored rows as float64 values: f16 rows, int8 codes, or packed 4-bit codes (byte j of a
    16-byte block: element j low, element j + 16 high, minus 8)."""
    if scales is None:
        return rows.double()
    if rows.shape[-1] == head_dim:
        codes = rows.double()
    else:
        b = rows.view(*rows.shape[:-1], head_dim // 32, 16).int()
        codes = (torch.cat((b & 15, b >> 4), -1) - 8).double().flatten(-2)
    return codes * scales.double().repeat_interleave(32, -1)


def attend(q, k, v, lim, scale, rounded_k=False):
    """One sequence in 64 bits.  q [n][H][D]; k, v [cells][Hk][D] float64; lim [n]: token t sees the
    cells below lim[t].  Returns out, lse and the kernel's error bounds for both."""
    n, H, D = q.shape
    Hk = k.shape[1]
    G = H // Hk
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    ok = torch.arange(k.shape[0], device=q.device)[None, :] < lim[:, None]
    some = ok.any(1)
    for h in range(H):
        kk, vv = k[:, h // G], v[:, h // G]
        x = scale * (q[:, h].double() @ kk.T)
        x = torch.where(ok, x, -math.inf)
        l = torch.logsumexp(x, 1)
        p = torch.where(ok, torch.exp(x - torch.where(some, l, 0.0)[:, None]), 0.0)
        # elements of V that are not finite reach the rows that see them (any weight there is above
        # zero), and no others: not by way of 0 x inf
        wild = ~torch.isfinite(vv)
        pure = torch.where(wild, 0.0, vv)
        o = p @ pure
        for c in wild.any(1).nonzero().flatten().tolist():
            o = torch.where(ok[:, c, None] & wild[c], o + vv[c], o)
        # each score: fp32 products and sums of D terms, ex2 and its argument in fp32 (2^-18 of
        # the terms' magnitudes covers D / 2 accumulation steps of 2^-24 and the rest); the K of a
        # quantised cache enters rounded to half
        mag = abs(scale) * (q[:, h].double().abs() @ kk.abs().T)
        es = torch.where(ok, mag, 0.0) * ((HALF if rounded_k else 0.0) + 2.0 ** -18) + 2.0 ** -20
        worst = es.max(1).values if es.shape[1] else torch.zeros(n, dtype=torch.float64, device=q.device)
        a = p @ pure.abs()
        # p rounded to half (and V, from a quantised cache), the output rounded to half; a relative
        # error e of every weight moves the quotient by 2 e a at most
        tol_o[:, h] = a * (HALF * (2 if rounded_k else 1) + 2.0 ** -18) + 2 * worst[:, None] * a + o.abs() * HALF + HALF_MIN
        tol_l[:, h] = worst + 2.0 ** -20 * (1 + torch.where(some, l, 0.0).abs())
        out[:, h], lse[:, h] = torch.where(some[:, None], o, 0.0), torch.where(some, l, -math.inf)
    return out, lse, tol_o, tol_l


def check(got, want, tol, what):
    """Every element within its own bound; the same infinities, the same NaN."""
    got = got.double()
    assert got.shape == want.shape, what
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), finite), f"{what}: other places are finite"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: other places are NaN"
    assert torch.equal(got[~finite & ~torch.isnan(want)], want[~finite & ~torch.isnan(want)]), what
    if finite.any():
        over = (got - want).abs()[finite] - tol[finite]
        i = int(over.argmax())
        assert over[i] <= 0, (f"{what}: off by {(got - want).abs()[finite][i]:.3e}, allowed {tol[finite][i]:.3e} "
                              f"({int((over > 0).sum())} of {over.numel()} values)")


def offsets_of(lens, first=0):
    off = [first]
    for n in lens:
        off.append(off[-1] + n)
    return off


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def halves(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).half()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cache_planes(g, kind, cells, Hk, D):
    """Random planes of a cache: (k, v, k_scales, v_scales)."""
    def side(bits):
        if bits == 16:
            return halves(g, cells, Hk, D), None
        d = (torch.rand(cells, Hk, D // 32, generator=g, device="cuda") * (0.02 if bits == 8 else 0.3) + 0.001).half()
        if bits == 8:
            return torch.randint(-127, 128, (cells, Hk, D), generator=g, device="cuda", dtype=torch.int8), d
        return torch.randint(0, 256, (cells, Hk, D // 2), generator=g, device="cuda", dtype=torch.uint8), d
    kb, vb = {"f16": (16, 16), "q8_0": (8, 8), "q8_0_q4_0": (8, 4), "q4_0": (4, 4)}[kind]
    k, ks = side(kb)
    v, vs = side(vb)
    return k, v, ks, vs
