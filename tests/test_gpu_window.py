"""Attention with a sliding window and first tokens that stay visible, against the definition in 64
bits.  Tolerances: step_util.attend derives each element's from the kernels' roundings."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import step_util as W  # noqa: E402
from tests import test_gpu_prefill as P  # noqa: E402

ctas = P.ctas
KINDS = P.KINDS


def check_prompt(kv, lens, H, Hk, D, window, sinks, *, scale=None, seed=1, first=0, behind=0, edit=None):
    g = U.gen(seed)
    T = first + sum(lens) + behind
    x = U.halves(g, T, H + 2 * Hk, D)
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    if edit is not None:
        edit(q, k, v)
    off = U.offsets_of(lens, first)
    out = torch.full((T, H, D), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda")
    ws = kv.prefill_workspace(T, len(lens), H, Hk, D)
    kv.prefill(q, k, v, U.ints(off), scale=scale, window=window, sinks=sinks, out=out, lse=lse, ws=ws)
    assert kv.kvattn_workspace_status(ws) == 0
    for a, b in zip(off, off[1:]):
        if a < b:
            ok = W.window_mask(torch.arange(1, b - a + 1, device="cuda"), b - a, window, sinks)
            o, l, to, tl = W.attend(q[a:b], k[a:b].double(), v[a:b].double(), ok, 1.0 / math.sqrt(D) if scale is None else scale)
            U.check(out[a:b], o, to, f"out {a}")
            U.check(lse[a:b], l, tl, f"lse {a}")
    for a, b in ((0, first), (off[-1], T)):   # tokens of no sequence are left as they were
        assert bool((out[a:b] == 7.0).all()) and bool((lse[a:b] == 7.0).all())


def check_chunk(kv, c, window, sinks, **kw):
    out, lse = P.call_chunk(kv, c, window=window, sinks=sinks, **kw)
    W.check_chunk(c, out, lse, window, sinks, kw.get("scale"))
    return out, lse


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (64, 4), (127, 0), (128, 128), (129, 1), (200, 130), (300, 0),
                                          (500, 700), (1000, 5), (5000, 3)])
def test_prompt_windows(kvattn, window, sinks, D):
    check_prompt(kvattn, [700, 1, 0, 333], 8, 2, D, window, sinks)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 1), (3, 1), (6, 2), (7, 1), (8, 1), (40, 1), (70, 1), (128, 1)])
def test_prompt_heads(kvattn, H, Hk, D):
    check_prompt(kvattn, [61, 400], H, Hk, D, 90, 3, seed=2)


@pytest.mark.parametrize("D", [128, 256])
def test_prompt_long(kvattn, D):
    """Gaps of many tiles between the first tokens and the window."""
    check_prompt(kvattn, [2500], 4, 2, D, 150, 260)
    check_prompt(kvattn, [3000, 40], 4, 1, D, 1, 0)
    check_prompt(kvattn, [70, 3, 140], 4, 2, D, 33, 5, first=9, behind=21)


@pytest.mark.parametrize("scale", [0.0, -0.07, 0.5])
def test_prompt_scale(kvattn, scale):
    check_prompt(kvattn, [350, 20], 4, 2, 128, 100, 7, scale=scale)


@pytest.mark.parametrize("D,H", [(128, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(kvattn, D, H, value):
    """In the first tokens, at a window's beginning, in the middle and at the end: every other row stays
    clean, in front of it and behind it."""
    for at in (0, 3, 5, 50, 130, 250, 256, 383, 500, 699):
        def edit(q, k, v):
            v[at, 0, 3] = value
            v[at, 0, D - 1] = value
        check_prompt(kvattn, [700], H, 1, D, 130, 5, edit=edit)

    def many(q, k, v):
        v[100:420:7, 0, 1] = value
    check_prompt(kvattn, [700], H, 1, D, 61, 140, edit=many)


@pytest.mark.parametrize("D,H", [(128, 4), (256, 2)])
def test_keys_that_are_not_finite_are_not_seen_from_behind_the_window(kvattn, D, H):
    def edit(q, k, v):
        k[200, 0, 5] = float("nan")
    g = U.gen(1)
    x = U.halves(g, 600, H + 2, D)
    q, k, v = x[:, :H], x[:, H:H + 1], x[:, H + 1:]
    clean, _ = kvattn.prefill(q, k, v, U.ints([0, 600]), window=64, sinks=2)
    clean = clean.clone()
    edit(q, k, v)
    got, _ = kvattn.prefill(q, k, v, U.ints([0, 600]), window=64, sinks=2)
    torch.cuda.synchronize()
    assert torch.equal(got[:200], clean[:200]) and torch.equal(got[264:], clean[264:])
    assert bool(torch.isnan(got[200:264]).any(-1).all())


def test_prompt_growing_maximum(kvattn):
    def edit(q, k, v):
        q[..., 0] = 4.0
        k[..., 0] = (torch.arange(k.shape[0], device="cuda") / 8).half()[:, None]
    check_prompt(kvattn, [900], 4, 1, 128, 300, 4, edit=edit)

    def fall(q, k, v):   # a first token that outweighs the window by far
        q[..., 0] = 4.0
        k[..., 0] = 0.0
        k[0, :, 0] = 30.0
    check_prompt(kvattn, [900], 4, 1, 256, 300, 1, edit=fall)
    check_prompt(kvattn, [900], 4, 1, 128, 300, 0, edit=fall)


@pytest.mark.parametrize("n", [None, 0, 5, 37])
@pytest.mark.parametrize("plan,holes", [(False, 0.0), (True, 0.0), (True, 0.3)])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_chunk_kinds(kvattn, ctas, kind, D, plan, holes, n):
    c = P.make_chunk(kind, [70, 1, 0, 33, 1], [900, 513, 0, 33, 1100], 8, 2, D, plan, holes)
    ctas(n)
    check_chunk(kvattn, c, 200, 9)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 1), (100, 128), (128, 0), (250, 200), (640, 31), (4000, 0)])
@pytest.mark.parametrize("new,lens", [([1], [1]), ([1], [128]), ([1], [129]), ([3], [2]), ([200], [150]), ([300], [300]),
                                      ([5, 6, 7], [0, 6, 1000]), ([260], [1500]), ([1] * 9, [1, 5, 127, 128, 129, 300, 700, 1000, 2000])])
def test_chunk_lengths(kvattn, ctas, new, lens, window, sinks, D):
    check_chunk(kvattn, P.make_chunk("f16", new, lens, 6, 2, D, False), window, sinks)
    ctas(11)
    check_chunk(kvattn, P.make_chunk("q8_0", new, lens, 6, 2, D, True, 0.1), window, sinks)


@pytest.mark.parametrize("H,Hk", [(1, 1), (5, 1), (16, 2), (48, 3), (128, 1)])
def test_chunk_heads(kvattn, ctas, H, Hk):
    for D in (128, 256):
        check_chunk(kvattn, P.make_chunk("f16", [50, 90], [600, 90], H, Hk, D, True, 0.1), 70, 3)
        ctas(13)
        check_chunk(kvattn, P.make_chunk("q4_0", [50, 90], [600, 90], H, Hk, D, False), 70, 3)
        ctas(None)


@pytest.mark.parametrize("kind", KINDS)
def test_chunk_holes_where_the_window_lies(kvattn, ctas, kind):
    """Rows whose window and first tokens are all holes see nothing."""
    c = P.make_chunk(kind, [40, 2], [900, 700], 4, 2, 128, True, 0.2)
    c["plan"][0, 600:900] = -1
    c["plan"][0, :6] = -1
    c["plan"][1, 384:700] = -1
    for n in (None, 0, 9):
        ctas(n)
        out, lse = check_chunk(kvattn, c, 200, 6)
        assert bool((out[:40] == 0).all()) and bool(torch.isneginf(lse[:40]).all())
        assert bool(torch.isfinite(lse[40:]).all())
    check_chunk(kvattn, c, 200, 6, scale=-0.05)


@pytest.mark.parametrize("D", [128, 256])
def test_chunk_cells_in_any_order(kvattn, ctas, D):
    g = U.gen(9)
    for kind in ("f16", "q8_0", "q4_0"):
        c = P.make_chunk(kind, [90, 5], [800, 500], 4, 2, D, True, 0.2)
        for s, n in enumerate(c["L"]):
            c["plan"][s, :n] = c["plan"][s, torch.randperm(n, generator=g, device="cuda")]
        for n in (None, 7):
            ctas(n)
            check_chunk(kvattn, c, 260, 70)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_chunk_values_that_are_not_finite(kvattn, ctas, kind, value):
    """Also in cells that no row sees: below the windows, behind the end."""
    for plan in (False, True):
        c = P.make_chunk(kind, [60, 1], [700, 650], 4, 2, 128, plan)
        for s, places in ((0, (0, 100, 500, 540, 561, 600, 690)), (1, (2, 300, 449, 450, 600))):
            for at in places:
                cell = s * c["n_cells"] + at if c["plan"] is None else int(c["plan"][s, at])
                (c["v"] if c["vs"] is None else c["vs"])[cell, 0, 1] = value
        for n in (None, 6):
            ctas(n)
            got, lse = P.call_chunk(kvattn, c, window=200, sinks=3)
            a = 0
            for s, (m, L) in enumerate(zip(c["new"], c["L"])):
                k, v, there = W.rows_of(c, s)
                if c["vs"] is not None:   # a scale that is not finite makes its 32 elements NaN
                    v = torch.where(torch.isfinite(v), v, math.nan)
                    cells = s * c["n_cells"] + torch.arange(L, device="cuda") if c["plan"] is None else c["plan"][s, :L].long()
                    bad = ~torch.isfinite(c["vs"][cells.clamp(min=0)]).repeat_interleave(32, -1)
                    v = torch.where(bad, math.nan, v)
                ok = W.window_mask(torch.arange(m, device="cuda") + L - m + 1, L, 200, 3) & there
                o, l, to, tl = W.attend(c["q"][a:a + m], k, v, ok, 1 / math.sqrt(128), c["ks"] is not None)
                U.check(got[a:a + m], o, to, f"out of sequence {s}")
                U.check(lse[a:a + m], l, tl, f"lse of sequence {s}")
                a += m


def test_a_window_of_everything_is_none(kvattn):
    c = P.make_chunk("f16", [70, 1], [700, 513], 8, 2, 128, True, 0.1)
    want = P.call_chunk(kvattn, c)
    for window in (700, 10 ** 6, 2 ** 62):
        for sinks in (0, 5, 2 ** 62):
            got = P.call_chunk(kvattn, c, window=window, sinks=sinks)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # first tokens that are everything: no window either
    got = P.call_chunk(kvattn, c, window=1, sinks=2 ** 40)
    W.check_chunk(c, *got)


def test_no_lse_and_results_that_repeat(kvattn, ctas):
    c = P.make_chunk("q8_0", [100, 1, 7], [5000, 3000, 800], 8, 2, 128, True, 0.1)
    want, lse = P.call_chunk(kvattn, c, window=1000, sinks=4)
    ws = kvattn.prefill_chunk_workspace(108, 3, 8, 2, 128, 5000)
    ws[256:] = 0xff
    for _ in range(3):
        got, _ = P.call_chunk(kvattn, c, lse=False, window=1000, sinks=4, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert kvattn.kvattn_workspace_status(ws) == 0


def test_without_tensor_maps(kvattn):
    """KVATTN_TMA=0: K and V by ordinary loads (read once per process, so in a child of its own)."""
    import os
    import subprocess
    import sys
    code = ("from tests import test_gpu_window as T, test_gpu_prefill as P; from kv_cache_decode_02_gb300 import kvattn as kv\n"
            "for D in (128, 256):\n"
            "    T.check_prompt(kv, [300, 20], 4, 2, D, 90, 5)\n"
            "    for kind in P.KINDS:\n"
            "        T.check_chunk(kv, P.make_chunk(kind, [70, 1], [700, 513], 8, 2, D, False), 200, 9)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, KVATTN_TMA="0"), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
