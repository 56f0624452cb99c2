"""Values, keys and scales that are not finite in a shared prefix and behind it, rows that belong to no
sequence, and what a call computes after one whose wait ran out."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import step_util as W  # noqa: E402
from tests import test_gpu_prefill as P  # noqa: E402
from tests import test_gpu_shared_prefix as X  # noqa: E402

ctas = P.ctas
PREFIX = 512
NEW, OWN = [3, 1, 40], [200, 50, 300]


def cells(c, s, places):
    """Of places of sequence s, those in the prefix wherever it is stored."""
    if c["plan"] is not None:
        return [int(c["plan"][s, at]) for at in places]
    all_of = range(len(c["new"]))
    return [t * c["n_cells"] + at for at in places for t in (all_of if at < PREFIX else [s])]


def check(kv, c, out, lse):
    """As step_util.check_chunk; a scale that is not finite makes its 32 elements NaN."""
    a = 0
    for s, (n, L) in enumerate(zip(c["new"], c["L"])):
        k, v, there = W.rows_of(c, s)
        if c["vs"] is not None:
            at = s * c["n_cells"] + torch.arange(L, device="cuda") if c["plan"] is None else c["plan"][s, :L].long()
            for x, sc in ((k, c["ks"]), (v, c["vs"])):
                x[~torch.isfinite(sc[at]).repeat_interleave(32, -1)] = math.nan
        ok = W.window_mask(torch.arange(n, device="cuda") + L - n + 1, L, L + n + 1, 0) & there
        o, l, to, tl = W.attend(c["q"][a:a + n], k, v, ok, 1 / math.sqrt(c["D"]), c["ks"] is not None)
        U.check(out[a:a + n], o, to, f"out of sequence {s}")
        U.check(lse[a:a + n], l, tl, f"lse of sequence {s}")
        a += n


def run(kv, c):
    ws = kv.prefill_chunk_workspace(sum(NEW), len(NEW), c["H"], c["Hk"], c["D"], max(c["L"]), shared=1)
    ws[256:] = 0xff
    out, lse = P.call_chunk(kv, c, shared=PREFIX, ws=ws)
    assert kv.kvattn_workspace_status(ws) == 0
    check(kv, c, out, lse)
    return out, lse


@pytest.mark.parametrize("plan", [False, True])
@pytest.mark.parametrize("kind,D", [("f16", 128), ("f16", 256), ("q8_0", 128), ("q4_0", 128), ("q8_0", 256)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_in_the_prefix_reach_every_row(kvattn, ctas, kind, D, plan, value):
    for n in (None, 0, 6):
        ctas(n)
        for places, element in (((5,), 1), ((200,), 3), ((511,), 0), ((0, 130, 300), 2)):
            c = X.make(kind, PREFIX, NEW, OWN, 4, 2, D, plan)
            which = c["v"] if c["vs"] is None else c["vs"]
            for cell in cells(c, 0, places):
                which[cell, 0, element] = value
            out, _ = run(kvattn, c)
            wild = ~torch.isfinite(out)
            own = slice(element, element + 1) if c["vs"] is None else slice(32 * element, 32 * element + 32)
            assert bool(wild[:, :2, own].all()) and int(wild.sum()) == sum(NEW) * 2 * (own.stop - own.start)


@pytest.mark.parametrize("plan", [False, True])
@pytest.mark.parametrize("kind", ["f16", "q8_0", "q4_0"])
def test_keys_in_the_prefix_and_behind_it(kvattn, ctas, kind, plan):
    for n in (None, 0, 6):
        ctas(n)
        for s, at in ((0, 7), (0, 333), (0, 511), (1, 540), (2, 600), (2, 790), (0, 710)):
            c = X.make(kind, PREFIX, NEW, OWN, 4, 2, 128, plan)
            which = c["k"] if c["ks"] is None else c["ks"]
            for cell in cells(c, s, (at,)):
                which[cell, 1, 2] = math.nan
            out, lse = run(kvattn, c)
            # the rows that see the cell, of the KV head's two query heads
            first = 0
            for t, (m, L) in enumerate(zip(NEW, c["L"])):
                sees = torch.arange(m, device="cuda") + L - m + 1 > at
                if at >= PREFIX and t != s:
                    sees[:] = False
                assert torch.equal(torch.isnan(lse[first:first + m, 2]), sees) and torch.equal(torch.isnan(lse[first:first + m, 3]), sees)
                assert bool(torch.isfinite(lse[first:first + m, :2]).all())
                first += m


@pytest.mark.parametrize("offsets", [[-5, 20, 10, 99], [30, 10, 0, 50], [50, 50, 50, 50], [0, 0, 0, 0], [60, 70, 80, 90], [0, 50, 0, 50],
                                     [7, 7, 20, 31], [12, 5, 30, 30], [-9, -3, 0, 4], [45, 99, 99, 99], [20, 10, 5, 0]])
@pytest.mark.parametrize("how", [dict(window=30, sinks=2), dict(shared=300), dict()])
def test_rows_of_no_sequence_are_left(kvattn, ctas, offsets, how):
    """Clamped to [0, n_tok] and to non-decreasing, a sequence's rows are [a, e): the others stay."""
    g = U.gen(6)
    q, k, v = U.halves(g, 50, 4, 128), U.halves(g, 1200, 4, 128), U.halves(g, 1200, 4, 128)
    ws = kvattn.prefill_chunk_workspace(50, 3, 4, 4, 128, 400, shared=1)
    theirs = torch.zeros(60, dtype=torch.bool, device="cuda")
    for a, e in zip(offsets, offsets[1:]):
        a = min(max(a, 0), 50)
        theirs[a:max(min(e, 50), a)] = True
    for n in (None, 0, 9):
        ctas(n)
        ws[256:] = 0xff
        out = torch.full((60, 4, 128), 7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((60, 4), 7.0, dtype=torch.float32, device="cuda")
        kvattn.prefill_chunk(q, U.ints(offsets), k, v, U.ints([400, 390, 380]), n_cells=400, out=out[:50], lse=lse[:50], ws=ws, **how)
        torch.cuda.synchronize()
        assert bool((out[~theirs] == 7.0).all()) and bool((lse[~theirs] == 7.0).all())
        assert kvattn.kvattn_workspace_status(ws) == 0


@pytest.mark.parametrize("D", [128, 256])
def test_a_prompt_window_after_a_wait_that_ran_out(kvattn, monkeypatch, D):
    g = U.gen(8)
    q, k, v = U.halves(g, 256, 4, D), U.halves(g, 256, 2, D), U.halves(g, 256, 2, D)
    ws = kvattn.prefill_workspace(256, 1, 4, 2, D)
    monkeypatch.setenv("KVATTN_DEBUG_STALL_TX", "16")
    kvattn.prefill(q, k, v, U.ints([0, 256]), window=50, sinks=3, ws=ws)
    assert kvattn.kvattn_workspace_status(ws, clear=True) == kvattn.KVATTN_DEVICE_WAIT_TIMEOUT
    monkeypatch.delenv("KVATTN_DEBUG_STALL_TX")
    out, lse = torch.full_like(q, 7.0), torch.full((256, 4), 7.0, device="cuda")
    kvattn.prefill(q, k, v, U.ints([0, 256]), window=50, sinks=3, out=out, lse=lse, ws=ws)
    assert kvattn.kvattn_workspace_status(ws) == 0
    ok = W.window_mask(torch.arange(1, 257, device="cuda"), 256, 50, 3)
    o, l, to, tl = W.attend(q, k.double(), v.double(), ok, 1.0 / math.sqrt(D))
    U.check(out, o, to, "out")
    U.check(lse, l, tl, "lse")
