"""Attention of sequences that begin with the same cells, against the definition in 64 bits (which
knows nothing of what is shared).  Tolerances: step_util.attend derives each element's."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import step_util as W  # noqa: E402
from tests import test_gpu_prefill as P  # noqa: E402

ctas = P.ctas
KINDS = P.KINDS


def make(kind, prefix, new, own, H, Hk, D, plan, holes=0.0, seed=3):
    """A chunk whose sequences hold the same `prefix` cells and `own` of their own behind them."""
    c = P.make_chunk(kind, new, [prefix + n for n in own], H, Hk, D, plan, holes, seed)
    for s in range(1, len(new)):
        if plan:
            c["plan"][s, :prefix] = c["plan"][0, :prefix]
        else:
            for x in (c["k"], c["v"], c["ks"], c["vs"]):
                if x is not None:
                    x[s * c["n_cells"]:s * c["n_cells"] + prefix] = x[:prefix]
    return c


def check(kv, c, shared, **kw):
    T, S, H, Hk, D = sum(c["new"]), len(c["new"]), c["H"], c["Hk"], c["D"]
    ws = kv.prefill_chunk_workspace(T, S, H, Hk, D, max(c["L"]), shared=1)
    ws[256:] = 0xff
    out, lse = P.call_chunk(kv, c, shared=shared, ws=ws, **kw)
    W.check_chunk(c, out, lse, scale=kw.get("scale"))
    assert kv.kvattn_workspace_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("n", [None, 0, 1, 5, 37])
@pytest.mark.parametrize("plan,holes", [(False, 0.0), (True, 0.0), (True, 0.3)])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_kinds(kvattn, ctas, kind, D, plan, holes, n):
    c = make(kind, 700, [1, 40, 1, 3], [1, 200, 129, 3], 8, 2, D, plan, holes)
    ctas(n)
    check(kvattn, c, 700)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("prefix", [1, 127, 128, 129, 256, 1000, 2500])
@pytest.mark.parametrize("new,own", [([1, 1], [1, 1]), ([1] * 20, list(range(1, 200, 10))), ([300, 2], [300, 7]), ([5], [9]),
                                     ([16] * 5, [16, 17, 140, 300, 20])])
def test_prefixes_and_tokens(kvattn, ctas, prefix, new, own, D):
    check(kvattn, make("f16", prefix, new, own, 6, 2, D, False), prefix)
    ctas(13)
    check(kvattn, make("q8_0", prefix, new, own, 6, 2, D, True, 0.1), prefix)


@pytest.mark.parametrize("H,Hk", [(1, 1), (5, 1), (16, 2), (48, 3), (40, 1), (128, 1)])
def test_heads(kvattn, ctas, H, Hk):
    for D in (128, 256):
        check(kvattn, make("f16", 600, [1, 9, 30], [40, 9, 200], H, Hk, D, True, 0.1), 600)
        ctas(13)
        check(kvattn, make("q4_0", 600, [1, 9, 30], [40, 9, 200], H, Hk, D, False), 600)
        ctas(None)


def test_more_sequences_than_a_warp(kvattn, ctas):
    own = [1 + (37 * i) % 150 for i in range(70)]
    c = make("f16", 1100, [1] * 70, own, 4, 2, 128, True)
    for n in (None, 0, 3, 64):
        ctas(n)
        check(kvattn, c, 1100)


@pytest.mark.parametrize("shared", [0, 1, 127, 128, 300, 1000, 10 ** 9, 2 ** 62])
def test_any_number_said_to_be_shared(kvattn, ctas, shared):
    """Up to what is the same, in whole tiles; a sequence that holds less sets it for all."""
    c = make("f16", 1000, [1, 2, 1], [1, 2, 300], 4, 2, 128, True)
    if shared > 1000:
        c["plan"][2, :512] = c["plan"][0, :512]
        c["L"][1] = 514
        c["lens"][1] = 514   # (its two tokens see 513 and 514 cells: four tiles are in front of them)
    for n in (None, 5):
        ctas(n)
        if shared == 0:
            out, lse = P.call_chunk(kvattn, c, shared=0)
            W.check_chunk(c, out, lse)
        else:
            check(kvattn, c, shared)


def test_sequences_without_tokens_or_cells(kvattn, ctas):
    for new, own in (([0, 3, 0, 1], [0, 30, 0, 200]), ([0, 0], [4, 4]), ([1, 1], [1, 50])):
        c = make("f16", 400, new, own, 4, 2, 128, True)
        if new[0] == 0:    # it shares nothing and is not asked
            c["plan"][0] = -1
            c["L"][0] = 0
            c["lens"][0] = 0
        for n in (None, 0, 7):
            ctas(n)
            check(kvattn, c, 400)


def test_tokens_in_front_of_their_cells(kvattn, ctas):
    """More tokens than cells: the first ones see nothing, and nothing can be shared."""
    for n in (None, 0, 4):
        ctas(n)
        check(kvattn, P.make_chunk("f16", [5, 3], [3, 300], 4, 2, 128, False), 200)


def test_rows_outside_the_sequences_are_left(kvattn):
    c = make("f16", 512, [2, 3], [10, 40], 4, 2, 128, True)
    q = torch.cat((c["q"][:2] * 0 + 1, c["q"], c["q"][:3] * 0 + 2))
    out = torch.full((10, 4, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((10, 4), 7.0, device="cuda")
    kvattn.prefill_chunk(q, c["offsets"] + 2, c["k"], c["v"], c["lens"], n_cells=c["n_cells"], cell_plan=c["plan"], shared=512,
                         out=out, lse=lse, max_len=max(c["L"]))
    torch.cuda.synchronize()
    W.check_chunk(c, out[2:7], lse[2:7])
    for a, b in ((0, 2), (7, 10)):
        assert bool((out[a:b] == 7).all()) and bool((lse[a:b] == 7).all())


@pytest.mark.parametrize("kind", KINDS)
def test_holes_everywhere(kvattn, ctas, kind):
    c = make(kind, 512, [1, 4], [30, 140], 4, 2, 128, True, 0.2)
    c["plan"][:, :256] = -1                 # whole tiles of the prefix
    for n in (None, 9):
        ctas(n)
        check(kvattn, c, 512)
        check(kvattn, c, 512, scale=-0.05)
    c["plan"][:, :512] = -1                 # all of it
    check(kvattn, c, 512)
    c["plan"][:] = -1                       # nothing to see at all
    for n in (None, 0, 9):
        ctas(n)
        out, lse = check(kvattn, c, 512)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_values_that_are_not_finite(kvattn, ctas, value):
    """In the prefix every row sees them; in a sequence's own cells that sequence's rows do."""
    for n in (None, 6):
        ctas(n)
        c = make("f16", 512, [3, 1], [200, 50], 4, 2, 128, True)
        c["v"][int(c["plan"][0, 600]), 0, 3] = value      # seen by the first sequence's three tokens
        c["v"][int(c["plan"][0, 711]), 1, 5] = value      # by its last one
        check(kvattn, c, 512)


def test_scores_that_differ_by_much(kvattn, ctas):
    """One side outweighs the other by far, either way round."""
    for heavy in ("prefix", "own"):
        c = make("f16", 640, [1, 2], [100, 30], 4, 1, 128, True)
        c["q"][..., 0] = 8.0
        for s in range(2):
            row = c["plan"][s].long()
            at = row[:640] if heavy == "prefix" else row[640:c["L"][s]]
            c["k"][at[at >= 0], :, 0] = 40.0
        for n in (None, 4):
            ctas(n)
            check(kvattn, c, 640)


def test_results_repeat_and_no_lse(kvattn):
    c = make("q8_0", 5000, [1] * 30, [50 + i for i in range(30)], 16, 2, 128, True)
    want, lse = check(kvattn, c, 5000)
    ws = kvattn.prefill_chunk_workspace(30, 30, 16, 2, 128, max(c["L"]), shared=5000)
    for _ in range(3):
        got, _ = P.call_chunk(kvattn, c, lse=False, shared=5000, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_one_workspace_for_all_calls(kvattn):
    """Made for the largest call, used by smaller ones of either form in turn."""
    big = make("f16", 900, [40] * 4, [60, 70, 80, 90], 8, 2, 128, True)
    ws = kvattn.prefill_chunk_workspace(160, 4, 8, 2, 128, max(big["L"]), shared=1)
    small = make("q4_0", 300, [1, 2], [4, 30], 8, 2, 128, False)
    for _ in range(2):
        for c, shared in ((big, 900), (small, 300), (big, 128), (small, 299)):
            out, lse = P.call_chunk(kvattn, c, shared=shared, ws=ws)
            W.check_chunk(c, out, lse)


def test_captured_and_replayed_with_other_lengths(kvattn):
    a = make("f16", 640, [1] * 5, [30, 1, 200, 77, 128], 8, 2, 128, True)
    b = make("f16", 384, [1] * 5, [300, 99, 20, 333, 256], 8, 2, 128, True, seed=9)
    N = max(a["plan"].shape[1], b["plan"].shape[1])
    cells = max(a["n_cells"], b["n_cells"])
    k, v = (torch.zeros(cells, 2, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    plan = torch.full((5, N), -1, dtype=torch.int32, device="cuda")
    q, lens = a["q"].clone(), a["lens"].clone()
    out, lse = torch.zeros(5, 8, 128, dtype=torch.float16, device="cuda"), torch.zeros(5, 8, device="cuda")
    ws = kvattn.prefill_chunk_workspace(5, 5, 8, 2, 128, N, shared=1)
    off = U.ints([0, 1, 2, 3, 4, 5])

    def load(c):
        k[:c["n_cells"]].copy_(c["k"])
        v[:c["n_cells"]].copy_(c["v"])
        plan.fill_(-1)
        plan[:, :c["plan"].shape[1]].copy_(c["plan"])
        q.copy_(c["q"])
        lens.copy_(c["lens"])

    load(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):   # (384 cells are the same in both)
        kvattn.prefill_chunk(q, off, k, v, lens, cell_plan=plan, shared=384, out=out, lse=lse, ws=ws)
    for c in (b, a, b):
        load(c)
        graph.replay()
        torch.cuda.synchronize()
        W.check_chunk(c, out, lse)
