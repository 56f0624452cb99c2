"""Batches of windows over sequences of very different lengths: whole units or shares, as the lengths have
it, with the result of the definition either way."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import step_util as W  # noqa: E402
from tests import test_gpu_prefill as P  # noqa: E402

ctas = P.ctas


def cut_units(ws, n):
    """Units that a call's first n CTAs cut (the notes of csrc/prompt.cuh's PrefillCut in its workspace)."""
    return int((ws[256:256 + 32 * n].view(torch.int32)[2::8] > 0).sum())


@pytest.mark.parametrize("kind,plan", [("f16", False), ("f16", True), ("q8_0", False), ("q8_0", True)])
@pytest.mark.parametrize("new,lens,window,cut", [
    ([1] * 19, [9000] + [100] * 18, 4000, True),                          # a long one among short ones
    ([1] * 19, [100] * 18 + [9000], 4000, True),
    ([1] * 38, [4100 + 10 * i for i in range(38)], 4000, False),          # all alike: two full rounds of 152
    ([200, 1, 1, 0, 70], [6000, 50, 1, 0, 3000], 2500, True),
    ([1] * 5, [0, 0, 0, 0, 0], 4000, False),                              # nothing to see
])
def test_mixed_lengths(kvattn, ctas, kind, plan, new, lens, window, cut):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hk = 8
    c = P.make_chunk(kind, new, lens, 16, Hk, 128, plan)
    ws = kvattn.prefill_chunk_workspace(sum(new), len(new), 16, Hk, 128, 10000)
    got = {}
    for n in (None, 0, 37):
        ctas(n)
        ws[256:] = 0xff
        out, lse = P.call_chunk(kvattn, c, window=window, sinks=5, ws=ws, max_len=10000)
        assert kvattn.kvattn_workspace_status(ws) == 0
        W.check_chunk(c, out, lse, window, 5)
        got[n] = cut_units(ws, 8 * 5 if n is None and sum(new) == 5 else min(sms, 152))
    if sms == 152:
        assert (got[None] > 0) == cut
    assert got[0] == 0


def test_captured_and_replayed_with_other_lengths(kvattn):
    """One graph, whole units in one replay and shares in the next."""
    a = P.make_chunk("f16", [1] * 19, [5000 + i for i in range(19)], 16, 8, 128, False)
    b = P.make_chunk("f16", [1] * 19, [5018] + [60 + i for i in range(18)], 16, 8, 128, False, seed=5)
    assert a["n_cells"] == b["n_cells"]
    k, v, q, lens = (a[x].clone() for x in ("k", "v", "q", "lens"))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    ws = kvattn.prefill_chunk_workspace(19, 19, 16, 8, 128, 6000)
    kw = dict(n_cells=a["n_cells"], window=4000, sinks=5, max_len=6000, out=out, lse=lse, ws=ws)
    kvattn.prefill_chunk(q, a["offsets"], k, v, lens, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvattn.prefill_chunk(q, a["offsets"], k, v, lens, **kw)
    for c in (b, a, b):
        for x, name in ((k, "k"), (v, "v"), (q, "q"), (lens, "lens")):
            x.copy_(c[name])
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        W.check_chunk(c, out, lse, 4000, 5)
        if torch.cuda.get_device_properties(0).multi_processor_count == 152:
            assert (cut_units(ws, 152) > 0) == (c is b)
