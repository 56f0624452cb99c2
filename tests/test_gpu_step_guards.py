"""What windows and shared prefixes do with what should not be: bad plan entries, offsets out of order, a
wait that runs out."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import step_util as W  # noqa: E402
from tests import test_gpu_prefill as P  # noqa: E402
from tests import test_gpu_shared_prefix as X  # noqa: E402


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("how", [dict(window=200, sinks=20), dict(shared=256)])
def test_bad_plan_entries_are_masked_and_flagged(kvattn, kind, how):
    c = X.make(kind, 256, [20, 1], [40, 300], 4, 2, 128, True)
    good = c["plan"].clone()
    ws = kvattn.prefill_chunk_workspace(21, 2, 4, 2, 128, max(c["L"]), shared=1)
    places = [(0, 17, c["n_cells"]), (0, 140, -2), (1, 400, 2147483647), (1, 540, -2147483648)]
    for s, at, e in places:
        c["plan"][s, at] = e
        if at < 256 and "shared" in how:
            c["plan"][:, at] = e
    out, lse = P.call_chunk(kvattn, c, ws=ws, **how)
    assert kvattn.kvattn_workspace_status(ws, clear=True) == kvattn.KVATTN_DEVICE_BAD_PLAN_ENTRY
    c["plan"] = good
    for s, at, _ in places:
        c["plan"][s, at] = -1
        if at < 256 and "shared" in how:
            c["plan"][:, at] = -1
    want, wl = P.call_chunk(kvattn, c, ws=ws, **how)
    assert kvattn.kvattn_workspace_status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, wl)
    W.check_chunk(c, out, lse, how.get("window"), how.get("sinks", 0))


@pytest.mark.parametrize("offsets", [[-5, 20, 10, 99], [30, 10, 0, 50], [50, 50, 50, 50], [0, 0, 0, 0], [60, 70, 80, 90], [0, 50, 0, 50]])
def test_offsets_out_of_order_stay_in_bounds(kvattn, offsets):
    """Clamped to [0, n_tok] and to non-decreasing: no row outside is written."""
    g = U.gen(6)
    q, k, v = U.halves(g, 50, 4, 128), U.halves(g, 1200, 4, 128), U.halves(g, 1200, 4, 128)
    ws = kvattn.prefill_chunk_workspace(50, 3, 4, 4, 128, 400, shared=1)
    ws[256:] = 0xff
    for how in (dict(window=30, sinks=2), dict(shared=300)):
        out = torch.full((60, 4, 128), 7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((60, 4), 7.0, dtype=torch.float32, device="cuda")
        kvattn.prefill_chunk(q, U.ints(offsets), k, v, U.ints([400, 390, 380]), n_cells=400, out=out[:50], lse=lse[:50], ws=ws, **how)
        torch.cuda.synchronize()
        assert bool((out[50:] == 7.0).all()) and bool((lse[50:] == 7.0).all())
        assert kvattn.kvattn_workspace_status(ws) == 0


@pytest.mark.parametrize("kind", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("how", [dict(window=200, sinks=20), dict(shared=256), dict()])
def test_a_wait_that_runs_out_is_reported(kvattn, monkeypatch, kind, how):
    """More slots than the ring has: what waits for the first one's release is not let go by a product
    that its own wait did not allow (that filled the slot twice in one phase of its barrier)."""
    c = X.make(kind, 256, [20, 1], [40, 300], 4, 2, 128, True)
    ws = kvattn.prefill_chunk_workspace(21, 2, 4, 2, 128, max(c["L"]), shared=1)
    monkeypatch.setenv("KVATTN_DEBUG_STALL_TX", "16")
    P.call_chunk(kvattn, c, ws=ws, **how)
    assert kvattn.kvattn_workspace_status(ws, clear=True) == kvattn.KVATTN_DEVICE_WAIT_TIMEOUT
    monkeypatch.delenv("KVATTN_DEBUG_STALL_TX")
    out, lse = P.call_chunk(kvattn, c, ws=ws, **how)
    assert kvattn.kvattn_workspace_status(ws) == 0
    W.check_chunk(c, out, lse, how.get("window"), how.get("sinks", 0))


def test_a_prompt_window_whose_wait_runs_out_is_reported(kvattn, monkeypatch):
    g = U.gen(8)
    q, k, v = U.halves(g, 256, 4, 128), U.halves(g, 256, 2, 128), U.halves(g, 256, 2, 128)
    ws = kvattn.prefill_workspace(256, 1, 4, 2, 128)
    monkeypatch.setenv("KVATTN_DEBUG_STALL_TX", "16")
    kvattn.prefill(q, k, v, U.ints([0, 256]), window=50, sinks=3, ws=ws)
    assert kvattn.kvattn_workspace_status(ws, clear=True) == kvattn.KVATTN_DEVICE_WAIT_TIMEOUT
    monkeypatch.delenv("KVATTN_DEBUG_STALL_TX")
    kvattn.prefill(q, k, v, U.ints([0, 256]), window=50, sinks=3, ws=ws)
    assert kvattn.kvattn_workspace_status(ws) == 0


def test_a_shared_workspace_serves_calls_that_share_nothing(kvattn):
    """Few rows behind long caches: the plain form's notes need more room than the shared form's results."""
    for D in (128, 256):
        for T, S, H, Hk in ((1, 1, 1, 1), (1, 1, 4, 1), (2, 1, 1, 1), (3, 2, 2, 2), (64, 8, 8, 2)):
            for n in (0, 128, 5000, 100000, 2 ** 31 - 1):
                assert (kvattn.kvattn_prefill_chunk_shared_workspace_bytes(T, S, H, Hk, D, n) >=
                        kvattn.kvattn_prefill_chunk_workspace_bytes(T, S, H, Hk, D, n))
    c = X.make("f16", 100, [1], [200], 1, 1, 128, False)
    ws = kvattn.prefill_chunk_workspace(1, 1, 1, 1, 128, 100000, shared=1)
    for shared in (100, 128, 256):
        out, lse = P.call_chunk(kvattn, c, shared=shared, ws=ws, max_len=100000)
        assert kvattn.kvattn_workspace_status(ws) == 0
        W.check_chunk(c, out, lse)
