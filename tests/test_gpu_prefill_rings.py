"""The attention kernel's rings of slots, gone around thousands of times by one CTA: every piece's
result against the definition in 64 bits, and no wait that gave up."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import test_gpu_prefill as P  # noqa: E402


@pytest.mark.parametrize("n", ["1", "3"])
@pytest.mark.parametrize("kind,D,new,lens", [
    ("q8_0", 256, [9], [20000]),          # three slots, four of them taken per tile
    ("q8_0_q4_0", 256, [130], [6000]),    # several blocks one after the other
    ("q4_0", 256, [3], [20000]),
    ("q8_0", 128, [1, 70], [9000, 5000]),  # units of one row group and of both in turn
    ("f16", 256, [5, 1], [12000, 128]),   # ... of many tiles and of one
])
def test_one_cta_goes_around_its_rings(kvattn, monkeypatch, kind, D, new, lens, n):
    monkeypatch.setenv("KVATTN_PREFILL_CTAS", n)
    c = P.make_chunk(kind, new, lens, 4, 1, D, False)
    ws = kvattn.prefill_chunk_workspace(sum(new), len(new), 4, 1, D, max(lens))
    P.check_chunk(kvattn, c, ws=ws)
    assert kvattn.kvattn_workspace_status(ws) == 0
