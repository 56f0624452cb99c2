"""Shared prefixes behind which one sequence has more blocks of tokens than its line of shares can number
in 32 bits: such calls are dealt out in whole units."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import step_util as W  # noqa: E402


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,H,Hk,D", [(65600, 128, 1, 256), (70000, 192, 2, 256), (140000, 64, 1, 256)])
def test_more_blocks_than_the_line_holds(kvattn, n, H, Hk, D):
    g = U.gen(4)
    L = n + 256
    k, v = U.halves(g, L, Hk, D), U.halves(g, L, Hk, D)
    q = torch.empty(n, H, D, dtype=torch.float16, device="cuda").uniform_(-1, 1, generator=g)
    ws = kvattn.prefill_chunk_workspace(n, 1, H, Hk, D, L, shared=1)
    ws[256:] = 0xff
    out, lse = torch.full_like(q, 7.0), torch.full((n, H), 7.0, device="cuda")
    kvattn.prefill_chunk(q, U.ints([0, n]), k, v, U.ints([L]), n_cells=L, shared=256, out=out, lse=lse, ws=ws)
    assert kvattn.kvattn_workspace_status(ws) == 0
    assert bool(torch.isfinite(lse).all())
    at = torch.tensor(sorted({0, 1, 2, 127, 128, n // 3, n // 2, 32768, 46341, 65535, 65536, 65537, n - 130, n - 2, n - 1} & set(range(n))),
                      device="cuda")
    ok = W.window_mask(at + 257, L, L + 1, 0)
    o, l, to, tl = W.attend(q[at], k.double(), v.double(), ok, 1.0 / math.sqrt(D))
    U.check(out[at], o, to, "out")
    U.check(lse[at], l, tl, "lse")
    # every row has a result of its own: means of that many values lie near zero
    assert float(out[n // 2:].abs().amax()) < 0.25
