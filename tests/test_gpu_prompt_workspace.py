"""A chunk workspace made for the largest call serves every smaller one."""
import itertools

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import test_gpu_prefill as P  # noqa: E402


@pytest.mark.parametrize("H,Hk,D", [(32, 8, 128), (48, 8, 128), (16, 8, 256), (4, 1, 256)])
def test_sizes_do_not_shrink(kvattn, H, Hk, D):
    tokens = (1, 5, 64, 500, 4000, 16384, 200000)
    seqs = (1, 4, 64)
    lens = (1, 128, 513, 4096, 65536, 131072, 1 << 24, (1 << 31) - 1)
    size = {x: kvattn.kvattn_prefill_chunk_workspace_bytes(x[0], x[1], H, Hk, D, x[2]) for x in itertools.product(tokens, seqs, lens)}
    assert min(size.values()) >= 256 and max(size.values()) < 50_000_000
    for a, b in itertools.product(size, size):
        if all(x <= y for x, y in zip(a, b)):
            assert size[a] <= size[b], (a, b)


def test_one_workspace_for_all_calls(kvattn):
    H, Hk, D = 32, 8, 128
    ws = kvattn.prefill_chunk_workspace(16384, 4, H, Hk, D, 65536)
    for new, lens in (([512], [16384]), ([1, 1, 1, 1], [65536, 5, 700, 0]), ([70, 3], [900, 9000])):
        c = P.make_chunk("f16", new, lens, H, Hk, D, False)
        P.check_chunk(kvattn, c, ws=ws)
    assert kvattn.kvattn_workspace_status(ws) == 0
