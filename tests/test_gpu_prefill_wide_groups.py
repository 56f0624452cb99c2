"""65 to 128 query heads per KV head: a row group is one token, and at head_dim 256 so is a block,
which sees its sequence's last tile only in part unless it is the last one."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import test_gpu_prefill as P  # noqa: E402

ctas = P.ctas


@pytest.mark.parametrize("n", [None, 0, 7, 29])
@pytest.mark.parametrize("kind,plan,holes", [("f16", False, 0.0), ("f16", True, 0.1), ("q8_0", False, 0.0), ("q4_0", True, 0.1)])
@pytest.mark.parametrize("H", [65, 96, 128])
def test_chunk_tokens_across_a_tile_border(kvattn, ctas, H, kind, plan, holes, n):
    ctas(n)
    P.check_chunk(kvattn, P.make_chunk(kind, [64, 3], [4100, 130], H, 1, 256, plan, holes))


@pytest.mark.parametrize("n", [None, 0, 5])
@pytest.mark.parametrize("H,D", [(128, 128), (130, 128), (130, 256)])
def test_chunk_odd_counts_and_two_kv_heads(kvattn, ctas, H, D, n):
    ctas(n)
    P.check_chunk(kvattn, P.make_chunk("f16", [33, 1], [700, 500], H, 1 if H <= 128 else 2, D, False))


@pytest.mark.parametrize("H,D", [(65, 256), (128, 256), (128, 128)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_later_values_that_are_not_finite_stay_away(kvattn, ctas, H, D, value):
    def edit(q, k, v):
        v[50, 0, 3] = value
        v[135, 0, :] = value
        v[149, 0, D - 1] = value
    P.check_prefill(kvattn, [150], H, 1, D, edit=edit)
    for kind in ("f16", "q8_0"):
        for n in (0, 6):
            ctas(n)
            c = P.make_chunk(kind, [20], [650], H, 1, D, False)
            if kind == "f16":
                c["v"][640, 0, 9] = value
                c["v"][648, 0, :] = value
            else:
                c["vs"][640, 0, 1] = float("nan")
                c["vs"][648, 0, 3] = float("nan")
            P.check_chunk(kvattn, c)


def test_prefill_lengths(kvattn):
    for lens in ([1], [129], [5, 0, 257]):
        P.check_prefill(kvattn, lens, 128, 1, 256)
