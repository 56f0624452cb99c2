"""Windows and shared prefixes at the far end of what a call takes: plans of 2^31 - 1 entries, and caches
whose rows lie beyond 32 bits of bytes."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402

D = 128
h = dict(dtype=torch.float16)


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def cells_of_two_kinds():
    """Cells 0 to 127: score 0, value 1; cell 200: score 5, value 3."""
    k, v, q = (torch.zeros(n, 1, D, device="cuda", **h) for n in (256, 256, 1))
    q[..., 0] = 1.0
    v[:128] = 1.0
    k[200, 0, 0], v[200] = 5.0, 3.0
    return q, k, v


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 127, 2 ** 31 - 130])
def test_the_longest_plan_through_a_window(kvattn, length):
    q, k, v = cells_of_two_kinds()
    plan = torch.empty(1, length, dtype=torch.int32, device="cuda")
    whole = length // 128 * 128
    plan[0, :whole].view(-1, 128)[:] = torch.arange(128, dtype=torch.int32, device="cuda")
    plan[0, whole:] = 5
    W, K = 1000, 7
    for at, inside in ((length - 1, True), (length - W, True), (length - W - 1, False), (K - 1, True), (K, False), (length // 2, False)):
        was = int(plan[0, at])
        plan[0, at] = 200
        out, lse = kvattn.prefill_chunk(q, U.ints([0, 1]), k, v, U.ints([length]), cell_plan=plan, scale=1.0, window=W, sinks=K,
                                        lse=torch.empty(1, 1, device="cuda"))
        plan[0, at] = was
        heavy, light = (math.exp(5.0), W + K - 1) if inside else (0.0, W + K)
        want = (3 * heavy + light) / (heavy + light)
        assert abs(float(lse) - math.log(heavy + light)) <= 2.0 ** -16
        assert float((out.double() - want).abs().max()) <= want * (2.0 ** -10 + 2.0 ** -18), at


def test_the_longest_plan_behind_a_shared_prefix(kvattn):
    """One token behind a prefix of nearly 2^31 cells: 16.7 million tiles, shared among the SMs."""
    length = 2 ** 31 - 130
    q, k, v = cells_of_two_kinds()
    plan = torch.empty(1, length, dtype=torch.int32, device="cuda")
    plan[0, :length // 128 * 128].view(-1, 128)[:] = torch.arange(128, dtype=torch.int32, device="cuda")
    plan[0, length // 128 * 128:] = 5
    k[200, 0, 0] = 22.0
    for at in (length - 1, length // 2, 0):
        was = int(plan[0, at])
        plan[0, at] = 200
        out, lse = kvattn.prefill_chunk(q, U.ints([0, 1]), k, v, U.ints([length]), cell_plan=plan, scale=1.0, shared=length,
                                        lse=torch.empty(1, 1, device="cuda"))
        plan[0, at] = was
        heavy, light = math.exp(22.0), length - 1
        total = heavy + light
        want = (3 * heavy + light) / total
        # sums over a share's tiles, as for the plain form: l one addition a tile, O eight products
        tiles = math.ceil(math.ceil(length / 128) / torch.cuda.get_device_properties(0).multi_processor_count) + 1
        assert abs(float(lse) - math.log(total)) <= tiles * 2.0 ** -24 + 2.0 ** -16
        assert float((out.double() - want).abs().max()) <= want * (tiles * 9 * 2.0 ** -23 + 2.0 ** -11)


@pytest.mark.parametrize("how", ["window", "shared"])
def test_rows_beyond_32_bits(kvattn, how):
    """Caches of their own of 2^25 + 77 cells (8.6 GB a plane and sequence): the last sequence's last cells."""
    N, S = 2 ** 25 + 77, 2
    k, v = torch.zeros(S * N, 1, D, device="cuda", **h), torch.zeros(S * N, 1, D, device="cuda", **h)
    q = torch.zeros(S, 1, D, device="cuda", **h)
    q[..., 0] = 1.0
    for s in range(S):
        k[s * N + N - 3, 0, 0], v[s * N + N - 3] = 20.0, 2.0 + s     # e^20 = 4.9e8 against 3.4e7 others
        k[s * N + 1, 0, 0], v[s * N + 1] = 18.0, 6.0                 # e^18 = 6.6e7 (shared: the same in both)
    lens, W, K = [N, N - 2], 900, 2
    out, lse = kvattn.prefill_chunk(q, U.ints([0, 1, 2]), k, v, U.ints(lens), n_cells=N, scale=1.0, lse=torch.empty(2, 1, device="cuda"),
                                    **(dict(window=W, sinks=K) if how == "window" else dict(shared=N - 100)))
    for s, n in enumerate(lens):
        heavy = math.exp(20.0) if N - 3 < n else 0.0
        first = math.exp(18.0)
        light = (W + K if how == "window" else n) - 1 - (heavy > 0)
        total = heavy + first + light
        want = ((2.0 + s) * heavy + 6.0 * first) / total
        tiles = math.ceil(N / 128 / torch.cuda.get_device_properties(0).multi_processor_count) + 9
        assert abs(float(lse[s]) - math.log(total)) <= tiles * 2.0 ** -24 + 2.0 ** -16
        assert float((out[s].double() - want).abs().max()) <= want * (tiles * 9 * 2.0 ** -23 + 2.0 ** -10 + 2.0 ** -18)
