"""The longest sequence that a chunk call takes, 2^31 - 1 entries of a plan, by few cells named again
and again: the line of shares is numbered to its end."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 127, 2 ** 31 - 130])
def test_the_longest_plan(kvattn, length):
    D, cells = 128, 256
    h = dict(dtype=torch.float16, device="cuda")
    k, v = torch.zeros(cells, 1, D, **h), torch.zeros(cells, 1, D, **h)
    q = torch.zeros(1, 1, D, **h)
    q[..., 0] = 1.0
    # cells 0 to 127: score 0, value 1; cell 200: a score of 22 = ln(3.6e9), value 3
    v[:128] = 1.0
    k[200, 0, 0], v[200] = 22.0, 3.0
    plan = torch.empty(1, length, dtype=torch.int32, device="cuda")
    whole = length // 128 * 128
    plan[0, :whole].view(-1, 128)[:] = torch.arange(128, dtype=torch.int32, device="cuda")
    plan[0, whole:] = 5
    n = length
    for at in (None, length - 1, length // 2, 0):   # where the heavy cell stands
        if at is not None:
            was = int(plan[0, at])
            plan[0, at] = 200
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        out, lse = kvattn.prefill_chunk(q, U.ints([0, 1]), k, v, U.ints([length]), cell_plan=plan, scale=1.0,
                                        lse=torch.empty(1, 1, dtype=torch.float32, device="cuda"))
        end.record()
        torch.cuda.synchronize()
        assert begin.elapsed_time(end) < 3000   # (shared; one SM alone takes some 20 s)
        heavy = 0.0 if at is None else math.exp(22.0)
        light = n - (0 if at is None else 1)
        total = heavy + light
        # running sums in fp32 over a share's tiles: l takes one addition a tile (half a step, 2^-24, each),
        # O eight products (a whole step, 2^-23, where they are cut off); then the result's rounding
        tiles = math.ceil(math.ceil(n / 128) / torch.cuda.get_device_properties(0).multi_processor_count) + 1
        want = (3 * heavy + light) / total
        assert abs(float(lse) - math.log(total)) <= tiles * 2.0 ** -24 + 2.0 ** -16
        assert float((out.double() - want).abs().max()) <= want * (tiles * 9 * 2.0 ** -23 + 2.0 ** -11)
        if at is not None:
            plan[0, at] = was
    del plan
    torch.cuda.empty_cache()
