"""The decode wrappers launched on a stream that is not torch's current one, with no buffers given:
what they make belongs to that stream, and the current stream's late work does not reach it."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests.test_gpu_prompt_streams import owner  # noqa: E402


def calls(kv):
    g = U.gen(31)
    q, k, v = U.halves(g, 2, 8, 128), U.halves(g, 2, 3000, 2, 128), U.halves(g, 2, 3000, 2, 128)
    qm, lens = U.halves(g, 2, 3, 8, 128), U.ints([3000, 1700])
    parts = torch.randn(5, 16, 128, generator=g, device="cuda")
    lses = torch.randn(5, 16, generator=g, device="cuda")
    kt, vt = (U.halves(g, 512, 2, 128).cpu().pin_memory() for _ in range(2))
    tail, copies = kv.WindowTail(), torch.cuda.Stream()
    return {
        "decode": lambda stream: kv.decode(q, k, v, lens, split=128, stream=stream),
        "decode_multi": lambda stream: kv.decode_multi(qm, k, v, lens, split=128, stream=stream),
        "merge": lambda stream: kv.merge(parts, lses, stream=stream),
        "window and tail": lambda stream: tail(q[:1], k[0], v[0], kt, vt, split=128, tile_cells=128, tail_split=128,
                                               compute_stream=stream, copy_stream=copies),
        # (no copy stream named: the current one)
        "tail copies on the current stream": lambda stream: tail(
            q[:1], k[0], v[0], kt, vt, split=128, tile_cells=128, tail_split=128, compute_stream=stream,
            copy_stream=copies if stream is None else None),
    }


@pytest.mark.parametrize("name", ["decode", "decode_multi", "merge", "window and tail", "tail copies on the current stream"])
def test_a_busy_current_stream(kvattn, name):
    call = calls(kvattn)[name]
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made = [torch.empty_like(x) for x in want]
    ws = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (256, 1 << 20, 8 << 20)]
    torch.cuda._sleep(200_000_000)
    for x in made + ws:
        x.view(torch.uint8).fill_(0xff)
    del made, ws, x
    got = call(side)
    late = [torch.full_like(x, 3) for x in want]
    torch.cuda.synchronize()
    assert all(owner(x) == side.cuda_stream for x in got)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(bool((x == 3).all()) for x in late)
