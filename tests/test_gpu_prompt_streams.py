"""Prompt-side wrappers launched on a stream that is not torch's current one, with no buffers given:
what they make belongs to that stream, and the current stream's late work does not reach it."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import test_gpu_prefill as P  # noqa: E402

H, Hk, D = 8, 2, 128


def calls(kv):
    """name -> (call(stream), sizes in bytes that the call makes)."""
    g = U.gen(21)
    T = 300
    q, k, v = U.halves(g, T, H, D), U.halves(g, T, Hk, D), U.halves(g, T, Hk, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    off = U.ints([0, 100, T])
    table = kv.rope_table(D)
    c = P.make_chunk("q8_0", [70, 200], [3000, 3000], H, Hk, D, False)
    f = P.make_chunk("f16", [70, 200], [3000, 3000], H, Hk, D, True, 0.1)
    slots = torch.randperm(5000, generator=g, device="cuda")[:T].to(torch.int32)

    def chunk(c):
        return lambda stream: kv.prefill_chunk(c["q"], c["offsets"], c["k"], c["v"], c["lens"], n_cells=c["n_cells"],
                                               cell_plan=c["plan"], k_scales=c["ks"], v_scales=c["vs"], max_len=3000,
                                               stream=stream)[:1]

    def write(stream):   # (makes nothing itself; its buffers are in the stream's order here)
        with torch.cuda.stream(torch.cuda.current_stream() if stream is None else torch.cuda.ExternalStream(handle(stream))):
            planes = [torch.zeros_like(x) for x in (c["k"], c["v"], c["ks"], c["vs"])]
        kv.cache_write(k, v, slots, planes[0], planes[1], k_scales=planes[2], v_scales=planes[3], stream=stream)
        return planes
    return {
        "rope": lambda stream: kv.rope(q, k, pos, table, stream=stream),
        "write": write,
        "read": lambda stream: kv.cache_read(c["k"], c["v"], slots, head_dim=D, k_scales=c["ks"], v_scales=c["vs"], stream=stream),
        "prefill": lambda stream: kv.prefill(q, k, v, off, stream=stream),
        "chunk q8_0": chunk(c),
        "chunk plan": chunk(f),
    }


def handle(stream):
    return stream if isinstance(stream, int) else stream.cuda_stream


def owner(x):
    """The handle of the stream whose pool x's memory is from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= x.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no such segment")


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", ["rope", "write", "read", "prefill", "chunk q8_0", "chunk plan"])
def test_a_busy_current_stream(kvattn, name, as_handle, monkeypatch):
    call = calls(kvattn)[name]
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # the current stream falls behind, with late writes queued to every block that it may reuse
    made = [torch.empty_like(x) for x in want]
    ws = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (256, 1 << 20, 40 << 20)]
    torch.cuda._sleep(200_000_000)   # about 0.1 s
    for x in made + ws:
        x.view(torch.uint8).fill_(0xff)
    del made, ws, x
    zeroed = []
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: zeroed.append(torch.cuda.current_stream().cuda_stream) or zeros(*a, **kw))
    got = call(side.cuda_stream if as_handle else side)
    monkeypatch.undo()
    assert all(x == side.cuda_stream for x in zeroed) and (name != "prefill" or len(zeroed) == 1)
    assert torch.cuda.current_stream().cuda_stream != side.cuda_stream
    late = [torch.full_like(x, 3) for x in want]   # and what it allocates afterwards is written late too
    torch.cuda.synchronize()
    assert all(owner(x) == side.cuda_stream for x in got)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert all(bool((x == 3).all()) for x in late)


def test_given_buffers_on_another_stream_are_used_as_they_are(kvattn):
    c = P.make_chunk("f16", [70], [900], H, Hk, D, False)
    want, lse = P.call_chunk(kvattn, c)
    side = torch.cuda.Stream()
    out, l = torch.zeros_like(want), torch.zeros_like(lse)
    ws = kvattn.prefill_chunk_workspace(70, 1, H, Hk, D, 900)
    torch.cuda.synchronize()
    got, gl = kvattn.prefill_chunk(c["q"], c["offsets"], c["k"], c["v"], c["lens"], n_cells=c["n_cells"], max_len=900, out=out,
                                   lse=l, ws=ws, stream=side)
    torch.cuda.synchronize()
    assert got is out and gl is l and torch.equal(out, want) and torch.equal(l, lse)


def test_the_default_stream_by_its_handles(kvattn):
    """A call for the default stream from under another one: by the handles 0 and 1."""
    q = U.halves(U.gen(5), 64, H, D)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    table = kvattn.rope_table(D)
    want, _ = kvattn.rope(q, None, pos, table)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [kvattn.rope(q, None, pos, table, stream=h)[0] for h in (0, 1)]
        torch.cuda.synchronize()
    assert all(owner(x) == 0 and torch.equal(x, want) for x in got)
