"""A serving program's steps with all of their operators in a run: maps made on the device, heads normed
and turned, rows stored by slot, attended to through a window and behind a shared prefix; against the
definitions in 64 bits, and captured and replayed with other steps, padded batches among them."""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import step_util as W  # noqa: E402

H, Hk, D, B = 8, 2, 128, 128
PREFIX, STRIDE = 2 * B, 8   # a system prompt of two blocks; entries of a table's row
WINDOW, SINKS = 150, 4


class Server:
    """The state that a program keeps: a cache in blocks, tables, lengths and the free list."""

    def __init__(self, kv, kind, S, seed, rows):
        g = U.gen(seed)
        self.kv, self.S, self.kind, self.rows = kv, S, kind, rows
        self.n_cells = (2 + S * (STRIDE - 2) + 3) * B
        k, v, ks, vs = U.cache_planes(g, kind, self.n_cells, Hk, D)
        self.cache = dict(k=k, v=v, ks=ks, vs=vs)     # (its first two blocks' contents are the prompt)
        ids = torch.randperm(self.n_cells // B - 2, generator=g, device="cuda").to(torch.int32) + 2
        self.free, self.n_free = ids, torch.tensor([ids.numel()], dtype=torch.int32, device="cuda")
        self.tables = torch.full((S, STRIDE), -1, dtype=torch.int32, device="cuda")
        self.tables[:, :2] = torch.arange(2, device="cuda")
        self.lens = torch.full((S,), PREFIX, dtype=torch.int32, device="cuda")
        self.plan = torch.full((S, STRIDE * B), -1, dtype=torch.int32, device="cuda")
        self.plan[:, :PREFIX] = torch.arange(PREFIX, device="cuda")
        self.maps = kv.step_maps_buffers(S, rows)
        self.table = kv.rope_table(D, base=1e6, sections=[16, 24, 24], order="cycle")
        self.weights = U.halves(g, D), U.halves(g, D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = kv.prefill_chunk_workspace(rows, S, H, Hk, D, STRIDE * B, shared=1)
        half = dict(dtype=torch.float16, device="cuda")
        self.q, self.k = torch.zeros(rows, H, D, **half), torch.zeros(rows, Hk, D, **half)
        self.out = [torch.full((rows, H, D), 7.0, **half) for _ in range(2)]
        self.lse = [torch.full((rows, H), 7.0, device="cuda") for _ in range(2)]
        self.pos = torch.zeros(3, rows, dtype=torch.int32, device="cuda")

    def step(self, x, new):
        """x: half [rows][H + 2 Hk][D], the step's projections; new: int32 [S]."""
        kv, m = self.kv, self.maps
        kv.step_maps(self.lens, new, self.tables, self.free, self.n_free, block_cells=B, n_cells=self.n_cells, plan=self.plan,
                     whole_plan=False, status=self.status, out=m)
        self.pos.copy_(m.positions)                   # (text: the same position on every axis)
        kv.norm_rope(x[:, :H], x[:, H:H + Hk], self.pos, self.table, q_weight=self.weights[0], k_weight=self.weights[1],
                     q_out=self.q, k_out=self.k)
        c = self.cache
        kv.cache_write(self.k, x[:, H + Hk:], m.slots, c["k"], c["v"], k_scales=c["ks"], v_scales=c["vs"], status=self.status)
        for i, how in enumerate((dict(window=WINDOW, sinks=SINKS), dict(shared=PREFIX))):
            kv.prefill_chunk(self.q, m.offsets, c["k"], c["v"], m.seq_lens, cell_plan=self.plan, k_scales=c["ks"], v_scales=c["vs"],
                             out=self.out[i], lse=self.lse[i], ws=self.ws, **how)
        self.lens.copy_(m.seq_lens)
        self.n_free.copy_(m.n_free)


@pytest.mark.parametrize("kind", ["f16", "q8_0", "q8_0_q4_0", "q4_0"])
def test_steps_against_the_definitions(kvattn, kind):
    S, rows = 3, 260
    s = Server(kvattn, kind, S, 5, rows)
    held, start = [PREFIX] * S, s.n_free.item()
    for i, new in enumerate([[200, 37, 1], [1, 1, 1], [2, 0, 90], [1, 1, 1]]):
        x = U.halves(U.gen(50 + i), rows, H + 2 * Hk, D)
        before = [y.clone() for y in s.out]
        s.step(x, U.ints(new))
        torch.cuda.synchronize()
        T = sum(new)
        held = [n + t for n, t in zip(held, new)]
        assert s.status.item() == 0 and s.lens.tolist() == held and s.maps.offsets.tolist() == U.offsets_of(new)
        assert s.n_free.item() == start - sum(-(-n // B) - 2 for n in held)
        slots = s.maps.slots[:T].tolist()
        assert len(set(slots)) == T and min(slots) >= PREFIX and s.maps.slots[T:].eq(-1).all()
        # what was stored reads back as the turned keys and the values: half a step off at most
        back = kvattn.cache_read(s.cache["k"], s.cache["v"], s.maps.slots[:T].contiguous(), head_dim=D, k_scales=s.cache["ks"],
                                 v_scales=s.cache["vs"])
        for got, want, sc in zip(back, (s.k[:T], x[:T, H + Hk:]), (s.cache["ks"], s.cache["vs"])):
            if sc is None:
                assert torch.equal(got, want)
            else:
                d = sc[s.maps.slots[:T].long()].double().abs().repeat_interleave(32, -1)
                four = got is back[1] and kind != "q8_0" or kind == "q4_0"
                # (the 4-bit code 8 becomes 7: a whole step there); and the product's rounding to half
                assert bool(((got.double() - want.double()).abs() <= d * (1.0 if four else 0.5) + 2.0 ** -10 * want.double().abs() + 1e-6).all())
        c = dict(s.cache, new=new, L=held, D=D, H=H, Hk=Hk, q=s.q[:T], plan=s.plan, n_cells=s.n_cells)
        W.check_chunk(c, s.out[0][:T], s.lse[0][:T], WINDOW, SINKS)
        W.check_chunk(c, s.out[1][:T], s.lse[1][:T])
        for y, old in zip(s.out, before):          # rows behind the last token are left as they were
            assert torch.equal(y[T:], old[T:])
    assert kvattn.kvattn_workspace_status(s.ws) == 0


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_steps_captured_with_padded_rows(kvattn, kind):
    """One graph of a step for up to 12 tokens of 4 sequences, replayed with other counts (none at all
    too); two graphs share the workspace.  The same steps eagerly give the same bits."""
    S, rows = 4, 12
    rng = random.Random(8)
    a, b = Server(kvattn, kind, S, 6, rows), Server(kvattn, kind, S, 6, rows)
    x, new = torch.zeros(rows, H + 2 * Hk, D, dtype=torch.float16, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    b.step(x, new)                                 # (nothing yet: sets the kernels up)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            b.step(x, new)
    for i in range(14):
        counts = [0] * S if i == 5 else [rng.randint(0, 3) for _ in range(S)]
        xi = U.halves(U.gen(90 + i), rows, H + 2 * Hk, D)
        a.step(xi, U.ints(counts))
        x.copy_(xi)
        new.copy_(U.ints(counts))
        graphs[i & 1].replay()
        torch.cuda.synchronize()
        T = sum(counts)
        for p, q in zip(a.out + a.lse, b.out + b.lse):
            assert torch.equal(p[:T], q[:T]), i
        for name in ("lens", "n_free", "tables", "plan"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        for p, q in zip(a.cache.values(), b.cache.values()):
            assert p is None or torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    assert a.status.item() == 0 and b.status.item() == 0
    assert kvattn.kvattn_workspace_status(b.ws) == 0


def test_a_sequence_without_room_keeps_its_state(kvattn):
    """The free list runs out: who is not served keeps length, table and cells; the others go on."""
    s = Server(kvattn, "f16", 3, 7, 64)
    s.n_free.fill_(1)
    cells = s.cache["k"].clone()
    s.step(U.halves(U.gen(1), 64, H + 2 * Hk, D), U.ints([20, 20, 0]))
    torch.cuda.synchronize()
    assert s.lens.tolist() == [PREFIX + 20, PREFIX, PREFIX] and s.n_free.item() == 0
    assert s.status.item() == kvattn.KVATTN_DEVICE_NO_ROOM
    assert s.tables[1].tolist() == [0, 1] + [-1] * (STRIDE - 2)
    first = int(s.tables[0, 2]) * B
    assert s.maps.slots.tolist() == list(range(first, first + 20)) + [-1] * 44
    cells[first:first + 20] = s.k[:20]
    assert torch.equal(s.cache["k"], cells)
    c = dict(s.cache, new=[20], L=[PREFIX + 20], D=D, H=H, Hk=Hk, q=s.q[:20], plan=s.plan, n_cells=s.n_cells)
    W.check_chunk(c, s.out[0][:20], s.lse[0][:20], WINDOW, SINKS)
    # the two unserved rows' tokens see what their lengths leave; whatever that is, it is finite
    assert bool(torch.isfinite(s.out[0][20:40]).all()) and bool(torch.isfinite(s.out[1][20:40]).all())


def owner(x):
    """The handle of the stream whose pool x's memory is from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= x.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no such segment")


@pytest.mark.parametrize("name", ["norm_rope", "axes", "maps", "prompt window", "chunk window", "chunk shared"])
def test_a_busy_current_stream(kvattn, name):
    """Calls on a stream that is not torch's current one, with no buffers given: what they make is that
    stream's, and late work of the current one does not reach it."""
    kv, g = kvattn, U.gen(21)
    T = 300
    q, k, v, w = U.halves(g, T, H, D), U.halves(g, T, Hk, D), U.halves(g, T, Hk, D), U.halves(g, D)
    pos = torch.arange(3 * T, dtype=torch.int32, device="cuda").view(3, T)
    table, axes = kv.rope_table(D), kv.rope_table(D, sections=[20, 22, 22])
    from tests import test_gpu_prefill as P
    from tests import test_gpu_shared_prefix as X
    c, f = P.make_chunk("q8_0", [70, 200], [3000, 3000], H, Hk, D, False), X.make("f16", 2000, [70, 200], [100, 900], H, Hk, D, True)
    off = U.ints([0, 100, T])
    lens, new = U.ints([100, 50]), U.ints([30, 90])
    tables, free = U.ints([[3, -1, -1], [2, -1, -1]]), U.ints([0, 1, 4, 5, 6])
    first, count = tables.clone(), U.ints([5])

    def chunk(c, **how):
        return lambda stream: kv.prefill_chunk(c["q"], c["offsets"], c["k"], c["v"], c["lens"], n_cells=c["n_cells"],
                                               cell_plan=c["plan"], k_scales=c["ks"], v_scales=c["vs"], max_len=3000, stream=stream,
                                               **how)[:1]

    def maps(stream):
        m = kv.step_maps(lens, new, tables, free, count, block_cells=64, n_cells=64 * 7, n_tok=150, stream=stream)
        return m.offsets, m.seq_lens, m.positions, m.slots, m.n_free
    call = {"norm_rope": lambda stream: kv.norm_rope(q, k, pos[0], table, q_weight=w, k_weight=w, stream=stream),
            "axes": lambda stream: kv.rope(q, k, pos, axes, stream=stream), "maps": maps,
            "prompt window": lambda stream: kv.prefill(q, k, v, off, window=40, sinks=3, stream=stream),
            "chunk window": chunk(c, window=500, sinks=5), "chunk shared": chunk(f, shared=2000)}[name]
    want = [x.clone() for x in call(None)]
    tables.copy_(first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made = [torch.empty_like(x) for x in want]
    ws = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (256, 1 << 20, 60 << 20)]
    torch.cuda._sleep(200_000_000)   # about 0.1 s
    for x in made + ws:
        x.view(torch.uint8).fill_(0xff)
    del made, ws, x
    got = call(side)
    late = [torch.full_like(x, 3) for x in want]
    torch.cuda.synchronize()
    assert all(owner(x) == side.cuda_stream for x in got)
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert all(bool((x == 3).all()) for x in late)
