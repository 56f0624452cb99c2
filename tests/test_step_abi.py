"""Host side of a serving step's operators: refusals before any device work, workspace sizes and the
axes of pairs (no GPU needed)."""
import numpy as np
import pytest

A = 0x7f0000000000  # fake, aligned addresses: every check below fails before any use
B = A + (1 << 32)
INV, UNS, WS = -1, -2, -3


def norm(kvattn, **over):
    a = dict(q=A, qs=4096, H=32, qw=A, k=A, ks=1024, Hk=8, kw=A, eps=1e-6, pos=A, pos_stride=4, n_axes=1, axis=None, turns=A,
             gain=1.0, n_rot=128, layout=0, n_tok=4, D=128, qo=A, qos=4096, ko=A, kos=1024, stream=None)
    a.update(over)
    return kvattn.lib.kvattn_norm_rope(*a.values())


@pytest.mark.parametrize("over,want", [
    (dict(D=64), UNS), (dict(D=192), UNS), (dict(n_rot=120), UNS), (dict(n_rot=144), INV), (dict(n_rot=-16), INV),
    (dict(layout=2), INV), (dict(n_tok=-1), INV), (dict(gain=float("nan")), INV), (dict(eps=-1e-6), INV),
    (dict(eps=float("inf")), INV), (dict(eps=float("nan")), INV), (dict(n_axes=0), INV), (dict(n_axes=5), UNS),
    (dict(n_axes=2), INV), (dict(n_axes=2, axis=A + 4), INV), (dict(n_axes=2, axis=A, pos_stride=3), INV),
    (dict(qw=A + 8), INV), (dict(kw=A + 2), INV), (dict(q=None), INV), (dict(q=A + 8), INV), (dict(qs=4088), INV),
    (dict(kos=1023), INV), (dict(ko=None), INV), (dict(pos=None), INV), (dict(pos=A + 2), INV), (dict(turns=None), INV),
    (dict(turns=A + 4), INV), (dict(H=-1), INV), (dict(n_tok=1 << 40), UNS), (dict(H=65536), UNS), (dict(n_tok=0), 0),
    (dict(H=0, Hk=0), 0),
])
def test_norm_rope_refusals(kvattn, over, want):
    assert norm(kvattn, **over) == want


@pytest.mark.parametrize("args,want", [
    ((128, [64], 0), [0] * 64), ((8, [1, 3], 0), [0, 1, 1, 1]), ((8, [1, 3], 1), [0, 1, 1, 1]),
    ((12, [2, 3, 1], 1), [0, 1, 2, 0, 1, 1]), ((12, [0, 6], 0), [1] * 6), ((12, [3, 0, 3], 1), [0, 2, 0, 2, 0, 2]),
    ((16, [2, 2, 2, 2], 0), [0, 0, 1, 1, 2, 2, 3, 3]),
])
def test_axes_of_pairs(kvattn, args, want):
    n_rot, sections, order = args
    axis = np.full(n_rot // 2, 9, np.uint8)
    kvattn.kvattn_rope_axes(n_rot, np.array(sections, np.int32), len(sections), order, axis)
    assert axis.tolist() == want


@pytest.mark.parametrize("n_rot,sections,order,want", [
    (7, [3], 0, INV), (0, [0], 0, INV), (8, [3], 0, INV), (8, [5], 0, INV), (8, [5, -1], 0, INV), (8, [4], 2, INV),
    (10, [1, 1, 1, 1, 1], 0, UNS), (8, [2 ** 31 - 1, 2 ** 31 - 1], 1, INV),
])
def test_axes_refusals(kvattn, n_rot, sections, order, want):
    axis, s = np.zeros(16, np.uint8), np.array(sections, np.int32)
    assert kvattn.lib.kvattn_rope_axes(n_rot, s.ctypes.data, len(sections), order, axis.ctypes.data) == want
    assert kvattn.lib.kvattn_rope_axes(8, None, 1, 0, axis.ctypes.data) == INV
    assert kvattn.lib.kvattn_rope_axes(8, s.ctypes.data, 1, 0, None) == INV


def test_rope_table_of_axes(kvattn):
    """Frequencies of the pairs, or of each axis' own pairs; refusals by Python's names."""
    t = kvattn.rope_table(32, base=1e4, sections=[4, 12], order="cycle", device="cpu")
    plain = kvattn.rope_table(32, base=1e4, device="cpu")
    assert t.n_axes == 2 and t.axis.tolist() == [0, 1] * 4 + [1] * 8 and bool((t.turns == plain.turns).all())
    assert plain.axis is None and plain.n_axes == 1
    r = kvattn.rope_table(32, base=1e4, sections=[4, 12], order="cycle", restart=True, device="cpu")
    for a, n in enumerate([4, 12]):
        own = kvattn.rope_table(2 * n, base=1e4, device="cpu").turns
        assert bool((r.turns[r.axis == a] == own).all())
    with pytest.raises(kvattn.KvattnError):
        kvattn.rope_table(32, sections=[4, 4], device="cpu")
    with pytest.raises(KeyError):
        kvattn.rope_table(32, sections=[4, 12], order="random", device="cpu")


def maps(kvattn, **over):
    a = dict(lens=A, new=A + 4096, S=8, tables=B, stride=16, block=16, free=B, n_list=100, n_free=A, n_cells=4096, n_tok=64,
             offsets=A, seq_lens=A + 256, positions=A, slots=A, left=A + 64, plan=A, plan_stride=256, whole=1, status=A, stream=None)
    a.update(over)
    return kvattn.lib.kvattn_step_maps(*a.values())


@pytest.mark.parametrize("over,want", [
    (dict(S=-1), INV), (dict(S=16385), UNS), (dict(stride=-1), INV), (dict(block=0), INV), (dict(block=-4), INV), (dict(block=2), UNS),
    (dict(block=24), UNS), (dict(block=1 << 17), UNS), (dict(n_list=-1), INV), (dict(n_list=1 << 31), UNS), (dict(n_cells=-1), INV),
    (dict(n_cells=1 << 31), UNS), (dict(n_tok=-1), INV), (dict(n_tok=1 << 31), UNS), (dict(plan_stride=-1), INV),
    (dict(plan_stride=1 << 31), UNS), (dict(offsets=None), INV), (dict(offsets=A + 2), INV), (dict(lens=None), INV),
    (dict(new=None), INV), (dict(tables=None), INV), (dict(seq_lens=None), INV), (dict(slots=None), INV), (dict(slots=A + 1), INV),
    (dict(positions=A + 2), INV), (dict(plan=A + 2), INV), (dict(status=A + 2), INV), (dict(n_free=None), INV), (dict(left=None), INV),
    (dict(free=None), INV), (dict(free=None, n_free=None), INV), (dict(free=B + 2), INV), (dict(seq_lens=A), INV),
    (dict(seq_lens=A + 4096), INV), (dict(left=A), INV),
])
def test_step_maps_refusals(kvattn, over, want):
    assert maps(kvattn, **over) == want


def prompt(kvattn, **over):
    a = dict(q=A, qs=4096, k=A, ks=1024, v=A, vs=1024, off=A, S=2, T=64, H=32, Hk=8, D=128, scale=0.1, window=16, sinks=2, out=A,
             lse=A, ws=A, nb=4096, stream=None)
    a.update(over)
    return kvattn.lib.kvattn_prefill_window(*a.values())


@pytest.mark.parametrize("over,want", [
    (dict(window=0), INV), (dict(window=-1), INV), (dict(sinks=-1), INV), (dict(D=64), UNS), (dict(H=30), INV), (dict(Hk=0), INV),
    (dict(H=1032), UNS), (dict(scale=float("nan")), INV), (dict(q=A + 8), INV), (dict(k=None), INV), (dict(off=None), INV),
    (dict(out=None), INV), (dict(lse=A + 2), INV), (dict(ws=None), INV), (dict(ws=A + 64), INV), (dict(nb=128), WS),
    (dict(T=-1), INV), (dict(T=1 << 40), UNS), (dict(T=0), 0), (dict(S=0), 0),
])
def test_prompt_window_refusals(kvattn, over, want):
    assert prompt(kvattn, **over) == want


def chunk(kvattn, name, **over):
    a = dict(q=A, qs=4096, off=A, T=64, kc=A, vc=A, ksc=A, vsc=A, kv_type=1, n_cells=8192, plan=None, stride=0, lens=A, S=2,
             max_len=8192, H=32, Hk=8, D=128, scale=0.1)
    a.update({"window": 16, "sinks": 2} if name == "window" else {"prefix": 1024})
    a.update(out=A, lse=A, ws=A, nb=1 << 40, stream=None)
    a.update(over)
    return getattr(kvattn.lib, f"kvattn_prefill_chunk_{name}")(*a.values())


@pytest.mark.parametrize("name", ["window", "shared"])
@pytest.mark.parametrize("over,want", [
    (dict(D=64), UNS), (dict(H=30), INV), (dict(scale=float("inf")), INV), (dict(kv_type=4), INV), (dict(kv_type=0), INV),
    (dict(ksc=None), INV), (dict(vsc=A + 4), INV), (dict(kc=None), INV), (dict(n_cells=0), INV), (dict(max_len=-1), INV),
    (dict(max_len=1 << 31), UNS), (dict(n_cells=1 << 62, S=4), UNS), (dict(plan=A, stride=0), INV), (dict(plan=A + 2, stride=8192), INV),
    (dict(lens=None), INV), (dict(lens=A + 1), INV), (dict(off=None), INV), (dict(q=A + 8), INV), (dict(out=A + 8), INV),
    (dict(lse=A + 2), INV), (dict(ws=None), INV), (dict(ws=A + 128), INV), (dict(nb=64), WS), (dict(T=-1), INV), (dict(T=1 << 31), UNS),
    (dict(T=0), 0), (dict(S=0), 0),
])
def test_chunk_refusals(kvattn, name, over, want):
    assert chunk(kvattn, name, **over) == want


def test_chunk_refusals_of_their_own(kvattn):
    for over in (dict(window=0), dict(window=-5), dict(sinks=-1)):
        assert chunk(kvattn, "window", **over) == INV
    assert chunk(kvattn, "shared", prefix=-1) == INV


def test_shared_workspace_sizes(kvattn):
    f = kvattn.kvattn_prefill_chunk_shared_workspace_bytes
    for bad in ((-1, 1, 8, 2, 128, 100), (8, -1, 8, 2, 128, 100), (8, 1, 7, 2, 128, 100), (8, 1, 8, 2, 64, 100), (8, 1, 8, 2, 128, -1),
                (8, 1, 8, 2, 128, 1 << 31)):
        assert f(*bad) == 0
    last = 0
    for T in (1, 2, 63, 64, 65, 1000, 8192):   # one for the largest serves all
        for S in (1, 2, 64):
            for n in (0, 127, 128, 5000, 1 << 20):
                assert f(T, S, 32, 8, 128, n) >= last
        last = f(T, 64, 32, 8, 128, 1 << 20)
    # two results in 32 bits for each (token, head) and a note for each (token, KV head) are in it
    assert f(8192, 64, 32, 8, 128, 4096) >= 2 * 8192 * (32 * 129 * 4 + 8 * 32)
    # ... and one that the plain form takes when nothing can be shared
    assert f(64, 2, 32, 8, 128, 8192) >= kvattn.kvattn_prefill_chunk_workspace_bytes(64, 2, 32, 8, 128, 8192)


def test_wrappers_refuse_what_does_not_go_together(kvattn):
    torch = pytest.importorskip("torch")
    if kvattn._torch is None:
        kvattn._bind_torch()
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    i = lambda *x: torch.tensor(x, dtype=torch.int32)
    with pytest.raises(ValueError):
        kvattn.step_maps(i(1), i(1), i(1)[None], block_cells=16, n_cells=64)                       # neither n_tok nor out
    out = kvattn.step_maps_buffers(1, 4, device="cpu")
    with pytest.raises(ValueError, match="n_tok"):
        kvattn.step_maps(i(1), i(1), i(1)[None], block_cells=16, n_cells=64, n_tok=5, out=out)
    with pytest.raises(ValueError, match="lens"):
        kvattn.step_maps(i(1), i(1), i(1)[None], block_cells=16, n_cells=64, out=out, stream=7)    # a host tensor
    with pytest.raises(AttributeError):
        out.slots = i(1)
    assert [x.numel() for x in (out.offsets, out.seq_lens, out.positions, out.slots, out.n_free)] == [2, 1, 4, 4, 1]
    with pytest.raises(ValueError):
        kvattn.norm_rope(None, None, i(0), kvattn.RopeTable(torch.zeros(64, dtype=torch.int64), 1.0, 128))
    with pytest.raises(KeyError):
        kvattn.norm_rope(h(1, 1, 128), None, i(0), kvattn.RopeTable(torch.zeros(64, dtype=torch.int64), 1.0, 128), layout="x")
