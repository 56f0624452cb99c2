"""Host side of the prompt operators: refusals before any device work, the workspace sizes and the
angle table (no GPU needed)."""
import math

import numpy as np
import pytest

A = 0x7f0000000000  # fake, aligned addresses: every check below fails before any use
INV, UNS, WS = -1, -2, -3


def rope(kvattn, **over):
    a = dict(q=A, qs=4096, H=32, k=A, ks=1024, Hk=8, pos=A, turns=A, gain=1.0, n_rot=128, layout=0, n_tok=4, D=128, qo=A,
             qos=4096, ko=A, kos=1024, stream=None)
    a.update(over)
    return kvattn.lib.kvattn_rope(*a.values())


@pytest.mark.parametrize("over,want", [
    (dict(D=64), UNS), (dict(D=192), UNS), (dict(n_rot=120), UNS), (dict(n_rot=144), INV), (dict(n_rot=-16), INV),
    (dict(layout=2), INV), (dict(n_tok=-1), INV), (dict(gain=float("inf")), INV), (dict(q=None), INV), (dict(q=A + 8), INV),
    (dict(qs=4088), INV), (dict(qs=4100), INV), (dict(kos=1023), INV), (dict(ko=None), INV), (dict(pos=None), INV),
    (dict(pos=A + 2), INV), (dict(turns=None), INV), (dict(turns=A + 4), INV), (dict(H=-1), INV), (dict(n_tok=1 << 40), UNS),
    (dict(n_tok=0), 0), (dict(H=0, Hk=0), 0),
])
def test_rope_refusals(kvattn, over, want):
    assert rope(kvattn, **over) == want


@pytest.mark.parametrize("args,want", [
    ((127, 1e4, 0, 1.0, 0), INV), ((0, 1e4, 0, 1.0, 0), INV), ((128, 1.0, 0, 1.0, 0), INV), ((128, float("nan"), 0, 1.0, 0), INV),
    ((128, 1e4, 3, 1.0, 0), INV), ((128, 1e4, 1, 0.5, 0), INV), ((128, 1e4, 2, 2.0, 0), INV), ((128, 1e4, 0, 0.0, 0), 0),
])
def test_rope_table_refusals(kvattn, args, want):
    import ctypes
    turns, gain = np.zeros(64, np.uint64), ctypes.c_float(0)
    assert kvattn.lib.kvattn_rope_table(*args, turns.ctypes.data, ctypes.byref(gain)) == want
    assert kvattn.lib.kvattn_rope_table(128, 1e4, 0, 1.0, 0, None, ctypes.byref(gain)) == INV


@pytest.mark.parametrize("scaling,factor,original", [(0, 1.0, 0), (1, 4.0, 0), (2, 8.0, 4096)])
@pytest.mark.parametrize("n_rot,base", [(2, 10000.0), (128, 10000.0), (64, 1000000.0)])
def test_rope_table_is_the_angle_in_turns(kvattn, n_rot, base, scaling, factor, original):
    turns = np.zeros(n_rot // 2, np.uint64)
    gain = kvattn.kvattn_rope_table(n_rot, base, scaling, factor, original, turns)
    i = np.arange(n_rot // 2)
    theta = base ** (-2.0 * i / n_rot)
    if scaling == 1:
        theta = theta / factor
    if scaling == 2:
        keep = np.clip((original * theta / (2 * math.pi) - 1) / 31, 0, 1)
        theta = theta / factor * (1 - keep) + theta * keep
        assert abs(gain - (0.1 * math.log(factor) + 1)) < 1e-6
    else:
        assert gain == 1.0
    got = turns.astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    # doubles throughout (a few 2^-53), the last of 2^-63 turns
    assert np.all(np.abs(got - theta) <= theta * 2.0 ** -49 + 2.0 ** -60)


def write(kvattn, read=False, **over):
    a = dict(k=A, ks=1024, v=A, vs=1024, slots=A, n_tok=8, Hk=8, D=128, kv_type=1, kc=A, vc=A, ksc=A, vsc=A, n_cells=64,
             status=None, stream=None)
    a.update(over)
    if read:
        return kvattn.lib.kvattn_cache_read(a["kc"], a["vc"], a["ksc"], a["vsc"], a["kv_type"], a["n_cells"], a["slots"],
                                            a["n_tok"], a["Hk"], a["D"], a["k"], a["ks"], a["v"], a["vs"], a["status"], None)
    return kvattn.lib.kvattn_cache_write(*a.values())


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("over,want", [
    (dict(D=64), UNS), (dict(Hk=0), INV), (dict(n_tok=-1), INV), (dict(n_cells=0), INV), (dict(kv_type=4), INV),
    (dict(kv_type=-1), INV), (dict(kv_type=0), INV), (dict(ksc=None), INV), (dict(vsc=A + 4), INV), (dict(D=256, ks=2048, vs=2048, ksc=A + 8), INV),
    (dict(kc=None), INV), (dict(vc=A + 8), INV), (dict(k=None), INV), (dict(v=A + 4), INV), (dict(ks=1016), INV),
    (dict(vs=1028), INV), (dict(slots=A + 2), INV), (dict(slots=None, n_tok=65), INV), (dict(status=A + 1), INV),
    (dict(n_tok=1 << 30), UNS), (dict(n_tok=1 << 62), UNS), (dict(n_tok=0), 0),
])
def test_cache_refusals(kvattn, over, want, read):
    assert write(kvattn, read, **over) == want


def prefill(kvattn, **over):
    a = dict(q=A, qs=4096, k=A, ks=1024, v=A, vs=1024, off=A, n_seq=2, n_tok=100, H=32, Hk=8, D=128, scale=0.1, out=A, lse=A,
             ws=A, ws_bytes=1 << 20, stream=None)
    a.update(over)
    return kvattn.lib.kvattn_prefill(*a.values())


@pytest.mark.parametrize("over,want", [
    (dict(D=64), UNS), (dict(H=30), INV), (dict(Hk=0), INV), (dict(H=129, Hk=1), UNS), (dict(n_tok=-1), INV), (dict(n_seq=-1), INV),
    (dict(scale=float("nan")), INV), (dict(q=None), INV), (dict(q=A + 8), INV), (dict(qs=4088), INV), (dict(ks=1020), INV),
    (dict(vs=1025), INV), (dict(off=None), INV), (dict(off=A + 2), INV), (dict(out=None), INV), (dict(out=A + 8), INV),
    (dict(lse=A + 2), INV), (dict(ws=None), INV), (dict(ws=A + 128), INV), (dict(ws_bytes=255), WS), (dict(n_tok=1 << 31), UNS),
    (dict(n_tok=1 << 27), UNS), (dict(n_tok=0), 0), (dict(n_seq=0), 0),
])
def test_prefill_refusals(kvattn, over, want):
    assert prefill(kvattn, **over) == want


def chunk(kvattn, **over):
    a = dict(q=A, qs=4096, off=A, n_tok=100, k=A, v=A, ksc=None, vsc=None, kv_type=0, n_cells=4096, plan=None, stride=0, lens=A,
             n_seq=2, max_len=4096, H=32, Hk=8, D=128, scale=0.1, out=A, lse=None, ws=A, ws_bytes=1 << 40, stream=None)
    a.update(over)
    return kvattn.lib.kvattn_prefill_chunk(*a.values())


@pytest.mark.parametrize("over,want", [
    (dict(D=64), UNS), (dict(H=30), INV), (dict(H=129, Hk=1), UNS), (dict(n_cells=1 << 62, n_seq=4), UNS),
    (dict(max_len=-1), INV), (dict(max_len=1 << 31), UNS), (dict(n_cells=0), INV), (dict(plan=A), INV), (dict(plan=A + 2, stride=128), INV),
    (dict(kv_type=5), INV), (dict(kv_type=1), INV), (dict(ksc=A, vsc=A), INV), (dict(kv_type=1, ksc=A, vsc=A + 4), INV),
    (dict(k=None), INV), (dict(v=A + 8), INV), (dict(q=A + 2), INV), (dict(qs=4090), INV), (dict(off=None), INV),
    (dict(lens=None), INV), (dict(lens=A + 1), INV), (dict(out=A + 4), INV), (dict(ws=None), INV), (dict(scale=float("inf")), INV),
    (dict(ws_bytes=0), WS), (dict(n_tok=0), 0), (dict(n_seq=0), 0),
])
def test_chunk_refusals(kvattn, over, want):
    assert chunk(kvattn, **over) == want


def test_workspaces(kvattn, monkeypatch):
    f, g = kvattn.kvattn_prefill_workspace_bytes, kvattn.kvattn_prefill_chunk_workspace_bytes
    assert f(100, 2, 32, 8, 128) == 256 and f(100, 2, 30, 8, 128) == 0 and f(100, 2, 32, 8, 96) == 0
    assert g(100, 1, 32, 8, 128, 128) == 256                         # units of one tile are not cut
    assert g(100, 1, 32, 8, 128, -1) == 0 and g(100, 1, 32, 8, 128, 1 << 31) == 0 and g(100, 1, 31, 8, 128, 128) == 0
    monkeypatch.setenv("KVATTN_PREFILL_CTAS", "0")
    assert g(100, 1, 32, 8, 128, 1 << 20) == 256


def test_wrapper_checks(kvattn):
    torch = pytest.importorskip("torch")
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        kvattn.prefill(h(4, 4, 128), h(4, 2, 128), h(4, 2, 256), off)
    with pytest.raises(ValueError):
        kvattn.prefill(h(4, 4, 128).float(), h(4, 2, 128), h(4, 2, 128), off)
    with pytest.raises(ValueError):
        kvattn.prefill(h(4, 128, 4).transpose(1, 2), h(4, 2, 128), h(4, 2, 128), off)
    with pytest.raises(ValueError):
        kvattn.prefill(h(4, 4, 128), h(4, 2, 128), h(4, 2, 128), off.long())
    with pytest.raises(ValueError):
        kvattn.prefill_chunk(h(4, 4, 128), off, h(9, 2, 128), h(9, 2, 128), off[:1], n_cells=10)
    with pytest.raises(ValueError):
        kvattn.prefill_chunk(h(4, 4, 128), off, h(9, 2, 64), h(9, 2, 64), off[:1])
    with pytest.raises(ValueError):
        kvattn.cache_write(h(4, 2, 128), h(4, 2, 128), off, h(9, 2, 128), h(9, 2, 128))     # two slots for four tokens
    with pytest.raises(ValueError):
        kvattn.cache_read(torch.zeros(9, 2, 128, dtype=torch.int8), torch.zeros(9, 2, 128, dtype=torch.int8), off, head_dim=128)
    with pytest.raises(ValueError):
        kvattn.rope(h(4, 4, 128), h(5, 2, 128), torch.zeros(4, dtype=torch.int32), kvattn.RopeTable(off, 1.0, 128))
    for kw in (dict(q_out=h(4, 2, 128)), dict(k_out=h(3, 2, 128)), dict(q_out=h(4, 4, 128).float())):
        with pytest.raises(ValueError):
            kvattn.rope(h(4, 4, 128), h(4, 2, 128), torch.zeros(4, dtype=torch.int32), kvattn.RopeTable(off, 1.0, 128), **kw)
    with pytest.raises(ValueError):
        kvattn.rope(None, None, torch.zeros(4, dtype=torch.int32), kvattn.RopeTable(off, 1.0, 128))


def test_wrappers_refuse_host_tensors(kvattn):
    torch = pytest.importorskip("torch")
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    off, slots = torch.tensor([0, 4], dtype=torch.int32), torch.arange(4, dtype=torch.int32)
    calls = [lambda: kvattn.prefill(h(4, 4, 128), h(4, 2, 128), h(4, 2, 128), off),
             lambda: kvattn.prefill_chunk(h(4, 4, 128), off, h(9, 2, 128), h(9, 2, 128), off[1:]),
             lambda: kvattn.cache_write(h(4, 2, 128), h(4, 2, 128), slots, h(9, 2, 128), h(9, 2, 128)),
             lambda: kvattn.cache_read(h(9, 2, 128), h(9, 2, 128), slots, head_dim=128),
             lambda: kvattn.rope(h(4, 4, 128), h(4, 2, 128), slots, kvattn.RopeTable(off, 1.0, 128))]
    for call in calls:
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
