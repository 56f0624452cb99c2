"""Causal attention of packed prompts and of chunks over caches, against the definition in 64 bits.
Tolerances: prompt_util.attend derives each element's from the kernels' roundings."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402

KINDS = ("f16", "q8_0", "q8_0_q4_0", "q4_0")


def run_prefill(kv, lens, H, Hk, D, scale=None, seed=1, first=0, behind=0, fused=False, edit=None):
    g = U.gen(seed)
    T = first + sum(lens) + behind
    if fused:  # q, k and v as slices of one projection
        x = U.halves(g, T, H + 2 * Hk, D)
        q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    else:
        q, k, v = U.halves(g, T, H, D), U.halves(g, T, Hk, D), U.halves(g, T, Hk, D)
    if edit is not None:
        edit(q, k, v)
    off = U.offsets_of(lens, first)
    out = torch.full((T, H, D), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda")
    kv.prefill(q, k, v, U.ints(off), scale=scale, out=out, lse=lse)
    torch.cuda.synchronize()
    s = 1.0 / math.sqrt(D) if scale is None else scale
    for a, b in zip(off, off[1:]):
        if a < b:
            lim = torch.arange(1, b - a + 1, device="cuda")
            o, l, to, tl = U.attend(q[a:b], k[a:b].double(), v[a:b].double(), lim, s)
            yield (a, b), (out[a:b], o, to), (lse[a:b], l, tl)
    for a, b in ((0, first), (off[-1], T)):  # tokens of no sequence are left as they were
        assert bool((out[a:b] == 7.0).all()) and bool((lse[a:b] == 7.0).all())


def check_prefill(*args, **kw):
    for where, o, l in run_prefill(*args, **kw):
        U.check(*o, f"out {where}")
        U.check(*l, f"lse {where}")


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255, 256, 257], [0, 5, 0, 300, 1, 0], [1000], [640, 33]])
def test_prefill_lengths(kvattn, lens, D):
    check_prefill(kvattn, lens, 8, 2, D)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 2), (3, 1), (5, 1), (6, 2), (7, 1), (8, 1), (12, 4), (40, 1)])
def test_prefill_heads(kvattn, H, Hk, D):
    check_prefill(kvattn, [61, 200], H, Hk, D, seed=2)


@pytest.mark.parametrize("D", [128, 256])
def test_prefill_strided_rows_and_tokens_of_no_sequence(kvattn, D):
    check_prefill(kvattn, [70, 3, 140], 4, 2, D, first=9, behind=21, fused=True)


@pytest.mark.parametrize("scale", [0.0, -0.07, 0.5])
def test_prefill_scale(kvattn, scale):
    check_prefill(kvattn, [150, 20], 4, 2, 128, scale=scale)


@pytest.mark.parametrize("D", [128, 256])
def test_prefill_growing_maximum(kvattn, D):
    # scores grow along the cells, so the running maximum moves in every tile
    def edit(q, k, v):
        n = k.shape[0]
        q[..., 0] = 4.0
        k[..., 0] = (torch.arange(n, device="cuda") / 8).half()[:, None]
    check_prefill(kvattn, [900], 4, 1, D, edit=edit)
    # ... or fall from a first cell that outweighs the rest by far
    def edit2(q, k, v):
        q[..., 0] = 4.0
        k[..., 0] = 0.0
        k[0, :, 0] = 30.0
    check_prefill(kvattn, [500], 4, 1, D, edit=edit2)


def test_prefill_many_small_weights(kvattn):
    # one heavy cell and thousands 2^-15 as heavy: half of the mass lies in the small ones
    def edit(q, k, v):
        q[:] = 0.0
        q[..., 0] = 1.0
        k[:] = 0.0
        k[0, :, 0] = 15 * math.log(2.0) * math.sqrt(128)
    check_prefill(kvattn, [4096], 1, 1, 128, edit=edit)


@pytest.mark.parametrize("D,H", [(128, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
def test_prefill_later_values_that_are_not_finite_stay_away_from_earlier_rows(kvattn, D, H, value):
    def edit(q, k, v):
        v[50, 0, 3] = value
        v[200, 0, D - 1] = value
        v[201, 0, :] = value
    check_prefill(kvattn, [260], H, 1, D, edit=edit)

    def edit_k(q, k, v):  # a key that is not finite: rows before it do not notice
        k[131, 0, 5] = value
    for where, (o, want, tol), (l, wl, tl) in run_prefill(kvattn, [200], H, 1, D, edit=edit_k):
        U.check(o[:131], want[:131], tol[:131], "out")
        U.check(l[:131], wl[:131], tl[:131], "lse")


def test_prefill_a_query_that_is_not_finite_spoils_its_own_row_only(kvattn):
    def edit(q, k, v):
        q[77, 1, 3] = float("nan")
    for where, (o, want, tol), (l, wl, tl) in run_prefill(kvattn, [130], 4, 2, 128, edit=edit):
        assert bool(torch.isnan(o[77, 1]).all()) and bool(torch.isnan(l[77, 1]))
        keep = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
        keep[77, 1] = False
        U.check(o[keep], want[keep], tol[keep], "out")


def make_chunk(kind, new, lens, H, Hk, D, plan, holes=0.0, seed=3, spare=2):
    """Inputs of a chunk call; cells no sequence owns hold NaN."""
    g = U.gen(seed)
    S = len(new)
    c = {"q": U.halves(g, max(sum(new), 1), H, D)[:sum(new)], "offsets": U.ints(U.offsets_of(new)), "lens": U.ints(lens),
         "new": new, "L": lens, "H": H, "Hk": Hk, "D": D, "plan": None}
    if plan:
        recs = [-(-n // 128) for n in lens]
        pool = sum(recs) + spare
        perm = torch.randperm(pool, generator=g, device="cuda")
        stride = 128 * max(max(recs), 1)
        table = torch.full((S, stride), -1, dtype=torch.int32, device="cuda")
        at = 0
        for s, n in enumerate(lens):
            ids = perm[at:at + recs[s]].sort().values
            at += recs[s]
            cells = (ids[:, None] * 128 + torch.arange(128, device="cuda")).flatten()[:n].to(torch.int32)
            drop = torch.rand(n, generator=g, device="cuda") < holes
            table[s, :n] = torch.where(drop, -1, cells)
        c["plan"], cells = table, pool * 128
        owned = torch.zeros(cells, dtype=torch.bool, device="cuda")
        owned[table[table >= 0].long()] = True
    else:
        cells = max(lens) + 5
        owned = (torch.arange(cells, device="cuda")[None, :] < torch.tensor(lens, device="cuda")[:, None]).flatten()
    total = owned.numel()
    k, v, ks, vs = U.cache_planes(g, kind, total, Hk, D)
    for rows, sc in ((k, ks), (v, vs)):
        (rows if sc is None else sc)[~owned] = float("nan")
    c |= {"n_cells": cells, "k": k, "v": v, "ks": ks, "vs": vs}
    return c


@pytest.fixture
def ctas(monkeypatch):
    """Sets how many CTAs share a chunk call's work (None: the library's choice, 0: whole units)."""
    def set_(n):
        if n is None:
            monkeypatch.delenv("KVATTN_PREFILL_CTAS", raising=False)
        else:
            monkeypatch.setenv("KVATTN_PREFILL_CTAS", str(n))
    return set_


def call_chunk(kv, c, lse=True, **kw):
    T, H, D = c["q"].shape
    out = torch.full((T, H, D), 7.0, dtype=torch.float16, device="cuda")
    l = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda") if lse else None
    kv.prefill_chunk(c["q"], c["offsets"], c["k"], c["v"], c["lens"], n_cells=c["n_cells"], cell_plan=c["plan"],
                     k_scales=c["ks"], v_scales=c["vs"], out=out, lse=l, **({"max_len": max(c["L"])} | kw))
    return out, l


def expect_chunk(c, s, scale):
    n, L, D = c["new"][s], c["L"][s], c["D"]
    if c["plan"] is None:
        cells = s * c["n_cells"] + torch.arange(L, device="cuda")
        lim = torch.arange(n, device="cuda") + L - n + 1
    else:
        row = c["plan"][s, :L].long()
        cells = row[row >= 0]
        # the valid cells among the first L - n + 1 + t entries
        count = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), (row >= 0).cumsum(0)))
        lim = count[(torch.arange(n, device="cuda") + L - n + 1).clamp(0, L)]
    k = U.dequant(c["k"][cells], None if c["ks"] is None else c["ks"][cells], D)
    v = U.dequant(c["v"][cells], None if c["vs"] is None else c["vs"][cells], D)
    a = sum(c["new"][:s])
    return U.attend(c["q"][a:a + n], k, v, lim, scale, rounded_k=c["ks"] is not None)


def check_chunk(kv, c, **kw):
    out, lse = call_chunk(kv, c, **kw)
    scale = kw.get("scale") or 1.0 / math.sqrt(c["D"])
    a = 0
    for s, n in enumerate(c["new"]):
        if n:
            o, l, to, tl = expect_chunk(c, s, scale)
            U.check(out[a:a + n], o, to, f"out of sequence {s}")
            U.check(lse[a:a + n], l, tl, f"lse of sequence {s}")
        a += n
    return out, lse


@pytest.mark.parametrize("n", [None, 0, 5, 37])
@pytest.mark.parametrize("plan,holes", [(False, 0.0), (True, 0.0), (True, 0.3)])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_chunk_kinds(kvattn, ctas, kind, D, plan, holes, n):
    c = make_chunk(kind, [70, 1, 0, 33], [700, 513, 0, 33], 8, 2, D, plan, holes)
    ctas(n)
    check_chunk(kvattn, c)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new,lens", [([1], [1]), ([1], [128]), ([1], [129]), ([3], [2]), ([200], [150]), ([300], [300]),
                                      ([128, 128], [128, 256]), ([5, 6, 7], [0, 6, 1000]), ([260], [1500])])
def test_chunk_lengths(kvattn, ctas, new, lens, D):
    check_chunk(kvattn, make_chunk("f16", new, lens, 6, 2, D, False))
    ctas(11)
    check_chunk(kvattn, make_chunk("q8_0", new, lens, 6, 2, D, True, 0.1))


@pytest.mark.parametrize("H,Hk", [(1, 1), (5, 1), (16, 2), (7, 7), (48, 3)])
def test_chunk_heads(kvattn, ctas, H, Hk):
    check_chunk(kvattn, make_chunk("f16", [50, 90], [400, 90], H, Hk, 128, True, 0.1))
    ctas(13)
    check_chunk(kvattn, make_chunk("q4_0", [50, 90], [400, 90], H, Hk, 128, False))


@pytest.mark.parametrize("kind", KINDS)
def test_chunk_all_holes_and_scales(kvattn, ctas, kind):
    c = make_chunk(kind, [40], [600], 4, 2, 128, True, 0.2)
    c["plan"][0, :256] = -1          # whole tiles of holes
    check_chunk(kvattn, c)
    ctas(9)
    check_chunk(kvattn, c, scale=-0.05)
    c["plan"][:] = -1                # nothing to see at all
    for n in (9, 0):
        ctas(n)
        out, lse = call_chunk(kvattn, c)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("D", [128, 256])
def test_chunk_cells_in_any_order(kvattn, ctas, D):
    """Plans whose tiles are no run of cells: entries shuffled, with and without holes."""
    g = U.gen(9)
    for kind in ("f16", "q8_0"):
        c = make_chunk(kind, [90, 5], [500, 300], 4, 2, D, True, 0.2)
        for s, n in enumerate(c["L"]):
            c["plan"][s, :n] = c["plan"][s, torch.randperm(n, generator=g, device="cuda")]
        check_chunk(kvattn, c)
        ctas(7)
        check_chunk(kvattn, c)
        ctas(None)


def test_without_tensor_maps(kvattn):
    """KVATTN_TMA=0: K and V by ordinary loads (read once per process, so in a child of its own)."""
    import subprocess
    import sys
    code = ("from kv_cache_decode_02_gb300 import kvattn as K\n"
            "from tests import test_gpu_prefill as t\n"
            "t.check_prefill(K, [300, 70], 8, 2, 128)\n"
            "t.check_chunk(K, t.make_chunk('f16', [60], [400], 4, 1, 256, True, 0.1))\n"
            "t.check_chunk(K, t.make_chunk('q8_0_q4_0', [60], [400], 4, 1, 256, True, 0.1))\n"
            "t.check_chunk(K, t.make_chunk('q4_0', [60], [400], 4, 1, 128, False))\n")
    import os
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, KVATTN_TMA="0"), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_results_do_not_depend_on_how_the_work_is_cut(kvattn, ctas):
    c = make_chunk("f16", [130, 1, 40], [3000, 2000, 40], 8, 2, 128, True, 0.1)
    got = []
    for n in (0, 2, 5, 40, 150):
        ctas(n)
        got.append(check_chunk(kvattn, c))
        again = call_chunk(kvattn, c)
        assert torch.equal(got[-1][0], again[0]) and torch.equal(got[-1][1], again[1])


@pytest.mark.parametrize("H", [12, 4])
@pytest.mark.parametrize("n", [2, 7, 40, 150])
def test_blocks_of_one_and_two_row_groups_share_the_line(kvattn, ctas, n, H):
    """Contiguous f16 caches, where a tile for one row group counts less: sequences whose last block
    has one group, both, and is alone, cut in few and many shares."""
    ctas(n)
    check_chunk(kvattn, make_chunk("f16", [130, 1, 45, 22, 64], [2500, 1900, 45, 3100, 1000], H, 2, 128, False))


@pytest.mark.parametrize("kind,plan,D", [("f16", False, 128), ("f16", True, 256), ("q8_0", True, 128), ("q4_0", False, 256)])
@pytest.mark.parametrize("n", [3, 8, 29])
def test_pieces_that_go_around(kvattn, ctas, kind, plan, D, n):
    """Several blocks of a KV head: a piece's whole tiles begin somewhere inside it.  A score that
    rules its row sits in the first tiles, so what is added after them has to be small."""
    ctas(n)
    c = make_chunk(kind, [300], [4000], 8, 2, D, plan, 0.1)
    if kind == "f16":
        c["k"][(c["plan"][0, 64:72].clamp(min=0).long() if plan else torch.arange(64, 72, device="cuda"))] *= 4
    check_chunk(kvattn, c)


def test_rows_that_a_block_does_not_have(kvattn, ctas):
    """A call full of queries that are not finite, then calls whose blocks leave rows of a group
    empty (their rows of shared memory may still hold those): nothing of them shows."""
    for n in (None, 4):
        ctas(n)
        c = make_chunk("f16", [200], [900], 6, 1, 128, False)
        c["q"][:] = float("nan")
        out, _ = call_chunk(kvattn, c)
        assert bool(torch.isnan(out).all())
        check_chunk(kvattn, make_chunk("f16", [3], [900], 6, 1, 128, False))
        check_chunk(kvattn, make_chunk("q8_0", [1, 23], [900, 700], 5, 1, 128, True, 0.1))
        c["q"][:] = float("inf")
        call_chunk(kvattn, c)
        check_chunk(kvattn, make_chunk("f16", [3, 30], [900, 30], 3, 1, 256, False))


@pytest.mark.parametrize("kind", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("n", [0, 6])
def test_chunk_values_that_are_not_finite(kvattn, ctas, kind, n):
    ctas(n)
    # in cells that only the later new tokens see
    c = make_chunk(kind, [60], [500], 4, 1, 128, False)
    if kind == "f16":
        c["v"][470, 0, 9] = float("inf")
        c["v"][495, 0, :] = float("nan")
    else:
        c["vs"][470, 0, 1] = float("nan")
        c["vs"][495, 0, 3] = float("nan")
    check_chunk(kvattn, c)


def test_chunk_agrees_with_decode(kvattn):
    # one token per sequence: the decode entry point's result, rounded to half
    c = make_chunk("f16", [1, 1, 1], [1000, 129, 1], 8, 2, 128, True, 0.1)
    out, lse = call_chunk(kvattn, c)
    want, wl = kvattn.decode(c["q"], c["k"], c["v"], c["lens"], split=256, cell_plan=c["plan"])
    torch.cuda.synchronize()
    assert float((out.float() - want).abs().max()) <= 4e-3   # both within 2e-3 of the definition here
    assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
    some = ~torch.isneginf(wl)
    assert float((lse[some] - wl[some]).abs().max()) <= 2e-4


def test_chunk_of_a_whole_prompt_agrees_with_prefill(kvattn, ctas):
    ctas(0)
    g = U.gen(5)
    T, H, Hk, D = 600, 8, 2, 128
    q, k, v = U.halves(g, T, H, D), U.halves(g, T, Hk, D), U.halves(g, T, Hk, D)
    off = U.ints([0, T])
    a, la = kvattn.prefill(q, k, v, off)
    lse = torch.empty((T, H), dtype=torch.float32, device="cuda")
    b, lb = kvattn.prefill_chunk(q, off, k, v, U.ints([T]), lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)         # the same tiles in the same order


def test_chunk_long_cache(kvattn):
    c = make_chunk("q8_0_q4_0", [130], [40000], 4, 1, 128, False)
    check_chunk(kvattn, c)
    c = make_chunk("f16", [17, 1], [30011, 9000], 4, 1, 256, True, 0.1)
    check_chunk(kvattn, c)


def test_chunk_bad_plan_entries_are_masked_and_flagged(kvattn):
    c = make_chunk("f16", [20], [300], 4, 2, 128, True, 0.0)
    good = c["plan"].clone()
    c["plan"][0, 17] = c["n_cells"]
    c["plan"][0, 140] = -2
    c["plan"][0, 141] = 2147483647
    ws = kvattn.prefill_chunk_workspace(20, 1, 4, 2, 128, 300)
    out, lse = call_chunk(kvattn, c, ws=ws)
    assert kvattn.kvattn_workspace_status(ws, clear=True) == kvattn.KVATTN_DEVICE_BAD_PLAN_ENTRY
    c["plan"] = good
    for i in (17, 140, 141):
        c["plan"][0, i] = -1
    want, wl = call_chunk(kvattn, c, ws=ws)
    assert kvattn.kvattn_workspace_status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_offsets_out_of_order_stay_in_bounds(kvattn):
    # clamped to [0, n_tok] and to non-decreasing: no row outside is read or written
    g = U.gen(6)
    q, k, v = U.halves(g, 50, 4, 128), U.halves(g, 50, 4, 128), U.halves(g, 50, 4, 128)
    out = torch.full((60, 4, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((60, 4), 7.0, dtype=torch.float32, device="cuda")
    kvattn.prefill(q, k, v, U.ints([-5, 20, 10, 99]), out=out[:50], lse=lse[:50])
    torch.cuda.synchronize()
    assert bool((out[50:] == 7.0).all()) and bool((lse[50:] == 7.0).all())


def test_prefill_in_a_graph_on_another_stream(kvattn):
    g = U.gen(7)
    T, H, Hk, D = 300, 8, 2, 128
    q, k, v = U.halves(g, T, H, D), U.halves(g, T, Hk, D), U.halves(g, T, Hk, D)
    off = U.ints([0, 100, 300])
    ws = kvattn.prefill_workspace(T, 2, H, Hk, D)
    want, _ = kvattn.prefill(q, k, v, off)
    c = make_chunk("q8_0", [70], [3000], 8, 2, 128, False)
    cws = kvattn.prefill_chunk_workspace(70, 1, 8, 2, 128, 3000)
    cwant, clse = call_chunk(kvattn, c)
    out, lse = torch.zeros_like(want), torch.zeros((T, H), dtype=torch.float32, device="cuda")
    cout, cl = torch.zeros_like(cwant), torch.zeros_like(clse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvattn.prefill(q, k, v, off, out=out, lse=lse, ws=ws)
        kvattn.prefill_chunk(c["q"], c["offsets"], c["k"], c["v"], c["lens"], n_cells=c["n_cells"], k_scales=c["ks"],
                             v_scales=c["vs"], max_len=3000, out=cout, lse=cl, ws=cws)
    for _ in range(3):
        out.zero_()
        cout.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(cout, cwant)
    # two streams at once, a workspace each
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(cwant) for _ in range(2)]
    wss = [kvattn.prefill_chunk_workspace(70, 1, 8, 2, 128, 3000) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for st, o, w in ((s1, outs[0], wss[0]), (s2, outs[1], wss[1])):
            kvattn.prefill_chunk(c["q"], c["offsets"], c["k"], c["v"], c["lens"], n_cells=c["n_cells"], k_scales=c["ks"],
                                 v_scales=c["vs"], max_len=3000, out=o, ws=w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, cwant) for o in outs)


def test_a_wait_that_runs_out_is_reported(kvattn, monkeypatch):
    g = U.gen(8)
    q, k, v = U.halves(g, 256, 4, 128), U.halves(g, 256, 2, 128), U.halves(g, 256, 2, 128)
    ws = kvattn.prefill_workspace(256, 1, 4, 2, 128)
    monkeypatch.setenv("KVATTN_DEBUG_STALL_TX", "16")
    kvattn.prefill(q, k, v, U.ints([0, 256]), ws=ws)
    assert kvattn.kvattn_workspace_status(ws, clear=True) == kvattn.KVATTN_DEVICE_WAIT_TIMEOUT
    monkeypatch.delenv("KVATTN_DEBUG_STALL_TX")
    kvattn.prefill(q, k, v, U.ints([0, 256]), ws=ws)
    assert kvattn.kvattn_workspace_status(ws) == 0
