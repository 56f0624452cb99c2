"""Calls that the prompt-side operators allow and that are easy to get wrong: many sequences, cells
named twice, runs that begin before the first cell or end behind the last, caches beyond 2^31
elements, lengths and offsets outside their range."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import test_gpu_prefill as P  # noqa: E402

ctas = P.ctas


def many(n_seq, top, seed):
    g = torch.Generator().manual_seed(seed)
    return [0 if int(torch.randint(0, 4, (1,), generator=g)) == 0 else int(torch.randint(1, top, (1,), generator=g))
            for _ in range(n_seq)]


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n_seq", [31, 32, 33, 64, 65, 150])
def test_prefill_many_sequences(kvattn, n_seq, D):
    P.check_prefill(kvattn, many(n_seq, 60, n_seq), 4, 2, D)
    P.check_prefill(kvattn, [0] * (n_seq - 1) + [140], 4, 2, D)


@pytest.mark.parametrize("n", [None, 0, 3, 41])
@pytest.mark.parametrize("kind,plan", [("f16", False), ("q8_0", True)])
@pytest.mark.parametrize("n_seq", [33, 70])
def test_chunk_many_sequences(kvattn, ctas, n_seq, kind, plan, n):
    ctas(n)
    new = many(n_seq, 40, n_seq)
    old = many(n_seq, 900, n_seq + 1)
    P.check_chunk(kvattn, P.make_chunk(kind, new, [a + b for a, b in zip(new, old)], 4, 1, 128, plan, 0.1))


def pool(kind, cells, Hk, D, plan, new, seed=13):
    """A chunk call of one sequence over `plan` (cells, -1: hole) of a pool."""
    g = U.gen(seed)
    k, v, ks, vs = U.cache_planes(g, kind, cells, Hk, D)
    table = torch.tensor(plan, dtype=torch.int32, device="cuda")[None]
    return {"q": U.halves(g, new, 2 * Hk, D), "offsets": U.ints([0, new]), "lens": U.ints([len(plan)]), "new": [new],
            "L": [len(plan)], "H": 2 * Hk, "Hk": Hk, "D": D, "plan": table, "n_cells": cells, "k": k, "v": v, "ks": ks, "vs": vs}


@pytest.mark.parametrize("kind", P.KINDS)
@pytest.mark.parametrize("D", [128, 256])
def test_runs_over_both_ends_of_the_cache(kvattn, ctas, kind, D):
    for n in (None, 4):
        ctas(n)
        # the run of the first tile would begin at cell -5, the second's at -100
        P.check_chunk(kvattn, pool(kind, 400, 2, D, [-1] * 5 + list(range(123)) + [-1] * 100 + list(range(28)) + list(range(200, 290)), 30))
        # the last tiles' would end behind the last cell
        P.check_chunk(kvattn, pool(kind, 300, 2, D, list(range(172, 300)) + [-1] * 3 + list(range(270, 300)) + [-1] * 95, 30))


@pytest.mark.parametrize("kind", P.KINDS)
def test_cells_named_twice(kvattn, ctas, kind):
    for n in (None, 3):
        ctas(n)
        P.check_chunk(kvattn, pool(kind, 40, 2, 128, [7] * 200 + [i % 40 for i in range(300)] + [39, 39], 20))


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_cells_beyond_32_bits(kvattn, kind):
    """The last cells of a cache of more than 2^31 elements, as runs and one by one."""
    cells, Hk, D = 1_060_000, 8, 256
    g = U.gen(17)
    used = 2000
    small = U.cache_planes(g, kind, used, Hk, D)
    big = []
    for x in small:
        if x is None:
            big.append(None)
            continue
        y = torch.empty((cells,) + x.shape[1:], dtype=x.dtype, device="cuda")
        y[-used:] = x
        big.append(y)
    assert big[0].numel() > 2 ** 31
    run = list(range(100, 900))
    for order in (run, [int(i) for i in torch.randperm(used, generator=torch.Generator().manual_seed(1))[:700]]):
        c = pool(kind, used, Hk, D, order, 25)
        c |= dict(zip(("k", "v", "ks", "vs"), small))
        want, wl = P.check_chunk(kvattn, c)
        far = c | {"plan": torch.where(c["plan"] >= 0, c["plan"] + (cells - used), -1).to(torch.int32), "n_cells": cells}
        far |= dict(zip(("k", "v", "ks", "vs"), big))
        got, gl = P.call_chunk(kvattn, far)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    del big, far
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [None, 0, 6])
def test_lengths_outside_the_cache(kvattn, ctas, n):
    """A length below zero is none, one above the cache (or max_len) is all of it."""
    ctas(n)
    c = P.make_chunk("f16", [20, 30, 10], [400, 400, 400], 4, 2, 128, False)
    c["k"].nan_to_num_(0.5)
    c["v"].nan_to_num_(0.5)
    c["lens"] = U.ints([-7, 2147483647, 405])
    out, lse = P.call_chunk(kvattn, c, max_len=1 << 20)
    c["lens"], c["L"] = U.ints([0, 405, 405]), [0, 405, 405]
    want, wl = P.call_chunk(kvattn, c, max_len=1 << 20)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    assert bool((out[:20] == 0).all()) and bool(torch.isneginf(lse[:20]).all())
    o, l, to, tl = P.expect_chunk(c, 1, 1 / math.sqrt(128))
    U.check(out[20:50], o, to, "out")
    U.check(lse[20:50], l, tl, "lse")


@pytest.mark.parametrize("n", [None, 0, 6])
def test_chunk_offsets_out_of_order_stay_in_bounds(kvattn, ctas, n):
    ctas(n)
    g = U.gen(6)
    q = U.halves(g, 50, 4, 128)
    c = P.make_chunk("f16", [50, 1, 1], [3000, 3000, 3000], 4, 2, 128, False)
    out = torch.full((60, 4, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((60, 4), 7.0, dtype=torch.float32, device="cuda")
    ws = kvattn.prefill_chunk_workspace(50, 3, 4, 2, 128, 3000)
    kvattn.prefill_chunk(q, U.ints([-5, 20, 10, 99]), c["k"], c["v"], c["lens"], n_cells=c["n_cells"], max_len=3000, out=out[:50],
                         lse=lse[:50], ws=ws)
    assert kvattn.kvattn_workspace_status(ws) == 0
    assert bool((out[50:] == 7.0).all()) and bool((lse[50:] == 7.0).all())


def test_nothing_to_do(kvattn):
    """No tokens, or no sequences: nothing is launched or written."""
    h = dict(dtype=torch.float16, device="cuda")
    q, k = torch.empty(0, 4, 128, **h), torch.empty(0, 2, 128, **h)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    cache = torch.ones(9, 2, 128, **h)
    a, b = kvattn.rope(q, k, none, kvattn.rope_table(128))
    assert a.shape == q.shape and b.shape == k.shape
    for slots in (none, None):
        kvattn.cache_write(k, k, slots, cache, cache)
    assert bool((cache == 1).all())
    a, b = kvattn.cache_read(cache, cache, none, head_dim=128)
    assert a.shape == b.shape == k.shape
    out, lse = kvattn.prefill(q, k, k, U.ints([0]))
    assert out.shape == q.shape and lse.shape == (0, 4)
    kvattn.prefill(q, k, k, U.ints([0, 0, 0]))
    kvattn.prefill_chunk(q, U.ints([0, 0]), cache, cache, U.ints([9]))
    x = torch.full((3, 4, 128), 7.0, **h)   # three tokens of no sequence
    for off, lens in ((U.ints([0]), none), (U.ints([3, 3]), U.ints([9]))):
        out = x.clone()
        kvattn.prefill_chunk(x, off, cache, cache, lens, out=out)
        kvattn.prefill(x, x[:, :2], x[:, :2], off, out=out)
        assert bool((out == 7.0).all())
    torch.cuda.synchronize()
