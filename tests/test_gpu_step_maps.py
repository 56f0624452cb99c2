"""A step's maps against a walk over the sequences on the host: whole numbers, equal everywhere."""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests import step_util as W  # noqa: E402


def rows(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(kv, lens, new, tables, free, n_free, block, n_cells, n_tok, plan=None, whole=True, status=True):
    want, bits = W.maps(lens, new, tables, free, n_free, block, n_cells, n_tok, plan, whole)
    S = len(lens)
    t = rows(tables).view(S, -1)
    pl = None if plan is None else rows(plan).view(S, -1)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = [x.clone() for x in (rows(lens), rows(new))]
    out = kv.step_maps_buffers(S, n_tok)
    for x in (out.offsets, out.seq_lens, out.positions, out.slots, out.n_free):
        x.fill_(-99)
    ls, ns = keep[0].clone(), keep[1].clone()
    kv.step_maps(ls, ns, t, None if free is None else rows(free), None if free is None else rows([n_free]), block_cells=block,
                 n_cells=n_cells, plan=pl, whole_plan=whole, status=word if status else None, out=out)
    torch.cuda.synchronize()
    got = {"tables": t, "offsets": out.offsets, "seq_lens": out.seq_lens, "positions": out.positions, "slots": out.slots}
    if plan is not None:
        got["plan"] = pl
    for name, x in got.items():
        assert x.tolist() == want[name], name
    assert out.n_free.item() == (-99 if free is None else want["n_free"])
    assert not status or word.item() == bits
    assert torch.equal(ls, keep[0]) and torch.equal(ns, keep[1])


def draw(rng, S, block, top, most, spare=4, tight=False):
    """Sequences that hold scattered blocks of a pool; the rest of it is free."""
    lens = [rng.randint(0, top) for _ in range(S)]
    new = [rng.randint(0, most) for _ in range(S)]
    stride = -(-(top + most) // block) + rng.randint(0, 2)
    ids = list(range(S * stride + spare))
    rng.shuffle(ids)
    tables = [[ids.pop() if e * block < n else -1 for e in range(stride)] for n in lens]
    need = sum(-(-(n + t) // block) - -(-n // block) for n, t in zip(lens, new))
    n_free = rng.randint(0, need) if tight else len(ids)
    return lens, new, tables, ids, n_free, (S * stride + spare) * block


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("block", [4, 16, 128, 512])
@pytest.mark.parametrize("S", [1, 2, 33, 257, 600])
def test_sequences_and_blocks(kvattn, S, block, whole):
    rng = random.Random(S * block)
    lens, new, tables, free, n_free, cells = draw(rng, S, block, 700 if S < 100 else 150, 40)
    stride = len(tables[0]) * block
    plan = [[rng.randint(-1, 50) for _ in range(stride)] for _ in range(S)]
    check(kvattn, lens, new, tables, free, n_free, block, cells, sum(new) + rng.randint(0, 50), plan, whole)


@pytest.mark.parametrize("seed", range(12))
def test_a_free_list_that_runs_out(kvattn, seed):
    rng = random.Random(seed)
    lens, new, tables, free, n_free, cells = draw(rng, rng.choice([3, 40, 300]), 16, 100, 60, tight=True)
    plan = [[7] * (len(tables[0]) * 16) for _ in lens]
    check(kvattn, lens, new, tables, free, n_free, 16, cells, sum(new), plan, seed % 2 == 0)


@pytest.mark.parametrize("stride", [1, 2, 3, 4, 5, 127, 130, 1001])
def test_plan_rows_of_any_length(kvattn, stride):
    """Rows that begin off 16 bytes, and end inside a block; sequences that pass them are not served."""
    rng = random.Random(stride)
    lens, new, tables, free, n_free, cells = draw(rng, 9, 8, max(stride - 2, 0), 4)
    check(kvattn, lens, new, tables, free, n_free, 8, cells, sum(new) + 3, [[5] * stride for _ in lens], True)
    check(kvattn, lens, new, tables, free, n_free, 8, cells, sum(new) + 3, [[5] * stride for _ in lens], False)


def test_lengths_and_rows_outside_their_range(kvattn):
    big = 2 ** 31 - 1
    tables = [[3, 1, -1, -1], [0, 2, 5, 4], [6, -1, -1, -1], [-1, -1, -1, -1], [7, -1, -1, -1]]
    free = [8, 9, 10, 11, 12, 13, 14, 15]
    for lens, new in [([20, 60, -5, 0, 3], [3, 5, 2, -7, 0]), ([20, 999, 5, 0, big], [3, 0, big, 1, big]),
                      ([-big, big, 0, 0, 0], [big, big, big, big, big]), ([16, 32, 48, 64, 0], [0, 0, 0, 0, 0])]:
        for n_tok in (0, 1, 6, 100):
            for n_free in (-3, 0, 2, 8, 99):
                check(kvattn, lens, new, tables, free, n_free, 16, 16 * 16, n_tok, [[1] * 64 for _ in lens], n_tok % 2 == 0)


def test_tables_that_are_complete(kvattn):
    """Nothing is taken: the tables hold every block; entries outside the cache are found."""
    tables = [[2, 0, 1, -1], [3, 99, 4, 5], [-2, 6, 7, 8]]
    for whole in (True, False):
        check(kvattn, [20, 16, 0], [20, 40, 33], tables, None, 0, 16, 9 * 16, 100, [[4] * 64 for _ in tables], whole)
    check(kvattn, [20, 16, 0], [20, 40, 33], tables, None, 0, 16, 9 * 16, 93, status=False)


def test_an_empty_free_list(kvattn):
    check(kvattn, [16, 3], [1, 4], [[0, -1], [1, -1]], [], 0, 16, 64, 5, [[9] * 32] * 2, True)


def test_no_sequences(kvattn):
    out = kvattn.step_maps_buffers(0, 5)
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    kvattn.step_maps(empty, empty, empty.view(0, 4), rows([1, 2, 3]), rows([2]), block_cells=16, n_cells=64, out=out)
    torch.cuda.synchronize()
    assert out.offsets.tolist() == [0] and out.positions.tolist() == [0] * 5 and out.slots.tolist() == [-1] * 5
    assert out.n_free.tolist() == [2]


def test_long_rows_and_many_new_tokens(kvattn):
    rng = random.Random(3)
    lens, new, tables, free, n_free, cells = draw(rng, 3, 128, 100000, 20000)
    plan = [[-1] * (len(tables[0]) * 128) for _ in lens]
    check(kvattn, lens, new, tables, free, n_free, 128, cells, sum(new), plan, True)
    check(kvattn, lens, new, tables, free, n_free, 128, cells, sum(new), plan, False)


def test_steps_one_after_the_other_captured(kvattn):
    """The step as a graph: lengths, free count and plan carried on by the program between replays."""
    rng = random.Random(5)
    S, block, n_tok = 6, 16, 24
    lens, new, tables, free, n_free, cells = draw(rng, S, block, 60, 4, spare=40)
    tables = [r + [-1] * 8 for r in tables]
    stride = len(tables[0]) * block
    plan = W.maps(lens, [0] * S, tables, free, n_free, block, cells, 0, [[0] * stride for _ in lens])[0]["plan"]
    d_lens, d_new, d_free, d_count = rows(lens), rows(new), rows(free), rows([n_free])
    d_tables, d_plan, out = rows(tables), rows(plan), kvattn.step_maps_buffers(S, n_tok)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    before = d_tables.clone()
    with torch.cuda.graph(graph):
        kvattn.step_maps(d_lens, d_new, d_tables, d_free, d_count, block_cells=block, n_cells=cells, plan=d_plan, whole_plan=False,
                         out=out)
        d_lens.copy_(out.seq_lens)
        d_count.copy_(out.n_free)
    assert torch.equal(d_tables, before)
    for step in range(10):
        d_new.copy_(rows(new))
        graph.replay()
        want, _ = W.maps(lens, new, tables, free, n_free, block, cells, n_tok, plan, False)
        lens, tables, plan, n_free = want["seq_lens"], want["tables"], want["plan"], want["n_free"]
        torch.cuda.synchronize()
        assert d_lens.tolist() == lens and d_tables.tolist() == tables and d_plan.tolist() == plan and d_count.item() == n_free
        assert out.slots.tolist() == want["slots"] and out.offsets.tolist() == want["offsets"]
        new = [rng.randint(0, 4) for _ in range(S)]
