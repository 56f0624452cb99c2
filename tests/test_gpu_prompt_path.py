"""A prompt's whole way through a layer's cache: positions, the cache written in its type,
attention of each chunk over it, then single tokens through the decode entry point."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402


@pytest.mark.parametrize("kind", ["f16", "q8_0", "q8_0_q4_0", "q4_0"])
def test_two_prompts_in_chunks_then_decode(kvattn, kind):
    g = U.gen(11)
    H, Hk, D = 8, 2, 128
    records = 12
    cells = records * 128
    # two sequences in one pool: every second record each, so the plan is not one run
    lens = [700, 500]
    steps = [[300, 500], [256, 0], [144, 0]]
    owned = [torch.arange(s, records, 2, device="cuda") for s in range(2)]
    plan = torch.full((2, 6 * 128), -1, dtype=torch.int32, device="cuda")
    for s in range(2):
        plan[s] = (owned[s][:, None] * 128 + torch.arange(128, device="cuda")).flatten().to(torch.int32)
    k, v, ks, vs = U.cache_planes(g, kind, cells, Hk, D)
    for rows, sc in ((k, ks), (v, vs)):
        (rows if sc is None else sc).fill_(float("nan"))          # nothing is there yet
    table = kvattn.rope_table(128, base=1000000.0)
    x = [U.halves(g, n + 3, H + 2 * Hk, D) for n in lens]           # each sequence's fused projections
    done = [0, 0]
    got = [[], []]

    def step(new):
        qkv = torch.cat([x[s][done[s]:done[s] + new[s]] for s in range(2)])
        pos = torch.cat([torch.arange(done[s], done[s] + new[s], device="cuda") for s in range(2)]).to(torch.int32)
        slots = torch.cat([plan[s, done[s]:done[s] + new[s]] for s in range(2)])
        for s in range(2):
            done[s] += new[s]
        q, kk, vv = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        kvattn.rope(q, kk, pos, table, q_out=q, k_out=kk)            # in place, in the projection
        kvattn.cache_write(kk, vv, slots, k, v, k_scales=ks, v_scales=vs)
        return q

    for new in steps:
        q = step(new)
        out, _ = kvattn.prefill_chunk(q, U.ints(U.offsets_of(new)), k, v, U.ints(done), cell_plan=plan, k_scales=ks, v_scales=vs)
        a = 0
        for s in range(2):
            got[s].append((q[a:a + new[s]].clone(), out[a:a + new[s]]))
            a += new[s]
    for s in range(2):
        cells_s = plan[s, :lens[s]].long()
        kd = U.dequant(k[cells_s], None if ks is None else ks[cells_s], D)
        vd = U.dequant(v[cells_s], None if vs is None else vs[cells_s], D)
        q = torch.cat([a for a, _ in got[s]])
        o = torch.cat([b for _, b in got[s]])
        lim = torch.arange(1, lens[s] + 1, device="cuda")
        want, _, tol, _ = U.attend(q, kd, vd, lim, 1 / math.sqrt(D), rounded_k=ks is not None)
        U.check(o, want, tol, f"sequence {s}")
    # the next tokens: the decode kernels read what was written
    q = step([1, 1])
    out, _ = kvattn.decode(q.contiguous(), k, v, U.ints(done), split=128, cell_plan=plan, k_scales=ks, v_scales=vs)
    both, _ = kvattn.prefill_chunk(q, U.ints([0, 1, 2]), k, v, U.ints(done), cell_plan=plan, k_scales=ks, v_scales=vs)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())
    assert float((out - both.float()).abs().max()) <= 6e-3
