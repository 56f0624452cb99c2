"""A layer's prompt path captured once and replayed with other inputs: turn, store, attend, and a single
token through the decode entry point, as the same calls give them eagerly; two graphs share a workspace."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402

H, Hk, D = 8, 2, 128


def inputs(seed, new, done, plan):
    """A step's projections, positions, slots and lengths: `new` tokens of each sequence behind `done`."""
    g = U.gen(seed)
    return {"qkv": U.halves(g, sum(new), H + 2 * Hk, D),
            "pos": torch.cat([torch.arange(d, d + n, device="cuda") for n, d in zip(new, done)]).to(torch.int32),
            "slots": torch.cat([plan[s, d:d + n] for s, (n, d) in enumerate(zip(new, done))]),
            "lens": U.ints([d + n for n, d in zip(new, done)])}


def layer(kv, x, cache, plan, offsets, table, ws, out, lse, dec=None):
    k, v, ks, vs = cache
    q, kk, vv = x["qkv"][:, :H], x["qkv"][:, H:H + Hk], x["qkv"][:, H + Hk:]
    kv.rope(q, kk, x["pos"], table, q_out=q, k_out=kk)
    kv.cache_write(kk, vv, x["slots"], k, v, k_scales=ks, v_scales=vs)
    kv.prefill_chunk(q, offsets, k, v, x["lens"], cell_plan=plan, k_scales=ks, v_scales=vs, out=out, lse=lse, ws=ws)
    if dec is not None:
        qd = dec["q"]
        qd.copy_(q)
        kv.decode(qd, k, v, x["lens"], split=128, cell_plan=plan, k_scales=ks, v_scales=vs, out=dec["out"], lse=dec["lse"],
                  ws=dec["ws"])


@pytest.mark.parametrize("kind", ["f16", "q8_0", "q8_0_q4_0", "q4_0"])
def test_the_path_replayed(kvattn, kind):
    g = U.gen(41)
    records = 12
    plan = torch.stack([(torch.arange(s, records, 2, device="cuda")[:, None] * 128 + torch.arange(128, device="cuda")).flatten()
                        for s in range(2)]).to(torch.int32)
    empty = U.cache_planes(g, kind, records * 128, Hk, D)
    table = kvattn.rope_table(D, base=1000000.0)
    steps = [([200, 37], [0, 0]), ([200, 37], [200, 37]), ([200, 37], [400, 74])]
    tokens = [([1, 1], [600, 111]), ([1, 1], [601, 112])]
    off, off1 = U.ints([0, 200, 237]), U.ints([0, 1, 2])
    ws = kvattn.prefill_chunk_workspace(237, 2, H, Hk, D, plan.shape[1])
    half = dict(dtype=torch.float16, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")

    def buffers():
        return {"out": torch.zeros(237, H, D, **half), "lse": torch.zeros(237, H, **f32), "out1": torch.zeros(2, H, D, **half),
                "lse1": torch.zeros(2, H, **f32),
                "dec": {"q": torch.zeros(2, H, D, **half), "out": torch.zeros(2, H, D, **f32), "lse": torch.zeros(2, H, **f32),
                        "ws": kvattn.decode_workspace(2, H, D, plan.shape[1], 128)}}

    def walk(run):
        got = []
        for i, (new, done) in enumerate(steps):
            got += run("prompt", inputs(50 + i, new, done, plan))
        for i, (new, done) in enumerate(tokens):
            got += run("token", inputs(60 + i, new, done, plan))
        return got

    def results(b, what):
        return [x.clone() for x in ((b["out"], b["lse"]) if what == "prompt" else
                                    (b["out1"], b["lse1"], b["dec"]["out"], b["dec"]["lse"]))]

    b, cache = buffers(), [None if x is None else x.clone() for x in empty]

    def eager(what, x):
        if what == "prompt":
            layer(kvattn, x, cache, plan, off, table, ws, b["out"], b["lse"])
        else:
            layer(kvattn, x, cache, plan, off1, table, ws, b["out1"], b["lse1"], b["dec"])
        return results(b, what)
    want = walk(eager)

    c, kept = buffers(), [None if x is None else x.clone() for x in empty]
    held = {"prompt": inputs(1, *steps[0], plan), "token": inputs(1, *tokens[0], plan)}
    graphs = {what: torch.cuda.CUDAGraph() for what in held}
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs["prompt"]):
        layer(kvattn, held["prompt"], kept, plan, off, table, ws, c["out"], c["lse"])
    with torch.cuda.graph(graphs["token"]):
        layer(kvattn, held["token"], kept, plan, off1, table, ws, c["out1"], c["lse1"], c["dec"])

    def replay(what, x):
        for name, y in held[what].items():
            y.copy_(x[name])
        graphs[what].replay()
        return results(c, what)
    got = walk(replay)
    torch.cuda.synchronize()
    assert kvattn.kvattn_workspace_status(ws) == 0
    for i, (a, w) in enumerate(zip(got, want)):
        assert bool(torch.isfinite(w).all()) and torch.equal(a, w), i
    for a, w in zip(kept, cache):
        assert a is None or torch.equal(a.view(torch.uint8), w.view(torch.uint8))
