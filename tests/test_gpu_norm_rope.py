"""Norms of the heads with the rotation in the same pass, and rotations by positions of several axes,
against the formulas in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402


def frequencies(n_rot, base, sections, order, restart):
    """(axis, theta) of every pair."""
    axis = []
    if order == "blocks":
        for a, n in enumerate(sections):
            axis += [a] * n
    else:
        for i in range(max(sections, default=0)):
            axis += [a for a, n in enumerate(sections) if i < n]
    seen, theta = [0] * len(sections), []
    for i, a in enumerate(axis):
        theta.append(base ** (-seen[a] / sections[a]) if restart else base ** (-2 * i / n_rot))
        seen[a] += 1
    return (torch.tensor(axis, dtype=torch.long, device="cuda"),
            torch.tensor(theta, dtype=torch.float64, device="cuda"))


def expected(x, weight, eps, pos, axis, theta, gain, layout):
    y = x.double()
    rel = torch.zeros((), dtype=torch.float64, device="cuda")
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
        # the squares' sum (D / 16 terms a lane, four shuffles), mean, root and two products: fewer
        # than 2^5 roundings of 2^-24
        rel = rel + 2.0 ** -19
    y = y.clone()
    size = y.abs() * rel
    n = 2 * theta.numel()
    i = torch.arange(n // 2, device="cuda")
    a, b = (i, i + n // 2) if layout == "half" else (2 * i, 2 * i + 1)
    ang = pos[axis].T.double()[:, None, :] * theta
    c, s = ang.cos() * gain, ang.sin() * gain
    u, w = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * c - w * s, u * s + w * c
    # as for the rotation alone (fp32 cosines, products and sums; the angle's rounding), and the norm's
    size[..., a] = size[..., b] = (u.abs() + w.abs()) * gain * (2.0 ** -20 + rel)
    tol = size + y.abs() * U.HALF + U.HALF_MIN
    if weight is None:
        tol[..., n:] = 0
    return y, tol


def run(kv, T, H, Hk, D, n_rot, *, layout="half", norm="both", sections=None, order="blocks", restart=False, base=10000.0,
        eps=1e-6, far=4096, fused=False, in_place=False, scale=1.0, seed=1):
    g = U.gen(seed)
    x = U.halves(g, T, H + 2 * Hk, D, scale=scale)
    q, k = (x[:, :H], x[:, H:H + Hk]) if fused else (x[:, :H].contiguous(), x[:, H:H + Hk].contiguous())
    axes = 1 if sections is None else len(sections)
    pos = torch.randint(0, far, (axes, T), generator=g, device="cuda", dtype=torch.int32)
    table = kv.rope_table(n_rot, base=base, sections=sections, order=order, restart=restart)
    axis, theta = frequencies(n_rot, base, [n_rot // 2] if sections is None else sections, order, restart)
    qw = U.halves(g, D) if norm in ("both", "q") else None
    kw = U.halves(g, D) if norm in ("both", "k") else None
    want = [expected(y, w, eps, pos, axis, theta, table.gain, layout) for y, w in ((q, qw), (k, kw))]
    rest = x[:, H + Hk:].clone()
    got = kv.norm_rope(q, k, pos if axes > 1 else pos[0], table, q_weight=qw, k_weight=kw, eps=eps, layout=layout,
                       **({"q_out": q, "k_out": k} if in_place else {}))
    torch.cuda.synchronize()
    for y, (w, tol), name in zip(got, want, "qk"):
        U.check(y, w, tol, name)
    assert torch.equal(x[:, H + Hk:], rest)
    return got


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", ["both", "q", "k", "none"])
@pytest.mark.parametrize("D,n_rot", [(128, 128), (128, 16), (128, 80), (256, 256), (256, 64)])
def test_sides_and_widths(kvattn, D, n_rot, norm, layout):
    run(kvattn, 37, 6, 2, D, n_rot, layout=layout, norm=norm)


@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (1, 32, 8), (3, 5, 1), (64, 32, 8), (130, 7, 7), (2000, 3, 1), (1, 128, 1)])
@pytest.mark.parametrize("D", [128, 256])
def test_tokens_and_heads(kvattn, T, H, Hk, D):
    run(kvattn, T, H, Hk, D, D, seed=T)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("restart", [False, True])
@pytest.mark.parametrize("order", ["blocks", "cycle"])
@pytest.mark.parametrize("sections", [[64], [16, 24, 24], [1, 63], [0, 32, 32], [20, 4, 30, 10], [64, 0]])
def test_axes(kvattn, sections, order, restart, layout):
    for norm in ("none", "both"):
        run(kvattn, 41, 4, 2, 128, 128, sections=sections, order=order, restart=restart, layout=layout, norm=norm, far=100000)


def test_rope_takes_a_table_of_axes(kvattn):
    g = U.gen(4)
    q, k = U.halves(g, 50, 4, 128), U.halves(g, 50, 2, 128)
    pos = torch.randint(0, 3000, (3, 50), generator=g, device="cuda", dtype=torch.int32)
    table = kvattn.rope_table(96, sections=[10, 20, 18])
    a = kvattn.rope(q, k, pos, table)
    b = kvattn.norm_rope(q, k, pos, table)
    # the same position on every axis is the rotation of one axis
    same = pos[:1].expand(3, -1).contiguous()
    c = kvattn.rope(q, k, same, table)
    d = kvattn.rope(q, k, pos[0].contiguous(), kvattn.rope_table(96))
    torch.cuda.synchronize()
    for x, y in zip(a + c, b + d):
        assert torch.equal(x, y)


def test_one_side_alone(kvattn):
    g = U.gen(5)
    q, k, w = U.halves(g, 9, 6, 128), U.halves(g, 9, 2, 128), U.halves(g, 128)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    table = kvattn.rope_table(128)
    both = kvattn.norm_rope(q, k, pos, table, q_weight=w, k_weight=w)
    only_q = kvattn.norm_rope(q, None, pos, table, q_weight=w)
    only_k = kvattn.norm_rope(None, k, pos, table, k_weight=w)
    torch.cuda.synchronize()
    assert only_q[1] is None and only_k[0] is None
    assert torch.equal(only_q[0], both[0]) and torch.equal(only_k[1], both[1])


def test_strided_rows_and_in_place(kvattn):
    for D in (128, 256):
        run(kvattn, 61, 8, 2, D, 64, fused=True)
        run(kvattn, 61, 8, 2, D, D, fused=True, in_place=True, sections=[D // 4, D // 4])
        run(kvattn, 61, 8, 2, D, 64, in_place=True, layout="interleaved")


@pytest.mark.parametrize("scale", [2.0 ** -24, 1e-4, 1.0, 4000.0])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-2])
def test_small_and_large_heads(kvattn, scale, eps):
    if scale == 2.0 ** -24 and eps == 0.0:
        eps = 1e-12        # (heads of zeros alone would be 0 / 0)
    run(kvattn, 20, 4, 2, 128, 128, scale=scale, eps=eps)


def test_heads_that_are_zero_or_not_finite_stay_alone(kvattn):
    g = U.gen(6)
    q, k, w = U.halves(g, 4, 8, 128), U.halves(g, 4, 2, 128), U.halves(g, 128)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    table = kvattn.rope_table(128)
    clean = kvattn.norm_rope(q, k, pos, table, q_weight=w, k_weight=w)[0].clone()
    q[1, 3] = 0.0
    q[2, 5, 7] = float("inf")
    q[3, 0, 100] = float("nan")
    got = kvattn.norm_rope(q, k, pos, table, q_weight=w, k_weight=w)[0]
    torch.cuda.synchronize()
    assert bool((got[1, 3] == 0).all())
    # infinity over infinity and its pair are NaN, the other elements of that head 0
    assert int(torch.isnan(got[2, 5]).sum()) == 2 and bool((got[2, 5][~torch.isnan(got[2, 5])] == 0).all())
    assert bool(torch.isnan(got[3, 0]).all())
    keep = torch.ones(4, 8, dtype=torch.bool, device="cuda")
    keep[1, 3] = keep[2, 5] = keep[3, 0] = False
    assert torch.equal(got[keep], clean[keep])


def test_far_and_negative_positions(kvattn):
    g = U.gen(7)
    q = U.halves(g, 6, 2, 128)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789], [5, -7, 2 ** 30, -3, 0, 99]], dtype=torch.int32, device="cuda")
    table = kvattn.rope_table(128, base=1e6, sections=[40, 24])
    got, _ = kvattn.rope(q, None, pos, table)
    # the table's own angles (2^-64 turns), as integers: what is left is fp32
    turns = [int(x) & (2 ** 64 - 1) for x in table.turns.tolist()]
    axis = table.axis.tolist()
    frac = torch.tensor([[((p * t + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 64 for t, p in
                          zip(turns, [int(pos[a, i]) for a in axis])] for i in range(6)], dtype=torch.float64, device="cuda")
    c, s = (frac * 2 * math.pi).cos()[:, None], (frac * 2 * math.pi).sin()[:, None]
    a, b = q[..., :64].double(), q[..., 64:].double()
    want = torch.cat((a * c - b * s, a * s + b * c), -1)
    size = torch.cat((a.abs() + b.abs(),) * 2, -1)
    torch.cuda.synchronize()
    U.check(got, want, size * 2.0 ** -20 + want.abs() * U.HALF + U.HALF_MIN, "q")


def test_an_axis_beyond_the_last_turns_by_position_zero(kvattn):
    g = U.gen(8)
    q = U.halves(g, 5, 3, 128)
    pos = torch.randint(1, 900, (2, 5), generator=g, device="cuda", dtype=torch.int32)
    table = kvattn.rope_table(128, sections=[32, 32])
    table.axis[40:] = 200
    table.axis[10] = 3
    got, _ = kvattn.rope(q, None, pos, table)
    table.axis[40:] = 0
    table.axis[10] = 0
    zero = pos.clone()
    want, _ = kvattn.rope(q, None, zero, table)
    torch.cuda.synchronize()
    still = [10] + list(range(40, 64))
    for i in still:
        assert torch.equal(got[..., i], q[..., i]) and torch.equal(got[..., i + 64], q[..., i + 64])
    moved = [i for i in range(64) if i not in still]
    assert torch.equal(got[..., moved], want[..., moved])


def test_no_rotation_is_the_norm_alone(kvattn):
    g = U.gen(9)
    q, w = U.halves(g, 7, 5, 256), U.halves(g, 256)
    table = kvattn.RopeTable(torch.zeros(0, dtype=torch.int64, device="cuda"), 1.0, 0)
    got, _ = kvattn.norm_rope(q, None, torch.zeros(7, dtype=torch.int32, device="cuda"), table, q_weight=w, eps=1e-5)
    y = q.double()
    want = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-5) * w.double()
    torch.cuda.synchronize()
    U.check(got, want, want.abs() * (U.HALF + 2.0 ** -19) + U.HALF_MIN, "q")


def test_another_stream_and_a_graph(kvattn):
    g = U.gen(10)
    q, k, w = U.halves(g, 64, 8, 128), U.halves(g, 64, 2, 128), U.halves(g, 128)
    pos = torch.arange(128, dtype=torch.int32, device="cuda").view(2, 64)
    table = kvattn.rope_table(128, sections=[30, 34])
    want = [x.clone() for x in kvattn.norm_rope(q, k, pos, table, q_weight=w, k_weight=w)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = kvattn.norm_rope(q, k, pos, table, q_weight=w, k_weight=w, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvattn.norm_rope(q, k, pos, table, q_weight=w, k_weight=w, q_out=qo, k_out=ko)
    q.copy_(q.flip(0))
    pos.copy_(pos.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want[0].flip(0))
