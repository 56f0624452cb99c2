"""Rotary positions against the rotation in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402


def theta(n_rot, base, scaling, factor, original):
    i = torch.arange(n_rot // 2, dtype=torch.float64, device="cuda")
    t = base ** (-2 * i / n_rot)
    if scaling == "linear":
        t = t / factor
    if scaling == "yarn":
        keep = ((original * t / (2 * math.pi) - 1) / 31).clamp(0, 1)
        t = t * keep + t / factor * (1 - keep)
    return t


def rotated(x, pos, t, gain, layout):
    n = 2 * t.numel()
    y = x.double().clone()
    i = torch.arange(n // 2, device="cuda")
    a, b = (i, i + n // 2) if layout == "half" else (2 * i, 2 * i + 1)
    ang = pos.double()[:, None, None] * t
    c, s = ang.cos() * gain, ang.sin() * gain
    u, w = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * c - w * s, u * s + w * c
    # fp32 cosines, products and sums (a few 2^-24 of the terms), the angle's 2^-32 turns and the
    # frequency's rounding to 64 bits, then half
    size = torch.zeros_like(y)
    size[..., a] = size[..., b] = (u.abs() + w.abs()) * gain
    tol = size * 2.0 ** -20 + y.abs() * U.HALF + U.HALF_MIN
    tol[..., n:] = 0
    return y, tol


def check_rope(kv, T, H, Hk, D, n_rot, layout, *, base=10000.0, scaling="none", factor=1.0, original=4096, far=None, pos=None,
               fused=False, in_place=False):
    g = U.gen(T + H + n_rot)
    if fused:
        x = U.halves(g, T, H + 2 * Hk, D)
        q, k = x[:, :H], x[:, H:H + Hk]
    else:
        q, k = U.halves(g, T, H, D), U.halves(g, T, Hk, D)
    if pos is None:
        pos = torch.randint(0, far or 4096, (T,), generator=g, device="cuda", dtype=torch.int32)
    table = kv.rope_table(n_rot, base=base, scaling=scaling, factor=factor, original=original)
    t = theta(n_rot, base, scaling, factor, original)
    gain = 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0
    assert abs(table.gain - gain) <= gain * 2.0 ** -23
    want = [rotated(y, pos, t, table.gain, layout) for y in (q, k)]
    keep = x[:, H + Hk:].clone() if fused else None
    out = kv.rope(q, k, pos, table, layout=layout, **({"q_out": q, "k_out": k} if in_place else {}))
    torch.cuda.synchronize()
    for got, (w, tol), name in zip(out, want, "qk"):
        U.check(got, w, tol, name)
    if fused:
        assert torch.equal(x[:, H + Hk:], keep)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,n_rot", [(128, 128), (128, 16), (128, 48), (128, 96), (256, 256), (256, 64), (256, 208)])
def test_rope_shapes(kvattn, D, n_rot, layout):
    for T, H, Hk in ((1, 1, 1), (5, 3, 1), (64, 32, 8), (1030, 6, 2)):
        check_rope(kvattn, T, H, Hk, D, n_rot, layout)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling,factor,original", [("linear", 4.0, 0), ("yarn", 8.0, 4096), ("yarn", 2.0, 32768)])
def test_rope_scalings(kvattn, scaling, factor, original, layout):
    check_rope(kvattn, 100, 4, 2, 128, 64, layout, base=500000.0, scaling=scaling, factor=factor, original=original, far=131072)


def test_rope_far_and_negative_positions(kvattn):
    pos = U.ints([0, 1, -1, 1000000, -1000003, 16777217, 2147483647, -2147483648, 1 << 30])
    # the reference's own fp64 angle is off by 2^-53 of 2^31 rad, far below the tolerance
    check_rope(kvattn, 9, 4, 2, 128, 128, "half", pos=pos)
    check_rope(kvattn, 9, 4, 2, 256, 32, "interleaved", pos=pos, base=1000000.0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_slices_in_place(kvattn, layout):
    check_rope(kvattn, 77, 5, 2, 128, 64, layout, fused=True, in_place=True)
    check_rope(kvattn, 77, 5, 2, 128, 128, layout, fused=True)


def test_rope_one_tensor_and_position_zero(kvattn):
    g = U.gen(3)
    q = U.halves(g, 10, 4, 128)
    table = kvattn.rope_table(128)
    out, none = kvattn.rope(q, None, torch.zeros(10, dtype=torch.int32, device="cuda"), table)
    assert none is None and torch.equal(out, q)
    none, out = kvattn.rope(None, q, torch.zeros(10, dtype=torch.int32, device="cuda"), table, layout="interleaved")
    assert none is None and torch.equal(out, q)


def test_rope_values_that_are_not_finite(kvattn):
    g = U.gen(4)
    q = U.halves(g, 3, 2, 128)
    pos = U.ints([5, 6, 7])
    table = kvattn.rope_table(64)
    want, _ = kvattn.rope(q, None, pos, table)
    x = q.clone()
    x[1, 0, 3] = float("nan")
    x[2, 1, 100] = float("inf")     # beyond the rotated part: copied
    out, _ = kvattn.rope(x, None, pos, table)
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[1, 0, 3] = hit[1, 0, 35] = hit[2, 1, 100] = True
    assert bool(torch.isnan(out[1, 0, [3, 35]]).all()) and float(out[2, 1, 100]) == float("inf")
    assert torch.equal(out[~hit], want[~hit])
