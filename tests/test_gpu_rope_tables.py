"""The angle itself, to the bound that holds at every position, and tables of a program's own frequencies."""
from fractions import Fraction
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402
from tests.test_gpu_rope import rotated  # noqa: E402

TWO_PI = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def test_angles_next_to_whole_turns(kvattn):
    """Positions whose angle for the first pair (one radian each) is next to a whole number of turns,
    where the sine, made large by the gain, shows an absolute error of the angle."""
    near = []   # numerators of the continued fraction of 2 pi, and small multiples of them
    a, p0, p1 = TWO_PI, 0, 1
    while True:
        n = math.floor(a)
        p0, p1 = p1, n * p1 + p0
        if p1 >= 2 ** 31:
            break
        near += [p1 * m for m in (1, 2, 3) if p1 * m < 2 ** 31]
        a = 1 / (a - n)
    near = sorted(x for x in set(near) if x > 100)
    assert len(near) > 10 and max(near) > 2 ** 29
    gain = 2.0 ** 14
    table = kvattn.rope_table(128)
    table = kvattn.RopeTable(table.turns, gain, 128)
    q = torch.zeros(2 * len(near), 1, 128, dtype=torch.float16, device="cuda")
    q[:, 0, 64] = 1.0
    pos = near + [-x for x in near]
    out, _ = kvattn.rope(q, None, U.ints(pos), table)
    for p, got in zip(pos, out[:, 0, 0].double().tolist()):
        turns = p / TWO_PI
        r = float((turns - round(turns)) * TWO_PI)   # the angle, less whole turns
        want = -math.sin(r) * gain
        # the table's double (2^-54 turns per position), the 32 bits of the fraction of a turn that are
        # kept, the angle's and the sine's roundings to fp32, the result's to half
        off = 2 * math.pi * (abs(p) * 2.0 ** -54 + 2.0 ** -32) + abs(r) * 2.0 ** -22
        assert abs(got - want) <= off * gain + abs(want) * U.HALF + U.HALF_MIN, p


def test_a_table_of_other_frequencies(kvattn):
    """The ramp in the pair's number between rounded bounds, with a gain of its own."""
    n, base, factor, original = 128, 1000000.0, 4.0, 32768

    def pair(turns):
        return n * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = math.floor(pair(32.0)), math.ceil(pair(1.0))
    i = torch.arange(n // 2, dtype=torch.float64)
    theta = base ** (-2 * i / n)
    mix = ((i - lo) / (hi - lo)).clamp(0, 1)
    theta = theta / factor * mix + theta * (1 - mix)
    turns = torch.tensor([round(t / (2 * math.pi) * 2.0 ** 64) for t in theta.tolist()], dtype=torch.int64, device="cuda")
    gain = 0.75
    g = U.gen(3)
    q, k = U.halves(g, 90, 4, n), U.halves(g, 90, 2, n)
    pos = torch.randint(0, 131072, (90,), generator=g, device="cuda", dtype=torch.int32)
    for layout in ("half", "interleaved"):
        got = kvattn.rope(q, k, pos, kvattn.RopeTable(turns, gain, n), layout=layout)
        for y, x in zip(got, (q, k)):
            want, tol = rotated(x, pos, theta.cuda(), gain, layout)
            U.check(y, want, tol, layout)
