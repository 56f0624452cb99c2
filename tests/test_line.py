"""The line that equal shares of attention are cut from (csrc/line.cuh, compiled for the host): where the
host says that it fits, 32 bits hold it, whatever the sequences' lengths; and the rule by which units of a
window are dealt out whole (no GPU needed)."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_decode_02_gb300", "csrc")
CODE = r"""
#include "line.cuh"
using namespace kvattn;
extern "C" {
uint32_t upto(uint32_t a, uint32_t step, uint32_t blocks, uint32_t less, uint32_t b) { return Line{a, step, blocks, less}.upto(b); }
uint32_t of(uint32_t a, uint32_t step, uint32_t blocks, uint32_t less, uint32_t b) { return Line{a, step, blocks, less}.of(b); }
uint32_t step(int block_tokens) { return line_step(block_tokens); }
int fits(int64_t n_tok, int n_seq, int n_head_kv, int group, int head_dim, int64_t max_len, int64_t prefix) {
    return shared_line_fits(n_tok, n_seq, n_head_kv, group, head_dim, max_len, prefix);
}
int whole(uint32_t units, uint64_t tiles, uint32_t longest, uint32_t n, uint32_t base, uint32_t more, uint32_t sms) {
    return whole_units(units, tiles, longest, n, WholeRule{base, more, sms});
}
uint32_t rule(int64_t n_tok, int n_seq, int fast, int merged) {
    const WholeRule r = whole_rule(n_tok, n_seq, fast != 0, merged != 0, 152);
    return r.base << 16 | r.more;
}
}
"""


@pytest.fixture(scope="module")
def line(tmp_path_factory):
    d = tmp_path_factory.mktemp("line")
    (d / "line.cpp").write_text(CODE)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "line.so"), str(d / "line.cpp")])
    lib = ctypes.CDLL(str(d / "line.so"))
    lib.upto.argtypes = lib.of.argtypes = [ctypes.c_uint32] * 5
    lib.upto.restype = lib.of.restype = ctypes.c_uint32
    lib.step.argtypes, lib.step.restype = [ctypes.c_int], ctypes.c_uint32
    lib.fits.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64]
    lib.whole.argtypes = [ctypes.c_uint32, ctypes.c_uint64] + [ctypes.c_uint32] * 5
    lib.rule.argtypes, lib.rule.restype = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int], ctypes.c_uint32
    return lib


def block(group, D):
    return 128 // group * (2 if D == 128 else 1)


def lines(new, lens, Hk, group, D, prefix):
    """(first block's length, step, blocks) of each sequence and of the prefix, as the schedulers have them."""
    bt = block(group, D)
    held = [max(L - n, 0) for n, L in zip(new, lens) if n]
    tiles = min(min(held), prefix) // 128 if held else 0
    out = []
    for n, L in zip(new, lens):
        lim = max(L - n, 0) + min(n, bt)
        out.append((8 * (2 + -(-lim // 128) - tiles), -(-bt // 16), -(-n // bt)))
    out.append((8 * (2 + tiles), 0, -(-sum(new) // bt) if tiles else 0))
    return out


def check(line, new, lens, Hk, group, D, prefix, max_len):
    """A line that is said to fit does, in whole numbers of any size, and Line agrees with those."""
    if not line.fits(sum(new), len(new), Hk, group, D, max_len, prefix):
        return False
    total = 0
    for a, step, blocks in lines(new, lens, Hk, group, D, prefix):
        if blocks:
            last = a + step * (blocks - 1)
            for less in (0, last - (last * 5 >> 3)):
                own = a * blocks + step * (blocks * (blocks - 1) // 2) - less
                assert line.upto(a, step, blocks, less, blocks) == own
                assert line.of(a, step, blocks, less, blocks - 1) == last - less
                for b in (0, 1, blocks // 2, blocks - 1):
                    assert line.upto(a, step, blocks, less, b) == a * b + step * (b * (b - 1) // 2) - (less if b == blocks else 0)
            total += Hk * (a * blocks + step * (blocks * (blocks - 1) // 2))
    assert total < 2 ** 31
    return True


# tokens of one sequence behind 256 shared cells
@pytest.mark.parametrize("n,group,Hk,D,fits", [
    (65600, 128, 1, 256, False), (65535, 128, 1, 256, False), (50000, 128, 1, 256, True), (65000, 128, 2, 256, False),
    (140000, 64, 1, 256, False), (140000, 128, 1, 128, False), (270000, 32, 1, 256, False), (270000, 64, 1, 128, False),
    (70000, 96, 2, 256, False), (70000, 64, 1, 256, True), (65600, 4, 8, 128, True), (8192, 4, 8, 128, True),
    (131072, 16, 1, 256, True), (2 ** 24, 4, 8, 128, False), (2 ** 31 - 1, 1, 1, 128, False),
])
def test_one_long_sequence(line, n, group, Hk, D, fits):
    assert check(line, [n], [n + 256], Hk, group, D, 256, n + 256) == fits


def test_steps_of_blocks(line):
    """An eighth of a tile is 16 cells."""
    for bt in (1, 2, 15, 16, 17, 42, 128, 256):
        assert line.step(bt) == -(-bt // 16)


def test_many_lengths(line):
    rng = random.Random(11)
    said = 0
    for _ in range(4000):
        group, D, Hk = rng.choice([1, 2, 4, 6, 8, 16, 40, 64, 96, 128]), rng.choice([128, 256]), rng.choice([1, 1, 2, 8])
        S = int(2 ** rng.uniform(0, 8))
        most = 2 ** rng.uniform(0, 19)
        new = [int(most * rng.random() ** 3) for _ in range(S)]
        prefix = int(2 ** rng.uniform(0, 31))
        lens = [max(0, min(2 ** 31 - 1, n + int(2 ** rng.uniform(-1, 31)) - rng.choice([0, 0, 0, n]))) for n in new]
        if sum(new) * group * Hk >= 2 ** 31 or sum(new) == 0:
            continue
        said += check(line, new, lens, Hk, group, D, prefix, max(lens))
    assert said > 500


@pytest.mark.parametrize("blocks", [1, 46340, 46341, 65535, 65536, 65537, 92681])
def test_a_line_of_its_largest_number_of_blocks(line, blocks):
    """b (b - 1) in 32 bits, wherever the host lets it come to that."""
    for D, group in ((256, 128), (256, 64), (128, 128), (128, 64), (128, 16)):
        bt = block(group, D)
        fits = check(line, [blocks * bt], [blocks * bt], 1, group, D, 128, blocks * bt)
        assert fits == (8 * blocks * (2 + -(-blocks * bt // 128)) + -(-bt // 16) * (blocks * (blocks - 1) // 2) + 8 * blocks * 3 < 2 ** 31)


# (single tokens, f16 rows of 128 without a plan, units, tiles of each, us whole, us in shares) of equal
# units on 152 SMs, where the two differ by more than a tenth.
MEASURED = [
    (1, 1, 160, 33, 89, 66), (1, 1, 152, 17, 31, 35), (1, 1, 128, 32, 45, 54), (1, 1, 128, 17, 28, 36), (1, 1, 128, 12, 22, 30),
    (1, 1, 128, 9, 19, 26), (1, 1, 128, 6, 15, 22), (1, 1, 96, 17, 27, 30), (1, 1, 96, 12, 21, 26), (1, 1, 96, 9, 18, 23),
    (1, 1, 96, 6, 14, 20), (1, 1, 64, 32, 43, 34), (1, 1, 64, 9, 17, 19), (1, 1, 64, 6, 14, 19), (1, 1, 48, 32, 43, 29),
    (1, 1, 48, 17, 27, 22), (1, 1, 48, 12, 21, 18), (1, 1, 48, 6, 14, 19), (1, 1, 32, 32, 43, 24), (1, 1, 32, 17, 26, 19),
    (1, 1, 32, 12, 21, 18), (1, 1, 32, 6, 14, 19), (1, 1, 24, 32, 42, 21), (1, 1, 24, 17, 26, 18), (1, 1, 24, 12, 21, 17),
    (1, 1, 24, 6, 14, 18), (1, 1, 16, 32, 42, 19), (1, 1, 16, 17, 26, 18), (1, 1, 16, 12, 20, 16), (1, 1, 16, 6, 14, 18),
    (1, 1, 8, 32, 42, 18), (1, 1, 8, 17, 26, 16), (1, 1, 8, 12, 20, 16), (1, 1, 8, 6, 14, 18), (1, 0, 352, 19, 99, 88),
    (1, 0, 160, 17, 89, 68), (1, 0, 160, 11, 44, 37), (1, 0, 160, 11, 41, 36), (1, 0, 160, 9, 40, 34), (1, 0, 128, 32, 82, 96),
    (1, 0, 128, 19, 41, 46), (1, 0, 128, 17, 49, 58), (1, 0, 128, 17, 38, 42), (1, 0, 128, 14, 29, 34), (1, 0, 128, 12, 37, 47),
    (1, 0, 128, 12, 29, 34), (1, 0, 128, 11, 24, 30), (1, 0, 128, 9, 30, 39), (1, 0, 128, 9, 24, 29), (1, 0, 128, 8, 19, 26),
    (1, 0, 128, 6, 24, 30), (1, 0, 128, 6, 18, 23), (1, 0, 96, 34, 61, 49), (1, 0, 96, 32, 63, 52), (1, 0, 96, 12, 34, 38),
    (1, 0, 96, 9, 28, 32), (1, 0, 96, 8, 19, 24), (1, 0, 96, 6, 22, 27), (1, 0, 96, 6, 18, 23), (1, 0, 64, 34, 60, 39),
    (1, 0, 64, 32, 72, 55), (1, 0, 64, 32, 63, 39), (1, 0, 64, 19, 36, 27), (1, 0, 64, 17, 43, 36), (1, 0, 64, 17, 37, 27),
    (1, 0, 64, 14, 28, 24), (1, 0, 64, 12, 34, 29), (1, 0, 64, 12, 28, 23), (1, 0, 64, 6, 21, 26), (1, 0, 64, 6, 18, 23),
    (1, 0, 48, 34, 60, 32), (1, 0, 48, 32, 72, 44), (1, 0, 48, 32, 63, 32), (1, 0, 48, 19, 36, 24), (1, 0, 48, 17, 43, 30),
    (1, 0, 48, 17, 37, 23), (1, 0, 48, 14, 28, 21), (1, 0, 48, 12, 33, 25), (1, 0, 48, 12, 28, 21), (1, 0, 48, 11, 22, 20),
    (1, 0, 48, 9, 27, 24), (1, 0, 48, 6, 21, 26), (1, 0, 48, 6, 18, 22), (1, 0, 32, 34, 59, 26), (1, 0, 32, 32, 72, 36),
    (1, 0, 32, 32, 62, 27), (1, 0, 32, 19, 35, 21), (1, 0, 32, 17, 43, 26), (1, 0, 32, 17, 36, 21), (1, 0, 32, 14, 27, 19),
    (1, 0, 32, 12, 33, 23), (1, 0, 32, 12, 28, 21), (1, 0, 32, 11, 22, 19), (1, 0, 32, 9, 27, 23), (1, 0, 32, 6, 21, 26),
    (1, 0, 32, 6, 18, 22), (1, 0, 24, 34, 59, 23), (1, 0, 24, 32, 72, 30), (1, 0, 24, 32, 62, 23), (1, 0, 24, 19, 33, 20),
    (1, 0, 24, 17, 43, 24), (1, 0, 24, 17, 36, 21), (1, 0, 24, 14, 25, 19), (1, 0, 24, 12, 33, 23), (1, 0, 24, 12, 28, 20),
    (1, 0, 24, 11, 21, 19), (1, 0, 24, 9, 27, 23), (1, 0, 24, 9, 23, 21), (1, 0, 24, 6, 21, 25), (1, 0, 24, 6, 18, 22),
    (1, 0, 16, 34, 56, 22), (1, 0, 16, 32, 72, 26), (1, 0, 16, 32, 62, 21), (1, 0, 16, 19, 32, 19), (1, 0, 16, 17, 42, 23),
    (1, 0, 16, 17, 36, 21), (1, 0, 16, 14, 25, 18), (1, 0, 16, 12, 33, 22), (1, 0, 16, 12, 28, 20), (1, 0, 16, 11, 21, 18),
    (1, 0, 16, 9, 27, 23), (1, 0, 16, 9, 23, 20), (1, 0, 16, 6, 21, 25), (1, 0, 16, 6, 17, 22), (1, 0, 8, 34, 56, 20),
    (1, 0, 8, 32, 72, 25), (1, 0, 8, 32, 62, 21), (1, 0, 8, 19, 33, 18), (1, 0, 8, 17, 42, 22), (1, 0, 8, 17, 36, 20),
    (1, 0, 8, 14, 25, 18), (1, 0, 8, 12, 33, 22), (1, 0, 8, 12, 28, 20), (1, 0, 8, 11, 21, 18), (1, 0, 8, 9, 27, 23),
    (1, 0, 8, 6, 21, 25), (1, 0, 8, 6, 17, 22), (0, 0, 800, 5, 88, 106), (0, 0, 800, 5, 87, 104), (0, 0, 512, 9, 88, 100),
    (0, 0, 512, 5, 70, 79), (0, 0, 400, 11, 91, 111), (0, 0, 320, 9, 65, 72), (0, 0, 256, 11, 63, 80), (0, 0, 256, 9, 52, 68),
    (0, 0, 256, 9, 49, 65), (0, 0, 240, 17, 96, 113), (0, 0, 240, 17, 83, 92), (0, 0, 160, 19, 113, 94),
    (0, 0, 160, 19, 105, 85), (0, 0, 160, 19, 92, 79), (0, 0, 160, 17, 80, 71), (0, 0, 128, 35, 104, 122),
    (0, 0, 128, 33, 89, 116), (0, 0, 128, 19, 49, 69), (0, 0, 128, 17, 53, 74), (0, 0, 128, 17, 45, 62),
    (0, 0, 128, 17, 40, 61), (0, 0, 128, 11, 34, 54), (0, 0, 128, 9, 34, 52), (0, 0, 128, 9, 29, 48), (0, 0, 128, 9, 27, 47),
    (0, 0, 120, 19, 57, 71), (0, 0, 120, 17, 45, 60), (0, 0, 96, 19, 49, 57), (0, 0, 96, 17, 45, 59), (0, 0, 96, 17, 44, 51),
    (0, 0, 96, 17, 39, 51), (0, 0, 96, 11, 34, 47), (0, 0, 96, 9, 30, 42), (0, 0, 96, 9, 29, 41), (0, 0, 96, 9, 26, 41),
    (0, 0, 64, 34, 77, 58), (0, 0, 64, 32, 74, 66), (0, 0, 64, 32, 73, 54), (0, 0, 64, 32, 62, 52), (0, 0, 64, 12, 30, 37),
    (0, 0, 64, 11, 33, 38), (0, 0, 64, 9, 29, 33), (0, 0, 64, 9, 28, 34), (0, 0, 64, 9, 25, 34), (0, 0, 64, 8, 27, 34),
    (0, 0, 64, 6, 23, 30), (0, 0, 64, 6, 22, 30), (0, 0, 64, 6, 20, 29), (0, 0, 48, 34, 77, 47), (0, 0, 48, 32, 74, 54),
    (0, 0, 48, 32, 72, 44), (0, 0, 48, 32, 62, 43), (0, 0, 48, 19, 48, 39), (0, 0, 48, 17, 44, 38), (0, 0, 48, 17, 44, 35),
    (0, 0, 48, 14, 38, 34), (0, 0, 48, 12, 35, 32), (0, 0, 48, 9, 28, 32), (0, 0, 48, 9, 25, 32), (0, 0, 48, 8, 26, 31),
    (0, 0, 48, 6, 23, 28), (0, 0, 48, 6, 22, 29), (0, 0, 48, 6, 20, 27), (0, 0, 32, 34, 77, 40), (0, 0, 32, 32, 74, 43),
    (0, 0, 32, 32, 72, 38), (0, 0, 32, 32, 62, 37), (0, 0, 32, 19, 48, 35), (0, 0, 32, 17, 45, 31), (0, 0, 32, 17, 43, 32),
    (0, 0, 32, 17, 38, 32), (0, 0, 32, 14, 39, 30), (0, 0, 32, 12, 35, 27), (0, 0, 32, 12, 34, 29), (0, 0, 32, 9, 25, 29),
    (0, 0, 32, 8, 26, 30), (0, 0, 32, 6, 23, 27), (0, 0, 32, 6, 22, 28), (0, 0, 32, 6, 20, 26), (0, 0, 24, 34, 77, 36),
    (0, 0, 24, 32, 74, 37), (0, 0, 24, 32, 72, 34), (0, 0, 24, 32, 62, 33), (0, 0, 24, 19, 47, 36), (0, 0, 24, 17, 44, 27),
    (0, 0, 24, 17, 43, 31), (0, 0, 24, 17, 38, 30), (0, 0, 24, 14, 38, 28), (0, 0, 24, 12, 35, 26), (0, 0, 24, 12, 34, 28),
    (0, 0, 24, 12, 30, 26), (0, 0, 24, 9, 25, 28), (0, 0, 24, 6, 22, 27), (0, 0, 24, 6, 20, 25), (0, 0, 16, 34, 77, 32),
    (0, 0, 16, 32, 74, 31), (0, 0, 16, 32, 72, 31), (0, 0, 16, 32, 62, 30), (0, 0, 16, 19, 48, 32), (0, 0, 16, 17, 44, 26),
    (0, 0, 16, 17, 43, 29), (0, 0, 16, 17, 38, 28), (0, 0, 16, 14, 38, 28), (0, 0, 16, 12, 34, 27), (0, 0, 16, 12, 34, 25),
    (0, 0, 16, 12, 29, 25), (0, 0, 16, 11, 32, 29), (0, 0, 16, 9, 28, 25), (0, 0, 16, 6, 23, 27), (0, 0, 16, 6, 22, 27),
    (0, 0, 16, 6, 19, 25), (0, 0, 8, 34, 75, 29), (0, 0, 8, 32, 73, 27), (0, 0, 8, 32, 71, 29), (0, 0, 8, 32, 62, 27),
    (0, 0, 8, 19, 47, 30), (0, 0, 8, 17, 44, 26), (0, 0, 8, 17, 42, 28), (0, 0, 8, 17, 37, 27), (0, 0, 8, 14, 37, 26),
    (0, 0, 8, 12, 34, 25), (0, 0, 8, 12, 33, 25), (0, 0, 8, 12, 30, 23), (0, 0, 8, 11, 31, 27), (0, 0, 8, 9, 28, 25),
    (0, 0, 8, 6, 22, 27), (0, 0, 8, 6, 21, 27), (0, 0, 8, 6, 19, 25),
]


def whole(line, units, tiles, longest, single, fast, merged=0):
    rule = line.rule(*((8, 8) if single else (64, 8)), fast, merged)
    n = min(152, max(units, -(-tiles // 4)))
    return bool(line.whole(units, tiles, longest, n, rule >> 16, rule & 0xffff, 152))


@pytest.mark.parametrize("merged", [0, 1])
def test_whole_units_where_they_were_measured_to_take_less(line, merged):
    for single, fast, units, tiles, us_whole, us_shares in MEASURED:
        n = min(152, max(units, units * tiles / 4))
        us_whole += merged * (1.2 + (0.8 if single else 2.4) * n / 152)   # a merge that finds nothing
        if abs(us_whole / us_shares - 1) > 0.11:
            assert whole(line, units, units * tiles, tiles, single, fast, merged) == (us_whole < us_shares), (single, fast, units, tiles)


def test_whole_units_are_compared_in_whole_numbers(line):
    """No part of a tile is rounded away: 256 units of 33 tiles on 152 SMs lose 10.42."""
    assert not line.whole(256, 256 * 33, 33, 152, 10, 0, 152) and line.whole(256, 256 * 33, 33, 152, 11, 0, 152)
    assert line.whole(256, 256 * 33, 33, 152, 3, 8, 152) and not line.whole(76, 76 * 33, 33, 152, 8, 16, 152)   # (76 lose 16.5)
    assert line.whole(76, 76 * 33, 33, 152, 9, 16, 152)
    assert line.whole(304, 304 * 10 ** 6, 10 ** 6, 152, 1, 0, 152)        # full rounds lose nothing
    assert line.whole(0, 0, 0, 152, 10, 0, 152)
    assert line.whole(2 ** 11, 2 ** 11 * 2 ** 24, 2 ** 24, 2 ** 8, 1, 0, 2 ** 8)
    assert not line.whole(2 ** 11 + 1, 2 ** 11 * 2 ** 24, 2 ** 24, 2 ** 8, 1, 0, 2 ** 8)


@pytest.mark.parametrize("tiles_of,want", [
    ([65] * 8 + [1] * 144, False),                 # one long sequence among short ones: 8 of 152 SMs would work
    ([33] * 8 + [1] * 1000, False), ([33] * 304, True), ([33] * 152 + [1] * 152, False), ([20] * 304 + [19] * 304, True),
])
def test_units_of_several_lengths(line, tiles_of, want):
    for single, fast in ((1, 1), (1, 0), (0, 0)):
        assert whole(line, len(tiles_of), sum(tiles_of), max(tiles_of), single, fast, 1) == want
