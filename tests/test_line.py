"""The line that equal shares of attention are cut from (csrc/line.cuh, compiled for the host): where the
host says that it fits, 32 bits hold it, whatever the sequences' lengths (no GPU needed)."""
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
