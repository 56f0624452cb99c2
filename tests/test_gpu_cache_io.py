"""The cache written in its stored type and read back, bit for bit against the format's definition
in 64 bits: scales are exact halves, codes the exact quotient's nearest whole number."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests import prompt_util as U  # noqa: E402

KINDS = ("f16", "q8_0", "q8_0_q4_0", "q4_0")
BITS = {"f16": (16, 16), "q8_0": (8, 8), "q8_0_q4_0": (8, 4), "q4_0": (4, 4)}


def up_to_half(x):
    """|x| rounded up to a half, with x's sign (float64)."""
    mag = x.abs()
    step = torch.exp2(torch.floor(torch.log2(torch.where(mag > 0, mag, 1.0))).clamp(min=-14) - 10)
    return torch.copysign(torch.ceil(mag / step) * step, x)


def stored(x, bits):
    """(rows, scales) that half rows [T][Hk][D] become."""
    if bits == 16:
        return x, None
    b = x.double().unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], 0.0, b)
    mag = b.abs()
    if bits == 8:
        d = up_to_half(mag.amax(-1) / 127.0)
    else:
        first = torch.where(mag == mag.amax(-1, keepdim=True), torch.arange(32, device=x.device), 99).amin(-1, keepdim=True)
        d = up_to_half(b.gather(-1, first)[..., 0] / -8.0)
    c = torch.where(d[..., None] == 0, 0.0, torch.round(b / torch.where(d == 0, 1.0, d)[..., None]))
    if bits == 4:
        c = c.clamp(max=7.0)
    assert float(c.abs().max()) <= (127 if bits == 8 else 8)
    d = torch.where(bad, float("nan"), d).half()
    if bits == 8:
        return c.flatten(-2).to(torch.int8), d
    u = (c + 8).to(torch.uint8)
    return (u[..., :16] | (u[..., 16:] << 4)).flatten(-2), d


def same_scales(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])


def blank(kind, cells, Hk, D, fill=0x55):
    planes = []
    for bits in BITS[kind]:
        shape = (cells, Hk, D * bits // 8)
        raw = torch.full(shape, fill, dtype=torch.uint8, device="cuda")
        planes.append((raw.view(torch.float16) if bits == 16 else raw.view(torch.int8) if bits == 8 else raw,
                       None if bits == 16 else torch.full((cells, Hk, D // 32), 1.5, dtype=torch.float16, device="cuda")))
    (k, ks), (v, vs) = planes
    return k, v, ks, vs


def check_write(kv, kind, k, v, slots, cells, D):
    Hk = k.shape[1]
    kc, vc, ks, vs = blank(kind, cells, Hk, D)
    before = [None if x is None else x.clone() for x in (kc, vc, ks, vs)]
    kv.cache_write(k, v, slots, kc, vc, k_scales=ks, v_scales=vs)
    torch.cuda.synchronize()
    at = torch.arange(k.shape[0], device="cuda") if slots is None else slots.long()
    live = (at >= 0) & (at < cells)
    for x, bits, rows, scales, rows0, scales0 in ((k, BITS[kind][0], kc, ks, before[0], before[2]),
                                                  (v, BITS[kind][1], vc, vs, before[1], before[3])):
        want, d = stored(x, bits)
        rows0[at[live]] = want[live]
        as_bytes = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
        assert torch.equal(as_bytes(rows), as_bytes(rows0))    # other cells keep their bytes
        if d is not None:
            scales0[at[live]] = d[live]
            assert same_scales(scales, scales0)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("Hk", [1, 3, 8])
@pytest.mark.parametrize("kind", KINDS)
def test_write(kvattn, kind, Hk, D):
    g = U.gen(1)
    for T in (1, 2, 37, 700):
        cells = T + 11
        slots = torch.randperm(cells, generator=g, device="cuda")[:T].to(torch.int32)
        check_write(kvattn, kind, U.halves(g, T, Hk, D), U.halves(g, T, Hk, D), slots, cells, D)
    x = U.halves(g, 50, 3 * Hk + 1, D)   # slices of a fused projection, cells in order
    check_write(kvattn, kind, x[:, 1:Hk + 1], x[:, 2 * Hk:3 * Hk], None, 60, D)


@pytest.mark.parametrize("kind", KINDS)
def test_write_values(kvattn, kind):
    """Ties, signed ties of the largest magnitude, zeros, subnormal and the largest halves, values
    that are not finite."""
    g = U.gen(2)
    D, Hk, T = 128, 2, 64
    k = U.halves(g, T, Hk, D)
    k[0] = 0.0
    k[1] = -0.0
    k[2] = 65504.0
    k[3] = 6e-8                                     # 2^-24
    k[4] = (torch.arange(128, device="cuda") - 64).half()[None] * 2.0 ** -24
    k[5] = (torch.arange(128, device="cuda") - 64).half()[None] * 0.5
    k[6] = torch.where(torch.arange(128, device="cuda") % 2 == 0, 3.0, -3.0).half()
    k[7] = torch.where(torch.arange(128, device="cuda") % 2 == 0, -3.0, 3.0).half()
    k[8] = 1.0
    k[8, :, 5] = float("inf")
    k[9, :, 40] = float("nan")
    k[10, :, 127] = -float("inf")
    k[11] = (torch.arange(128, device="cuda") - 64).half()[None] * 127.0
    k[12] = (torch.arange(128, device="cuda") % 17 - 8).half()[None] * 2.5
    k[13, :, 0] = 60000.0
    # every quotient half-way between codes: 254 and odd numbers below it
    k[14] = torch.where(torch.arange(128, device="cuda") % 32 == 0, 254.0, (torch.arange(128, device="cuda") * 2 + 1) % 254).half()
    k[15] = torch.where(torch.arange(128, device="cuda") % 32 == 0, -16.0, torch.arange(128, device="cuda") % 32 - 15.0).half()
    check_write(kvattn, kind, k, k.flip(0).contiguous(), None, T, D)


@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
def test_write_all_quotients(kvattn, kind):
    """Half magnitudes against many block maxima: the code without a division is the exact one."""
    g = U.gen(3)
    T, Hk, D = 4096, 1, 256
    bits = torch.randint(0, 0x7c00, (T, Hk, D), generator=g, device="cuda", dtype=torch.int16)
    bits = torch.where(torch.rand(bits.shape, generator=g, device="cuda") < 0.5, bits, bits | -32768)
    x = bits.view(torch.float16)
    # ... whose blocks lie within a few powers of two, so that most codes are not zero
    e = torch.randint(-6, 6, (T, Hk, D // 32), generator=g, device="cuda").repeat_interleave(32, -1)
    y = torch.ldexp(U.halves(g, T, Hk, D).float(), e).half()
    check_write(kvattn, kind, x, y, None, T, D)


def test_write_skips_and_flags(kvattn):
    g = U.gen(4)
    k, v = U.halves(g, 6, 2, 128), U.halves(g, 6, 2, 128)
    slots = U.ints([3, -1, 9, 100, 0, -7])
    check_write(kvattn, "q8_0_q4_0", k, v, slots, 10, 128)
    kc, vc, ks, vs = blank("q8_0", 10, 2, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvattn.cache_write(k, v, U.ints([3, -1, 9, 1, 0, 2]), kc, vc, k_scales=ks, v_scales=vs, status=status)
    assert int(status) == 0
    kvattn.cache_write(k, v, slots, kc, vc, k_scales=ks, v_scales=vs, status=status)
    assert int(status) == kvattn.KVATTN_DEVICE_BAD_PLAN_ENTRY
    ko, vo = kvattn.cache_read(kc, vc, slots, head_dim=128, k_scales=ks, v_scales=vs, status=status)
    assert bool((ko[[1, 3, 5]] == 0).all()) and bool((vo[[1, 3, 5]] == 0).all())


def values(rows, scales, D):
    x = U.dequant(rows, scales, D)
    if scales is None:
        return rows
    return torch.where(torch.isnan(x), x, x.clamp(-65504.0, 65504.0)).half()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_read(kvattn, kind, D):
    g = U.gen(5)
    for Hk, cells, T in ((1, 5, 1), (3, 300, 700), (8, 1000, 257)):
        k, v, ks, vs = U.cache_planes(g, kind, cells, Hk, D)
        if ks is not None:
            ks[1, 0, 0] = 600.0                      # products beyond the largest half
            vs[2, 0, 1] = float("nan")
            vs[3, 0, 2] = -0.0
        slots = torch.randint(-1, cells, (T,), generator=g, device="cuda", dtype=torch.int32)  # some twice, some holes
        ko, vo = kvattn.cache_read(k, v, slots, head_dim=D, k_scales=ks, v_scales=vs)
        torch.cuda.synchronize()
        hole = (slots < 0)[:, None, None]
        for got, rows, scales in ((ko, k, ks), (vo, v, vs)):
            want = torch.where(hole, 0.0, values(rows, scales, D)[slots.clamp(min=0).long()].float())
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(got.float().nan_to_num(), want.nan_to_num())
        ko, vo = kvattn.cache_read(k, v, head_dim=D, k_scales=ks, v_scales=vs)
        assert ko.shape == (cells, Hk, D) and torch.equal(ko.nan_to_num(), values(k, ks, D).nan_to_num())


@pytest.mark.parametrize("kind,step", [("q8_0", 1 / 254), ("q4_0", 1 / 8)])
def test_written_then_read(kvattn, kind, step):
    g = U.gen(6)
    k, v = U.halves(g, 500, 4, 128), U.halves(g, 500, 4, 128, scale=1e-6)   # (v: subnormal halves)
    kc, vc, ks, vs = blank(kind, 600, 4, 128)
    slots = torch.randperm(600, generator=g, device="cuda")[:500].to(torch.int32)
    kvattn.cache_write(k, v, slots, kc, vc, k_scales=ks, v_scales=vs)
    x = torch.zeros(500, 9, 128, dtype=torch.float16, device="cuda")           # strided results
    ko, vo = kvattn.cache_read(kc, vc, slots, head_dim=128, k_scales=ks, v_scales=vs, k_out=x[:, :4], v_out=x[:, 5:])
    torch.cuda.synchronize()
    for a, b, s in ((k, ko, ks), (v, vo, vs)):
        d = s[slots.long()].double().abs().repeat_interleave(32, -1)
        # half a step (a whole one where the 4-bit +8 became 7) and the result's own rounding
        assert bool(((a.double() - b.double()).abs() <= d * (0.5 if kind == "q8_0" else 1.0) + a.double().abs() * U.HALF * 2
                     + 2.0 ** -24).all())
    assert bool((x[:, 4] == 0).all())


def test_offsets_beyond_32_bits(kvattn):
    """A plane of more than 2^32 bytes: the last cells are written and read, the first ones not."""
    Hk, D = 8, 256
    cells = (1 << 32) // (Hk * D) + 64
    g = U.gen(7)
    k, v = U.halves(g, 32, Hk, D), U.halves(g, 32, Hk, D)
    kc = torch.zeros(cells, Hk, D, dtype=torch.int8, device="cuda")
    vc = torch.zeros(cells, Hk, D, dtype=torch.int8, device="cuda")
    ks = torch.zeros(cells, Hk, D // 32, dtype=torch.float16, device="cuda")
    vs = torch.zeros_like(ks)
    slots = (cells - 1 - torch.arange(32, device="cuda")).to(torch.int32)
    kvattn.cache_write(k, v, slots, kc, vc, k_scales=ks, v_scales=vs)
    ko, _ = kvattn.cache_read(kc, vc, slots, head_dim=D, k_scales=ks, v_scales=vs)
    torch.cuda.synchronize()
    want, d = stored(k, 8)
    assert torch.equal(kc[slots.long()], want) and torch.equal(ks[slots.long()], d)
    assert torch.equal(ko, values(want, d, D))
    assert not bool(kc[:64].any())


def test_graph_and_streams(kvattn):
    g = U.gen(8)
    k, v = U.halves(g, 40, 2, 128), U.halves(g, 40, 2, 128)
    slots = torch.randperm(100, generator=g, device="cuda")[:40].to(torch.int32)
    kc, vc, ks, vs = blank("q4_0", 100, 2, 128)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvattn.cache_write(k, v, slots, kc, vc, k_scales=ks, v_scales=vs)
        kvattn.cache_read(kc, vc, slots, head_dim=128, k_scales=ks, v_scales=vs, k_out=ko, v_out=vo)
    for i in range(3):
        k.copy_(U.halves(g, 40, 2, 128))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ko, values(*stored(k, 4), 128))
