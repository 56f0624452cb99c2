// Causal attention of many query tokens per sequence on the fifth-generation tensor cores:
// whole packed prompts over their own K and V, and chunks of new tokens over a cache that
// already holds them (f16, Q8_0, Q8_0 + Q4_0, Q4_0; contiguous or through a cell plan).
//
// Rows.  For each KV head the G query heads of a token are neighbouring rows, so that every row
// of a work unit reads the same K and V: a row group is floor(128 / G) tokens x G rows (at most
// the 128 TMEM lanes), a block is two groups at head_dim 128 and one at 256, and a unit is a
// block and a KV head.  Token t of a sequence sees the cells below lim(t) = L - n_q + 1 + t.
//
//     S = Q K^T,  x = scale S (masked: -inf),  m = max x,  p = exp(x - m),
//     l = sum p,  O = sum p V,  out = O / l,  lse = m + ln l,
//
// one pass over the cells in tiles of 128 with a running m and l per row (32 bits; p is rounded
// to f16 for the matrix product only, l sums the unrounded p).
//
// Work.  The kernel is persistent, one CTA per SM.  Its schedulers cut the work in one of two
// ways: whole units dealt out in alternating directions, from the last sequence's last block (its
// longest) to the first's first (prompts, where units are many; with ragged prompts the order of
// the sequences decides how even that is); or (chunks) the concatenation of all units' tiles cut into equal contiguous shares,
// one per CTA, wherever the cuts fall.  A unit that is cut leaves partials (O_p, lse_p) in the
// workspace, two at most per CTA, and the merge kernel joins them.  The shares follow from the
// lengths alone, so results do not depend on timing.
//
// Sixteen warps with fixed roles:
//
//  * softmax (warps 0-7): threads t and t + 128 hold row t of a row group, which is TMEM lane t,
//    and half of a tile's columns each; they take the row groups' tiles in turn.  A thread reads
//    its scores from tensor memory, masks, and writes p over them as f16 pairs.  p is scaled by
//    2^7 (it cancels in O / l): with the lazily moved maximum below p stays under 2^15, and p of
//    2^-21 of a row's largest still has all its f16 bits.
//  * loader (warps 8-11): fills a ring of 32 KB slots, each 128 cells x 128 dims of K or V in
//    two 128-byte-swizzled planes.  f16: warp 8 issues a TMA box for each slot whose cells are
//    one physical run (holes and the end of a sequence included); warps 9-11 mend V slots that
//    need it afterwards, and copy the slots of tiles that are no run.  Quantised: warp 14 brings codes (TMA) and
//    scales (cp.async) into a ring of raw bytes, and these four turn them into f16.
//  * MMA (warp 12): one elected lane issues tcgen05.mma.  The 512 TMEM columns hold two buffers
//    of S, over which p is written, and O (2 x 128 columns, or 256).  With both row groups at
//    work each has a buffer, and a group's products run under the other's softmax; with one (256,
//    or at most 128 rows) its tiles take the buffers in turn, and S of the next tile runs under
//    the softmax of this one.
//  * scheduler (warp 13): finds the next unit's sequence, block and tiles while the others work,
//    and issues the TMA of its query rows once the last S of the unit before is complete.
//
// The running maximum moves only when it grows by more than 2^8 (in p), so that O is rescaled
// a few times per row at most; the softmax thread does it in tensor memory itself.
//
// Masked places: a score is replaced (not added to) before it is used, so whatever K holds there
// is dropped.  V is multiplied by p = 0 there, and 0 x inf is NaN on the tensor cores, so V rows
// that no row may see are zeroed in shared memory, and in a tile that only some rows see whole,
// elements of V that are not finite become zeros too and are added at the end to the rows that
// do see the cell (any p > 0 times an infinity is that infinity).
//
// What bounds it.  At head_dim 128 a tile of both row groups takes about 3450 clocks: two chains
// of that length turn in step, the softmax warps' (per group 550 clocks of exponentials at the
// special-function rate, the rest scores from and p to tensor memory, maxima, packing, a barrier)
// and each group's p -> P V -> S -> p; the four products alone take 2123.  A prompt of 8192 tokens
// (32 / 8 heads) takes 390 us, 1409 TFLOP/s (74 % of cuBLAS bf16) with pauses between the calls and
// 407 one after the other; 16 / 8 heads of 256, where one group's tiles follow each other, 428 with
// pauses.  Two row groups and halves of the columns for two warps
// are there for this: one warp per 32 rows and all columns took 3 % more over an 8-bit cache at
// 128, 28 % at 256.
// Chunks: 512 tokens over 16384 f16 cells 114 us (62 %).  Quantised caches: the turning of codes
// into f16, about 1500 clocks a slot, shares the issue slots with the softmax: 100 tokens over
// 131072 8-bit cells 240 us (47 %).
//
// Every wait is bounded, as in the decode kernels; a wait that gives up sets a flag that the
// others see, and KVATTN_DEVICE_WAIT_TIMEOUT in the workspace.
#include <climits>
#include <cmath>
#include <cstddef>
#include <mutex>

#include "prompt.cuh"

namespace kvattn {

namespace {

constexpr int kThreads = 512;
constexpr int kPlaneBytes = 128 * 128;        // 128 cells (or rows) x 128 bytes
constexpr int kSlotBytes = 2 * kPlaneBytes;   // 128 cells x 128 dims of f16
constexpr int kQTileBytes = 2 * kPlaneBytes;  // 128 rows x 128 dims of f16
constexpr int kMaxSlots = 5;
constexpr int kHeaderBytes = 3 * 1024;
constexpr int kRing = 4;                      // pieces of work whose plans are kept
constexpr int kMasks = 2;                     // tiles whose masks are
constexpr int kRawStages = 3;                 // quantised: slots of raw bytes in flight
constexpr int kCutTiles = 3;                  // tiles that only some of a unit's (<= 256) tokens see whole
constexpr float kSlack = 8.f;                 // lazy maximum
constexpr float kLift = 7.f;                  // p is scaled by 2^kLift
constexpr float kLn2 = 0.69314718055994530942f;
constexpr uint32_t kNoMore = 0xffffffffu;
constexpr int kUnitCost = 2;                  // a unit's fixed cost in tiles, for the equal shares

// f16 slots in the ring: what the 227 KB hold beside the queries (64 KB) and, for quantised
// caches, the raw ring (17 KB a stage with 8-bit rows, 9 KB with 4-bit ones)
template <int KBITS>
struct Memory {
    static constexpr int kSlots = KBITS == 16 ? 5 : (KBITS == 8 ? 3 : 4);
    static constexpr int kRawBytes = KBITS == 16 ? 0 : 128 * 8 * KBITS * 2 + 1024;  // codes, then scales
    static constexpr int kBytes = 2 * kQTileBytes + kSlots * kSlotBytes + kRawStages * kRawBytes + kHeaderBytes;
    static_assert(kBytes <= 232448, "227 KB");
};

// What the scheduler tells the others of a piece of work.
struct Seg {
    long long q_tok;     // first token of the block, in the packed rows
    long long cell0;     // first cell of the sequence (no plan)
    long long len;       // cells of the sequence
    long long lim0;      // lim of the block's first token
    int seq, g;
    int n_tok;           // tokens of the block; < 0: no more work
    int j0, n[2];        // first tile; tiles of the row groups from there
    int first_cut;       // from this tile on (from j0) some row does not see the tile whole
    int part;            // partial slot, or -1: the whole unit
    int whole, turn;     // the first `whole` tiles, which every row sees whole, are taken from tile `turn` on
};

// f16: a slot that warps 9-11 mend or copy, or the end of a unit.
struct Job {
    uint32_t n;          // slot number
    int32_t j;           // tile, from the piece's first
    uint32_t word;       // type | V << 2 | half << 3 | unit << 8
};
constexpr uint32_t kJobMend = 0, kJobCopy = 1, kJobUnit = 2, kJobEnd = 3;

struct Header {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t mended[kMaxSlots];  // a V slot that is mended after it landed
    uint64_t raw_full[kRawStages], raw_empty[kRawStages];  // quantised: a slot's raw bytes; they are turned
    uint64_t q_full, q_empty;    // the unit's query rows; its last S is complete
    uint64_t s_full[2], p_full[2];  // an S buffer holds S, or p
    uint64_t pv_done[2];         // its P V is complete
    uint64_t mask_full[kMasks], mask_empty[kMasks];  // through a plan: a tile's bias and holes are written, read
    uint64_t load_done[kRing];   // every slot of a unit is filled, its bad_cells are complete
    uint64_t seg_full[kRing], seg_empty[kRing];
    uint64_t job_full[kRing], job_empty[kRing];
    uint32_t tmem;
    int abort_flag;
    alignas(16) uint32_t bad_cells[kRing][kCutTiles][4];  // of a unit: cells of its cut tiles with V that is not finite
    uint32_t holes[kMasks];                   // whether the tile has any
    uint32_t slot_mend[kMaxSlots];            // whether the slot is one
    uint32_t raw_word[kRawStages];  // of a raw slot: V, cut, its unit's last, no slot at all | cut tile << 4 | unit << 8
    Seg seg[kRing];
    Job job[kRing];
    float meet[2][128];                       // what two threads of a row tell each other
    alignas(16) float bias[kMasks][kPrefillTile];  // through a plan: +inf, or -inf for a hole
};
static_assert(sizeof(Header) <= kHeaderBytes && offsetof(Header, bias) % 16 == 0 && offsetof(Header, bad_cells) % 16 == 0, "header");

// Shared-memory matrix descriptor: start address, leading and stride byte offsets, the
// descriptor version of this architecture family, 128-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor of kind::f16: f32 accumulator, f16 A and B, operand majors (1: the
// M/N dimension is contiguous), N and M.
constexpr uint32_t instr_desc(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kIdQK = instr_desc(128, 128, 0, 0);
constexpr uint32_t kIdPV = instr_desc(128, 128, 0, 1);

// byte (row r, byte b) of a 128-byte-swizzled plane whose base is 1024-byte aligned
__device__ __forceinline__ uint32_t swz(int r, int b) {
    return (uint32_t)(r * 128 + ((((b >> 4) & 7) ^ (r & 7)) << 4) + (b & 15));
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a_tmem), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t pred;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(pred));
    return pred != 0;
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 consecutive 32-bit TMEM columns of the warp's 32 lanes (one per thread)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                 "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                 "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_box4(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
// arrives on bar when this thread's cp.async so far are complete (adds itself to the phase's
// pending arrivals first: the phase must be held open by an arrival that comes later)
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 bytes, one sector where the address allows it
__device__ __forceinline__ void st_sector(void* at, const uint32_t* r, bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                     "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(at)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        reinterpret_cast<uint4*>(at)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// two fp32 operations per instruction
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// mbar_wait_bounded in fewer instructions: the kernel has some forty waits, and its sixteen warps'
// roles together are at the edge of what the instruction caches hold.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    if (mbar_test(bar, parity)) return true;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!mbar_test(bar, parity)) {
        if (*abort != 0 || global_ns() - t0 > limit_ns) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
// The OR of a predicate over the 64 threads that name this barrier; the barrier orders their
// shared-memory accesses.
__device__ __forceinline__ bool bar_or(int id, bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"((uint32_t)x)
                 : "memory");
    return r != 0u;
}
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Two 4-bit codes - 8 as halves, from bits 0-3 or 4-7 of both 16-bit halves of w: under the
// exponent of 1024, or of 64, a code stands in the mantissa with weight one.
__device__ __forceinline__ uint32_t nib_lo(uint32_t w) {
    return as_u32(__hsub2(as_h2((w & 0x000f000fu) | 0x64006400u), as_h2(0x64086408u)));
}
__device__ __forceinline__ uint32_t nib_hi(uint32_t w) {
    return as_u32(__hsub2(as_h2((w & 0x00f000f0u) | 0x54005400u), as_h2(0x54805480u)));
}
// Whether eight halves are all finite: adding 1 to an exponent of ones carries into the sign.
__device__ __forceinline__ bool finite8(const uint4& w) {
    const uint32_t a = (w.x & 0x7c007c00u) + 0x04000400u, b = (w.y & 0x7c007c00u) + 0x04000400u;
    const uint32_t c = (w.z & 0x7c007c00u) + 0x04000400u, d = (w.w & 0x7c007c00u) + 0x04000400u;
    return ((a | b | c | d) & 0x80008000u) == 0u;
}
// Zeros in place of the halves that are not finite; `bad` is set when there was one.
__device__ __forceinline__ uint32_t finite2(uint32_t w, bool& bad) {
    if ((w & 0x7c00u) == 0x7c00u) {
        w &= 0xffff0000u;
        bad = true;
    }
    if ((w & 0x7c000000u) == 0x7c000000u) {
        w &= 0xffffu;
        bad = true;
    }
    return w;
}

// Stored value = scale x code, rounded once to half: the type of an f16 cache (2^-11 of the
// value, where the 8-bit code itself is off by up to 2^-8 of the block's largest).  Scales
// above 515 could pass the largest half; those products are kept at it (as cache_read does).  In
// a cut tile what is not finite is dropped and its cell noted.  Both are done to 16 bytes of a
// slot after they were stored, and rarely.
constexpr uint32_t kBigScale = 0x6006u;   // 515
__device__ __forceinline__ void amend(unsigned char* at, uint32_t scale, bool cut, uint32_t* bad_row, int cell) {
    const __half2 top = __halves2half2(__ushort_as_half(0x7bffu), __ushort_as_half(0x7bffu));
    uint4 w = *reinterpret_cast<uint4*>(at);
    uint32_t o[4] = {w.x, w.y, w.z, w.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i] = as_u32(__hmax2_nan(__hmin2_nan(as_h2(o[i]), top), __hneg2(top)));
        if ((scale & 0x7c00u) == 0x7c00u) o[i] = 0x7fff7fffu;   // not finite: the whole block is NaN
        if (cut) o[i] = finite2(o[i], bad);
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
    if (bad) atomicOr(&bad_row[cell >> 5], 1u << (cell & 31));
}

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : (x > hi ? hi : x); }

// ------------------------------------ work ------------------------------------

template <int D>
struct Geometry {
    static constexpr int kGroups = D == 128 ? 2 : 1;
    static constexpr int kHalves = D / 128;     // slots per tile of K or V
};

// A sequence as the schedulers see it.
struct Sequence {
    int32_t q0, n_q, len;
    uint32_t blocks;
};
__device__ __forceinline__ Sequence read_sequence(const PrefillParams& p, int s) {
    Sequence x = {};
    if (s < 0 || s >= p.n_seq) return x;
    const int32_t n_tok = (int32_t)p.n_tok;
    const int32_t a = __ldg(p.offsets + s), e = __ldg(p.offsets + s + 1);
    x.q0 = min(max(a, 0), n_tok);
    x.n_q = min(max(e, x.q0), n_tok) - x.q0;
    x.len = x.n_q;
    if (p.seq_lens != nullptr) {
        const int64_t cap = p.plan != nullptr ? p.plan_stride : p.n_cells;
        x.len = (int32_t)clamp64(__ldg(p.seq_lens + s), 0, cap < p.max_len ? cap : p.max_len);
    }
    x.blocks = ((uint32_t)x.n_q + (uint32_t)p.block_tokens - 1u) / (uint32_t)p.block_tokens;
    return x;
}
// Tiles that the first n tokens of a block see.
__device__ __forceinline__ int32_t tiles_seen(int64_t lim0, int32_t n) {
    const int64_t lim = n > 0 ? lim0 + n - 1 : 0;
    return lim > 0 ? (int32_t)((lim + kPrefillTile - 1) / kPrefillTile) : 0;
}

// The units of all sequences in one line, in eighths of a tile: each a unit's fixed cost, then
// its tiles (by a rule that is linear in the block's number, so that sums have a closed form; the
// last share of a unit takes what is left).  CTA c of n takes [share(c), share(c + 1)) of it.
// Order: sequence, KV head, block.  The host sees to it that the line fits 32 bits.
// (With f16 rows and no plan a tile for one row group of two takes about 0.55 of one for both,
// 1900 clocks to 3450: a last block of one group counts 5 / 8 (units of 1 to 256 tokens over 8192
// to 65536 cells: 243 -> 229 us).  Through a plan, or from quantised rows, it waits for its loader
// and counts as a whole one: 5 / 8 there took 267 -> 302 us.)
struct Line {
    uint32_t a, step;       // length of block b: a + step b,
    uint32_t blocks, less;  // the last one's less this
    __device__ __forceinline__ uint32_t of(uint32_t b) const { return a + step * b - (b + 1u == blocks ? less : 0u); }
    __device__ __forceinline__ uint32_t upto(uint32_t b) const {
        return a * b + step * (b * (b - 1u) / 2u) - (b == blocks ? less : 0u);
    }
};
// Length of a tile of a block of n tokens in the line.
__device__ __forceinline__ int32_t tile_length(const PrefillParams& p, int32_t n_tok) {
    return n_tok <= p.group_tokens ? p.single_length : 8;
}
__device__ __forceinline__ Line line_of(const PrefillParams& p, const Sequence& x) {
    const int32_t lim = max(x.len - x.n_q, 0) + min(x.n_q, p.block_tokens);  // of the first block's last token, or above
    const int32_t tiles = lim / kPrefillTile + (lim % kPrefillTile != 0 ? 1 : 0);   // (lim can be 2^31 - 1)
    Line l{8u * (uint32_t)(kUnitCost + tiles), (uint32_t)(p.block_tokens + 15) / 16u, x.blocks, 0u};
    if (x.blocks != 0u) {
        const uint32_t whole = l.of(x.blocks - 1u);
        l.less = whole - (whole * (uint32_t)tile_length(p, x.n_q - (int32_t)(x.blocks - 1u) * p.block_tokens) >> 3);
    }
    return l;
}
struct Shares {
    uint32_t total, each, left, n;
    __device__ __forceinline__ void set(uint32_t total_, uint32_t n_) {
        total = total_;
        n = n_;
        each = total / n;
        left = total - each * n;
    }
    __device__ __forceinline__ uint32_t of(uint32_t c) const { return each * c + left * c / n; }
};
__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {  // inclusive, over the lanes
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}
__device__ __forceinline__ uint32_t length_of(const PrefillParams& p, const Sequence& x) {
    return x.blocks != 0u ? line_of(p, x).upto(x.blocks) * (uint32_t)p.n_head_kv : 0u;
}
__device__ __forceinline__ uint32_t total_of(const PrefillParams& p) {
    uint32_t sum = 0;
    for (int s = threadIdx.x & 31; s < p.n_seq; s += 32) sum += length_of(p, read_sequence(p, s));
    return __reduce_add_sync(0xffffffffu, sum);
}
__device__ __forceinline__ Sequence from_lane(const Sequence& x, int l) {
    Sequence y;
    y.q0 = __shfl_sync(0xffffffffu, x.q0, l);
    y.n_q = __shfl_sync(0xffffffffu, x.n_q, l);
    y.len = __shfl_sync(0xffffffffu, x.len, l);
    y.blocks = __shfl_sync(0xffffffffu, x.blocks, l);
    return y;
}
// The unit that holds position `at` of the line (at < total), the same in all lanes.
struct Place {
    Sequence x;
    Line line;
    int seq;
    uint32_t g, block, start, end;  // start, end: the unit's part of the line
    __device__ __forceinline__ int32_t tok0(const PrefillParams& p) const { return (int32_t)block * p.block_tokens; }
    __device__ __forceinline__ int32_t tokens(const PrefillParams& p) const { return min(x.n_q - tok0(p), p.block_tokens); }
    __device__ __forceinline__ int32_t tiles(const PrefillParams& p) const {
        return tiles_seen((int64_t)x.len - x.n_q + 1 + tok0(p), tokens(p));
    }
};
// The tile that position y of a unit of that length and n tiles of length `each` falls on.
__device__ __forceinline__ int32_t tile_at(uint32_t y, uint32_t length, int32_t n, int32_t each) {
    const int32_t t = ((int32_t)y - each * (int32_t)kUnitCost) / each;
    return y >= length ? n : min(max(t, 0), n);
}
__device__ __forceinline__ Place place_of(const PrefillParams& p, uint32_t at) {
    Place r = {};
    uint32_t base = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += 32) {
        const Sequence x = read_sequence(p, s0 + (threadIdx.x & 31));
        const uint32_t own = length_of(p, x), sum = warp_scan(own);
        const uint32_t hit = __ballot_sync(0xffffffffu, at < base + sum);
        if (hit != 0u) {
            const int l = __ffs(hit) - 1;
            r.seq = s0 + l;
            r.x = from_lane(x, l);
            base += __shfl_sync(0xffffffffu, sum - own, l);
            break;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (r.x.blocks == 0u) return r;   // (no such place: offsets that overlap can pass the line's 32 bits)
    r.line = line_of(p, r.x);
    const uint32_t per = r.line.upto(r.x.blocks);
    uint32_t y = at - base;
    r.g = y / per;
    y -= r.g * per;
    uint32_t lo = 0, hi = r.x.blocks - 1u;  // the last block that starts at or before y
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1u) / 2u;
        if (r.line.upto(mid) <= y)
            lo = mid;
        else
            hi = mid - 1u;
    }
    r.block = lo;
    r.start = at - (y - r.line.upto(lo));
    r.end = r.start + r.line.of(lo);
    return r;
}

// Fills in a piece of work: tiles [first, last) of a block.
template <int D>
__device__ __forceinline__ void make_seg(const PrefillParams& p, const Sequence& x, int seq, int g, uint32_t block, int32_t first,
                                         int32_t last, int part, int from, Seg& s) {
    constexpr int kGroups = Geometry<D>::kGroups;
    const int32_t tok0 = (int32_t)block * p.block_tokens;
    s.seq = seq;
    s.g = g;
    s.n_tok = min(x.n_q - tok0, p.block_tokens);
    s.q_tok = x.q0 + tok0;
    s.cell0 = p.seq_lens != nullptr ? (int64_t)seq * p.n_cells : (int64_t)x.q0;
    s.len = x.len;
    s.lim0 = (int64_t)x.len - x.n_q + 1 + tok0;
    s.j0 = first;
    s.part = part;
    int n_max = 0;
    s.n[1] = 0;
#pragma unroll
    for (int t = 0; t < kGroups; ++t) {
        const int32_t in = min(s.n_tok, (t + 1) * p.group_tokens);
        const int32_t tiles = min(in > t * p.group_tokens ? tiles_seen(s.lim0, in) : 0, last);
        s.n[t] = max(tiles - first, 0);
        n_max = max(n_max, s.n[t]);
    }
    // (the sequence's last token alone: its rows see all that is there.  With more than 64 heads per
    // KV head at 256 every token is alone, and the others' last tile holds cells that they do not see)
    const int64_t cut = (s.lim0 > 0 ? s.lim0 : 0) / kPrefillTile - first;
    s.first_cut = ((s.n_tok == 1 && s.lim0 >= s.len) || cut > n_max) ? n_max : (cut < 0 ? 0 : (int)cut);
    s.whole = min(s.first_cut, (int)clamp64(x.len / kPrefillTile - first, 0, n_max));
    if (s.n[1] > 0) s.whole = min(s.whole, min(s.n[0], s.n[1]));
    s.turn = from < s.whole ? from : 0;
}

// A warp's walk over its CTA's pieces.
template <int D>
struct Walk {
    // whole units
    uint32_t round;
    // shares
    uint32_t at, end;
    Shares sh;
    Place r;
    bool started;

    __device__ __forceinline__ void begin(const PrefillParams& p) {
        round = 0;
        started = false;
        if (p.shares) {
            sh.set(total_of(p), gridDim.x);
            at = sh.of(blockIdx.x);
            end = sh.of(blockIdx.x + 1u);
            if ((threadIdx.x & 31) == 0) p.cuts[blockIdx.x].n_parts = 0;
        }
    }
    // The next piece in s; false: none left.
    __device__ __forceinline__ bool next(const PrefillParams& p, Seg& s) {
        int32_t first = 0, last = INT_MAX;
        int part = -1, from = 0;
        if (!(p.shares ? next_share(p, first, last, part, from) : next_whole(p))) return false;
        make_seg<D>(p, r.x, r.seq, (int)r.g, r.block, first, last, part, from, s);
        return true;
    }

    // Unit number i counts from the last sequence's last block (the longest rows of a prompt
    // first), KV heads fastest; round r deals them out forwards or backwards.
    __device__ __forceinline__ bool next_whole(const PrefillParams& p) {
        const uint32_t n = gridDim.x, c = blockIdx.x;
        const uint32_t i = round * n + ((round & 1u) ? n - 1u - c : c);
        if (i < round * n) return false;  // (beyond 32 bits)
        ++round;
        const uint32_t b = i / (uint32_t)p.n_head_kv, g = i - b * (uint32_t)p.n_head_kv;
        uint32_t seen = 0;
        for (int top = p.n_seq; top > 0; top -= 32) {
            const Sequence x = read_sequence(p, top - 1 - (int)(threadIdx.x & 31));
            const uint32_t sum = warp_scan(x.blocks);
            const uint32_t hit = __ballot_sync(0xffffffffu, b < seen + sum);
            if (hit != 0u) {
                const int l = __ffs(hit) - 1;
                r.x = from_lane(x, l);
                r.seq = top - 1 - l;
                r.g = g;
                r.block = r.x.blocks - 1u - (b - (seen + __shfl_sync(0xffffffffu, sum, l) - r.x.blocks));
                return true;
            }
            seen += __shfl_sync(0xffffffffu, sum, 31);
        }
        return false;
    }

    // Blocks of one KV head read the same cells, in pieces that begin anywhere.  So that a tile's
    // readers come by at about the same time, and find it in L2, every CTA takes tile t of any
    // unit at about time t modulo the length of a share: a piece's whole tiles begin at the one
    // whose time it is when the piece begins, and go around (`from`).
    __device__ __forceinline__ bool next_share(const PrefillParams& p, int32_t& first, int32_t& last, int& part, int& from) {
        while (at < end) {
            if (!started || (r.block + 1u == r.x.blocks && r.g + 1u == (uint32_t)p.n_head_kv)) {
                r = place_of(p, at);
                started = true;
            } else {  // the next unit of the sequence
                if (++r.block == r.x.blocks) {
                    r.block = 0;
                    ++r.g;
                }
                r.start = r.end;
                r.end = r.start + r.line.of(r.block);
            }
            if (r.end <= at) break;
            const uint32_t a = at, b = min(r.end, end);
            at = b;
            const int32_t tiles = r.tiles(p), each = tile_length(p, r.tokens(p));
            first = tile_at(a - r.start, r.end - r.start, tiles, each);
            last = tile_at(b - r.start, r.end - r.start, tiles, each);
            // a unit whose first piece is here and whose last is not: the merge joins its parts
            if (a == r.start && b != r.end && tiles > 0 && (threadIdx.x & 31) == 0) {
                PrefillCut* cut = p.cuts + blockIdx.x;
                int parts = 1;
                while (blockIdx.x + (uint32_t)parts < gridDim.x && sh.of(blockIdx.x + (uint32_t)parts) < r.end) ++parts;
                cut->q_tok = r.x.q0 + r.tok0(p);
                cut->n_tok = r.tokens(p);
                cut->g = (int32_t)r.g;
                cut->tiles = tiles;
                cut->start = r.start;
                cut->end = r.end;
                cut->n_parts = parts;
            }
            if (tiles == 0 ? a != r.start : first == last) continue;  // (a unit that sees nothing: its first piece)
            part = first == 0 && last == tiles ? -1 : 2 * (int)blockIdx.x + (a > r.start ? 0 : 1);
            if (r.x.blocks > 1u) {
                const int32_t period = max((int32_t)(sh.each >> 3), 1);
                from = ((int32_t)((a - sh.of(blockIdx.x)) >> 3) - first) % period;
                if (from < 0) from += period;
            }
            return true;
        }
        return false;
    }
};

// The order in which the MMA warp takes a piece's slots, HALVES (128 of the dims each) per tile of
// K or V: with both row groups at work K0 V0 K1 V1 .., with one K0 K1 V0 K2 V1 ...
template <int HALVES>
__device__ __forceinline__ void slot_number(int step, int n_max, bool dual, bool& v_side, int& j, int& half) {
    const int q = step / HALVES;
    half = step % HALVES;
    if (dual) {
        v_side = q & 1;
        j = q >> 1;
    } else if (q == 0 || q == 2 * n_max - 1) {
        v_side = q != 0;
        j = q == 0 ? 0 : n_max - 1;
    } else {
        v_side = !(q & 1);
        j = v_side ? (q >> 1) - 1 : (q >> 1) + 1;
    }
}

// A tile's cells, in a warp: lane l holds cells l, l + 32, l + 64, l + 96.
struct Tile {
    int32_t e[4];     // physical cells (no plan: from the tile's first), -1: none
    int64_t base;     // first physical cell when a run
    bool run, holes;  // the cells that are there lie at base + their number; some are not
};
template <bool PLAN>
__device__ __forceinline__ Tile read_tile(const PrefillParams& p, const Seg& s, int j) {
    Tile t;
    const int lane = threadIdx.x & 31;
    int at = j;
    if (j < s.whole) {
        at += s.turn;
        if (at >= s.whole) at -= s.whole;
    }
    const int64_t i0 = (int64_t)(s.j0 + at) * kPrefillTile;
    const int n_max = s.n[0] > s.n[1] ? s.n[0] : s.n[1];
    const int left = j < n_max ? (int)clamp64(s.len - i0, 0, kPrefillTile) : 0;
    t.run = true;
    t.holes = left < kPrefillTile;
    t.base = s.cell0 + i0;
    const int32_t* row = PLAN ? p.plan + (int64_t)s.seq * p.plan_stride + i0 : nullptr;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = 32 * k + lane;
        t.e[k] = -1;
        if (c < left) t.e[k] = row != nullptr ? __ldg(row + c) : c;
    }
    return t;
}
// Checks a plan tile's entries and whether they are one run; true: all entries are in range.
template <bool PLAN>
__device__ __forceinline__ bool settle(const PrefillParams& p, Tile& t) {
    if (!PLAN) return true;
    const int lane = threadIdx.x & 31;
    int lo = INT_MAX, hi = INT_MIN;
    bool hole = false, good = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (t.e[k] < -1 || (int64_t)t.e[k] >= p.n_cells) {
            good = false;
            t.e[k] = -1;
        }
        if (t.e[k] >= 0) {
            const int d = t.e[k] - (32 * k + lane);
            lo = min(lo, d);
            hi = max(hi, d);
        } else {
            hole = true;
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    t.run = lo >= hi;   // (no cell at all: lo > hi)
    t.base = lo <= hi ? lo : 0;
    t.holes = __any_sync(0xffffffffu, hole);
    return good;
}
// Physical cell of the tile's cell c (which may differ from lane to lane), -1: none.
template <bool PLAN>
__device__ __forceinline__ int64_t cell_of(const Tile& t, int c) {
    const int32_t v0 = __shfl_sync(0xffffffffu, t.e[0], c & 31);
    const int32_t v1 = __shfl_sync(0xffffffffu, t.e[1], c & 31);
    const int32_t v2 = __shfl_sync(0xffffffffu, t.e[2], c & 31);
    const int32_t v3 = __shfl_sync(0xffffffffu, t.e[3], c & 31);
    const int32_t v = (c & 64) ? ((c & 32) ? v3 : v2) : ((c & 32) ? v1 : v0);
    return (!PLAN && v >= 0) ? t.base + v : v;
}

// ------------------------------------- the kernel -------------------------------------

// PLAN: through a cell plan (a kernel of its own: the masks' code slowed the others by 2 %).
template <int D, int KBITS, int VBITS, bool PLAN>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillParams p) {
    constexpr int kGroups = Geometry<D>::kGroups, kHalves = Geometry<D>::kHalves;
    constexpr bool kQuant = KBITS != 16;
    constexpr int kSlots = Memory<KBITS>::kSlots;
    // TMEM columns: two buffers of S, over which p is written; O of the row groups
    constexpr uint32_t kColS1 = 128, kColO = 256;
    // the swizzled planes want a 1024-byte aligned base; with no static shared memory the window
    // starts on one, and nothing is left to align it with
    extern __shared__ __align__(1024) unsigned char q_tiles[];
    unsigned char* slots = q_tiles + 2 * kQTileBytes;
    unsigned char* raws = slots + kSlots * kSlotBytes;
    Header* h = reinterpret_cast<Header*>(raws + kRawStages * Memory<KBITS>::kRawBytes);
    volatile int* abort_flag = &h->abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((smem_addr(q_tiles) & 1023u) != 0u) {
        if (tid == 0) atomicOr(p.status, KVATTN_DEVICE_WAIT_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(smem_addr(&h->full[i]), kQuant ? 4 : 1);  // the loader's warps, or warp 8
            mbar_init(smem_addr(&h->empty[i]), 1);              // the MMA lane's commit
            mbar_init(smem_addr(&h->mended[i]), 3);             // warps 9-11
        }
        for (int i = 0; i < kMasks; ++i) {
            mbar_init(smem_addr(&h->mask_full[i]), 1);
            mbar_init(smem_addr(&h->mask_empty[i]), 8);
        }
        for (int i = 0; i < kRawStages; ++i) {
            mbar_init(smem_addr(&h->raw_full[i]), 1);
            mbar_init(smem_addr(&h->raw_empty[i]), 4);
        }
        mbar_init(smem_addr(&h->q_full), 1);
        mbar_init(smem_addr(&h->q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&h->s_full[i]), 1);
            mbar_init(smem_addr(&h->p_full[i]), 8);
            mbar_init(smem_addr(&h->pv_done[i]), 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_addr(&h->load_done[i]), kQuant ? 4 : 3);
            mbar_init(smem_addr(&h->job_full[i]), 1);
            mbar_init(smem_addr(&h->job_empty[i]), 3);
            mbar_init(smem_addr(&h->seg_full[i]), 1);
            mbar_init(smem_addr(&h->seg_empty[i]), (kQuant ? 2 : 5) + 8);  // loader, MMA and softmax warps
        }
        h->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&h->tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = h->tmem;
    pdl_wait();
    const int G = p.group;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_bar(smem_addr(bar), parity, abort_flag, p.wait_limit_ns));
    };
    // piece number i (in the order of the scheduler); false: no more, or a wait that gave up
    auto take = [&](uint32_t i, Seg& s) -> bool {
        if (!wait_all(&h->seg_full[i % kRing], (i / kRing) & 1u)) return false;
        s = h->seg[i % kRing];
        return s.n_tok >= 0;
    };
    auto give_back = [&](uint32_t i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&h->seg_empty[i % kRing]));
    };

    // a plan tile's holes, for the softmax (tile number T of the CTA), from one warp
    auto put_mask = [&](const Tile& t, uint32_t T) -> bool {
        const uint32_t r = T % kMasks;
        if (T >= kMasks && !wait_all(&h->mask_empty[r], (T / kMasks - 1u) & 1u)) return false;
#pragma unroll
        for (int k = 0; k < 4; ++k) h->bias[r][32 * k + lane] = t.e[k] < 0 ? -INFINITY : INFINITY;
        if (lane == 0) h->holes[r] = t.holes ? 1u : 0u;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&h->mask_full[r]));
        return true;
    };

    if (warp >= 8 && warp < 12) {
        // (the four warpgroups' shares add up to the 4 x 128 registers of the launch)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        // ------------------------------------ loader ------------------------------------
        const int lt = tid - 256;       // 0 .. 127
        bool bad_entry = false, ok = true;
        uint32_t filled = 0;            // slots
        uint32_t n = 0;                 // quantised: raw slots turned
        Seg s = {};
        auto wait_slot_empty = [&]() -> bool {
            const uint32_t use = filled / kSlots;
            return use == 0 || wait_all(&h->empty[filled % kSlots], (use - 1) & 1u);
        };
        auto slot_ready = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(bar));
            ++filled;
        };
        auto stall_hook = [&](uint64_t* bar) {
            if (filled == 0 && p.stall_tx != 0u && lt == 0) mbar_expect_tx(smem_addr(bar), p.stall_tx);
        };

        if constexpr (!kQuant) {
            if (warp == 8) {
                // ---- f16: fills the slots by TMA, and leaves jobs to warps 9-11 ----
                uint32_t jobs = 0, T = 0;     // jobs given, tiles begun
                auto give_job = [&](uint32_t word, int j) -> bool {
                    const uint32_t e = jobs % kRing;
                    if (jobs >= kRing && !wait_all(&h->job_empty[e], (jobs / kRing - 1u) & 1u)) return false;
                    if (lane == 0) {
                        h->job[e] = Job{filled, j, word};
                        mbar_arrive(smem_addr(&h->job_full[e]));
                    }
                    __syncwarp();
                    ++jobs;
                    return true;
                };
                for (uint32_t i = 0; ok; ++i) {
                    if (!take(i, s)) break;
                    const int n_max = s.n[0] > s.n[1] ? s.n[0] : s.n[1];
                    const uint32_t unit = (i & 0xffffu) << 8;
                    Tile tk = read_tile<PLAN>(p, s, 0), tv = tk, next = read_tile<PLAN>(p, s, 1);
#pragma unroll 1
                    for (int step = 0; step < 2 * kHalves * n_max && ok; ++step) {
                        bool v_side;
                        int j, half;
                        slot_number<kHalves>(step, n_max, s.n[1] > 0, v_side, j, half);
                        if (!v_side && half == 0) {   // a tile begins (its V may come after the next one's K)
                            if (j > 0) {
                                tv = tk;
                                tk = next;
                                next = read_tile<PLAN>(p, s, j + 1);
                            }
                            if (!settle<PLAN>(p, tk)) bad_entry = true;
                            if (PLAN && !(ok = put_mask(tk, T))) break;
                            ++T;
                        }
                        if (v_side && (s.n[1] > 0 || j + 1 == n_max)) tv = tk;
                        const bool run = (v_side ? tv.run : tk.run) && p.use_tma != 0;
                        const bool job = !run || (v_side && (j >= s.first_cut || tv.holes));
                        if (!(ok = wait_slot_empty())) break;
                        const uint32_t st = filled % kSlots;
                        if (lane == 0) {
                            const uint32_t bar = smem_addr(&h->full[st]);
                            h->slot_mend[st] = job ? 1u : 0u;
                            if (filled == 0 && p.stall_tx != 0u) mbar_expect_tx(bar, p.stall_tx);
                            if (run) {
                                mbar_expect_tx(bar, (uint32_t)kSlotBytes);
                                tma_box4(smem_addr(slots + st * kSlotBytes), v_side ? &p.tmap_v : &p.tmap_k, 0,
                                         (int)(v_side ? tv.base : tk.base), 2 * half, s.g, bar);
                            }
                            mbar_arrive(bar);
                        }
                        __syncwarp();
                        if (job && !(ok = give_job(unit | (run ? kJobMend : kJobCopy) | (v_side ? 4u : 0u) | (half ? 8u : 0u), j))) break;
                        ++filled;
                    }
                    ok = ok && give_job(unit | kJobUnit, 0);
                    give_back(i);
                }
                if (ok) give_job(kJobEnd, 0);
            } else {
                // ---- warps 9-11: rows that TMA cannot bring, or that are mended after it did ----
                for (uint32_t k = 0;; ++k) {
                    const uint32_t e = k % kRing;
                    if (!wait_all(&h->job_full[e], (k / kRing) & 1u)) break;
                    const Job job = h->job[e];
                    const uint32_t type = job.word & 3u;
                    if (type == kJobEnd) break;
                    const uint32_t i = (job.word >> 8) & 0xffffu;   // (kRing divides 65536)
                    if (type == kJobUnit) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&h->load_done[i % kRing]));
                        give_back(i);
                    } else {
                        s = h->seg[i % kRing];                      // (not given back yet)
                        const bool v_side = job.word & 4u, cut = v_side && job.j >= s.first_cut;
                        const int half = (job.word >> 3) & 1u;
                        Tile t = read_tile<PLAN>(p, s, job.j);
                        settle<PLAN>(p, t);
                        const uint32_t st = job.n % kSlots;
                        const int sub = lane >> 4, b = (lane & 15) * 16;      // 16 lanes a row
                        unsigned char* plane = slots + st * kSlotBytes + (b >> 7) * kPlaneBytes;
                        uint32_t* bad_row = h->bad_cells[i % kRing][cut ? (job.j - s.first_cut) % kCutTiles : 0];
                        if (type == kJobMend) {
                            // (MMA waits for the mended slot, so this use of it is not over)
                            if (!wait_all(&h->full[st], (job.n / kSlots) & 1u)) break;
                            // (cells below the first token's end are seen by all rows: nothing to keep apart)
                            const int64_t seen = s.lim0 - (int64_t)(s.j0 + job.j) * kPrefillTile;
#pragma unroll 1
                            for (int k4 = 0; k4 < 4; ++k4) {                  // 32 cells at a time
                                const int32_t e = k4 < 2 ? (k4 ? t.e[1] : t.e[0]) : (k4 == 2 ? t.e[2] : t.e[3]);
                                const uint32_t gone = __ballot_sync(0xffffffffu, e < 0);
                                if ((!cut || seen >= 32 * k4 + 32) && gone == 0u) continue;
                                unsigned char* cells = plane + 4096 * k4;
#pragma unroll
                                for (int q = 0; q < 6; ++q) {
                                    const int c = 2 * (3 * q + warp - 9) + sub;
                                    if (c >= 32) continue;
                                    uint4* at = reinterpret_cast<uint4*>(cells + swz(c, b & 127));
                                    if ((gone >> c) & 1u) {
                                        *at = make_uint4(0u, 0u, 0u, 0u);
                                    } else if (cut) {
                                        uint4 w = *at;
                                        if (!finite8(w)) {
                                            bool bad;
                                            w = make_uint4(finite2(w.x, bad), finite2(w.y, bad), finite2(w.z, bad), finite2(w.w, bad));
                                            *at = w;
                                            atomicOr(&bad_row[k4], 1u << c);
                                        }
                                    }
                                }
                            }
                        } else {
                            const char* rows = reinterpret_cast<const char*>(static_cast<const __half*>(v_side ? p.v : p.k) +
                                                                             (int64_t)s.g * D + half * 128) + b;
                            const int64_t row_bytes = (v_side ? p.v_stride : p.k_stride) * 2;
#pragma unroll 1
                            for (int r0 = 2 * (warp - 9); r0 < 128; r0 += 24) {   // four rows in flight
                                uint4 w[4];
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const int64_t cell = cell_of<PLAN>(t, min(r0 + 6 * q, 126) + sub);
                                    w[q] = make_uint4(0u, 0u, 0u, 0u);
                                    if (cell >= 0) w[q] = __ldg(reinterpret_cast<const uint4*>(rows + cell * row_bytes));
                                }
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const int c = r0 + 6 * q + sub;
                                    if (c >= 128) continue;
                                    if (cut && !finite8(w[q])) {
                                        bool bad;
                                        w[q] = make_uint4(finite2(w[q].x, bad), finite2(w[q].y, bad), finite2(w[q].z, bad),
                                                          finite2(w[q].w, bad));
                                        atomicOr(&bad_row[c >> 5], 1u << (c & 31));
                                    }
                                    *reinterpret_cast<uint4*>(plane + swz(c, b & 127)) = w[q];
                                }
                            }
                        }
                        fence_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&h->mended[st]));
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&h->job_empty[e]));
                }
            }
        } else {
            // ---- quantised: turns the raw slots that warp 14 brings ----
            for (;; ++n) {
                const uint32_t r = n % kRawStages;
                // (both waits with one vote: a word that was read after a lost one is not used)
                bool got = wait_bar(smem_addr(&h->raw_full[r]), (n / kRawStages) & 1u, abort_flag, p.wait_limit_ns);
                const uint32_t word = h->raw_word[r];
                if (!(word & 8u) && filled >= kSlots)
                    got = wait_bar(smem_addr(&h->empty[filled % kSlots]), (filled / kSlots - 1) & 1u, abort_flag,
                                   p.wait_limit_ns) && got;
                if (!(ok = __all_sync(0xffffffffu, got)) || word == kNoMore) break;
                const bool v_side = word & 1u, cut = (word >> 1) & 1u;
                const uint32_t unit = (word >> 8) & 0xffffu;
                if (!(word & 8u)) {
                    stall_hook(&h->full[filled % kSlots]);
                    const int bits = v_side ? VBITS : KBITS;
                    const unsigned char* stage = raws + r * Memory<KBITS>::kRawBytes;
                    const unsigned short* scales = reinterpret_cast<const unsigned short*>(stage + Memory<KBITS>::kRawBytes - 1024);
                    unsigned char* slot = slots + (filled % kSlots) * kSlotBytes;
                    uint32_t* bad_row = h->bad_cells[unit % kRing][(word >> 4) & 3u];
                    if (bits == 8) {
                        const int piece = lt & 7;  // halves 16 piece .. of the row: bytes 32 piece ..
                        unsigned char* plane = slot + (piece >> 2) * kPlaneBytes;
                        const int c0 = lt >> 3;    // cells c0, c0 + 16, ..: the same place in the swizzle
                        const uint32_t oa = swz(c0, (piece & 3) * 32), ob = oa ^ 16u;
                        // (the upper plane's lanes store in the other order: eight lanes, eight bank groups)
                        const bool upper = piece >= 4;
                        unsigned char* d0 = plane + (upper ? ob : oa);
                        unsigned char* d1 = plane + (upper ? oa : ob);
                        const unsigned char* src = stage + 16 * lt;
                        const unsigned short* sc = scales + 4 * c0 + (piece >> 1);
                        // four cells at a time, loads first: the stores cannot be seen not to alias them
#pragma unroll 1
                        for (int k0 = 0; k0 < 8; k0 += 4) {
                            uint4 w[4];
                            uint32_t ds[4], big = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                w[k] = *reinterpret_cast<const uint4*>(src + 2048 * (k0 + k));
                                ds[k] = sc[64 * (k0 + k)];
                                big = max(big, ds[k]);   // (a negative one, which no write makes, counts as big)
                            }
                            const bool odd = cut || big > kBigScale;   // rare: a loop of its own below
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t d = prmt_b32(ds[k], 0u, 0x1010u);
                                const uint32_t x[4] = {(upper ? w[k].z : w[k].x) ^ 0x80808080u, (upper ? w[k].w : w[k].y) ^ 0x80808080u,
                                                       (upper ? w[k].x : w[k].z) ^ 0x80808080u, (upper ? w[k].y : w[k].w) ^ 0x80808080u};
                                uint32_t o[8];
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    o[2 * q] = hmul2_u32(i8x2_lo(x[q]), d);
                                    o[2 * q + 1] = hmul2_u32(i8x2_hi(x[q]), d);
                                }
                                *reinterpret_cast<uint4*>(d0 + 2048 * (k0 + k)) = make_uint4(o[0], o[1], o[2], o[3]);
                                *reinterpret_cast<uint4*>(d1 + 2048 * (k0 + k)) = make_uint4(o[4], o[5], o[6], o[7]);
                            }
                            if (odd)
#pragma unroll 1
                                for (int k = k0; k < k0 + 4; ++k) {
                                    amend(d0 + 2048 * k, sc[64 * k], cut, bad_row, c0 + 16 * k);
                                    amend(d1 + 2048 * k, sc[64 * k], cut, bad_row, c0 + 16 * k);
                                }
                        }
                    } else {
                        const int piece = lt & 3;  // block `piece`: halves 32 piece .., bytes 64 piece ..
                        unsigned char* plane = slot + (piece >> 1) * kPlaneBytes;
                        const int c0 = lt >> 2;    // cells c0, c0 + 32, ..
                        const int b = (piece & 1) * 64;
#pragma unroll 1
                        for (int k0 = 0; k0 < 4; k0 += 2) {
                            uint4 w[2];
                            uint32_t ds[2], big = 0;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                w[k] = *reinterpret_cast<const uint4*>(stage + 16 * lt + 2048 * (k0 + k));
                                ds[k] = scales[4 * c0 + piece + 128 * (k0 + k)];
                                big = max(big, ds[k] & 0x7fffu);
                            }
                            const bool odd = cut || big > kBigScale;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t d = prmt_b32(ds[k], 0u, 0x1010u);
                                const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                                uint32_t o[16];  // elements 0-15 and 16-31 of the block
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const uint32_t a = prmt_b32(x[q], 0u, 0x4140u), e = prmt_b32(x[q], 0u, 0x4342u);
                                    o[2 * q] = hmul2_u32(nib_lo(a), d);
                                    o[2 * q + 1] = hmul2_u32(nib_lo(e), d);
                                    o[8 + 2 * q] = hmul2_u32(nib_hi(a), d);
                                    o[9 + 2 * q] = hmul2_u32(nib_hi(e), d);
                                }
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    *reinterpret_cast<uint4*>(plane + swz(c0, b + 16 * q) + 4096 * (k0 + k)) =
                                        make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                            }
                            if (odd)
#pragma unroll 1
                                for (int i = 0; i < 8; ++i)
                                    amend(plane + swz(c0, b + 16 * (i & 3)) + 4096 * (k0 + (i >> 2)),
                                          scales[4 * c0 + piece + 128 * (k0 + (i >> 2))], cut, bad_row, c0 + 32 * (k0 + (i >> 2)));
                        }
                    }
                    fence_async();
                    slot_ready(&h->full[filled % kSlots]);
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&h->raw_empty[r]));
                    if (word & 4u) mbar_arrive(smem_addr(&h->load_done[unit % kRing]));  // the unit's last slot
                }
            }
        }
        if (__any_sync(0xffffffffu, bad_entry) && lane == 0 && warp == 8) atomicOr(p.status, KVATTN_DEVICE_BAD_PLAN_ENTRY);
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        if (warp == 13) {
            // ---------------------------------- scheduler ----------------------------------
            Walk<D> walk;
            walk.begin(p);
            uint32_t q_uses = 0;
            for (uint32_t i = 0;; ++i) {
                Seg s;
                if (!walk.next(p, s)) s.n_tok = -1;
                if (i >= kRing && !wait_all(&h->seg_empty[i % kRing], ((i / kRing) - 1) & 1u)) break;
                if (lane < 4 * kCutTiles) h->bad_cells[i % kRing][lane >> 2][lane & 3] = 0u;
                __syncwarp();
                if (lane == 0) {
                    h->seg[i % kRing] = s;
                    mbar_arrive(smem_addr(&h->seg_full[i % kRing]));
                }
                __syncwarp();
                if (s.n_tok < 0) break;
                if (s.n[0] > 0 || s.n[1] > 0) {
                    // its query rows, once the last S of the unit before is complete
                    if (q_uses > 0 && !wait_all(&h->q_empty, (q_uses - 1) & 1u)) break;
                    ++q_uses;
                    if (lane == 0) {
                        const uint32_t bar = smem_addr(&h->q_full);
                        const uint32_t box = 128u * (uint32_t)(p.group_tokens * G);
                        const int n_grp = (kGroups == 2 && s.n[1] > 0) ? 2 : 1;
                        mbar_expect_tx(bar, box * 2u * (uint32_t)(kHalves * n_grp));
                        for (int t = 0; t < n_grp * kHalves; ++t)
                            for (int pl = 0; pl < 2; ++pl)
                                tma_box(smem_addr(q_tiles) + t * kQTileBytes + pl * kPlaneBytes, &p.tmap_q,
                                        (kGroups == 2 ? 0 : t * 128) + pl * 64, s.g * G,
                                        (int)s.q_tok + (kGroups == 2 ? t * p.group_tokens : 0), bar);
                        mbar_arrive(bar);
                    }
                    __syncwarp();
                }
            }
        } else if (kQuant && warp == 14) {
            // ------------------------------- raw bytes, quantised -------------------------------
            uint32_t ahead = 0, T = 0;    // slots brought, tiles begun
            bool bad_entry = false, ok = true;
            Seg s = {};
            auto stage_free = [&]() -> bool {
                return ahead < kRawStages || wait_all(&h->raw_empty[ahead % kRawStages], (ahead / kRawStages - 1u) & 1u);
            };
            auto publish = [&](uint32_t word) {
                const uint32_t r = ahead % kRawStages;
                if (lane == 0) h->raw_word[r] = word;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&h->raw_full[r]));
                ++ahead;
            };
            auto bring = [&](const Tile& t, bool v_side, int half, uint32_t word) {
                if (!(ok = stage_free())) return;
                const int bits = v_side ? VBITS : KBITS;
                const uint32_t bar = smem_addr(&h->raw_full[ahead % kRawStages]);
                const uint32_t stage = smem_addr(raws + (ahead % kRawStages) * Memory<KBITS>::kRawBytes);
                const int64_t Hk = p.n_head_kv;
                if (t.run && p.use_tma != 0) {
                    if (lane == 0) {
                        mbar_expect_tx(bar, 128u * 16u * (uint32_t)bits);
                        tma_box(stage, v_side ? &p.tmap_v : &p.tmap_k, half * 16 * bits, s.g, (int)t.base, bar);
                    }
                } else {   // 16-byte pieces of the cells' 128 dims, `bits` a cell
                    const char* rows = static_cast<const char*>(v_side ? p.v : p.k);
#pragma unroll 1
                    for (int i = lane; i < 128 * bits; i += 32) {
                        const int c = i / bits, piece = i - c * bits;
                        const int64_t cell = cell_of<PLAN>(t, c);
                        if (cell >= 0)
                            cp_async_16_cg(stage + 16 * i, rows + (cell * Hk + s.g) * (D * bits / 8) + half * 16 * bits + 16 * piece);
                    }
                }
                // scales: a cell's four blocks; zeros where there is no cell, so that whatever its
                // codes are it stands for zeros
                const __half* scales = (v_side ? p.v_scale : p.k_scale) + half * 4;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t dst = stage + Memory<KBITS>::kRawBytes - 1024 + 8 * (32 * k + lane);
                    const int64_t cell = !PLAN ? t.base + t.e[k] : t.e[k];
                    if (t.e[k] >= 0)
                        cp_async_8(dst, scales + (cell * Hk + s.g) * (D / 32));
                    else
                        asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(dst), "r"(0u) : "memory");
                }
                cp_async_arrive(bar);
                publish(word);
            };
            for (uint32_t i = 0; ok; ++i) {
                if (!take(i, s)) break;
                const int n_max = s.n[0] > s.n[1] ? s.n[0] : s.n[1];
                const uint32_t unit = (i & 0xffffu) << 8;
                if (n_max == 0) {    // (the turning warps still sign the unit off)
                    if ((ok = stage_free())) publish(unit | 12u);
                    give_back(i);
                    continue;
                }
                Tile tk = read_tile<PLAN>(p, s, 0), tv = tk, next = read_tile<PLAN>(p, s, 1);
#pragma unroll 1
                for (int step = 0; step < 2 * kHalves * n_max && ok; ++step) {
                    bool v_side;
                    int j, half;
                    slot_number<kHalves>(step, n_max, s.n[1] > 0, v_side, j, half);
                    if (!v_side && half == 0) {
                        if (j > 0) {
                            tv = tk;
                            tk = next;
                            next = read_tile<PLAN>(p, s, j + 1);
                        }
                        if (!settle<PLAN>(p, tk)) bad_entry = true;
                        if (PLAN && !(ok = put_mask(tk, T))) break;
                        ++T;
                    }
                    if (v_side && (s.n[1] > 0 || j + 1 == n_max)) tv = tk;
                    const bool cut = v_side && j >= s.first_cut;
                    bring(v_side ? tv : tk, v_side, half,
                          unit | (v_side ? 1u : 0u) | (cut ? 2u | ((uint32_t)(j - s.first_cut) << 4) : 0u) |
                              (step + 1 == 2 * kHalves * n_max ? 4u : 0u));
                }
                give_back(i);
            }
            if (ok && stage_free()) publish(kNoMore);
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (__any_sync(0xffffffffu, bad_entry) && lane == 0) atomicOr(p.status, KVATTN_DEVICE_BAD_PLAN_ENTRY);
        } else if (warp == 12) {
            // ------------------------------------- MMA -------------------------------------
            // (every operand is the same in all lanes, and known to be: values from shared memory
            // are broadcast from lane 0)
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t slot0 = smem_addr(slots), q_addr = smem_addr(q_tiles);
            const bool leader = elect_one();
            uint32_t mends = 0;               // a bit per slot: parity of its mended barrier
            uint32_t st = 0, use = 0;         // the next slot, and the parity of its use
            // This warp's own instructions, one after the other, set the pace of everything: a wait
            // is a test by every lane, without a vote (a lane whose wait gave up is noticed by the
            // vote at the end of a tile; until then it goes on, over data that nobody will use).
            // The lanes meet once per slot, before the leader gives its products out: without that
            // one could still test the barrier of a slot (or read its slot_mend) when the products are
            // done and the loader fills it again, and would wait for a phase that is over.  A barrier
            // of p, or of the queries, moves on only after products that come after the next meeting.
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = wait_bar(smem_addr(bar), parity, abort_flag, p.wait_limit_ns) && ok;
            };
            auto wait_slot = [&](bool check) {
                wait(&h->full[st], use);
                if (check && h->slot_mend[st] != 0u) {
                    wait(&h->mended[st], (mends >> st) & 1u);
                    mends ^= 1u << st;
                }
                __syncwarp();
            };
            auto next_slot = [&]() {
                ++st;
                if (st == kSlots) {
                    st = 0;
                    use ^= 1u;
                }
            };
            // S (+)= Q K^T over 128 dims: 8 steps of 16, 32 bytes of the swizzled rows each
            auto issue_s = [&](uint32_t d, uint32_t q_tile, uint32_t slot, bool acc) {
                const uint64_t qd = smem_desc(q_tile, 16, 1024), kd = smem_desc(slot0 + slot * kSlotBytes, 16, 1024);
                mma_ss(d, qd, kd, kIdQK, acc ? 1u : 0u);
#pragma unroll
                for (int k = 1; k < 8; ++k) {
                    const uint64_t off = (uint64_t)(((k >> 2) * kPlaneBytes + 32 * (k & 3)) >> 4);
                    mma_ss(d, qd + off, kd + off, kIdQK, 1u);
                }
            };
            // O (+)= P V over 128 cells: 8 steps of 16 cells; A = f16 pairs in TMEM
            auto issue_pv = [&](uint32_t d, uint32_t a, uint32_t slot, bool acc) {
                const uint64_t vd = smem_desc(slot0 + slot * kSlotBytes, kPlaneBytes, 1024);
                mma_ts(d, a, vd, kIdPV, acc ? 1u : 0u);
#pragma unroll
                for (int k = 1; k < 8; ++k) mma_ts(d, a + 8 * k, vd + (uint64_t)((2048 * k) >> 4), kIdPV, 1u);
            };
            uint32_t uses0 = 0, uses1 = 0;    // of the S buffers
            uint32_t q_uses = 0;              // of the query rows
            for (uint32_t i = 0;; ++i) {
                if (!wait_all(&h->seg_full[i % kRing], (i / kRing) & 1u)) break;
                const Seg& s = h->seg[i % kRing];
                const int n_tok = __shfl_sync(0xffffffffu, s.n_tok, 0);
                const int n0 = __shfl_sync(0xffffffffu, s.n[0], 0), n1 = __shfl_sync(0xffffffffu, s.n[1], 0);
                // (the tiles whose slots may be mended: cut ones, and a sequence's last; through a plan any)
                const int whole = (int)clamp64(s.len / kPrefillTile - s.j0, 0, INT_MAX);
                const int mend_from = PLAN || p.use_tma == 0 ? 0 : __shfl_sync(0xffffffffu, min(s.first_cut, whole), 0);
                if (n_tok < 0) break;
                give_back(i);
                const int n_max = n0 > n1 ? n0 : n1;
                if (n_max == 0) continue;
                wait(&h->q_full, q_uses & 1u);
                ++q_uses;
                tc_fence_after();
                if (kGroups == 2 && n1 > 0) {
                    // both row groups, a buffer each: a group's S and P V run under the other's softmax
                    uint32_t vs = 0;          // V of the tile before
#pragma unroll 1
                    for (int j = 0; j <= n_max; ++j) {
                        const uint32_t ks = st;
                        const bool check = !kQuant && j >= mend_from;
                        if (j < n_max) {
                            wait_slot(check);
                            next_slot();
                            tc_fence_after();
                            if (leader && j < n0) {
                                issue_s(tm, q_addr, ks, false);
                                mma_commit(smem_addr(&h->s_full[0]));
                            }
                        }
                        if (j > 0) {
                            if (j - 1 < n1) wait(&h->p_full[1], (uses1 + j - 1) & 1u);
                            tc_fence_after();
                            if (leader) {
                                if (j - 1 < n1) {
                                    issue_pv(tm + kColO + 128, tm + kColS1, vs, j > 1);
                                    if (j == n1) mma_commit(smem_addr(&h->pv_done[1]));
                                }
                                mma_commit(smem_addr(&h->empty[vs]));
                            }
                        }
                        if (!__all_sync(0xffffffffu, ok) || j == n_max) break;
                        if (leader) {
                            if (j < n1) {
                                issue_s(tm + kColS1, q_addr + kQTileBytes, ks, false);
                                mma_commit(smem_addr(&h->s_full[1]));
                            }
                            mma_commit(smem_addr(&h->empty[ks]));
                            if (j + 1 == n_max) mma_commit(smem_addr(&h->q_empty));
                        }
                        vs = st;
                        wait_slot(check);
                        next_slot();
                        if (j < n0) {
                            wait(&h->p_full[0], (uses0 + j) & 1u);
                            tc_fence_after();
                            if (leader) {
                                issue_pv(tm + kColO, tm, vs, j > 0);
                                if (j + 1 == n0) mma_commit(smem_addr(&h->pv_done[0]));
                            }
                        }
                    }
                    uses0 += n0;
                    uses1 += n1;
                } else {
                    // one row group, buffers in turn: S of the next tile runs under this one's softmax
#pragma unroll 1
                    for (int j = -1; j < n_max; ++j) {
                        if (j + 1 < n_max) {
                            const uint32_t buf = (j + 1) & 1;
#pragma unroll 1
                            for (int half = 0; half < kHalves; ++half) {   // of the dims
                                wait_slot(!kQuant && j + 1 >= mend_from);
                                tc_fence_after();
                                if (leader) {
                                    issue_s(tm + kColS1 * buf, q_addr + half * kQTileBytes, st, half > 0);
                                    mma_commit(smem_addr(&h->empty[st]));
                                    if (half + 1 == kHalves) {
                                        mma_commit(smem_addr(&h->s_full[buf]));
                                        if (j + 2 == n_max) mma_commit(smem_addr(&h->q_empty));
                                    }
                                }
                                next_slot();
                            }
                        }
                        if (!__all_sync(0xffffffffu, ok)) break;
                        if (j < 0) continue;
                        const uint32_t buf = j & 1;
                        wait(&h->p_full[buf], ((buf ? uses1 : uses0) + (j >> 1)) & 1u);
#pragma unroll 1
                        for (int half = 0; half < kHalves; ++half) {
                            wait_slot(!kQuant && j >= mend_from);
                            tc_fence_after();
                            if (leader) {
                                issue_pv(tm + kColO + 128 * half, tm + kColS1 * buf, st, j > 0);
                                mma_commit(smem_addr(&h->empty[st]));
                                if (half + 1 == kHalves) mma_commit(smem_addr(&h->pv_done[buf]));
                            }
                            next_slot();
                        }
                    }
                    uses0 += (n_max + 1) >> 1;
                    uses1 += n_max >> 1;
                }
                if (!__all_sync(0xffffffffu, ok)) break;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
        // ------------------------------------ softmax ------------------------------------
        // Warps w and w + 4 share 32 rows: a thread has one row (its TMEM lane) and half of a
        // tile's columns, then half of O's.  They meet in a named barrier once per tile, which
        // also ORs what either saw: a maximum that grew, or a wait that gave up (which both then
        // leave together: a named barrier has no bound of its own).
        const int half = warp >> 2;
        const int row_in = tid & 127;                // TMEM lane
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        auto pair_any = [&](bool x) -> bool { return bar_or(2 + (warp & 3), x); };
        // (scale <= 0: scores are scaled before the maximum is taken)
        const bool pre = !(p.scale_log2 > 0.f);
        const float sc = pre ? 1.f : p.scale_log2;
        const int tok_in = row_in / G, head_in = row_in - tok_in * G;
        uint32_t uses0 = 0, uses1 = 0;               // of the S buffers
        uint32_t done0 = 0, done1 = 0;               // of pv_done: once a piece with a buffer each, else per tile
        uint32_t masks = 0;                          // tiles of the CTA so far
        for (uint32_t i = 0;; ++i) {
            if (pair_any(!wait_all(&h->seg_full[i % kRing], (i / kRing) & 1u))) break;
            const Seg& s = h->seg[i % kRing];        // (kept until it is given back)
            if (s.n_tok < 0) break;
            const int n0 = s.n[0], n1 = s.n[1], n_max = n0 > n1 ? n0 : n1;
            const bool dual = kGroups == 2 && n1 > 0;
            // first cell of the piece that the thread's row of a group does not see, from its first.  A
            // row that is not there sees all, so that no tile is a cut one for its sake (what it
            // computes goes nowhere; letting warps without any row skip theirs slowed the others'
            // code: a prompt of 8192 tokens 421 -> 440 us)
            int rel[2] = {INT_MAX, INT_MAX};
            {
                const int64_t r0 = s.lim0 + tok_in - (int64_t)s.j0 * kPrefillTile;
                if (tok_in < p.group_tokens && tok_in < s.n_tok) rel[0] = (int)clamp64(r0, 0, INT_MAX);
                if (tok_in < p.group_tokens && tok_in + p.group_tokens < s.n_tok)
                    rel[1] = (int)clamp64(r0 + p.group_tokens, 0, INT_MAX);
            }
            // a row's running maximum (of both halves) and sum (of this one), per group
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            uint32_t use0 = uses0, use1 = uses1;
            bool lost = false;                       // a wait gave up
            int masked = -1;                         // the tile whose mask is there,
            bool holes = false;                      // and whether it has holes
#pragma unroll 1
            for (int x = 0; x < (dual ? 2 * n_max : n_max); ++x) {
                const int g = dual ? x & 1 : 0, j = dual ? x >> 1 : x;
                const int buf = dual ? g : j & 1;
                if (j < (g ? n1 : n0)) {
                    const uint32_t par = (buf ? use1 : use0) & 1u;
                    if (buf)
                        ++use1;
                    else
                        ++use0;
                    const uint32_t t_s = tmem + lane_base + (buf ? kColS1 : 0u);
                    if (PLAN && j != masked) {   // (once for both groups, and while S is on its way)
                        const uint32_t t = masks + j;
                        masked = j;
                        lost = lost || !wait_all(&h->mask_full[t % kMasks], (t / kMasks) & 1u);
                        holes = h->holes[t % kMasks] != 0u;
                    }
                    // (without a vote: the barrier below ORs what a lane lost)
                    lost = lost || !wait_bar(smem_addr(&h->s_full[buf]), par, abort_flag, p.wait_limit_ns);
                    __syncwarp();
                    tc_fence_after();
                    const int left = (g ? rel[1] : rel[0]) - j * kPrefillTile - 64 * half;
                    if (pre || !__all_sync(0xffffffffu, left >= 64)) {
                        // (the rare tiles: scaled, masked and put back by a loop of its own, which keeps
                        // the code of the others short)
#pragma unroll 1
                        for (int c0 = 0; c0 < 64; c0 += 32) {
                            uint32_t v[32];
                            tmem_ld32(t_s + 64 * half + c0, v);
                            tc_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                const float f = __uint_as_float(v[c]);
                                v[c] = c0 + c >= left ? 0xff800000u : __float_as_uint(pre ? f * p.scale_log2 : f);
                            }
                            tmem_st32(t_s + 64 * half + c0, v);
                        }
                        tc_wait_st();
                    }
                    uint32_t sv[64];
                    tmem_ld32(t_s + 64 * half, sv);
                    tmem_ld32(t_s + 64 * half + 32, sv + 32);
                    tc_wait_ld();
                    if (PLAN) {
                        const uint32_t t = masks + j;
                        if (holes) {
                            // the minimum of the score and -inf for a hole, +inf for a cell: a NaN that
                            // stands in a hole goes too (a bit for each cell and a select took longer)
                            const float4* bias = reinterpret_cast<const float4*>(h->bias[t % kMasks]) + 16 * half;
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const float4 f = bias[c];
                                sv[4 * c] = __float_as_uint(fminf(__uint_as_float(sv[4 * c]), f.x));
                                sv[4 * c + 1] = __float_as_uint(fminf(__uint_as_float(sv[4 * c + 1]), f.y));
                                sv[4 * c + 2] = __float_as_uint(fminf(__uint_as_float(sv[4 * c + 2]), f.z));
                                sv[4 * c + 3] = __float_as_uint(fminf(__uint_as_float(sv[4 * c + 3]), f.w));
                            }
                        }
                    }

                    float mx[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) mx[k] = fmaxf(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1]));
#pragma unroll
                    for (int c = 8; c < 64; c += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mx[k] = max3(mx[k], __uint_as_float(sv[c + 2 * k]), __uint_as_float(sv[c + 2 * k + 1]));
                    const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                    float m_run = g ? m[1] : m[0];
                    // (both have read their scores: p of one is written over the other's)
                    tc_fence_before();
                    const bool turn = pair_any(tmax > m_run + kSlack || lost);
                    tc_fence_after();
                    if (turn) {
                        h->meet[half][row_in] = lost ? INFINITY : tmax;
                        const bool gone = pair_any(lost);          // (and both values are there)
                        if (gone) {
                            lost = true;
                            break;
                        }
                        const float both = fmaxf(tmax, h->meet[half ^ 1][row_in]);
                        pair_any(false);                           // (they are read)
                        float alpha = 1.f;
                        if (both > m_run + kSlack) {
                            alpha = fast_exp2(m_run - both);       // (0 from a maximum of -inf)
                            m_run = both;
                            if (g) {
                                m[1] = m_run;
                                l[1] *= alpha;
                            } else {
                                m[0] = m_run;
                                l[0] *= alpha;
                            }
                        }
                        // rows whose maximum moved rescale their O (each thread its half of it) once the
                        // last P V is complete.  (With buffers in turn S of this tile came after the P V
                        // before that, so the barrier is in its phase or the next.)
                        if (j > 0) {
                            // (with a buffer each, S of this tile came after it)
                            if (!dual) lost = !wait_all(&h->pv_done[buf ^ 1], ((buf ? done0 : done1) + ((j - 1) >> 1)) & 1u);
                            tc_fence_after();
                            const uint32_t t_o = tmem + lane_base + kColO + (uint32_t)(128 * g + D / 2 * half);
#pragma unroll 1
                            for (int c0 = 0; c0 < D / 2; c0 += 32) {
                                uint32_t ov[32];
                                tmem_ld32(t_o + c0, ov);
                                tc_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
                                tmem_st32(t_o + c0, ov);
                            }
                        }
                    }
                    const float nm = (m_run == -INFINITY) ? 0.f : kLift - m_run;
                    uint64_t sum[2] = {0ull, 0ull};
                    const uint64_t sc2 = pack2(sc, sc), nm2 = pack2(nm, nm);
#pragma unroll
                    for (int c0 = 0; c0 < 64; c0 += 32) {
                        uint32_t pw[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float a, b;
                            unpack2(fma2(pack2(__uint_as_float(sv[c0 + c]), __uint_as_float(sv[c0 + c + 1])), sc2, nm2), a, b);
                            a = fast_exp2(a);
                            b = fast_exp2(b);
                            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(a, b));
                            pw[c >> 1] = pack_half2(a, b);
                        }
                        tmem_st16(t_s + 32 * half + (c0 >> 1), pw);
                    }
                    float s0, s1, s2, s3;
                    unpack2(sum[0], s0, s1);
                    unpack2(sum[1], s2, s3);
                    if (g)
                        l[1] += (s0 + s1) + (s2 + s3);
                    else
                        l[0] += (s0 + s1) + (s2 + s3);
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&h->p_full[buf]));
                }
                if (PLAN && g == (dual ? 1 : 0)) {   // every warp, for every tile
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&h->mask_empty[(masks + j) % kMasks]));
                }
            }
            masks += n_max;
            if (pair_any(lost)) break;
            // ---- the piece's result: a thread has its row and half of the columns of each group ----
#pragma unroll 1
            for (int g = 0; g < kGroups && g * p.group_tokens < s.n_tok; ++g) {
                const int n_tiles = g ? n1 : n0;
                const int tok = g * p.group_tokens + tok_in;
                const bool row_ok = tok_in < p.group_tokens && tok < s.n_tok;
                const float m_run = g ? m[1] : m[0];
                float l_run = g ? l[1] : l[0];
                bool fix = false;   // V that was kept apart: cells that this row sees
                if (n_tiles > 0) {
                    const int buf = dual ? g : (n_tiles - 1) & 1;
                    const uint32_t uses = dual ? 0u : (uint32_t)(n_tiles - 1) >> 1;   // before the last in this piece
                    lost = lost || !wait_all(&h->pv_done[buf], ((buf ? done1 : done0) + uses) & 1u);
                    lost = lost || !wait_all(&h->load_done[i % kRing], (i / kRing) & 1u);
                    tc_fence_after();
                    uint32_t any = 0;
#pragma unroll
                    for (int t = 0; t < kCutTiles; ++t) {
                        const uint4 bad = *reinterpret_cast<const uint4*>(h->bad_cells[i % kRing][t]);
                        any |= bad.x | bad.y | bad.z | bad.w;
                    }
                    fix = any != 0u && row_ok;
                }
                h->meet[half][row_in] = l_run;
                lost = pair_any(lost);
                if (lost) break;
                l_run += h->meet[half ^ 1][row_in];
                pair_any(false);                                   // (they are read)
                const bool none = n_tiles == 0 || l_run == 0.f;    // (a NaN sum stays)
                const float inv = none ? 0.f : 1.f / l_run;
                const int64_t out_row = (s.q_tok + tok) * p.n_head + s.g * G + head_in;
                const int64_t part_row = ((int64_t)s.part * kGroups + g) * 128 + row_in;
                constexpr int kCols = D / 2;
                const int d0 = kCols * half;
                const uint32_t t_o = tmem + lane_base + kColO + (uint32_t)(128 * g + d0);
                // (a thread stores its part of a row in whole 32-byte sectors: turning rows among lanes
                // first, to store whole lines, took longer)
                char* to = s.part >= 0 ? reinterpret_cast<char*>(p.part_o + part_row * D + d0)
                                       : reinterpret_cast<char*>(p.out + out_row * D + d0);
                const bool sectors = p.out_sectors != 0;
#pragma unroll 1
                for (int c0 = 0; c0 < kCols; c0 += 32) {
                    if (s.part >= 0 && n_tiles == 0) break;      // (its lse says that nothing is there)
                    uint32_t ov[32];
                    if (n_tiles > 0) {
                        tmem_ld32(t_o + c0, ov);
                        tc_wait_ld();
                    } else {   // (written on both ways: else its registers live through the tiles' loop)
#pragma unroll
                        for (int k = 0; k < 32; ++k) ov[k] = 0u;
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        ov[k] = none ? 0u : __float_as_uint(__uint_as_float(ov[k]) * inv);
                    if (fix) {
#pragma unroll 1
                        for (int t = 0; t < kCutTiles; ++t)
#pragma unroll 1
                            for (int c = 0; c < 128; ++c) {
                                if (!((h->bad_cells[i % kRing][t][c >> 5] >> (c & 31)) & 1u)) continue;
                                const int64_t at = (int64_t)(s.j0 + s.first_cut + t) * kPrefillTile + c;
                                if (at >= s.lim0 + tok) continue;
                                const int64_t cell = PLAN ? (int64_t)__ldg(p.plan + (int64_t)s.seq * p.plan_stride + at)
                                                                       : s.cell0 + at;
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const int d = d0 + c0 + k;
                                    __half x;
                                    if (VBITS == 16) {
                                        x = static_cast<const __half*>(p.v)[cell * p.v_stride + (int64_t)s.g * D + d];
                                    } else {  // (only the scale is not finite)
                                        x = p.v_scale[(cell * p.n_head_kv + s.g) * (D / 32) + d / 32];
                                        if (__hisinf(x)) x = __ushort_as_half(0x7fffu);  // (as the loader has it)
                                    }
                                    if (__hisinf(x) || __hisnan(x)) ov[k] = __float_as_uint(__uint_as_float(ov[k]) + __half2float(x));
                                }
                            }
                    }
                    if (!row_ok) continue;
                    if (s.part >= 0) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) st_sector(to + 4 * c0 + 32 * k, ov + 8 * k, true);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) ov[k] = pack_half2(__uint_as_float(ov[2 * k]), __uint_as_float(ov[2 * k + 1]));
                        st_sector(to + 2 * c0, ov, sectors);
                        st_sector(to + 2 * c0 + 32, ov + 8, sectors);
                    }
                }
                if (row_ok && half == 0) {
                    const float v = none ? -INFINITY : (m_run - kLift + fast_log2(l_run)) * kLn2;
                    if (s.part >= 0)
                        p.part_lse[part_row] = v;
                    else if (p.lse != nullptr)
                        p.lse[out_row] = v;
                }
            }
            if (lost) break;
            uses0 = use0;
            uses1 = use1;
            done0 += dual ? (n0 > 0 ? 1 : 0) : (n_max + 1) >> 1;
            done1 += dual ? 1 : n_max >> 1;
            tc_fence_before();   // (O is read: the next piece's first P, which follows, lets it be written)
            give_back(i);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag != 0) {
        if (threadIdx.x == 0) atomicOr(p.status, KVATTN_DEVICE_WAIT_TIMEOUT);
        // an MMA or copy issued before the wait that gave up finishes long before this
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < p.wait_limit_ns / 8) {
        }
    }
    tc_fence_after();
    if (warp == 12)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Joins the partials of the units that were cut: weights exp(lse_p - max lse).  blockIdx.x is the
// CTA that began the unit (and noted it in cuts); its parts are one of each share that the unit's
// line meets and that holds tiles of it.  blockIdx.y and the warps take its rows, the lanes a
// row's dims.
constexpr int kMergeWarps = 4;
constexpr int kMaxCtas = 1024;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prefill_merge_kernel(const __grid_constant__ PrefillParams p, int n_ctas) {
    constexpr int kGroups = Geometry<D>::kGroups, kBatch = 512 / D;
    __shared__ int slot[kMaxCtas];   // part i's partial slot, -1: it holds no tile
    pdl_wait();
    const PrefillCut cut = p.cuts[blockIdx.x];
    if (cut.n_parts == 0) return;
    const int lane = threadIdx.x & 31;
    Shares sh;
    sh.set(total_of(p), (uint32_t)n_ctas);
    // `whole`: one share holds all its tiles and has written the result itself
    bool whole = false;
    for (int i = threadIdx.x; i < cut.n_parts; i += 32 * kMergeWarps) {
        const uint32_t cta = blockIdx.x + (uint32_t)i;
        const uint32_t x0 = sh.of(cta), a = max(x0, cut.start), b = min(sh.of(cta + 1u), cut.end);
        const int32_t each = tile_length(p, cut.n_tok);
        const int32_t first = tile_at(a - cut.start, cut.end - cut.start, cut.tiles, each);
        const int32_t last = tile_at(b - cut.start, cut.end - cut.start, cut.tiles, each);
        whole = whole || (first == 0 && last == cut.tiles);
        slot[i] = first == last ? -1 : 2 * (int)cta + (x0 > cut.start ? 0 : 1);
    }
    if (__syncthreads_or(whole)) return;
    const int parts = cut.n_parts, G = p.group;
    const int step = kMergeWarps * gridDim.y;
    for (int row = (int)blockIdx.y * kMergeWarps + (threadIdx.x >> 5); row < 128 * kGroups; row += step) {
        const int grp = row >> 7, in = row & 127;
        const int tok_in = in / G, tok = grp * p.group_tokens + tok_in;
        if (tok_in >= p.group_tokens || tok >= cut.n_tok) continue;
        // maximum over the parts, a lane each
        auto lse_of = [&](int i) -> float {
            const int sl = i < parts ? slot[i] : -1;
            return sl < 0 ? -INFINITY : p.part_lse[(int64_t)sl * kGroups * 128 + row];
        };
        float m = -INFINITY;
        for (int i = lane; i < parts; i += 32) {
            const float v = lse_of(i);
            m = v > m || v != v ? v : m;  // (a NaN stays)
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float v = __shfl_xor_sync(0xffffffffu, m, o);
            m = v > m || v != v ? v : m;
        }
        float acc[D / 32] = {};
        float sum = 0.f;
        if (m != -INFINITY) {
            for (int i0 = 0; i0 < parts; i0 += 32) {
                // (a part without a cell that the row sees has weight 0 and an O that was not written)
                const float v = lse_of(i0 + lane);
                const float w = v == -INFINITY ? 0.f : exp2f((v - m) * 1.4426950408889634f);
                sum += w;
                uint32_t left = __ballot_sync(0xffffffffu, v != -INFINITY);
                while (left != 0u) {   // the rows of kBatch parts on their way at once
                    float4 f[kBatch][D / 128];
                    float wk[kBatch];
                    int at[kBatch];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {   // (past the last one: weight 0, nothing loaded)
                        const int i = left != 0u ? __ffs(left) - 1 : 0;
                        wk[b] = __shfl_sync(0xffffffffu, w, i);
                        at[b] = left != 0u ? slot[i0 + i] : -1;
                        left &= left - 1u;
                    }
#pragma unroll
                    for (int b = 0; b < kBatch; ++b)
#pragma unroll
                        for (int k = 0; k < D / 128; ++k)
                            f[b][k] = at[b] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                : reinterpret_cast<const float4*>(p.part_o + ((int64_t)at[b] * kGroups * 128 + row) * D)[32 * k + lane];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b)
#pragma unroll
                        for (int k = 0; k < D / 128; ++k) {
                            acc[4 * k] += wk[b] * f[b][k].x;
                            acc[4 * k + 1] += wk[b] * f[b][k].y;
                            acc[4 * k + 2] += wk[b] * f[b][k].z;
                            acc[4 * k + 3] += wk[b] * f[b][k].w;
                        }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        const float inv = m == -INFINITY ? 0.f : 1.f / sum;
        const int64_t out_row = (cut.q_tok + tok) * p.n_head + cut.g * G + (in - tok_in * G);
        uint2* d = reinterpret_cast<uint2*>(p.out + out_row * D);
#pragma unroll
        for (int k = 0; k < D / 128; ++k)
            d[32 * k + lane] = make_uint2(pack_half2(acc[4 * k] * inv, acc[4 * k + 1] * inv),
                                          pack_half2(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
        if (lane == 0 && p.lse != nullptr) p.lse[out_row] = m == -INFINITY ? -INFINITY : m + logf(sum);
    }
}

template <int D, bool PLAN>
const void* kernel_of(int kv_type) {
    switch (kv_type) {
    case KVATTN_KV_F16: return (const void*)prefill_kernel<D, 16, 16, PLAN>;
    case KVATTN_KV_Q8_0: return (const void*)prefill_kernel<D, 8, 8, PLAN>;
    case KVATTN_KV_Q8_0_Q4_0: return (const void*)prefill_kernel<D, 8, 4, PLAN>;
    default: return (const void*)prefill_kernel<D, 4, 4, PLAN>;
    }
}
const void* kernel_of(int kv_type, int head_dim, bool plan) {
    if (head_dim == 128) return plan ? kernel_of<128, true>(kv_type) : kernel_of<128, false>(kv_type);
    return plan ? kernel_of<256, true>(kv_type) : kernel_of<256, false>(kv_type);
}
int smem_of(int kv_type) {
    return kv_type == KVATTN_KV_F16 ? Memory<16>::kBytes : (kv_type == KVATTN_KV_Q4_0 ? Memory<4>::kBytes : Memory<8>::kBytes);
}

// Per device and kernel, once: its shared memory.
cudaError_t prefill_setup(int kv_type, int head_dim, bool plan) {
    static std::mutex mu;
    static bool done[64][4][2][2];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    bool& d = done[dev & 63][kv_type][head_dim == 256][plan];
    if (!d) {
        e = cudaFuncSetAttribute(kernel_of(kv_type, head_dim, plan), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 smem_of(kv_type));
        d = e == cudaSuccess;
    }
    return e;
}

cudaError_t launch(const void* f, dim3 grid, unsigned threads, size_t smem, void** args, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, f, args);
}

}  // namespace

cudaError_t launch_prefill(const PrefillParams& p, int kv_type, int head_dim, int n_ctas, cudaStream_t stream, bool pdl) {
    cudaError_t e = prefill_setup(kv_type, head_dim, p.plan != nullptr);
    if (e != cudaSuccess) return e;
    void* args[] = {const_cast<PrefillParams*>(&p), &n_ctas};
    e = launch(kernel_of(kv_type, head_dim, p.plan != nullptr), dim3((unsigned)n_ctas), kThreads, (size_t)smem_of(kv_type),
               args, stream, pdl);
    if (e != cudaSuccess || !p.shares || n_ctas < 2) return e;
    if (n_ctas > kMaxCtas) return cudaErrorInvalidValue;
    // two rows a warp (one at head_dim 256), so that a merge of a few units fills the device
    return launch(head_dim == 128 ? (const void*)prefill_merge_kernel<128> : (const void*)prefill_merge_kernel<256>,
                  dim3((unsigned)n_ctas, 32), 32 * kMergeWarps, 0, args, stream, pdl);
}

}  // namespace kvattn
