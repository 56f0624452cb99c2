// Causal attention of many query tokens per sequence on the fifth-generation tensor cores:
// whole packed prompts over their own K and V, and chunks of new tokens over a cache that
// already holds them (f16, Q8_0, Q8_0 + Q4_0, Q4_0; contiguous or through a cell plan).
//
// For each KV head the G x n_q query rows of a sequence are packed flat (row = token x G +
// query head), so that every row of a work unit reads the same K and V.  Row r sees the cells
// below lim(r) = L - n_q + 1 + r / G.  A unit is a block of rows (256 at head_dim 128, 128 at
// 256), a KV head and a range of 128-cell tiles (all of them, or one of n_split parts):
//
//     S = Q K^T,  x = scale S (masked: -inf),  m = max x,  p = exp(x - m),
//     l = sum p,  O = sum p V,  out = O / l,  lse = m + ln l,
//
// one pass over the cells with a running m and l per row (kept in 32 bits; p is rounded to f16
// for the matrix product only, l sums the unrounded p).  Sixteen warps with fixed roles:
//
//  * softmax (warps 0-3 and 4-7, 128 threads each): thread t holds row t, which is TMEM lane
//    t: a row's maximum and sum need no exchange between threads.  At head_dim 128 each group
//    has its own 128 rows; at 256 the first group has the unit's 128 rows and the second is
//    idle.  The thread reads its row of S from tensor memory, masks, and writes p over it as
//    f16 pairs.  p is scaled by 2^7 (it cancels in O / l): with the lazily moved maximum below
//    p stays under 2^15, and p of 2^-21 of a row's largest still has all its f16 bits.
//  * loader (warps 8-11): fills a ring of five 32 KB slots, each 128 cells x 128 dims of K or
//    V in two 128-byte-swizzled planes.  A tile of f16 cells that are one physical run comes
//    by TMA; other tiles by 16-byte cp.async per row with zeros for missing cells; quantised
//    tiles are read into registers one slot ahead, turned into f16 there and stored.
//  * MMA (warp 12): one elected lane issues tcgen05.mma.  S of one row group is computed while
//    the softmax of the other runs (head_dim 128: two S and two O accumulators fill the 512
//    TMEM columns), or S of the next tile while the softmax of this one runs (256: two S and
//    a 256-column O).
//
// The running maximum moves only when it grows by more than 2^8 (in p), so that O is rescaled
// a few times per row at most; the softmax thread does it in tensor memory itself.
//
// Masked places: a score is masked before it is used, so whatever K holds there is dropped.  V
// is multiplied by p = 0 there, and 0 x inf is NaN on the tensor cores, so cells that no row
// may see are zeros in shared memory (a tile with any is not loaded by TMA), and in a tile that
// only some rows see, elements of V that are not finite become zeros too and are added at the
// end to the rows that do see the cell (any p > 0 times an infinity is that infinity).
//
// Every wait is bounded, as in the decode kernels; a wait that gives up sets a flag that the
// others see, and KVATTN_DEVICE_WAIT_TIMEOUT in the workspace.
#include <climits>
#include <cmath>
#include <mutex>

#include "prompt.cuh"

namespace kvattn {

namespace {

constexpr int kThreads = 512;
constexpr int kSlots = 5;
constexpr int kPlaneBytes = 128 * 128;        // 128 cells (or rows) x 128 bytes
constexpr int kSlotBytes = 2 * kPlaneBytes;   // 128 cells x 128 dims of f16
constexpr int kQTileBytes = 2 * kPlaneBytes;  // 128 rows x 128 dims of f16
constexpr int kHeaderBytes = 3072;
constexpr int kRing = 4;                      // tiles whose masks are kept
constexpr int kSmemBytes = 2 * kQTileBytes + kSlots * kSlotBytes + kHeaderBytes;  // all of the 227 KB
constexpr float kSlack = 8.f;                 // lazy maximum
constexpr float kLift = 7.f;                  // p is scaled by 2^kLift
constexpr float kLn2 = 0.69314718055994530942f;

struct Header {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full;       // the unit's query rows are in shared memory
    uint64_t s_full[2];    // S is in TMEM (of row group t, or of buffer b)
    uint64_t p_full[2];    // p is
    uint64_t pv_done;      // head_dim 256: P V of a tile is complete
    uint64_t o_full[2];    // a row group's last P V is complete
    uint64_t mask_full[kRing];  // through a plan: a tile's bias and holes are written
    uint64_t load_done;    // every slot is filled, bad_cells is complete
    uint32_t tmem;
    int abort_flag;
    uint32_t bad_cells[4][4];              // cells of the last (partly seen) tiles with non-finite V
    float bias[kRing][kPrefillTile];       // through a plan: 0, or -inf for a hole
    uint32_t holes[kRing];                 // whether the tile has any
};
static_assert(sizeof(Header) <= kHeaderBytes, "header");

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
// arrives on bar when this thread's cp.async so far are complete (adds itself to the phase's
// pending arrivals first: the phase must be held open by an arrival that comes later)
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A work unit, the same in every thread of the CTA.
struct Unit {
    int64_t q0;        // first token of the sequence
    int64_t cell0;     // its first cell (no plan)
    int64_t len;       // its cells
    int64_t lim0;      // lim of row r = lim0 + r / G
    int64_t rows;      // its rows for a KV head
    int64_t row0;      // first row of the unit
    int seq, g, split;
    int j0;            // first tile of the split
    int n[2];          // tiles of the row groups (from j0)
    int n_max;
    bool any;
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Finds block number `b` of the sequences' row blocks counted from the last sequence's last
// block (the longest rows of a prompt come first), a warp at a time.
template <int D>
__device__ __forceinline__ Unit find_unit(const PrefillParams& p) {
    constexpr int kRows = D == 128 ? 256 : 128, kGroups = D == 128 ? 2 : 1;
    Unit u = {};
    const int lane = threadIdx.x & 31;
    uint32_t id = blockIdx.x, b;
    if (p.n_split == 1) {  // KV heads side by side: the longest units first
        u.g = (int)(id % (uint32_t)p.n_head_kv);
        b = id / (uint32_t)p.n_head_kv;
    } else {               // the row blocks that read the same cells side by side
        b = id % (uint32_t)p.n_blocks;
        id /= (uint32_t)p.n_blocks;
        u.g = (int)(id % (uint32_t)p.n_head_kv);
        u.split = (int)(id / (uint32_t)p.n_head_kv);
    }
    const int G = p.group;
    uint32_t seen = 0;
    u.seq = -1;
    for (int top = p.n_seq; top > 0; top -= 32) {
        const int s = top - 1 - lane;
        int64_t a = 0, e = 0;
        if (s >= 0) {
            a = clamp64(__ldg(p.offsets + s), 0, p.n_tok);
            e = clamp64(__ldg(p.offsets + s + 1), a, p.n_tok);
        }
        const uint32_t blocks = (uint32_t)(((e - a) * G + kRows - 1) / kRows);
        uint32_t sum = blocks;  // inclusive over the lanes so far
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, b < seen + sum);
        if (hit != 0u) {
            const int l = __ffs(hit) - 1;
            u.seq = top - 1 - l;
            u.q0 = __shfl_sync(0xffffffffu, a, l);
            const int64_t end = __shfl_sync(0xffffffffu, e, l);
            const uint32_t n_blocks = __shfl_sync(0xffffffffu, blocks, l);
            const uint32_t before = seen + __shfl_sync(0xffffffffu, sum, l) - n_blocks;
            u.rows = (end - u.q0) * G;
            u.row0 = (int64_t)(n_blocks - 1 - (b - before)) * kRows;
            break;
        }
        seen += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (u.seq < 0) return u;
    const int64_t nq = u.rows / G;
    if (p.seq_lens != nullptr) {
        const int64_t cap = p.plan != nullptr ? p.plan_stride : p.n_cells;
        int64_t L = clamp64(__ldg(p.seq_lens + u.seq), 0, p.max_len);
        u.len = L < cap ? L : cap;
        u.cell0 = (int64_t)u.seq * p.n_cells;
    } else {
        u.len = nq;
        u.cell0 = u.q0;
    }
    u.lim0 = u.len - nq + 1;
    u.j0 = u.split * p.split_tiles;
#pragma unroll
    for (int t = 0; t < kGroups; ++t) {
        const int64_t first = u.row0 + 128 * t;
        const int64_t last = (first + 127 < u.rows ? first + 127 : u.rows - 1);
        int64_t tiles = 0;
        if (first < u.rows) {
            const int64_t lim = u.lim0 + last / G;  // (at most len)
            tiles = lim > 0 ? (lim + kPrefillTile - 1) / kPrefillTile : 0;
        }
        if (p.n_split > 1 && tiles > u.j0 + p.split_tiles) tiles = u.j0 + p.split_tiles;
        u.n[t] = tiles > u.j0 ? (int)(tiles - u.j0) : 0;
    }
    if (kGroups == 1) u.n[1] = 0;
    u.n_max = u.n[0] > u.n[1] ? u.n[0] : u.n[1];
    u.any = true;
    return u;
}

// ------------------------------- quantised rows in registers -------------------------------

// The raw bytes of a thread's part of a slot.  8-bit: 8 cells' 16-byte pieces (half a block
// each); 4-bit: 4 cells' 16-byte blocks.  scale: the halves of their blocks, two per word.
struct Raw {
    uint4 w[8];
    uint32_t d[4];
};

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Stored value = scale x code, rounded once to half: the type of an f16 cache (2^-11 of the
// value, where the 8-bit code itself is off by up to 2^-8 of the block's largest).  Scales
// above 515 could pass the largest half; those products are kept at it (as cache_read does).
__device__ __forceinline__ uint32_t dequant(uint32_t codes, __half2 d, bool big) {
    __half2 r = __hmul2_rn(as_h2(codes), d);
    if (big) {
        const __half2 top = __halves2half2(__ushort_as_half(0x7bffu), __ushort_as_half(0x7bffu));
        r = __hmax2_nan(__hmin2_nan(r, top), __hneg2(top));
    }
    return as_u32(r);
}
__device__ __forceinline__ bool big_scale(uint32_t d) { return (d & 0x7fffu) > 0x6006u; }  // 515
// a scale that is not finite makes its whole block NaN
__device__ __forceinline__ __half2 scale2(uint32_t d) {
    if ((d & 0x7c00u) == 0x7c00u) d = 0x7fffu;
    return as_h2(d | (d << 16));
}
__device__ __forceinline__ uint32_t nib2(uint32_t n) {
    return as_u32(__hsub2(as_h2(n | 0x64006400u), as_h2(0x64086408u)));
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

// ------------------------------------- the kernel -------------------------------------

template <int D, int KBITS, int VBITS>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillParams p) {
    constexpr int kGroups = D == 128 ? 2 : 1;   // row groups of 128
    constexpr int kHalves = D / 128;            // slots per tile of K or V
    constexpr bool kQuant = KBITS != 16;
    constexpr uint32_t kColS1 = 128, kColO = 256;
    // the swizzled planes want a 1024-byte aligned base; with no static shared memory the window
    // starts on one, and nothing is left to align it with
    extern __shared__ __align__(1024) unsigned char q_tiles[];
    unsigned char* slots = q_tiles + 2 * kQTileBytes;
    Header* h = reinterpret_cast<Header*>(slots + kSlots * kSlotBytes);
    volatile int* abort_flag = &h->abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((smem_addr(q_tiles) & 1023u) != 0u) {
        if (tid == 0) atomicOr(p.status, KVATTN_DEVICE_WAIT_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_addr(&h->full[i]), 4);   // a lane of each loader warp (and its copies)
            mbar_init(smem_addr(&h->empty[i]), 1);  // the MMA lane's commit
        }
        mbar_init(smem_addr(&h->q_full), 128 * kGroups);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&h->s_full[i]), 1);
            mbar_init(smem_addr(&h->p_full[i]), 128);
            mbar_init(smem_addr(&h->o_full[i]), 1);
        }
        mbar_init(smem_addr(&h->pv_done), 1);
        for (int i = 0; i < kRing; ++i) mbar_init(smem_addr(&h->mask_full[i]), 1);
        mbar_init(smem_addr(&h->load_done), 4);
        h->abort_flag = 0;
        for (int i = 0; i < 16; ++i) h->bad_cells[i >> 2][i & 3] = 0u;
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
    const Unit u = find_unit<D>(p);
    const int G = p.group;
    // first tile (of the unit) that some row of it does not see whole: from here V's elements
    // that are not finite are kept apart
    const int64_t lim_first = u.lim0 + u.row0 / G;
    const int64_t first_cut64 = (lim_first > 0 ? lim_first : 0) / kPrefillTile - u.j0;
    const int first_cut = first_cut64 < 0 ? 0 : (first_cut64 > u.n_max ? u.n_max : (int)first_cut64);
    // (at most 256 rows: with G = 1 a unit's limits lie in up to 256 cells, 3 tiles)

    if (warp >= 8 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        // ------------------------------------ loader ------------------------------------
        const int lt = tid - 256;       // 0 .. 127
        const int64_t Hk = p.n_head_kv;
        bool bad_entry = false;
        if (u.any && u.n_max > 0) {
            const int32_t* prow = p.plan != nullptr ? p.plan + (int64_t)u.seq * p.plan_stride : nullptr;
            // plan entries of a tile: lane l holds those of cells l, l + 32, l + 64, l + 96
            struct Tile {
                int32_t e[4];     // physical cells, -1: none
                int64_t base;     // first physical cell when whole
                bool whole;       // 128 cells in one run
            };
            auto read_tile = [&](int j) {
                Tile t;
                const int64_t i0 = (int64_t)(u.j0 + j) * kPrefillTile;
                t.whole = i0 + kPrefillTile <= u.len;
                t.base = u.cell0 + i0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t i = i0 + 32 * k + lane;
                    t.e[k] = -1;
                    if (j < u.n_max && i < u.len) t.e[k] = prow != nullptr ? __ldg(prow + i) : 32 * k + lane;
                }
                return t;
            };
            // checks a plan tile's entries and whether they are one run; writes its holes
            auto settle = [&](Tile& t, int j) {
                if (prow == nullptr) return;
                bool run = t.whole, hole = false;
                const int32_t first = __shfl_sync(0xffffffffu, t.e[0], 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (t.e[k] < -1 || (int64_t)t.e[k] >= p.n_cells) {
                        bad_entry = true;
                        t.e[k] = -1;
                    }
                    run = run && t.e[k] >= 0 && t.e[k] - first == 32 * k + lane;
                    hole = hole || t.e[k] < 0;
                }
                t.whole = __all_sync(0xffffffffu, run);
                t.base = first;
                const bool holes = __any_sync(0xffffffffu, hole);
                if (warp == 8) {
                    const int r = j % kRing;
#pragma unroll
                    for (int k = 0; k < 4; ++k) h->bias[r][32 * k + lane] = t.e[k] < 0 ? -INFINITY : 0.f;
                    if (lane == 0) h->holes[r] = holes ? 1u : 0u;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&h->mask_full[r]));
                }
            };
            // physical cell of the tile's cell c (any lane's), -1: none
            auto cell_of = [&](const Tile& t, int c) -> int64_t {
                if (prow == nullptr) {
                    const int64_t i = (int64_t)c;
                    return i < u.len - (t.base - u.cell0) ? t.base + i : -1;
                }
                int32_t v = __shfl_sync(0xffffffffu, t.e[0], c & 31);
                const int32_t v1 = __shfl_sync(0xffffffffu, t.e[1], c & 31);
                const int32_t v2 = __shfl_sync(0xffffffffu, t.e[2], c & 31);
                const int32_t v3 = __shfl_sync(0xffffffffu, t.e[3], c & 31);
                v = (c & 64) ? ((c & 32) ? v3 : v2) : ((c & 32) ? v1 : v);
                return v;
            };
            // The raw bytes of this thread's part of a slot (bits of the side, half of the dims)
            auto fetch = [&](const Tile& t, bool v_side, int half, Raw& raw) {
                const int bits = v_side ? VBITS : KBITS;
                const char* rows = static_cast<const char*>(v_side ? p.v : p.k);
                const __half* scales = v_side ? p.v_scale : p.k_scale;
                if (bits == 8) {
                    const int piece = lt & 7;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t c = cell_of(t, (lt >> 3) + 16 * i);
                        raw.w[i] = make_uint4(0u, 0u, 0u, 0u);
                        uint32_t d = 0u;
                        if (c >= 0) {
                            const int64_t row = c * Hk + u.g;
                            raw.w[i] = __ldg(reinterpret_cast<const uint4*>(rows + row * D + half * 128 + 16 * piece));
                            d = __ldg(reinterpret_cast<const unsigned short*>(scales) + row * (D / 32) + half * 4 + (piece >> 1));
                        }
                        raw.d[i >> 1] = (i & 1) ? (raw.d[i >> 1] | (d << 16)) : d;
                    }
                } else if (bits == 4) {
                    const int piece = lt & 3;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int64_t c = cell_of(t, (lt >> 2) + 32 * i);
                        raw.w[i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
                        uint32_t d = 0u;
                        if (c >= 0) {
                            const int64_t row = c * Hk + u.g;
                            raw.w[i] = __ldg(reinterpret_cast<const uint4*>(rows + row * (D / 2) + half * 64 + 16 * piece));
                            d = __ldg(reinterpret_cast<const unsigned short*>(scales) + row * (D / 32) + half * 4 + piece);
                        }
                        raw.d[i] = d;
                    }
                }
            };
            // Bits of V that are not finite are dropped from the slot and their cells noted.
            auto note = [&](int j, int c, bool bad) {
                if (bad) atomicOr(&h->bad_cells[(j - first_cut) & 3][c >> 5], 1u << (c & 31));
            };
            auto store_raw = [&](unsigned char* slot, const Raw& raw, bool v_side, bool cut, int j) {
                const int bits = v_side ? VBITS : KBITS;
                if (bits == 8) {
                    const int piece = lt & 7;  // halves 16 piece .. of the row: bytes 32 piece ..
                    unsigned char* plane = slot + (piece >> 2) * kPlaneBytes;
                    const int b = (piece & 3) * 32;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = (lt >> 3) + 16 * i;
                        const uint32_t ds = (raw.d[i >> 1] >> (16 * (i & 1))) & 0xffffu;
                        const __half2 d = scale2(ds);
                        const bool big = big_scale(ds);
                        const uint32_t x[4] = {raw.w[i].x ^ 0x80808080u, raw.w[i].y ^ 0x80808080u,
                                               raw.w[i].z ^ 0x80808080u, raw.w[i].w ^ 0x80808080u};
                        uint32_t o[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            o[2 * k] = dequant(i8x2_lo(x[k]), d, big);
                            o[2 * k + 1] = dequant(i8x2_hi(x[k]), d, big);
                        }
                        if (cut) {
                            bool bad = false;
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = finite2(o[k], bad);
                            note(j, c, bad);
                        }
                        *reinterpret_cast<uint4*>(plane + swz(c, b)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(plane + swz(c, b + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                } else if (bits == 4) {
                    const int piece = lt & 3;  // block `piece`: halves 32 piece .., bytes 64 piece ..
                    unsigned char* plane = slot + (piece >> 1) * kPlaneBytes;
                    const int b = (piece & 1) * 64;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = (lt >> 2) + 32 * i;
                        const uint32_t ds = raw.d[i];
                        const __half2 d = scale2(ds);
                        const bool big = big_scale(ds);
                        const uint32_t x[4] = {raw.w[i].x, raw.w[i].y, raw.w[i].z, raw.w[i].w};
                        uint32_t lo[8], hi[8];  // elements 0-15 and 16-31 of the block
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t a = prmt_b32(x[k], 0u, 0x4140u), e = prmt_b32(x[k], 0u, 0x4342u);
                            lo[2 * k] = dequant(nib2(a & 0x000f000fu), d, big);
                            lo[2 * k + 1] = dequant(nib2(e & 0x000f000fu), d, big);
                            hi[2 * k] = dequant(nib2((a >> 4) & 0x000f000fu), d, big);
                            hi[2 * k + 1] = dequant(nib2((e >> 4) & 0x000f000fu), d, big);
                        }
                        if (cut) {
                            bool bad = false;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                lo[k] = finite2(lo[k], bad);
                                hi[k] = finite2(hi[k], bad);
                            }
                            note(j, c, bad);
                        }
                        *reinterpret_cast<uint4*>(plane + swz(c, b)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        *reinterpret_cast<uint4*>(plane + swz(c, b + 16)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                        *reinterpret_cast<uint4*>(plane + swz(c, b + 32)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(plane + swz(c, b + 48)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                    }
                }
            };
            // f16 rows of a slot by the whole group: 16 lanes a row, one row per 8 cells and warp half
            auto copy_rows = [&](unsigned char* slot, const Tile& t, bool v_side, int half) {
                const int64_t stride = v_side ? p.v_stride : p.k_stride;
                const __half* rows = static_cast<const __half*>(v_side ? p.v : p.k) + (int64_t)u.g * D + half * 128;
                const int b = (lt & 15) * 16;
                const uint32_t plane = smem_addr(slot) + (b >> 7) * kPlaneBytes;
                for (int i = 0; i < 16; ++i) {
                    const int c = (lt >> 4) + 8 * i;
                    const int64_t cell = cell_of(t, c);
                    const uint32_t dst = plane + swz(c, b & 127);
                    if (cell >= 0)
                        cp_async_16_cg(dst, rows + cell * stride + b / 2);
                    else
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0u) : "memory");
                }
            };
            // ... V of a tile that only some rows see whole: through registers
            auto copy_rows_finite = [&](unsigned char* slot, const Tile& t, int half, int j) {
                const __half* rows = static_cast<const __half*>(p.v) + (int64_t)u.g * D + half * 128;
                const int b = (lt & 15) * 16;
                unsigned char* plane = slot + (b >> 7) * kPlaneBytes;
#pragma unroll 1
                for (int i0 = 0; i0 < 16; i0 += 8) {
                    uint4 w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t cell = cell_of(t, (lt >> 4) + 8 * (i0 + i));
                        w[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (cell >= 0) w[i] = __ldg(reinterpret_cast<const uint4*>(rows + cell * p.v_stride + b / 2));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = (lt >> 4) + 8 * (i0 + i);
                        bool bad = false;
                        w[i].x = finite2(w[i].x, bad);
                        w[i].y = finite2(w[i].y, bad);
                        w[i].z = finite2(w[i].z, bad);
                        w[i].w = finite2(w[i].w, bad);
                        note(j, c, bad);
                        *reinterpret_cast<uint4*>(plane + swz(c, b & 127)) = w[i];
                    }
                }
            };

            // The order in which the MMA warp needs the slots: at head_dim 128 K0 V0 K1 V1 ..,
            // at 256 K0 K1 V0 K2 V1 .. (two slots each).
            uint32_t n = 0;  // slots filled
            bool ok = true;
            Raw cur, nxt;
            Tile tk = read_tile(0), tv = tk, tnext = read_tile(1);
            settle(tk, 0);
            tv = tk;
            auto fill = [&](const Tile& t, bool v_side, int half, int j) {
                const int st = (int)(n % kSlots);
                const uint32_t use = n / kSlots;
                if (use > 0) {
                    const bool got = mbar_wait_bounded(smem_addr(&h->empty[st]), (use - 1) & 1u, abort_flag, p.wait_limit_ns);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        return;
                    }
                }
                unsigned char* slot = slots + st * kSlotBytes;
                const uint32_t bar = smem_addr(&h->full[st]);
                const bool cut = v_side && j >= first_cut;
                if (n == 0 && p.stall_tx != 0u && lt == 0) mbar_expect_tx(bar, p.stall_tx);
                if (kQuant) {
                    store_raw(slot, cur, v_side, cut, j);
                    fence_async();
                } else if (cut) {
                    copy_rows_finite(slot, t, half, j);
                    fence_async();
                } else if (t.whole && p.use_tma != 0) {
                    if (lt == 0) {
                        mbar_expect_tx(bar, (uint32_t)kSlotBytes);
                        const CUtensorMap* map = v_side ? &p.tmap_v : &p.tmap_k;
                        tma_box(smem_addr(slot), map, half * 128, u.g, (int)t.base, bar);
                        tma_box(smem_addr(slot) + kPlaneBytes, map, half * 128 + 64, u.g, (int)t.base, bar);
                    }
                } else {
                    copy_rows(slot, t, v_side, half);
                    cp_async_arrive(bar);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
                ++n;
            };
            if (kHalves == 1) {
                if (kQuant) fetch(tk, false, 0, cur);
                for (int j = 0; j < u.n_max && ok; ++j) {
                    if (kQuant) fetch(tk, true, 0, nxt);
                    fill(tk, false, 0, j);
                    if (!ok) break;
                    tv = tk;
                    if (j + 1 < u.n_max) {
                        tk = tnext;
                        settle(tk, j + 1);
                        tnext = read_tile(j + 2);
                    }
                    if (kQuant) {
                        cur = nxt;
                        if (j + 1 < u.n_max) fetch(tk, false, 0, nxt);
                    }
                    fill(tv, true, 0, j);
                    if (kQuant) cur = nxt;
                }
            } else {
                // (K of tile j + 1 before V of tile j; each in two halves)
                if (kQuant) fetch(tk, false, 0, cur);
                for (int j = -1; j < u.n_max && ok; ++j) {
                    const int jk = j + 1;
                    if (jk < u.n_max) {
                        if (jk > 0) {
                            tv = tk;
                            tk = tnext;
                            settle(tk, jk);
                            tnext = read_tile(jk + 1);
                            if (kQuant) fetch(tk, false, 0, cur);
                        }
#pragma unroll 1
                        for (int half = 0; half < 2 && ok; ++half) {
                            if (kQuant && half == 0) fetch(tk, false, 1, nxt);
                            fill(tk, false, half, jk);
                            if (kQuant) cur = nxt;
                        }
                    } else {
                        tv = tk;
                    }
                    if (j >= 0 && ok) {
                        if (kQuant) fetch(tv, true, 0, cur);
#pragma unroll 1
                        for (int half = 0; half < 2 && ok; ++half) {
                            if (kQuant && half == 0) fetch(tv, true, 1, nxt);
                            fill(tv, true, half, j);
                            if (kQuant) cur = nxt;
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&h->load_done));
        if (__any_sync(0xffffffffu, bad_entry) && lane == 0 && warp == 8) atomicOr(p.status, KVATTN_DEVICE_BAD_PLAN_ENTRY);
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 12 && u.any && u.n_max > 0) {
            // ------------------------------------- MMA -------------------------------------
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(bar), parity, abort_flag, p.wait_limit_ns));
            };
            uint32_t n = 0;  // slots consumed
            auto wait_slot = [&](uint32_t s) -> bool {
                if (!wait_all(&h->full[s % kSlots], (s / kSlots) & 1u)) return false;
                fence_async();  // rows that ordinary stores or cp.async wrote
                tc_fence_after();
                return true;
            };
            // S (+)= Q K^T over 128 dims: 8 steps of 16, 32 bytes of the swizzled rows each
            auto issue_s = [&](uint32_t d, uint32_t q_addr, uint32_t slot, bool acc) {
                const uint64_t qd = smem_desc(q_addr, 16, 1024);
                const uint64_t kd = smem_desc(smem_addr(slots + (slot % kSlots) * kSlotBytes), 16, 1024);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t off = (uint64_t)(((k >> 2) * kPlaneBytes + 32 * (k & 3)) >> 4);
                    mma_ss(d, qd + off, kd + off, kIdQK, (acc || k > 0) ? 1u : 0u);
                }
            };
            // O (+)= P V over 128 cells: 8 steps of 16 cells; A = f16 pairs in TMEM
            auto issue_pv = [&](uint32_t d, uint32_t a, uint32_t slot, bool acc) {
                const uint64_t vd = smem_desc(smem_addr(slots + (slot % kSlots) * kSlotBytes), kPlaneBytes, 1024);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_ts(d, a + 8 * k, vd + (uint64_t)((2048 * k) >> 4), kIdPV, (acc || k > 0) ? 1u : 0u);
            };
            const uint32_t q_addr = smem_addr(q_tiles);
            bool ok = wait_all(&h->q_full, 0u);
            tc_fence_after();
            if (kGroups == 2) {
                for (int j = 0; j <= u.n_max && ok; ++j) {
                    const uint32_t ks = n, vs = n + 1, v_last = n - 1;
                    if (j < u.n_max) {
                        if (!(ok = wait_slot(ks))) break;
                        if (j < u.n[0] && elect_one()) {
                            issue_s(tm, q_addr, ks, false);
                            mma_commit(smem_addr(&h->s_full[0]));
                        }
                        __syncwarp();
                    }
                    if (j > 0) {
                        if (j - 1 < u.n[1] && !(ok = wait_all(&h->p_full[1], (j - 1) & 1u))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            if (j - 1 < u.n[1]) {
                                issue_pv(tm + kColO + 128, tm + kColS1, v_last, j > 1);
                                if (j == u.n[1]) mma_commit(smem_addr(&h->o_full[1]));
                            }
                            mma_commit(smem_addr(&h->empty[v_last % kSlots]));
                        }
                        __syncwarp();
                    }
                    if (j == u.n_max) break;
                    if (elect_one()) {
                        if (j < u.n[1]) {
                            issue_s(tm + kColS1, q_addr + kQTileBytes, ks, false);
                            mma_commit(smem_addr(&h->s_full[1]));
                        }
                        mma_commit(smem_addr(&h->empty[ks % kSlots]));
                    }
                    __syncwarp();
                    if (!(ok = wait_slot(vs))) break;
                    if (j < u.n[0]) {
                        if (!(ok = wait_all(&h->p_full[0], j & 1u))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_pv(tm + kColO, tm, vs, j > 0);
                            if (j + 1 == u.n[0]) mma_commit(smem_addr(&h->o_full[0]));
                        }
                        __syncwarp();
                    }
                    n += 2;
                }
            } else {
                // S of a tile into buffer j & 1, its two halves of the dims in turn
                auto issue_tile_s = [&](int j) -> bool {
#pragma unroll 1
                    for (int half = 0; half < 2; ++half, ++n) {
                        if (!wait_slot(n)) return false;
                        if (elect_one()) {
                            issue_s(tm + kColS1 * (j & 1), q_addr + half * kQTileBytes, n, half > 0);
                            mma_commit(smem_addr(&h->empty[n % kSlots]));
                            if (half == 1) mma_commit(smem_addr(&h->s_full[j & 1]));
                        }
                        __syncwarp();
                    }
                    return true;
                };
                ok = ok && issue_tile_s(0);
                for (int j = 0; j < u.n_max && ok; ++j) {
                    if (j + 1 < u.n_max && !(ok = issue_tile_s(j + 1))) break;
                    if (!(ok = wait_all(&h->p_full[j & 1], (j >> 1) & 1u))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int half = 0; half < 2; ++half, ++n) {
                        if (!(ok = wait_slot(n))) break;
                        if (elect_one()) {
                            issue_pv(tm + kColO + 128 * half, tm + kColS1 * (j & 1), n, j > 0);
                            mma_commit(smem_addr(&h->empty[n % kSlots]));
                            if (half == 1) {
                                mma_commit(smem_addr(&h->pv_done));
                                if (j + 1 == u.n_max) mma_commit(smem_addr(&h->o_full[0]));
                            }
                        }
                        __syncwarp();
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ------------------------------------ softmax ------------------------------------
        const int grp = warp >> 2;                   // row group
        const int row_in = tid & 127;                // TMEM lane
        const int64_t row = u.row0 + 128 * grp + row_in;
        if (u.any && grp < kGroups) {
            const bool row_ok = row < u.rows;
            const int64_t tok = row_ok ? row / G : 0;
            const int head = u.g * G + (row_ok ? (int)(row - tok * G) : 0);
            // Q rows in: each warp its 32 rows, 16 lanes a row of 128 dims
            if (u.n_max > 0) {
                const long long my_src = row_ok ? (long long)((u.q0 + tok) * p.q_stride + (int64_t)head * D) : -1ll;
#pragma unroll 1
                for (int half = 0; half < kHalves; ++half) {
                    unsigned char* qt = q_tiles + (kGroups == 2 ? grp : half) * kQTileBytes;
                    const int b = (lane & 15) * 16;
                    const uint32_t plane = smem_addr(qt) + (b >> 7) * kPlaneBytes;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int rl = 2 * i + (lane >> 4);
                        const long long src = __shfl_sync(0xffffffffu, my_src, rl);
                        const uint32_t dst = plane + swz(32 * (warp & 3) + rl, b & 127);
                        if (src >= 0)
                            cp_async_16_cg(dst, p.q + src + half * 128 + b / 2);
                        else
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0u) : "memory");
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_async();
                mbar_arrive(smem_addr(&h->q_full));
            }
            const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t t_o = tmem + lane_base + kColO + (kGroups == 2 ? 128u * grp : 0u);
            const int n_tiles = u.n[grp];
            // first cell of the split that this row does not see, from the split's first
            const int64_t rel0 = row_ok ? u.lim0 + tok - (int64_t)u.j0 * kPrefillTile : 0;
            float m_run = -INFINITY, l_run = 0.f;
            bool ok = true;
            // (scale <= 0: scores are scaled before the maximum is taken)
            const bool pre = !(p.scale_log2 > 0.f);
            const float sc = pre ? 1.f : p.scale_log2;
            for (int j = 0; j < n_tiles; ++j) {
                const int buf = kGroups == 2 ? grp : (j & 1);
                const uint32_t par = kGroups == 2 ? (j & 1u) : ((j >> 1) & 1u);
                const uint32_t t_s = tmem + lane_base + kColS1 * buf;
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&h->s_full[buf]), par, abort_flag, p.wait_limit_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t sv[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) tmem_ld32(t_s + c, sv + c);
                const int64_t rel = rel0 - (int64_t)j * kPrefillTile;
                tc_wait_ld();
                if (pre) {
                    const uint64_t f = pack2(p.scale_log2, p.scale_log2);
#pragma unroll
                    for (int c = 0; c < 128; c += 2) {
                        float a, b;
                        unpack2(mul2(pack2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), f), a, b);
                        sv[c] = __float_as_uint(a);
                        sv[c + 1] = __float_as_uint(b);
                    }
                }
                if (!__all_sync(0xffffffffu, rel >= kPrefillTile)) {
                    const int lim = rel < 0 ? 0 : (rel > 128 ? 128 : (int)rel);
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c >= lim) sv[c] = 0xff800000u;
                }
                bool holes = false;
                if (p.plan != nullptr) {
                    // (the loader's write, ordered by a barrier of its own; the tile's V slot is
                    // released after this thread's P, and the ring is deeper than the slots reach)
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&h->mask_full[j % kRing]), (j / kRing) & 1u,
                                                                   abort_flag, p.wait_limit_ns))) {
                        ok = false;
                        break;
                    }
                    holes = h->holes[j % kRing] != 0u;
                }
                if (holes) {
                    const float4* bias = reinterpret_cast<const float4*>(h->bias[j % kRing]);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float4 f = bias[c];
                        sv[4 * c] = __float_as_uint(__uint_as_float(sv[4 * c]) + f.x);
                        sv[4 * c + 1] = __float_as_uint(__uint_as_float(sv[4 * c + 1]) + f.y);
                        sv[4 * c + 2] = __float_as_uint(__uint_as_float(sv[4 * c + 2]) + f.z);
                        sv[4 * c + 3] = __float_as_uint(__uint_as_float(sv[4 * c + 3]) + f.w);
                    }
                }
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) mx[k] = fmaxf(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1]));
#pragma unroll
                for (int c = 8; c < 128; c += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = max3(mx[k], __uint_as_float(sv[c + 2 * k]), __uint_as_float(sv[c + 2 * k + 1]));
                const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                const bool grow = tmax > m_run + kSlack;
                if (__any_sync(0xffffffffu, grow)) {
                    float alpha = 1.f;
                    if (grow) {
                        alpha = fast_exp2(m_run - tmax);  // (0 from a maximum of -inf)
                        m_run = tmax;
                        l_run *= alpha;
                    }
                    // rows whose maximum moved rescale their O once the last P V is complete
                    // (head_dim 128: S of this tile came after it)
                    if (j > 0) {
                        if (kGroups == 1) {
                            if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&h->pv_done), (j - 1) & 1u, abort_flag,
                                                                           p.wait_limit_ns))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
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
                const uint64_t sc2 = pack2(sc, sc), nm2 = pack2(nm, nm);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c0 = 0; c0 < 128; c0 += 32) {
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
                    tmem_st16(t_s + (c0 >> 1), pw);
                }
                float s0, s1, s2, s3;
                unpack2(sum[0], s0, s1);
                unpack2(sum[1], s2, s3);
                l_run += (s0 + s1) + (s2 + s3);
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(smem_addr(&h->p_full[buf]));
            }
            // ---- the unit's result ----
            if (ok && n_tiles > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&h->o_full[grp]), 0u, abort_flag, p.wait_limit_ns));
                tc_fence_after();
            }
            if (ok) {
                const bool none = n_tiles == 0 || l_run == 0.f;  // (a NaN sum stays)
                const float inv = none ? 0.f : 1.f / l_run;
                const bool split = p.n_split > 1;
                const bool write = row_ok && !(split && n_tiles == 0);  // (the merge reads no such part)
                const int64_t out_row = (u.q0 + tok) * p.n_head + head;
                const int64_t part_row = (int64_t)u.split * p.n_tok * p.n_head + out_row;
                // V that was kept apart: cells that this row sees
                bool fix = false;
                if (n_tiles > 0 && mbar_wait_bounded(smem_addr(&h->load_done), 0u, abort_flag, p.wait_limit_ns) && row_ok)
                    for (int t = 0; t < 4; ++t)
                        fix = fix || (h->bad_cells[t][0] | h->bad_cells[t][1] | h->bad_cells[t][2] | h->bad_cells[t][3]) != 0u;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t ov[32];
                    if (n_tiles > 0) {
                        tmem_ld32(t_o + c0, ov);
                        tc_wait_ld();
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        ov[k] = none ? 0u : __float_as_uint(__uint_as_float(ov[k]) * inv);
                    if (fix) {
#pragma unroll 1
                        for (int t = 0; t < 4; ++t)
#pragma unroll 1
                            for (int c = 0; c < 128; ++c) {
                                if (!((h->bad_cells[t][c >> 5] >> (c & 31)) & 1u)) continue;
                                const int64_t at = (int64_t)(u.j0 + first_cut + t) * kPrefillTile + c;
                                if (at >= u.lim0 + tok) continue;
                                const int64_t cell = p.plan != nullptr ? (int64_t)__ldg(p.plan + (int64_t)u.seq * p.plan_stride + at)
                                                                       : u.cell0 + at;
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const int e = c0 + k;
                                    __half x;
                                    const int64_t vr = cell * p.n_head_kv + u.g;
                                    if (VBITS == 16) {
                                        x = static_cast<const __half*>(p.v)[cell * p.v_stride + (int64_t)u.g * D + e];
                                    } else {  // (only the scale is not finite)
                                        x = p.v_scale[vr * (D / 32) + e / 32];
                                        if (__hisinf(x)) x = __ushort_as_half(0x7fffu);  // (as the loader has it)
                                    }
                                    if (__hisinf(x) || __hisnan(x)) ov[k] = __float_as_uint(__uint_as_float(ov[k]) + __half2float(x));
                                }
                            }
                    }
                    if (write) {
                        if (split) {
                            float4* d = reinterpret_cast<float4*>(p.part_o + part_row * D + c0);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                d[k] = make_float4(__uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1]),
                                                   __uint_as_float(ov[4 * k + 2]), __uint_as_float(ov[4 * k + 3]));
                        } else {
                            uint4* d = reinterpret_cast<uint4*>(p.out + out_row * D + c0);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    w[i] = pack_half2(__uint_as_float(ov[8 * k + 2 * i]), __uint_as_float(ov[8 * k + 2 * i + 1]));
                                d[k] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                }
                if (write) {
                    const float v = none ? -INFINITY : (m_run - kLift + fast_log2(l_run)) * kLn2;
                    if (split)
                        p.part_lse[part_row] = v;
                    else if (p.lse != nullptr)
                        p.lse[out_row] = v;
                }
            }
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

// Merges a row's partials: weights exp(lse_p - max lse).  A warp per row; the parts that a row
// has follow from its limit, so nothing is read of the others.
template <int D>
__global__ void __launch_bounds__(128) prefill_merge_kernel(const __grid_constant__ PrefillParams p) {
    pdl_wait();
    const int64_t rows = p.n_tok * p.n_head;
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const int64_t tok = r / p.n_head;
    // the token's sequence: the last one that starts at or before it and ends after it
    int seq = -1;
    int64_t q0 = 0, end = 0;
    for (int s0 = 0; s0 < p.n_seq && seq < 0; s0 += 32) {
        const int s = s0 + lane;
        int64_t a = 0, e = 0;
        if (s < p.n_seq) {
            a = clamp64(__ldg(p.offsets + s), 0, p.n_tok);
            e = clamp64(__ldg(p.offsets + s + 1), a, p.n_tok);
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, tok >= a && tok < e);
        if (hit != 0u) {
            const int l = __ffs(hit) - 1;
            seq = s0 + l;
            q0 = __shfl_sync(0xffffffffu, a, l);
            end = __shfl_sync(0xffffffffu, e, l);
        }
    }
    if (seq < 0) return;  // a row behind the last sequence stays as it was
    const int64_t cap = p.plan != nullptr ? p.plan_stride : p.n_cells;
    int64_t L = clamp64(__ldg(p.seq_lens + seq), 0, p.max_len);
    L = L < cap ? L : cap;
    const int64_t lim = L - (end - q0) + 1 + (tok - q0);
    int64_t parts = lim > 0 ? ((lim + kPrefillTile - 1) / kPrefillTile + p.split_tiles - 1) / p.split_tiles : 0;
    if (parts > p.n_split) parts = p.n_split;
    // maximum and weights' sum over the parts, a lane each
    float m = -INFINITY;
    for (int64_t i = lane; i < parts; i += 32) {
        const float v = p.part_lse[i * rows + r];
        m = v > m || v != v ? v : m;  // (a NaN stays)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float v = __shfl_xor_sync(0xffffffffu, m, o);
        m = v > m || v != v ? v : m;
    }
    float acc[D / 32] = {};
    float total = 0.f;
    if (m != -INFINITY) {
        for (int64_t i = 0; i < parts; ++i) {
            const float v = p.part_lse[i * rows + r];
            if (v == -INFINITY) continue;
            const float w = exp2f((v - m) * 1.4426950408889634f);
            total += w;
            const float4* o = reinterpret_cast<const float4*>(p.part_o + (i * rows + r) * D);
#pragma unroll
            for (int k = 0; k < D / 128; ++k) {
                const float4 f = o[32 * k + lane];
                acc[4 * k] += w * f.x;
                acc[4 * k + 1] += w * f.y;
                acc[4 * k + 2] += w * f.z;
                acc[4 * k + 3] += w * f.w;
            }
        }
    }
    const float inv = m == -INFINITY ? 0.f : 1.f / total;
    uint2* d = reinterpret_cast<uint2*>(p.out + r * D);
#pragma unroll
    for (int k = 0; k < D / 128; ++k)
        d[32 * k + lane] = make_uint2(pack_half2(acc[4 * k] * inv, acc[4 * k + 1] * inv),
                                      pack_half2(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
    if (lane == 0 && p.lse != nullptr) p.lse[r] = m == -INFINITY ? -INFINITY : m + logf(total);
}

template <int D>
const void* kernel_of(int kv_type) {
    switch (kv_type) {
    case KVATTN_KV_F16: return (const void*)prefill_kernel<D, 16, 16>;
    case KVATTN_KV_Q8_0: return (const void*)prefill_kernel<D, 8, 8>;
    case KVATTN_KV_Q8_0_Q4_0: return (const void*)prefill_kernel<D, 8, 4>;
    default: return (const void*)prefill_kernel<D, 4, 4>;
    }
}

// Per device and kernel, once: its shared memory.
cudaError_t prefill_setup(int kv_type, int head_dim) {
    static std::mutex mu;
    static bool done[64][4][2];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    bool& d = done[dev & 63][kv_type][head_dim == 256];
    if (!d) {
        e = cudaFuncSetAttribute(head_dim == 128 ? kernel_of<128>(kv_type) : kernel_of<256>(kv_type),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        d = e == cudaSuccess;
    }
    return e;
}

cudaError_t launch(const void* f, unsigned grid, unsigned threads, size_t smem, void** args, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
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

cudaError_t launch_prefill(const PrefillParams& p, int kv_type, int head_dim, cudaStream_t stream, bool pdl) {
    const cudaError_t e = prefill_setup(kv_type, head_dim);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)p.n_blocks * p.n_head_kv * p.n_split;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    void* args[] = {const_cast<PrefillParams*>(&p)};
    return launch(head_dim == 128 ? kernel_of<128>(kv_type) : kernel_of<256>(kv_type), (unsigned)grid, kThreads, kSmemBytes,
                  args, stream, pdl);
}

cudaError_t launch_prefill_merge(const PrefillParams& p, int head_dim, cudaStream_t stream, bool pdl) {
    const int64_t grid = (p.n_tok * p.n_head + 3) / 4;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    void* args[] = {const_cast<PrefillParams*>(&p)};
    return launch(head_dim == 128 ? (const void*)prefill_merge_kernel<128> : (const void*)prefill_merge_kernel<256>,
                  (unsigned)grid, 128, 0, args, stream, pdl);
}

}  // namespace kvattn
