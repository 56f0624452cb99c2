// A step's maps from what a serving program knows of its requests: how many cells each holds and how
// many tokens it gets.  Sequence s needs
//
//     need_s = ceil((len_s + new_s) / B) - ceil(len_s / B)
//
// blocks of B cells more, taken_s = need_0 + .. + need_s; it is served when need_s = 0 or taken_s <=
// n_free, and its j-th new block is number taken_s - need_s + j of the free list from its end.  From
// that follow the block tables, the packed rows' offsets, positions and slots, the lengths, and the
// cell plan (entry i of a row is table[i / B] B + i % B).
//
// One launch, whatever the sizes: blocks of threads do not wait for one another, each makes the two
// running sums over the sequences itself (new tokens, then needed blocks) and finds new blocks in the
// free list, not in the tables that another one may be writing.  A few sequences and tokens are all
// latency; a whole plan is bytes (4 an entry, written in 16-byte pieces).
#include <cstdint>

#include "prompt.cuh"

namespace kvattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPieceEntries = 8192;   // of a plan row, for one block of threads
constexpr int kPieceTokens = 1024;

// Inclusive sum over the block's threads, added to `base`, which moves on by the whole sum.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t& base, int64_t* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    int64_t before = base;
    for (int i = 0; i < kWarps; ++i) {
        const int64_t w = part[i];
        if (i < warp) before += w;
        base += w;
    }
    __syncthreads();
    return before + v;
}

__global__ void __launch_bounds__(kThreads) step_maps_kernel(const __grid_constant__ StepMapsParams p) {
    __shared__ int64_t part[kWarps];
    __shared__ int64_t mine[5];   // of this block's sequence: length, new tokens, first row, blocks taken before, needed
    __shared__ int mine_served;
    __shared__ unsigned long long most;   // blocks taken in all
    pdl_wait();
    const int tid = threadIdx.x;
    const int seq = (int)(blockIdx.x / (unsigned)p.pieces), piece = (int)(blockIdx.x % (unsigned)p.pieces);
    const int shift = p.block_shift;
    const int64_t B = (int64_t)1 << shift;
    int64_t n_free = 0;
    if (p.free_list != nullptr) {
        n_free = __ldg(p.n_free);
        n_free = n_free < 0 ? 0 : (n_free > p.n_list ? p.n_list : n_free);
    }
    if (tid == 0) most = 0ull;
    __syncthreads();
    int64_t rows = 0, taken_all = 0;
    bool unserved = false;
    for (int s0 = 0; s0 < p.n_seq; s0 += kThreads) {
        const int s = s0 + tid;
        int64_t len = 0, n = 0;
        if (s < p.n_seq) {
            len = __ldg(p.lens + s);
            n = __ldg(p.n_new + s);
            len = len < 0 ? 0 : (len > p.max_len ? p.max_len : len);
            n = n < 0 ? 0 : n;
        }
        const int64_t end_row = block_sum(n, rows, part);
        const bool fits = n == 0 || (len + n <= p.max_len && end_row <= p.n_tok);
        const int64_t need = fits && p.free_list != nullptr ? ((len + n + B - 1) >> shift) - ((len + B - 1) >> shift) : 0;
        const int64_t taken = block_sum(need, taken_all, part);
        const bool served = fits && (need == 0 || taken <= n_free);
        unserved = unserved || !served;
        if (need > 0 && served) atomicMax(&most, (unsigned long long)taken);
        if (s == seq) {
            mine[0] = len;
            mine[1] = n;
            mine[2] = end_row - n;
            mine[3] = taken - need;
            mine[4] = need;
            mine_served = served ? 1 : 0;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) p.offsets[0] = 0;
    // rows behind the last token: no cell
    for (int64_t r = rows + (int64_t)blockIdx.x * kThreads + tid; r < p.n_tok; r += (int64_t)gridDim.x * kThreads) {
        if (p.positions != nullptr) p.positions[r] = 0;
        p.slots[r] = -1;
    }
    if (blockIdx.x == 0) {
        if (tid == 0 && p.n_free_out != nullptr) *p.n_free_out = (int32_t)(n_free - (int64_t)most);
        if (unserved && p.status != nullptr) atomicOr(p.status, KVATTN_DEVICE_NO_ROOM);
    }
    if (seq >= p.n_seq) return;

    const int64_t len = mine[0], n = mine[1], row0 = mine[2], before = mine[3], need = mine[4];
    const bool served = mine_served != 0;
    const int64_t after = served ? len + n : len;
    const int64_t held = (len + B - 1) >> shift;
    int32_t* table = p.tables + (int64_t)seq * p.table_stride;
    bool bad = false;
    // first cell of the sequence's block e, -1: none
    auto block_cell = [&](int64_t e) -> int32_t {
        const int32_t id = served && e >= held && e < held + need ? __ldg(p.free_list + (n_free - 1 - (before + e - held))) : table[e];
        if (id >= 0 && (((int64_t)id + 1) << shift) <= p.n_cells) return (int32_t)((int64_t)id << shift);
        bad = true;
        return -1;
    };
    auto cell_at = [&](int64_t i) -> int32_t {
        const int32_t c = block_cell(i >> shift);
        return c < 0 ? -1 : c + (int32_t)(i & (B - 1));
    };
    if (piece == 0) {
        if (tid == 0) {
            const int64_t end = row0 + n;
            p.offsets[seq + 1] = (int32_t)(end < p.n_tok ? end : p.n_tok);
            p.seq_lens[seq] = (int32_t)after;
        }
        if (served)
            for (int64_t j = tid; j < need; j += kThreads) table[held + j] = __ldg(p.free_list + (n_free - 1 - (before + j)));
    }
    int32_t* row = p.plan == nullptr ? nullptr : p.plan + (int64_t)seq * p.plan_stride;
    // (the tokens of a sequence that is served all have rows)
    const int64_t there = row0 + n <= p.n_tok ? n : (row0 < p.n_tok ? p.n_tok - row0 : 0);
    for (int64_t t = (int64_t)piece * kThreads + tid; t < there; t += (int64_t)p.pieces * kThreads) {
        const int32_t cell = served ? cell_at(len + t) : -1;
        if (p.positions != nullptr) p.positions[row0 + t] = len + t < INT32_MAX ? (int32_t)(len + t) : INT32_MAX;
        p.slots[row0 + t] = cell;
        if (row != nullptr && !p.whole && served) row[len + t] = cell;
    }
    if (row != nullptr && p.whole) {
        // (blocks hold a multiple of four cells: four entries that begin at a multiple of four have one
        // block; a row that does not lie on 16 bytes is written one by one)
        const bool wide = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
        for (int64_t i = 4 * ((int64_t)piece * kThreads + tid); i < p.plan_stride; i += 4 * (int64_t)p.pieces * kThreads) {
            const int32_t first = i < after ? block_cell(i >> shift) : -1;
            const int32_t c = first < 0 ? -1 : first + (int32_t)(i & (B - 1));
            int4 e;
            e.x = c;
            e.y = c < 0 || i + 1 >= after ? -1 : c + 1;
            e.z = c < 0 || i + 2 >= after ? -1 : c + 2;
            e.w = c < 0 || i + 3 >= after ? -1 : c + 3;
            if (wide && i + 4 <= p.plan_stride) {
                *reinterpret_cast<int4*>(row + i) = e;
            } else {
                row[i] = e.x;
                if (i + 1 < p.plan_stride) row[i + 1] = e.y;
                if (i + 2 < p.plan_stride) row[i + 2] = e.z;
                if (i + 3 < p.plan_stride) row[i + 3] = e.w;
            }
        }
    }
    if (bad && p.status != nullptr) atomicOr(p.status, KVATTN_DEVICE_BAD_PLAN_ENTRY);
}

}  // namespace

cudaError_t launch_step_maps(const StepMapsParams& p0, cudaStream_t stream, bool pdl) {
    StepMapsParams p = p0;
    const int64_t seqs = p.n_seq > 0 ? p.n_seq : 1;
    // a sequence's share of the rows and its plan row, a block of threads for each piece of them
    int64_t pieces = (p.n_tok / seqs + kPieceTokens - 1) / kPieceTokens;
    if (p.plan != nullptr && p.whole) {
        const int64_t of_plan = (p.plan_stride + kPieceEntries - 1) / kPieceEntries;
        pieces = pieces > of_plan ? pieces : of_plan;
    }
    pieces = pieces < 1 ? 1 : (pieces > 64 ? 64 : pieces);
    p.pieces = (int)pieces;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(seqs * pieces), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    void* args[] = {&p};
    return cudaLaunchKernelExC(&cfg, (const void*)step_maps_kernel, args);
}

}  // namespace kvattn
