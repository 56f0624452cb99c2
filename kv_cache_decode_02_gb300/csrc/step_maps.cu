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
// free list, not in the tables that another one may be writing.  One warp makes the sums, 128 sequences
// at a time, while the others write what does not depend on them: plan entries of cells held before.
// 64 rows of 131584 entries over blocks of 16 cells: 11.0 us (a fill of the same bytes takes 6.2; 15.6 with
// sums by all warps in front of everything); 64 single tokens 4.1 us, all latency.
#include <cstdint>

#include "prompt.cuh"

namespace kvattn {
namespace {

constexpr int kThreads = 256;
constexpr int kQuads = 8;                                // of plan entries, for one thread at a time
constexpr int kPieceEntries = 4 * kQuads * kThreads;     // of a plan row, for one block of threads
constexpr int kPieceTokens = 1024;
constexpr int64_t kMaxPieces = 1024;
constexpr int kLaneSequences = 4;

// Inclusive sum over the lanes.
__device__ __forceinline__ int64_t lane_sum(int64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

struct Mine {       // of the block's sequence
    int64_t len, n, row0, before, need;   // length, new tokens, first row, blocks taken before its own
    bool served;
};

__global__ void __launch_bounds__(kThreads) step_maps_kernel(const __grid_constant__ StepMapsParams p) {
    __shared__ Mine mine;
    __shared__ int64_t all_rows, all_taken;   // new tokens, blocks taken
    __shared__ int64_t free_count;
    pdl_wait();
    const int tid = threadIdx.x;
    const int seq = (int)(blockIdx.x / (unsigned)p.pieces), piece = (int)(blockIdx.x % (unsigned)p.pieces);
    const int shift = p.block_shift;
    const int64_t B = (int64_t)1 << shift;
    const bool whole = p.plan != nullptr && p.whole && seq < p.n_seq;
    int32_t* table = p.tables + (int64_t)seq * p.table_stride;
    int32_t* row = p.plan == nullptr ? nullptr : p.plan + (int64_t)seq * p.plan_stride;
    // (a row that does not lie on 16 bytes is written entry by entry)
    const bool wide = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    const uint32_t stride = (uint32_t)p.plan_stride, in_block = (1u << shift) - 1u;
    bool bad = false;
    auto first_of = [&](int32_t id) -> int32_t {   // cell of block `id`, -1: outside the cache
        if (id >= 0 && (((int64_t)id + 1) << shift) <= p.n_cells) return (int32_t)((int64_t)id << shift);
        bad = true;
        return -1;
    };
    auto quad = [&](uint32_t i0, int k) -> uint32_t { return i0 + 4u * (uint32_t)(tid + k * kThreads); };
    auto put4 = [&](uint32_t i, const int4& e) {
        if (wide && i + 4 <= stride) {
            *reinterpret_cast<int4*>(row + i) = e;
        } else {
            if (i < stride) row[i] = e.x;
            if (i + 1 < stride) row[i + 1] = e.y;
            if (i + 2 < stride) row[i + 2] = e.z;
            if (i + 3 < stride) row[i + 3] = e.w;
        }
    };
    // What a thread writes of a plan row is quads, four entries of one block (a block holds a multiple of
    // four cells).  Those below the sequence's length, and those that the step's tokens cannot reach, do
    // not depend on the sums.
    uint32_t held_cells = 0, most = 0;
    auto put_known = [&](uint32_t i0) {
        int32_t id[kQuads];
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            const uint32_t i = quad(i0, k);
            id[k] = i < held_cells ? table[i >> shift] : -1;
        }
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            const uint32_t i = quad(i0, k);
            if (i >= most) {
                put4(i, make_int4(-1, -1, -1, -1));
            } else if (i + 4 <= held_cells) {
                const int32_t first = first_of(id[k]), c = first + (int32_t)(i & in_block);
                put4(i, first < 0 ? make_int4(-1, -1, -1, -1) : make_int4(c, c + 1, c + 2, c + 3));
            }
        }
    };
    if (whole) {
        const int64_t l = __ldg(p.lens + seq), n = __ldg(p.n_new + seq);
        const int64_t held = l < 0 ? 0 : (l > p.max_len ? p.max_len : l), end = held + (n < 0 ? 0 : n);
        held_cells = (uint32_t)held;
        most = (uint32_t)(end > p.max_len ? held : end);   // (one that does not fit is not served)
        if (tid >= 32) put_known((uint32_t)piece * kPieceEntries);
    }

    if (tid < 32) {
        int64_t n_free = 0;
        if (p.free_list != nullptr) {
            n_free = __ldg(p.n_free);
            n_free = n_free < 0 ? 0 : (n_free > p.n_list ? p.n_list : n_free);
        }
        int64_t rows = 0, asked = 0, taken_all = 0;
        bool unserved = false;
        for (int s0 = 0; s0 < p.n_seq; s0 += 32 * kLaneSequences) {
            const int first = s0 + kLaneSequences * tid;
            int64_t len[kLaneSequences], n[kLaneSequences], need[kLaneSequences];
            int64_t sum = 0;
#pragma unroll
            for (int k = 0; k < kLaneSequences; ++k) {
                len[k] = n[k] = 0;
                if (first + k < p.n_seq) {
                    len[k] = __ldg(p.lens + first + k);
                    n[k] = __ldg(p.n_new + first + k);
                }
            }
#pragma unroll
            for (int k = 0; k < kLaneSequences; ++k) {
                len[k] = len[k] < 0 ? 0 : (len[k] > p.max_len ? p.max_len : len[k]);
                n[k] = n[k] < 0 ? 0 : n[k];
                sum += n[k];
            }
            const int64_t row_end = rows + lane_sum(sum);
            int64_t row = row_end - sum;
            bool fits[kLaneSequences];
            sum = 0;
#pragma unroll
            for (int k = 0; k < kLaneSequences; ++k) {
                row += n[k];
                fits[k] = n[k] == 0 || (len[k] + n[k] <= p.max_len && row <= p.n_tok);
                need[k] = fits[k] && p.free_list != nullptr ? ((len[k] + n[k] + B - 1) >> shift) - ((len[k] + B - 1) >> shift) : 0;
                sum += need[k];
            }
            const int64_t asked_end = asked + lane_sum(sum);
            int64_t taken = asked_end - sum;
            row = row_end;
#pragma unroll
            for (int k = kLaneSequences - 1; k >= 0; --k) row -= n[k];
#pragma unroll
            for (int k = 0; k < kLaneSequences; ++k) {
                taken += need[k];
                const bool served = fits[k] && (need[k] == 0 || taken <= n_free);
                if (need[k] > 0 && served) taken_all = taken;
                unserved = unserved || !served;
                if (first + k == seq && first + k < p.n_seq) mine = Mine{len[k], n[k], row, taken - need[k], need[k], served};
                row += n[k];
            }
            rows = __shfl_sync(0xffffffffu, row_end, 31);
            asked = __shfl_sync(0xffffffffu, asked_end, 31);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int64_t w = __shfl_xor_sync(0xffffffffu, taken_all, o);
            taken_all = w > taken_all ? w : taken_all;
        }
        unserved = __any_sync(0xffffffffu, unserved);
        if (tid == 0) {
            all_rows = rows;
            all_taken = taken_all;
            free_count = n_free;
            if (blockIdx.x == 0) {
                p.offsets[0] = 0;
                if (unserved && p.status != nullptr) atomicOr(p.status, KVATTN_DEVICE_NO_ROOM);
            }
        }
    }
    if (whole && tid < 32) put_known((uint32_t)piece * kPieceEntries);
    __syncthreads();
    const int64_t n_free = free_count;
    if (blockIdx.x == 0 && tid == 0 && p.n_free_out != nullptr) *p.n_free_out = (int32_t)(n_free - all_taken);
    // rows behind the last token: no cell
    for (int64_t r = all_rows + (int64_t)blockIdx.x * kThreads + tid; r < p.n_tok; r += (int64_t)gridDim.x * kThreads) {
        if (p.positions != nullptr) p.positions[r] = 0;
        p.slots[r] = -1;
    }
    if (seq >= p.n_seq) return;

    const int64_t len = mine.len, n = mine.n, row0 = mine.row0;
    const bool served = mine.served;
    const int64_t after = served ? len + n : len;
    const int64_t held = (len + B - 1) >> shift, fresh = served ? held + mine.need : held;
    // new block e is entry `from_end - e` of the free list
    const int64_t from_end = n_free - 1 - mine.before + held;
    // first cell of the sequence's block e, whose entry in the table is (or was) `id`; -1: none
    auto block_cell = [&](int64_t e, int32_t id) -> int32_t {
        return first_of(e >= held && e < fresh ? __ldg(p.free_list + (from_end - e)) : id);
    };
    if (piece == 0) {
        if (tid == 0) {
            const int64_t end = row0 + n;
            p.offsets[seq + 1] = (int32_t)(end < p.n_tok ? end : p.n_tok);
            p.seq_lens[seq] = (int32_t)after;
        }
        for (int64_t e = held + tid; e < fresh; e += kThreads) table[e] = __ldg(p.free_list + (from_end - e));
    }
    // (the tokens of a sequence that is served all have rows)
    const int64_t there = row0 + n <= p.n_tok ? n : (row0 < p.n_tok ? p.n_tok - row0 : 0);
    for (int64_t t = (int64_t)piece * kThreads + tid; t < there; t += (int64_t)p.pieces * kThreads) {
        int32_t cell = -1;
        if (served) {
            const int64_t e = (len + t) >> shift;
            cell = block_cell(e, e < held || e >= fresh ? table[e] : -1);   // (not one that is being written)
            if (cell >= 0) cell += (int32_t)((len + t) & (B - 1));
        }
        if (p.positions != nullptr) p.positions[row0 + t] = len + t < INT32_MAX ? (int32_t)(len + t) : INT32_MAX;
        p.slots[row0 + t] = cell;
        if (row != nullptr && !p.whole && served) row[len + t] = cell;
    }
    if (whole) {
        const uint32_t last = (uint32_t)after;
        for (uint32_t i0 = (uint32_t)piece * kPieceEntries; i0 < stride; i0 += (uint32_t)p.pieces * kPieceEntries) {
            if (i0 != (uint32_t)piece * kPieceEntries) put_known(i0);
            if (i0 + kPieceEntries <= held_cells || i0 >= most) continue;
            for (int k = 0; k < kQuads; ++k) {
                const uint32_t i = quad(i0, k);
                if (i >= most || i + 4 <= held_cells) continue;
                const int64_t e = (int64_t)(i >> shift);
                const int32_t first = i < last ? block_cell(e, e < held || e >= fresh ? table[e] : -1) : -1;
                const int32_t c = first + (int32_t)(i & in_block);
                const bool none = first < 0;
                put4(i, make_int4(none ? -1 : c, none || i + 1 >= last ? -1 : c + 1, none || i + 2 >= last ? -1 : c + 2,
                                  none || i + 3 >= last ? -1 : c + 3));
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
    pieces = pieces < 1 ? 1 : (pieces > kMaxPieces ? kMaxPieces : pieces);
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
