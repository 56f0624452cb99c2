// Attention of sequences that begin with the same cells: those are read once, for the rows of all
// sequences together, and each sequence's own for its rows.
//
// To the kernel the prefix is one more sequence, whose tokens are everybody's and whose tiles every
// row sees whole (prefix_of in prefill_kernel.cuh: whole tiles, as far as every sequence holds them);
// the sequences' own units begin behind it.  A row then has two results, (O_1, lse_1) over the prefix
// and (O_2, lse_2) over its sequence's own cells, each whole or in parts where the shares cut its unit,
// all in 32 bits; the merge weighs them by exp(lse - max lse) and rounds once.
//
// Why one launch for both: the prefix's units are few and long and bound by the products, the others
// many, short and bound by bytes; in one line of equal shares they fill the device together, where two
// launches each leave a tail.
#include "prefill_kernel.cuh"

namespace kvattn {

namespace {

// A warp joins a row's parts: lane i of a batch holds part i's weight, the lanes a row's dims.  The
// maximum runs along from batch to batch.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prefill_join_kernel(const __grid_constant__ PrefillParams p, int n_ctas) {
    constexpr int kGroups = Geometry<D>::kGroups, kBatch = 512 / D;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (row >= p.n_tok * p.n_head) return;
    const int64_t tok = row / p.n_head;
    const int head = (int)(row - tok * p.n_head), G = p.group, g = head / G;
    const int32_t most = (int32_t)p.n_tok;
    const int32_t first = min(max(__ldg(p.offsets), 0), most), last = min(max(__ldg(p.offsets + p.n_seq), 0), most);
    if (tok < first || tok >= last) return;
    const uint2 join = *p.join;   // the prefix's tiles, the length of the line (0: all units are whole)
    Shares sh;
    sh.set(join.y, (uint32_t)n_ctas);
    const int sides = join.x != 0u ? 2 : 1;   // the sequence's own cells, the prefix

    float m = -INFINITY, sum = 0.f;
    float acc[D / 32] = {};
    for (int side = 0; side < sides; ++side) {
        const int64_t whole_row = (int64_t)side * p.n_tok * p.n_head + row;
        PrefillNote note = {};
        int parts = 1, part_row = 0;
        bool whole = join.y == 0u;
        if (!whole) {
            note = p.notes[((int64_t)side * p.n_tok + tok) * p.n_head_kv + g];
            // (offsets that decrease leave tokens without a note: what stands there must not lead outside)
            note.cta = min(max(note.cta, 0), n_ctas - 1);
            while (note.cta + parts < n_ctas && sh.of((uint32_t)(note.cta + parts)) < note.end) ++parts;
            const int t = (int)tok - note.tok0, grp = t / p.group_tokens;
            part_row = min(max(128 * grp + (t - grp * p.group_tokens) * G + (head - g * G), 0), 128 * kGroups - 1);
            whole = note.tiles == 0;
        }
        // part i's place: 2 x CTA + (0: what it began with, 1: what it ended with); -1: it holds no tile
        auto slot_of = [&](int i, bool& all) -> int {
            if (i >= parts) return -1;
            const uint32_t cta = (uint32_t)(note.cta + i), x0 = sh.of(cta);
            const uint32_t a = max(x0, note.start), b = min(sh.of(cta + 1u), note.end);
            const int32_t each = tile_length(p, note.n_tok);
            const int32_t t0 = tile_at(a - note.start, note.end - note.start, note.tiles, each);
            const int32_t t1 = tile_at(b - note.start, note.end - note.start, note.tiles, each);
            all = t0 == 0 && t1 == note.tiles;
            return t0 == t1 ? -1 : 2 * (int)cta + (x0 > note.start ? 0 : 1);
        };
        if (!whole)   // (one part may hold all tiles, and wrote them as a whole unit)
            for (int i0 = 0; i0 < parts; i0 += 32) {
                bool all = false;
                slot_of(i0 + lane, all);
                whole = whole || __any_sync(0xffffffffu, all);
            }
        if (whole) parts = 1;
        for (int i0 = 0; i0 < parts; i0 += 32) {
            float v = -INFINITY;
            const float* from = nullptr;
            if (whole) {
                if (lane == 0) {
                    v = p.whole_lse[whole_row];
                    from = p.whole_o + whole_row * D;
                }
            } else {
                bool all;
                const int slot = slot_of(i0 + lane, all);
                if (slot >= 0) {
                    const int64_t at = (int64_t)slot * kGroups * 128 + part_row;
                    v = p.part_lse[at];
                    from = p.part_o + at * D;
                }
            }
            float top = v;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float w = __shfl_xor_sync(0xffffffffu, top, o);
                top = w > top || w != w ? w : top;   // (a NaN stays)
            }
            if (top == -INFINITY) continue;          // (no part with a cell: its O was not written)
            if (!(m >= top)) {                       // (a NaN too)
                const float old = m == -INFINITY ? 0.f : exp2f((m - top) * 1.4426950408889634f);
                sum *= old;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) acc[k] *= old;
                m = top;
            }
            const float w = v == -INFINITY ? 0.f : exp2f((v - m) * 1.4426950408889634f);
            sum += w;                                // (this lane's parts)
            uint32_t left = __ballot_sync(0xffffffffu, v != -INFINITY);
            while (left != 0u) {
                float4 f[kBatch][D / 128];
                float wk[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const bool in = left != 0u;
                    const int i = in ? __ffs(left) - 1 : 0;
                    wk[b] = __shfl_sync(0xffffffffu, w, i);
                    const float4* o = reinterpret_cast<const float4*>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), i));
                    left &= left - 1u;
#pragma unroll
                    for (int k = 0; k < D / 128; ++k) f[b][k] = in ? o[32 * k + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                }
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
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = m == -INFINITY ? 0.f : 1.f / sum;
    uint2* d = reinterpret_cast<uint2*>(p.out + row * D);
#pragma unroll
    for (int k = 0; k < D / 128; ++k)
        d[32 * k + lane] = make_uint2(pack_half2(acc[4 * k] * inv, acc[4 * k + 1] * inv),
                                      pack_half2(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
    if (lane == 0 && p.lse != nullptr) p.lse[row] = m == -INFINITY ? -INFINITY : m + logf(sum);
}

}  // namespace

cudaError_t launch_prefill_shared(const PrefillParams& p, int kv_type, int head_dim, int n_ctas, cudaStream_t stream, bool pdl) {
    cudaError_t e = run_prefill<kShared>(p, kv_type, head_dim, n_ctas, stream, pdl);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.n_tok * p.n_head + kMergeWarps - 1) / kMergeWarps;
    void* args[] = {const_cast<PrefillParams*>(&p), &n_ctas};
    return launch(head_dim == 128 ? (const void*)prefill_join_kernel<128> : (const void*)prefill_join_kernel<256>,
                  dim3((unsigned)blocks), 32 * kMergeWarps, 0, args, stream, pdl);
}

}  // namespace kvattn
