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
//
// What it measured: 64 single tokens behind 8192 f16 cells with 30 to 1038 of their own, through a plan,
// 32 / 8 heads of 128: 54 us (49 % of the copy rate; about 4000 clocks for each of 512 units beside its
// tiles); 16 behind 131072 8-bit cells 117 us (38 %; turning codes into halves); 8 x 4 tokens behind 4096
// cells at head_dim 256 22 us.  The join takes 3 to 5 us of each.
#include "prefill_kernel.cuh"

namespace kvattn {

namespace {

// A warp joins a row's parts: lane i of a batch holds the weights of part i over the row's own cells and of
// part i over the prefix, then the lanes hold the row's dims, with the rows of kBatch parts on their way
// at once.  The maximum runs along from batch to batch.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prefill_join_kernel(const __grid_constant__ PrefillParams p, int n_ctas) {
    constexpr int kGroups = Geometry<D>::kGroups, kBatch = 1536 / D;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (row >= p.n_tok * p.n_head) return;
    const int64_t tok = row / p.n_head;
    const int head = (int)(row - tok * p.n_head), G = p.group, g = head / G;
    const int32_t most = (int32_t)p.n_tok;
    const int32_t first = min(max(__ldg(p.offsets), 0), most), last = min(max(__ldg(p.offsets + p.n_seq), 0), most);
    const uint2 join = *p.join;   // the prefix's tiles, the length of the line (0: all units are whole)
    PrefillNote note[2];          // of the sequence's own cells, of the prefix
#pragma unroll
    for (int side = 0; side < 2; ++side) note[side] = p.notes[((int64_t)side * p.n_tok + tok) * p.n_head_kv + g];
    if (tok < first || tok >= last) return;
    Shares sh;
    sh.set(join.y, (uint32_t)n_ctas);
    const bool line = join.y != 0u;

    int parts[2], part_row[2];
    bool whole[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        PrefillNote& x = note[side];
        const bool there = side == 0 || join.x != 0u;
        // (offsets that decrease leave tokens without a note: what stands there must not lead outside)
        x.cta = min(max(x.cta, 0), n_ctas - 1);
        const int t = (int)tok - x.tok0, grp = t / p.group_tokens;
        part_row[side] = min(max(128 * grp + (t - grp * p.group_tokens) * G + (head - g * G), 0), 128 * kGroups - 1);
        whole[side] = !line || x.tiles == 0;
        parts[side] = !there ? 0 : (whole[side] ? 1 : min(max(x.parts, 1), n_ctas - x.cta));
    }
    // part i's place: 2 x CTA + (0: what it began with, 1: what it ended with); -1: it holds no tile
    auto slot_of = [&](int side, int i, bool& all) -> int {
        if (i >= parts[side]) return -1;
        const PrefillNote& x = note[side];
        const uint32_t cta = (uint32_t)(x.cta + i), x0 = sh.of(cta);
        const uint32_t a = max(x0, x.start), b = min(sh.of(cta + 1u), x.end);
        const int32_t each = tile_length(p, x.n_tok);
        const int32_t t0 = tile_at(a - x.start, x.end - x.start, x.tiles, each);
        const int32_t t1 = tile_at(b - x.start, x.end - x.start, x.tiles, each);
        all = t0 == 0 && t1 == x.tiles;
        return t0 == t1 ? -1 : 2 * (int)cta + (x0 > x.start ? 0 : 1);
    };

    float m = -INFINITY, sum = 0.f;
    float acc[D / 32] = {};
    for (int i0 = 0; i0 < max(parts[0], parts[1]); i0 += 32) {
        const float* from[2];
        float v[2];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            bool all = false;
            int slot = -1;
            if (!whole[side]) slot = slot_of(side, i0 + lane, all);
            if (line && __any_sync(0xffffffffu, all)) {   // one part holds all tiles, and wrote them as a whole unit
                whole[side] = true;
                parts[side] = i0 + 1;
            }
            v[side] = -INFINITY;
            from[side] = nullptr;
            if (whole[side]) {
                if (lane == 0 && i0 < parts[side]) {
                    const int64_t at = (int64_t)side * p.n_tok * p.n_head + row;
                    v[side] = p.whole_lse[at];
                    from[side] = p.whole_o + at * D;
                }
            } else if (slot >= 0) {
                const int64_t at = (int64_t)slot * kGroups * 128 + part_row[side];
                v[side] = p.part_lse[at];
                from[side] = p.part_o + at * D;
            }
        }
        float top = v[1] > v[0] || v[1] != v[1] ? v[1] : v[0];
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
        float w[2];
        uint32_t left[2];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            w[side] = v[side] == -INFINITY ? 0.f : exp2f((v[side] - m) * 1.4426950408889634f);
            sum += w[side];                      // (this lane's parts)
            left[side] = __ballot_sync(0xffffffffu, v[side] != -INFINITY);
        }
        while ((left[0] | left[1]) != 0u) {
            float4 f[kBatch][D / 128];
            float wk[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const bool second = left[0] == 0u, in = (left[0] | left[1]) != 0u;
                const uint32_t bits = second ? left[1] : left[0];
                const int i = in ? __ffs(bits) - 1 : 0;
                if (second)
                    left[1] &= left[1] - 1u;
                else
                    left[0] &= left[0] - 1u;
                wk[b] = __shfl_sync(0xffffffffu, second ? w[1] : w[0], i);
                const float4* o = reinterpret_cast<const float4*>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(second ? from[1] : from[0]), i));
#pragma unroll
                for (int k = 0; k < D / 128; ++k) f[b][k] = in ? o[32 * k + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                if (!in) wk[b] = 0.f;
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
