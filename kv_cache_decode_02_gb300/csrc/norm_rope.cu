// Norms of the heads of q and k with the rotation in the same pass, and rotations by positions of
// several axes.  A head x of D elements becomes
//
//     y = x w / sqrt(mean(x^2) + eps)      (each side that has weights w; else y = x),
//
// then pair i of its first n_rot elements is turned by pos[axis(i)] theta_i, as in rope.cu: (a, b)
// -> gain (a cos - b sin, a sin + b cos).  The sum of squares, its root and the products are in 32
// bits, and the result is rounded to half once (a norm that stores its result and a rotation that
// reads it round twice and move every element twice more).  Angles are 64-bit integer products of
// positions and fixed-point turns, as in rope.cu.
//
// Bound: bytes.  A lane holds 16 elements of a head (its 8 pairs, or 16 elements that are not
// turned), 8 or 16 lanes a head, which sum their squares in three or four shuffles; a warp keeps one
// token's cosines and sines and a side's weights in registers and walks the heads of q and k.  16384
// tokens of 16 / 8 heads of 256, 64 turned (403 MB): 67 us, 90 % of the measured copy rate; 8192 tokens
// of 32 / 8 heads of 128 by three axes, not normed (168 MB): 27.5 us, 91 %; 64 tokens 3.4 us in a graph.
#include <cstdint>

#include "prompt.cuh"

namespace kvattn {
namespace {

constexpr int kThreads = 128;
constexpr int kBlocksPerSm = 8;    // 64 registers: 67 us for the prompt above, 72 without the bound, 92 at ten
// A token is split among warps until there are this many for an SM: 8192 tokens of 32 / 8 heads of 128
// 28.0 us at 16, 27.5 at 64, 31.5 at 128 (every warp makes the token's angles).
constexpr int kWarpsPerSm = 64;

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}

// A warp serves one token and the groups of 512 / D heads [part, +parts, ...): lane l holds the
// elements of piece l % (D / 16) of head l / (D / 16) of a group.  Every lane stays to the end (heads
// meet in shuffles); a lane whose group ends before it repeats the last head and stores nothing.
template <int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_rope_kernel(const __grid_constant__ NormRopeParams p, int parts) {
    constexpr int kPieces = D / 16, kHeads = 32 / kPieces;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t tok = w / parts;
    const int part = (int)(w - tok * parts);
    if (tok >= p.r.n_tok) return;
    const int piece = lane % kPieces, sub = lane / kPieces;
    const bool turned = piece < p.r.n_rot / 16;
    // element offsets of the lane's two 16-byte pieces
    const int e0 = (INTERLEAVED || !turned) ? 16 * piece : 8 * piece;
    const int e1 = (INTERLEAVED || !turned) ? e0 + 8 : e0 + p.r.n_rot / 2;
    const int total = p.r.n_head[0] + p.r.n_head[1];
    // two heads in flight per lane, the first two under way before the angles are made
    uint4 x[2][2];
    __half* d[2];
    bool side[2];   // of k
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int j = min(base + u * parts * kHeads + sub, total - 1);
            side[u] = j >= p.r.n_head[0];
            const int s = side[u] ? 1 : 0;
            const int h = side[u] ? j - p.r.n_head[0] : j;
            const __half* from = p.r.src[s] + tok * p.r.src_stride[s] + (int64_t)h * D;
            d[u] = p.r.dst[s] + tok * p.r.dst_stride[s] + (int64_t)h * D;
            x[u][0] = *reinterpret_cast<const uint4*>(from + e0);
            x[u][1] = *reinterpret_cast<const uint4*>(from + e1);
        }
    };
    int base = part * kHeads;
    if (base >= total) return;
    load(base);
    // the weights of the side that the lane is at (a head's side changes once, from q to k)
    uint4 w0 = {}, w1 = {};
    bool normed = false, second = false;
    auto weights = [&](bool k) {
        second = k;
        const __half* at = p.weight[k ? 1 : 0];
        normed = at != nullptr;
        if (normed) {
            w0 = __ldg(reinterpret_cast<const uint4*>(at + e0));
            w1 = __ldg(reinterpret_cast<const uint4*>(at + e1));
        }
    };
    if (NORM) weights(side[0]);
    float cs[8], sn[8];
    if (turned) {
        int32_t pos[kMaxAxes];
#pragma unroll
        for (int a = 0; a < kMaxAxes; ++a) pos[a] = a < p.n_axes ? __ldg(p.r.pos + a * p.pos_stride + tok) : 0;
        uint2 axis = make_uint2(0u, 0u);
        if (p.n_axes > 1) axis = __ldg(reinterpret_cast<const uint2*>(p.axis) + piece);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = ((i < 4 ? axis.x : axis.y) >> (8 * (i & 3))) & 0xffu;
            int32_t at = 0;   // (an axis that is not there: position 0)
#pragma unroll
            for (int b = 0; b < kMaxAxes; ++b) at = a == (uint32_t)b ? pos[b] : at;
            const uint64_t turn = (uint64_t)(int64_t)at * __ldg(p.r.turns + 8 * piece + i);
            const float half_turns = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
            sincospif(half_turns, &sn[i], &cs[i]);
            cs[i] *= p.r.gain;
            sn[i] *= p.r.gain;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
    }
    while (true) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!NORM && !turned) continue;   // copied
            float f[16];
            unpack8(x[u][0], f);
            unpack8(x[u][1], f + 8);
            if (NORM) {
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i & 1] = fmaf(f[i], f[i], sum[i & 1]);
                float all = sum[0] + sum[1];
#pragma unroll
                for (int o = 1; o < kPieces; o <<= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
                if (side[u] != second) weights(side[u]);
                if (normed) {
                    const float r = rsqrtf(fmaf(all, 1.f / D, p.eps));
                    float g[8];
                    unpack8(w0, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= r * g[i];
                    unpack8(w1, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[8 + i] *= r * g[i];
                }
            }
            if (turned) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int ia = INTERLEAVED ? 2 * i : i, ib = INTERLEAVED ? ia + 1 : i + 8;
                    const float a = f[ia], b = f[ib];
                    f[ia] = a * cs[i] - b * sn[i];
                    f[ib] = a * sn[i] + b * cs[i];
                }
            }
            x[u][0] = pack8(f);
            x[u][1] = pack8(f + 8);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (base + u * parts * kHeads + sub < total) {
                *reinterpret_cast<uint4*>(d[u] + e0) = x[u][0];
                *reinterpret_cast<uint4*>(d[u] + e1) = x[u][1];
            }
        base += 2 * parts * kHeads;
        if (base >= total) break;
        load(base);
    }
}

template <int D>
const void* kernel_of(bool interleaved, bool norm) {
    if (interleaved) return norm ? (const void*)norm_rope_kernel<D, true, true> : (const void*)norm_rope_kernel<D, true, false>;
    return norm ? (const void*)norm_rope_kernel<D, false, true> : (const void*)norm_rope_kernel<D, false, false>;
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int sms, cudaStream_t stream, bool pdl) {
    const RopeParams& r = p.r;
    const int heads_per_warp = 512 / r.head_dim;
    const int groups = (r.n_head[0] + r.n_head[1] + heads_per_warp - 1) / heads_per_warp;
    int parts = 1;
    while (2 * parts < groups && r.n_tok * parts < (int64_t)sms * kWarpsPerSm) parts *= 2;
    const int64_t warps = r.n_tok * parts;
    const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    void* args[] = {const_cast<NormRopeParams*>(&p), &parts};
    const bool norm = p.weight[0] != nullptr || p.weight[1] != nullptr;
    return cudaLaunchKernelExC(&cfg, r.head_dim == 128 ? kernel_of<128>(r.interleaved, norm) : kernel_of<256>(r.interleaved, norm),
                               args);
}

}  // namespace kvattn
