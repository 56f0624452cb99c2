// Rotary positions: pair i of a head's first n_rot elements is turned by the angle
// pos x theta_i, (a, b) -> gain (a cos - b sin, a sin + b cos); the rest is copied.
//
// Angles: theta_i is kept as a fixed-point fraction of a turn (2^-64 turns, 64 bits), and
// pos x theta_i is a 64-bit integer product whose overflow drops whole turns, exactly what a
// periodic function may drop.  The top 32 bits, as a signed number of half turns, feed
// sincospif: no 64-bit floating-point arithmetic on the device and no range reduction.  The angle
// is off by the position times the table's rounding (made in doubles: 2^-54 turns), 2^-32 turns
// for the bits dropped, and 2^-25 of itself for the conversion to fp32 (at most 2^-26 turns): 2e-7
// rad at position 10^6, where a product in fp32 is off by 0.06 rad.
//
// Bound: bytes.  Every element is read and written once, 16 bytes per access; a warp keeps one
// token's cosines and sines (8 pairs per lane) in registers and walks the heads of q and k, so
// the 8 sincospif per lane are spread over all of the token's heads.  16384 tokens of 16 / 8 heads
// of 256 (403 MB): 62 us, 95 % of the measured copy rate; 64 tokens: 7.3 us with the launch, all
// latency (9.3 before the data was on its way while the angles are made).
#include <cstdint>

#include "prompt.cuh"

namespace kvattn {
namespace {

constexpr int kRopeThreads = 128;

struct Pairs {
    float c[8], s[8];
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}

// One lane's 16 elements of a head: 8 pairs (first, second in two 16-byte pieces, or
// interleaved in both).
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate16(uint4& w0, uint4& w1, const Pairs& t) {
    float x[8], y[8];
    unpack8(w0, x);
    unpack8(w1, y);
    if (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a0 = x[2 * i], b0 = x[2 * i + 1], a1 = y[2 * i], b1 = y[2 * i + 1];
            x[2 * i] = a0 * t.c[i] - b0 * t.s[i];
            x[2 * i + 1] = a0 * t.s[i] + b0 * t.c[i];
            y[2 * i] = a1 * t.c[4 + i] - b1 * t.s[4 + i];
            y[2 * i + 1] = a1 * t.s[4 + i] + b1 * t.c[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[i], b = y[i];
            x[i] = a * t.c[i] - b * t.s[i];
            y[i] = a * t.s[i] + b * t.c[i];
        }
    }
    w0 = pack8(x);
    w1 = pack8(y);
}

// A warp serves one token and the heads [part, +step, ...): lane l holds the 16 elements of
// piece l % (D / 16) of head l / (D / 16) of each group of 512 / D heads.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, int parts) {
    constexpr int kPieces = D / 16, kHeads = 32 / kPieces;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t tok = w / parts;
    const int part = (int)(w - tok * parts);
    if (tok >= p.n_tok) return;
    const int piece = lane % kPieces, sub = lane / kPieces;
    const int n_pieces = p.n_rot / 16;
    const bool turned = piece < n_pieces;
    // element offsets of the lane's two 16-byte pieces
    const int e0 = (INTERLEAVED || !turned) ? 16 * piece : 8 * piece;
    const int e1 = (INTERLEAVED || !turned) ? e0 + 8 : e0 + p.n_rot / 2;
    const int total = p.n_head[0] + p.n_head[1];
    auto place = [&](int j, const __half*& src, __half*& dst) {
        const int which = j >= p.n_head[0] ? 1 : 0;
        const int h = which ? j - p.n_head[0] : j;
        src = p.src[which] + tok * p.src_stride[which] + (int64_t)h * D;
        dst = p.dst[which] + tok * p.dst_stride[which] + (int64_t)h * D;
    };
    // two heads in flight per lane, the first two under way before the angles are made (a step of
    // a few tokens is all latency)
    uint4 x[2][2];
    __half* d[2];
    auto load = [&](int j0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int j = j0 + u * parts * kHeads;
            const __half* s;
            place(j < total ? j : j0, s, d[u]);
            x[u][0] = *reinterpret_cast<const uint4*>(s + e0);
            x[u][1] = *reinterpret_cast<const uint4*>(s + e1);
        }
    };
    int j0 = part * kHeads + sub;
    if (j0 >= total) return;
    load(j0);
    Pairs t;
    if (turned) {
        const uint64_t pos = (uint64_t)(int64_t)__ldg(p.pos + tok);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t turn = pos * __ldg(p.turns + 8 * piece + i);
            const float half_turns = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
            float s, c;
            sincospif(half_turns, &s, &c);
            t.c[i] = c * p.gain;
            t.s[i] = s * p.gain;
        }
    }
    while (true) {
        if (turned) {
            rotate16<INTERLEAVED>(x[0][0], x[0][1], t);
            rotate16<INTERLEAVED>(x[1][0], x[1][1], t);
        }
        *reinterpret_cast<uint4*>(d[0] + e0) = x[0][0];
        *reinterpret_cast<uint4*>(d[0] + e1) = x[0][1];
        if (j0 + parts * kHeads < total) {
            *reinterpret_cast<uint4*>(d[1] + e0) = x[1][0];
            *reinterpret_cast<uint4*>(d[1] + e1) = x[1][1];
        }
        j0 += 2 * parts * kHeads;
        if (j0 >= total) break;
        load(j0);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t stream, bool pdl) {
    const int heads_per_warp = 512 / p.head_dim;
    const int groups = (p.n_head[0] + p.n_head[1] + heads_per_warp - 1) / heads_per_warp;
    // Warps per token: one walks all heads when the tokens alone fill the device (16 warps per
    // SM); a few tokens spread theirs over up to a warp per two head groups.
    int parts = 1;
    while (2 * parts < groups && p.n_tok * parts < (int64_t)sms * 16) parts *= 2;
    const int64_t warps = p.n_tok * parts;
    const int64_t grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    void* args[] = {const_cast<RopeParams*>(&p), &parts};
    const void* f = p.head_dim == 128
                        ? (p.interleaved ? (const void*)rope_kernel<128, true> : (const void*)rope_kernel<128, false>)
                        : (p.interleaved ? (const void*)rope_kernel<256, true> : (const void*)rope_kernel<256, false>);
    return cudaLaunchKernelExC(&cfg, f, args);
}

}  // namespace kvattn
