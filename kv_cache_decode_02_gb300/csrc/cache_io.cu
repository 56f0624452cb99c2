// The cache as it is written and read back: half rows into cells of an f16, Q8_0, Q8_0 + Q4_0
// or Q4_0 cache, and cells back into half rows.  Slots name the cells (-1: no cell); a token's
// row of all KV heads is n_head_kv x head_dim elements, in blocks of 32 that share a scale.
//
// Stored scale: Q8_0 d = amax / 127, Q4_0 d = m / -8 with m the element of largest magnitude
// (the lowest index of equals), rounded to half AWAY from zero: then |x / d| <= 127 (or 8) for
// every element, so no code is clipped but the 4-bit +8, and the error of every other element
// is at most |d| / 2 also where d is subnormal.  Code: x / d rounded to the nearest whole
// number, ties to even, of the exact quotient (quantise below says how, without a division).
// A block with an infinity or a NaN gets the scale NaN, so that reading it shows it.
//
// Bound: bytes.  131072 Q8_0 cells of 8 heads x 256 read back (1.6 GB): 260 us, 93 % of the
// measured copy rate; 16384 tokens of 8 heads x 128 into Q8_0 + Q4_0 and back: 39 us for the two
// kernels, 71 % (46 before a row was loaded while its slot is).  A thread holds half a block (32
// bytes of halves); two neighbouring lanes meet in shuffles for the block's maximum, and for
// 4-bit rows, whose byte j holds elements j and j + 16, to pair their nibbles.  Offsets into the
// cache are 64-bit.
#include <cstdint>

#include "prompt.cuh"

namespace kvattn {
namespace {

constexpr int kIoThreads = 128;
constexpr uint32_t kFull = 0xffffffffu;

// The nearest whole number (ties to even) of x / d, in the low bits of a float's mantissa
// above `base` (1.5 x 2^23 + an offset), from r = 1 / d rounded to fp32.  x and d are halves
// and |x / d| <= 127.5: their quotient is half-way between two whole numbers, or at least 2^-12
// away from every half-way point (both are whole numbers below 2^11 times a power of two), and
// x * r is within 2^-16 of it.  So rounding x * r to a multiple of 2^-14 first (adding and
// subtracting 768, whose last place that is) restores exact ties and moves nothing across one.
__device__ __forceinline__ uint32_t quantise(float x, float r, float top, float base) {
    const float y = __fsub_rn(__fmaf_rn(x, r, 768.f), 768.f);
    return __float_as_uint(__fadd_rn(fminf(y, top), base));
}

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

struct Half16 {
    uint32_t w[8];  // 16 halves
};
__device__ __forceinline__ Half16 load16(const __half* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
    return Half16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// The largest magnitude of a block whose halves lie in lanes l and l ^ 1, as half bits; a NaN
// anywhere gives a NaN.
__device__ __forceinline__ uint32_t block_amax(const Half16& x) {
    __half2 m = __habs2(as_h2(x.w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(as_h2(x.w[i])));
    m = __hmax2_nan(m, __lowhigh2highlow(m));
    const uint32_t other = __shfl_xor_sync(kFull, as_u32(m), 1);
    m = __hmax2_nan(m, as_h2(other));
    return as_u32(m) & 0xffffu;
}

__device__ __forceinline__ float2 pair_f32(uint32_t w) { return __half22float2(as_h2(w)); }

// Reports slots outside [-1, n_cells) once per thread that saw one.
__device__ __forceinline__ int64_t slot_of(const CacheIoParams& p, int64_t tok) {
    if (p.slots == nullptr) return tok;
    const int32_t c = __ldg(p.slots + tok);
    if (c >= 0 && (int64_t)c < p.n_cells) return c;
    if (c != -1 && p.status != nullptr) atomicOr(p.status, KVATTN_DEVICE_BAD_PLAN_ENTRY);
    return -1;
}

// BITS: of this side's rows (16, 8, 4).  One thread: 16 elements of token tok's row.
template <int BITS>
__device__ __forceinline__ void write_item(const CacheIoParams& p, int side, int64_t tok, uint32_t item, int64_t cell,
                                           const Half16& x) {
    const int64_t row_elems = (int64_t)p.n_head_kv * p.head_dim;
    const bool live = cell >= 0;
    if (BITS == 16) {
        if (live) {
            uint4* d = reinterpret_cast<uint4*>(static_cast<__half*>(p.rows[side]) + cell * row_elems + 16 * item);
            d[0] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
            d[1] = make_uint4(x.w[4], x.w[5], x.w[6], x.w[7]);
        }
        return;
    }
    const uint32_t amax = block_amax(x);
    const bool bad = amax >= 0x7c00u;
    const float mag = __half2float(__ushort_as_half((unsigned short)amax));
    // the scale's magnitude, rounded up to half
    const __half dh = __float2half_ru(BITS == 8 ? __fdiv_rn(mag, 127.f) : mag * 0.125f);
    uint32_t dbits = __half_as_ushort(dh);
    if (BITS == 4) {
        // m > 0 makes the scale negative: the sign of the lowest element of magnitude amax
        // (bit 0: seen in this half of the block, bit 1: positive)
        uint32_t found = 0;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const uint32_t hi = x.w[i] >> 16, lo = x.w[i] & 0xffffu;
            if ((hi & 0x7fffu) == amax) found = 1u | ((~hi >> 14) & 2u);
            if ((lo & 0x7fffu) == amax) found = 1u | ((~lo >> 14) & 2u);
        }
        const uint32_t other = __shfl_xor_sync(kFull, found, 1);
        const uint32_t first = (item & 1u) ? other : found, second = (item & 1u) ? found : other;
        const uint32_t use = (first & 1u) ? first : second;
        if ((use & 2u) && amax != 0u) dbits |= 0x8000u;
    }
    const float d = __half2float(__ushort_as_half((unsigned short)dbits));
    // (a zero block and a bad one: r = 0, every code 0)
    const float r = (amax == 0u || bad) ? 0.f : __frcp_rn(d);
    if (bad) dbits = 0x7fffu;
    uint32_t q[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = pair_f32(x.w[i]);
        const float fx = bad ? 0.f : f.x, fy = bad ? 0.f : f.y;
        const float top = BITS == 8 ? 127.f : 7.f, base = BITS == 8 ? 12582912.f : 12582912.f + 8.f;
        q[2 * i] = quantise(fx, r, top, base);
        q[2 * i + 1] = quantise(fy, r, top, base);
    }
    uint32_t b[4];  // 16 bytes: the low byte of every code
#pragma unroll
    for (int i = 0; i < 4; ++i)
        b[i] = prmt_b32(prmt_b32(q[4 * i], q[4 * i + 1], 0x0040u), prmt_b32(q[4 * i + 2], q[4 * i + 3], 0x0040u), 0x5410u);
    if (BITS == 8) {
        if (live)
            *reinterpret_cast<uint4*>(static_cast<int8_t*>(p.rows[side]) + cell * row_elems + 16 * item) =
                make_uint4(b[0], b[1], b[2], b[3]);
    } else {
        // (a code's byte is 0x00 .. 0x0f: 1.5 x 2^23 + 8 + code ends in it)
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] &= 0x0f0f0f0fu;
        // the even lane packs bytes 0-7 of the block, the odd one bytes 8-15
        const bool odd = item & 1u;
        const uint32_t s0 = __shfl_xor_sync(kFull, odd ? b[0] : b[2], 1);
        const uint32_t s1 = __shfl_xor_sync(kFull, odd ? b[1] : b[3], 1);
        const uint32_t w0 = odd ? (s0 | (b[2] << 4)) : (b[0] | (s0 << 4));
        const uint32_t w1 = odd ? (s1 | (b[3] << 4)) : (b[1] | (s1 << 4));
        if (live)
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.rows[side]) + cell * (row_elems / 2) + 8 * item) =
                make_uint2(w0, w1);
    }
    if (live && !(item & 1u))
        p.scales[side][cell * (row_elems / 32) + item / 2] = __ushort_as_half((unsigned short)dbits);
}

// Products of two halves with the scale, each rounded once to half and kept at the largest
// finite half (a scale of 516 x 127 is beyond it); a NaN scale stays NaN.
__device__ __forceinline__ uint32_t scaled(uint32_t codes, __half2 d) {
    const __half2 top = __halves2half2(__ushort_as_half(0x7bffu), __ushort_as_half(0x7bffu));
    return as_u32(__hmax2_nan(__hmin2_nan(__hmul2_rn(as_h2(codes), d), top), __hneg2(top)));
}

// 4-bit codes - 8 as halves: a nibble under 0x6400 is the half 1024 + nibble
__device__ __forceinline__ uint32_t nib2(uint32_t n) {
    return as_u32(__hsub2(as_h2(n | 0x64006400u), as_h2(0x64086408u)));
}

template <int BITS>
__device__ __forceinline__ void read_item(const CacheIoParams& p, int side, int64_t tok, uint32_t item, int64_t cell) {
    const int64_t row_elems = (int64_t)p.n_head_kv * p.head_dim;
    __half* out = p.dst[side] + tok * p.stride[side];
    // the thread's two 16-byte pieces of the half row (4-bit: bytes 8t .. of a block hold its
    // elements 8t .. and 16 + 8t ..)
    const uint32_t e0 = BITS == 4 ? 32 * (item >> 1) + 8 * (item & 1u) : 16 * item;
    const uint32_t e1 = BITS == 4 ? e0 + 16 : e0 + 8;
    uint32_t w[8] = {};
    if (cell >= 0) {
        if (BITS == 16) {
            const Half16 x = load16(static_cast<const __half*>(p.rows[side]) + cell * row_elems + 16 * item);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = x.w[i];
        } else {
            __half d1 = p.scales[side][cell * (row_elems / 32) + item / 2];
            if (__hisinf(d1)) d1 = __ushort_as_half(0x7fffu);  // a scale that is not finite: the block is NaN
            const __half2 d = __half2half2(d1);
            if (BITS == 8) {
                const uint4 c = *reinterpret_cast<const uint4*>(static_cast<const int8_t*>(p.rows[side]) +
                                                                cell * row_elems + 16 * item);
                const uint32_t u[4] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[2 * i] = scaled(i8x2_lo(u[i]), d);
                    w[2 * i + 1] = scaled(i8x2_hi(u[i]), d);
                }
            } else {
                const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.rows[side]) +
                                                                cell * (row_elems / 2) + 8 * item);
                const uint32_t u[2] = {c.x, c.y};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t a = prmt_b32(u[i], 0u, 0x4140u), b = prmt_b32(u[i], 0u, 0x4342u);
                    w[2 * i] = scaled(nib2(a & 0x000f000fu), d);
                    w[2 * i + 1] = scaled(nib2(b & 0x000f000fu), d);
                    w[4 + 2 * i] = scaled(nib2((a >> 4) & 0x000f000fu), d);
                    w[5 + 2 * i] = scaled(nib2((b >> 4) & 0x000f000fu), d);
                }
            }
        }
    }
    *reinterpret_cast<uint4*>(out + e0) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(out + e1) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Threads count (token, 16-element piece of its row); blockIdx.y is the side (K, V).
template <int KBITS, int VBITS, bool WRITE>
__global__ void __launch_bounds__(kIoThreads) cache_io_kernel(const __grid_constant__ CacheIoParams p, uint32_t items) {
    pdl_wait();
    const uint32_t n = (uint32_t)p.n_tok * items;
    const uint32_t i = blockIdx.x * kIoThreads + threadIdx.x;
    const bool in = i < n;
    const uint32_t tok = in ? i / items : 0u;
    const uint32_t item = in ? i - tok * items : (threadIdx.x & 1u);
    const int side = blockIdx.y;
    if (WRITE) {  // (all lanes stay: the two halves of a block meet in shuffles)
        // (the row is on its way while its slot is read; a skipped token's is read for nothing)
        Half16 x = {};
        if (in) x = load16(p.src[side] + (int64_t)tok * p.stride[side] + 16 * (int64_t)item);
        const int64_t cell = in ? slot_of(p, tok) : -1;
        if (side == 0)
            write_item<KBITS>(p, 0, tok, item, cell, x);
        else
            write_item<VBITS>(p, 1, tok, item, cell, x);
    } else if (in) {
        const int64_t cell = slot_of(p, tok);
        if (side == 0)
            read_item<KBITS>(p, 0, tok, item, cell);
        else
            read_item<VBITS>(p, 1, tok, item, cell);
    }
}

template <bool WRITE>
cudaError_t launch_io(const CacheIoParams& p, int kv_type, cudaStream_t stream, bool pdl) {
    uint32_t items = (uint32_t)(p.n_head_kv * p.head_dim / 16);
    const int64_t n = p.n_tok * (int64_t)items;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n + kIoThreads - 1) / kIoThreads), 2, 1);
    cfg.blockDim = dim3(kIoThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    void* args[] = {const_cast<CacheIoParams*>(&p), &items};
    const void* f = kv_type == KVATTN_KV_F16    ? (const void*)cache_io_kernel<16, 16, WRITE>
                    : kv_type == KVATTN_KV_Q8_0 ? (const void*)cache_io_kernel<8, 8, WRITE>
                    : kv_type == KVATTN_KV_Q4_0 ? (const void*)cache_io_kernel<4, 4, WRITE>
                                                : (const void*)cache_io_kernel<8, 4, WRITE>;
    return cudaLaunchKernelExC(&cfg, f, args);
}

}  // namespace

cudaError_t launch_cache_write(const CacheIoParams& p, int kv_type, cudaStream_t stream, bool pdl) {
    return launch_io<true>(p, kv_type, stream, pdl);
}
cudaError_t launch_cache_read(const CacheIoParams& p, int kv_type, cudaStream_t stream, bool pdl) {
    return launch_io<false>(p, kv_type, stream, pdl);
}

}  // namespace kvattn
