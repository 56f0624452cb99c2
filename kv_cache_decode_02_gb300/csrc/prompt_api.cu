// C entry points of the prompt-side operators: host-side validation, how attention's
// work is cut, workspace carving and launches.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "prompt.cuh"

using namespace kvattn;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? KVATTN_OK : KVATTN_ERR_CUDA; }
bool known_type(int t) { return t >= KVATTN_KV_F16 && t <= KVATTN_KV_Q4_0; }
bool known_dim(int d) { return d == 128 || d == 256; }

constexpr int kMaxPrefillGroup = 128;

// Half rows of n_head x head_dim elements, `stride` elements apart: 16-byte pieces.
bool row_ok(const void* p, int64_t stride, int64_t n_head, int head_dim) {
    return p != nullptr && aligned(p, 16) && stride >= n_head * head_dim && stride % 8 == 0;
}

int check_cache(int kv_type, const void* k, const void* v, const void* ks, const void* vs, int head_dim) {
    if (!known_type(kv_type) || k == nullptr || v == nullptr || !aligned(k, 16) || !aligned(v, 16))
        return KVATTN_ERR_INVALID_ARG;
    if (kv_type == KVATTN_KV_F16) return ks == nullptr && vs == nullptr ? KVATTN_OK : KVATTN_ERR_INVALID_ARG;
    const size_t sa = head_dim == 128 ? 8 : 16;
    return ks != nullptr && vs != nullptr && aligned(ks, sa) && aligned(vs, sa) ? KVATTN_OK : KVATTN_ERR_INVALID_ARG;
}

// Units of all sequences together: at most one part-filled block per sequence.
int64_t unit_bound(int64_t n_tok, int n_seq, int n_head_kv, int group, int head_dim) {
    const int64_t per = (int64_t)(128 / group) * prefill_groups(head_dim);
    return std::min((n_tok + per - 1) / per + std::max(n_seq - 1, 0), n_tok) * n_head_kv;
}

// How a call's work is cut.  Units that are many and short are dealt out whole; few or long ones
// (chunks over long caches) are cut into equal shares, one per CTA: 16 units of 1024 tiles would
// otherwise keep 16 of 152 SMs busy.  A share costs its CTA a partial (written and read once
// more) and the call a merge, so a CTA gets at least four tiles' worth of the bound below.
struct Cut {
    bool shares;
    int n_ctas;
    size_t cuts_off, lse_off, o_off, total;
};

constexpr int64_t kMinShareTiles = 4;

// `bound`: of all calls with at most that many units and tiles (one of fewer units may be shared
// where this one is dealt out whole).
Cut cut_of(int64_t units, int64_t tiles, int head_dim, bool may_share, bool bound = false) {
    Cut c = {};
    // (KVATTN_PREFILL_CTAS: the CTAs that share the work, for tests; 0: dealt out whole)
    const char* env = std::getenv("KVATTN_PREFILL_CTAS");
    const int sms = device_sms();
    if (bound) units = std::min(units, 8 * (int64_t)sms - 1);
    c.shares = may_share && tiles > kMinShareTiles && units < 8 * (int64_t)sms;
    // (the kernel numbers the line of all tiles, in eighths, in 31 bits)
    const bool fits = bound || (units < INT32_MAX && (tiles + 18) * 8 < INT32_MAX / std::max<int64_t>(units, 1));
    int64_t n = units;
    if (c.shares) n = std::max(units, (units * tiles + kMinShareTiles - 1) / kMinShareTiles);
    c.n_ctas = (int)std::max<int64_t>(std::min<int64_t>(n, sms), 1);
    if (may_share && env != nullptr && *env != 0) {
        const int want = std::atoi(env);
        c.shares = want > 0;
        c.n_ctas = std::max(std::min(want > 0 ? want : c.n_ctas, sms), 1);
    }
    if (c.n_ctas == 1 || !fits) c.shares = false;
    size_t off = kStatusBytes;
    const size_t rows = c.shares ? (size_t)c.n_ctas * 2 * (size_t)prefill_groups(head_dim) * 128 : 0;
    c.cuts_off = off;
    off = align_up(off + (c.shares ? (size_t)c.n_ctas * sizeof(PrefillCut) : 0), kWsAlign);
    c.lse_off = off;
    off = align_up(off + rows * 4, kWsAlign);
    c.o_off = off;
    c.total = align_up(off + rows * (size_t)head_dim * 4, kWsAlign);
    return c;
}

Cut chunk_cut(int64_t n_tok, int n_seq, int n_head, int n_head_kv, int head_dim, int64_t max_len, bool bound = false) {
    return cut_of(unit_bound(n_tok, n_seq, n_head_kv, n_head / n_head_kv, head_dim),
                  (max_len + kPrefillTile - 1) / kPrefillTile, head_dim, true, bound);
}

// What the two attention entry points have in common.
int launch_attention(PrefillParams& p, const void* q, int64_t q_stride, int kv_type, int n_head, int n_head_kv, int head_dim,
                     int64_t rows, float scale, const Cut& c, const char* name, void* stream) {
    p.n_head = n_head;
    p.n_head_kv = n_head_kv;
    p.group = n_head / n_head_kv;
    p.group_tokens = 128 / p.group;
    p.block_tokens = p.group_tokens * prefill_groups(head_dim);
    p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    p.single_length = kv_type == KVATTN_KV_F16 && head_dim == 128 && p.plan == nullptr ? 5 : 8;
    p.shares = c.shares ? 1 : 0;
    p.out_sectors = aligned(p.out, 32) ? 1 : 0;
    debug_waits(&p.wait_limit_ns, &p.stall_tx);
    if (!encode_prefill_map(&p.tmap_q, q, p.n_tok, n_head, head_dim, q_stride, p.group, p.group_tokens)) return KVATTN_ERR_CUDA;
    if (kv_type == KVATTN_KV_F16) {
        p.use_tma = encode_planes_map(&p.tmap_k, p.k, rows, n_head_kv, head_dim, p.k_stride) &&
                    encode_planes_map(&p.tmap_v, p.v, rows, n_head_kv, head_dim, p.v_stride);
    } else {
        const int kb = kv_type == KVATTN_KV_Q4_0 ? 4 : 8, vb = kv_type == KVATTN_KV_Q8_0 ? 8 : 4;
        p.use_tma = encode_codes_map(&p.tmap_k, p.k, rows, n_head_kv, head_dim * kb / 8, 16 * kb, kPrefillTile) &&
                    encode_codes_map(&p.tmap_v, p.v, rows, n_head_kv, head_dim * vb / 8, 16 * vb, kPrefillTile);
    }
    if (!tma_enabled()) p.use_tma = 0;
    if (log_enabled()) {
        char buf[256];
        std::snprintf(buf, sizeof(buf), "%s kv_type=%d n_seq=%d n_tok=%lld n_head=%d/%d head_dim=%d plan=%d shares=%d grid=%d tma=%d",
                      name, kv_type, p.n_seq, (long long)p.n_tok, n_head, n_head_kv, head_dim, p.plan != nullptr, p.shares,
                      c.n_ctas, p.use_tma);
        log_text(buf);
    }
    return cuda_status(launch_prefill(p, kv_type, head_dim, c.n_ctas, static_cast<cudaStream_t>(stream), pdl_enabled()));
}

int check_heads(int64_t n_tok, int n_seq, int n_head, int n_head_kv, int head_dim) {
    if (n_tok < 0 || n_seq < 0 || n_head < 1 || n_head_kv < 1 || n_head % n_head_kv != 0) return KVATTN_ERR_INVALID_ARG;
    if (n_head / n_head_kv > kMaxPrefillGroup || !known_dim(head_dim)) return KVATTN_ERR_UNSUPPORTED;
    // tokens are numbered in 32 bits, (token, head) rows too
    if (n_tok > INT32_MAX || n_tok * n_head > (int64_t)INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    return KVATTN_OK;
}

}  // namespace

extern "C" {

int kvattn_rope_table(int n_rot, double base, int scaling, double factor, int64_t original_len, uint64_t* turns,
                      float* gain) {
    if (n_rot < 2 || n_rot % 2 != 0 || turns == nullptr || gain == nullptr || !(base > 1.0) || !std::isfinite(base))
        return KVATTN_ERR_INVALID_ARG;
    if (scaling < KVATTN_ROPE_PLAIN || scaling > KVATTN_ROPE_YARN) return KVATTN_ERR_INVALID_ARG;
    if (scaling != KVATTN_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return KVATTN_ERR_INVALID_ARG;
    if (scaling == KVATTN_ROPE_YARN && original_len < 1) return KVATTN_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    *gain = 1.f;
    for (int i = 0; i < n_rot / 2; ++i) {
        double theta = std::pow(base, -2.0 * i / n_rot);
        if (scaling == KVATTN_ROPE_LINEAR) theta /= factor;
        if (scaling == KVATTN_ROPE_YARN) {
            // turns that the pair makes over the original context: pairs below 1 are
            // interpolated, pairs above 32 kept, a ramp between
            const double rounds = (double)original_len * theta / two_pi;
            const double keep = std::min(std::max((rounds - 1.0) / 31.0, 0.0), 1.0);
            theta = theta / factor * (1.0 - keep) + theta * keep;
        }
        // (theta <= 1 rad: below 2^62 of the 2^64 parts of a turn)
        turns[i] = (uint64_t)std::llround(std::ldexp(theta / two_pi, 63)) * 2u;
    }
    if (scaling == KVATTN_ROPE_YARN) *gain = (float)(0.1 * std::log(factor) + 1.0);
    return KVATTN_OK;
}

int kvattn_rope(const void* q, int64_t q_stride, int n_head, const void* k, int64_t k_stride, int n_head_kv,
                const int32_t* positions, const uint64_t* turns, float gain, int n_rot, int layout, int64_t n_tok,
                int head_dim, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
    if (n_tok < 0 || n_head < 0 || n_head_kv < 0 || n_rot < 0 || !std::isfinite(gain)) return KVATTN_ERR_INVALID_ARG;
    if (layout != KVATTN_ROPE_HALF && layout != KVATTN_ROPE_INTERLEAVED) return KVATTN_ERR_INVALID_ARG;
    if (!known_dim(head_dim) || n_rot % 16 != 0) return KVATTN_ERR_UNSUPPORTED;
    if (n_rot > head_dim) return KVATTN_ERR_INVALID_ARG;
    if (n_tok > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    if ((n_head == 0 && n_head_kv == 0) || n_tok == 0) return KVATTN_OK;
    if ((int64_t)n_head + n_head_kv > 65536) return KVATTN_ERR_UNSUPPORTED;
    if (positions == nullptr || !aligned(positions, 4) || (n_rot > 0 && (turns == nullptr || !aligned(turns, 8))))
        return KVATTN_ERR_INVALID_ARG;
    if (n_head > 0 && !(row_ok(q, q_stride, n_head, head_dim) && row_ok(q_out, q_out_stride, n_head, head_dim)))
        return KVATTN_ERR_INVALID_ARG;
    if (n_head_kv > 0 && !(row_ok(k, k_stride, n_head_kv, head_dim) && row_ok(k_out, k_out_stride, n_head_kv, head_dim)))
        return KVATTN_ERR_INVALID_ARG;
    RopeParams p = {};
    p.src[0] = static_cast<const __half*>(q);
    p.src[1] = static_cast<const __half*>(k);
    p.dst[0] = static_cast<__half*>(q_out);
    p.dst[1] = static_cast<__half*>(k_out);
    p.src_stride[0] = q_stride;
    p.src_stride[1] = k_stride;
    p.dst_stride[0] = q_out_stride;
    p.dst_stride[1] = k_out_stride;
    p.n_head[0] = n_head;
    p.n_head[1] = n_head_kv;
    p.pos = positions;
    p.turns = turns;
    p.n_tok = n_tok;
    p.head_dim = head_dim;
    p.n_rot = n_rot;
    p.interleaved = layout == KVATTN_ROPE_INTERLEAVED;
    p.gain = gain;
    return cuda_status(launch_rope(p, device_sms(), static_cast<cudaStream_t>(stream), pdl_enabled()));
}

static int cache_io(bool write, const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int32_t* slots,
                    int64_t n_tok, int n_head_kv, int head_dim, int kv_type, const void* k_cache, const void* v_cache,
                    const void* k_scales, const void* v_scales, int64_t n_cells, uint32_t* status, void* stream) {
    if (n_tok < 0 || n_head_kv < 1 || n_cells < 1) return KVATTN_ERR_INVALID_ARG;
    if (!known_dim(head_dim)) return KVATTN_ERR_UNSUPPORTED;
    // (token, 16-element piece) pairs are numbered in 32 bits
    if (n_tok > INT32_MAX || (int64_t)n_head_kv * head_dim > INT32_MAX ||
        n_tok * ((int64_t)n_head_kv * head_dim / 16) > (int64_t)INT32_MAX)
        return KVATTN_ERR_UNSUPPORTED;
    const int st = check_cache(kv_type, k_cache, v_cache, k_scales, v_scales, head_dim);
    if (st != KVATTN_OK) return st;
    if (slots != nullptr ? !aligned(slots, 4) : n_tok > n_cells) return KVATTN_ERR_INVALID_ARG;
    if (status != nullptr && !aligned(status, 4)) return KVATTN_ERR_INVALID_ARG;
    if (n_tok == 0) return KVATTN_OK;
    if (!row_ok(k, k_stride, n_head_kv, head_dim) || !row_ok(v, v_stride, n_head_kv, head_dim)) return KVATTN_ERR_INVALID_ARG;
    CacheIoParams p = {};
    p.src[0] = static_cast<const __half*>(k);
    p.src[1] = static_cast<const __half*>(v);
    p.dst[0] = static_cast<__half*>(const_cast<void*>(k));
    p.dst[1] = static_cast<__half*>(const_cast<void*>(v));
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.rows[0] = const_cast<void*>(k_cache);
    p.rows[1] = const_cast<void*>(v_cache);
    p.scales[0] = static_cast<__half*>(const_cast<void*>(k_scales));
    p.scales[1] = static_cast<__half*>(const_cast<void*>(v_scales));
    p.slots = slots;
    p.status = status;
    p.n_tok = n_tok;
    p.n_cells = n_cells;
    p.n_head_kv = n_head_kv;
    p.head_dim = head_dim;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(write ? launch_cache_write(p, kv_type, s, pdl_enabled()) : launch_cache_read(p, kv_type, s, pdl_enabled()));
}

int kvattn_cache_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int32_t* slots,
                       int64_t n_tok, int n_head_kv, int head_dim, int kv_type, void* k_cache, void* v_cache,
                       void* k_scales, void* v_scales, int64_t n_cells, uint32_t* status, void* stream) {
    return cache_io(true, k, k_stride, v, v_stride, slots, n_tok, n_head_kv, head_dim, kv_type, k_cache, v_cache, k_scales,
                    v_scales, n_cells, status, stream);
}

int kvattn_cache_read(const void* k_cache, const void* v_cache, const void* k_scales, const void* v_scales, int kv_type,
                      int64_t n_cells, const int32_t* slots, int64_t n_tok, int n_head_kv, int head_dim, void* k,
                      int64_t k_stride, void* v, int64_t v_stride, uint32_t* status, void* stream) {
    return cache_io(false, k, k_stride, v, v_stride, slots, n_tok, n_head_kv, head_dim, kv_type, k_cache, v_cache, k_scales,
                    v_scales, n_cells, status, stream);
}

size_t kvattn_prefill_workspace_bytes(int64_t n_tok, int n_seq, int n_head, int n_head_kv, int head_dim) {
    return check_heads(n_tok, n_seq, n_head, n_head_kv, head_dim) == KVATTN_OK ? kStatusBytes : 0;
}

int kvattn_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                   const int32_t* offsets, int n_seq, int64_t n_tok, int n_head, int n_head_kv, int head_dim, float scale,
                   void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    const int st = check_heads(n_tok, n_seq, n_head, n_head_kv, head_dim);
    if (st != KVATTN_OK) return st;
    if (!std::isfinite(scale)) return KVATTN_ERR_INVALID_ARG;
    if (n_tok == 0 || n_seq == 0) return KVATTN_OK;
    if (!row_ok(q, q_stride, n_head, head_dim) || !row_ok(k, k_stride, n_head_kv, head_dim) ||
        !row_ok(v, v_stride, n_head_kv, head_dim) || offsets == nullptr || !aligned(offsets, 4) || out == nullptr ||
        !aligned(out, 16) || !aligned(lse, 4) || ws == nullptr || !aligned(ws, kWsAlign))
        return KVATTN_ERR_INVALID_ARG;
    if (ws_bytes < kStatusBytes) return KVATTN_ERR_WORKSPACE;
    const int64_t units = unit_bound(n_tok, n_seq, n_head_kv, n_head / n_head_kv, head_dim);
    if (units > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    PrefillParams p = {};
    p.k = k;
    p.v = v;
    p.offsets = offsets;
    p.out = static_cast<__half*>(out);
    p.lse = lse;
    p.status = static_cast<uint32_t*>(ws);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_tok = n_tok;
    p.n_cells = n_tok;
    p.max_len = n_tok;
    p.n_seq = n_seq;
    return launch_attention(p, q, q_stride, KVATTN_KV_F16, n_head, n_head_kv, head_dim, n_tok, scale,
                            cut_of(units, 1, head_dim, false), "prefill", stream);
}

size_t kvattn_prefill_chunk_workspace_bytes(int64_t n_tok, int n_seq, int n_head, int n_head_kv, int head_dim,
                                            int64_t max_len) {
    if (check_heads(n_tok, n_seq, n_head, n_head_kv, head_dim) != KVATTN_OK || max_len < 0 || max_len > INT32_MAX) return 0;
    return chunk_cut(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len, true).total;
}

int kvattn_prefill_chunk(const void* q, int64_t q_stride, const int32_t* offsets, int64_t n_tok, const void* k_cache,
                         const void* v_cache, const void* k_scales, const void* v_scales, int kv_type, int64_t n_cells,
                         const int32_t* cell_plan, int64_t plan_stride, const int32_t* seq_lens, int n_seq,
                         int64_t max_len, int n_head, int n_head_kv, int head_dim, float scale, void* out, float* lse,
                         void* ws, size_t ws_bytes, void* stream) {
    int st = check_heads(n_tok, n_seq, n_head, n_head_kv, head_dim);
    if (st != KVATTN_OK) return st;
    if (max_len < 0 || n_cells < 1 || !std::isfinite(scale) || (cell_plan != nullptr && plan_stride < 1))
        return KVATTN_ERR_INVALID_ARG;
    // (cells are numbered in 63 bits over all sequences)
    if (max_len > INT32_MAX || n_cells > INT64_MAX / std::max(n_seq, 1)) return KVATTN_ERR_UNSUPPORTED;
    st = check_cache(kv_type, k_cache, v_cache, k_scales, v_scales, head_dim);
    if (st != KVATTN_OK) return st;
    if (n_tok == 0 || n_seq == 0) return KVATTN_OK;
    if (!row_ok(q, q_stride, n_head, head_dim) || offsets == nullptr || !aligned(offsets, 4) || seq_lens == nullptr ||
        !aligned(seq_lens, 4) || !aligned(cell_plan, 4) || out == nullptr || !aligned(out, 16) || !aligned(lse, 4) ||
        ws == nullptr || !aligned(ws, kWsAlign))
        return KVATTN_ERR_INVALID_ARG;
    const Cut c = chunk_cut(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len);
    if (unit_bound(n_tok, n_seq, n_head_kv, n_head / n_head_kv, head_dim) > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    if (ws_bytes < c.total) return KVATTN_ERR_WORKSPACE;
    PrefillParams p = {};
    p.k = k_cache;
    p.v = v_cache;
    p.k_scale = static_cast<const __half*>(k_scales);
    p.v_scale = static_cast<const __half*>(v_scales);
    p.offsets = offsets;
    p.plan = cell_plan;
    p.seq_lens = seq_lens;
    p.out = static_cast<__half*>(out);
    p.lse = lse;
    char* wsb = static_cast<char*>(ws);
    p.status = reinterpret_cast<uint32_t*>(wsb);
    p.cuts = reinterpret_cast<PrefillCut*>(wsb + c.cuts_off);
    p.part_lse = reinterpret_cast<float*>(wsb + c.lse_off);
    p.part_o = reinterpret_cast<float*>(wsb + c.o_off);
    p.k_stride = p.v_stride = (int64_t)n_head_kv * head_dim;
    p.n_tok = n_tok;
    p.n_cells = n_cells;
    p.plan_stride = plan_stride;
    p.max_len = max_len;
    p.n_seq = n_seq;
    return launch_attention(p, q, q_stride, kv_type, n_head, n_head_kv, head_dim, cell_plan != nullptr ? n_cells : n_cells * n_seq,
                            scale, c, "prefill_chunk", stream);
}

}  // extern "C"
