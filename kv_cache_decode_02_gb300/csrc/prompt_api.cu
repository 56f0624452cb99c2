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

// How a call's work is cut.  Units that are many and short are dealt out whole; few or long ones
// (chunks over long caches) are cut into equal shares, one per CTA: 16 units of 1024 tiles would
// otherwise keep 16 of 152 SMs busy.  A share costs its CTA a partial (written and read once
// more) and the call a merge, so a CTA gets at least four tiles' worth of the bound below.
struct Cut {
    bool shares, forced;   // forced: by the environment
    int n_ctas;
    size_t cuts_off, lse_off, o_off, total;
};

constexpr int64_t kMinShareTiles = 4, kFewTiles = 13;

// `bound`: of all calls with at most that many units and tiles (one of fewer units may be shared
// where this one is dealt out whole).
//
// `whole`: with a window units are often about equal, and are dealt out whole where that takes no longer
// (whole_units).  The schedulers decide, who know how many blocks and cells the sequences have: one of 60000
// cells and 18 of 100 behind a window of 8192 take 78 us whole, on 8 SMs, and 23 in shares.  Units of few
// tiles lose little whatever their lengths: they are whole, without a merge to launch, where equal ones
// would be.
Cut cut_of(int64_t units, int64_t tiles, int head_dim, bool may_share, bool bound = false, WholeRule whole = {}) {
    Cut c = {};
    // (KVATTN_PREFILL_CTAS: the CTAs that share the work, for tests; 0: dealt out whole)
    const char* env = std::getenv("KVATTN_PREFILL_CTAS");
    const int sms = device_sms();
    if (bound) units = std::min(units, 8 * (int64_t)sms - 1);
    c.shares = may_share && tiles > kMinShareTiles && units < 8 * (int64_t)sms;
    c.forced = may_share && env != nullptr && *env != 0;
    // (the kernel numbers the line of all tiles, in eighths, in 31 bits)
    const bool fits = bound || (units < INT32_MAX && (tiles + 18) * 8 < INT32_MAX / std::max<int64_t>(units, 1));
    auto ctas = [&](int64_t n) { return (int)std::max<int64_t>(std::min<int64_t>(n, sms), 1); };
    c.n_ctas = ctas(c.shares ? std::max(units, (units * tiles + kMinShareTiles - 1) / kMinShareTiles) : units);
    if (c.shares && whole.base != 0u && tiles <= kFewTiles &&
        whole_units((uint32_t)units, (uint64_t)(units * tiles), (uint32_t)tiles, (uint32_t)c.n_ctas, whole)) {
        c.shares = false;
        c.n_ctas = ctas(units);
    }
    if (c.forced) {
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
    return cut_of(unit_bound(n_tok, n_seq, n_head_kv, block_tokens_of(n_head / n_head_kv, head_dim)),
                  (max_len + kPrefillTile - 1) / kPrefillTile, head_dim, true, bound);
}

// With a window: tiles that the first tokens and the windows of a block meet, at most (window_gap in
// prefill_kernel.cuh; through a plan the window begins anywhere in a tile).
int64_t window_tiles_of(int64_t window, int64_t sinks, int group, int head_dim, bool plan) {
    const int64_t front = plan ? (sinks + kPrefillTile - 1) / kPrefillTile * kPrefillTile + kPrefillTile - 1 : (sinks + 31) / 32 * 32;
    return (front + window + block_tokens_of(group, head_dim) - 1 + kPrefillTile - 1) / kPrefillTile;
}

// With a shared prefix: the line holds the sequences' units and the prefix's, however many, and is always
// cut into shares (a prefix's units are few and long beside the others), but where it would pass 31 bits
// (units are whole then: 65600 tokens, each a block of 128 heads that share one, make 2.15e9 eighths).
struct SharedCut {
    bool shares;
    int n_ctas;
    size_t join_off, note_off, whole_lse_off, whole_o_off, lse_off, o_off, total;
};

SharedCut shared_cut(int64_t n_tok, int n_seq, int n_head, int n_head_kv, int head_dim, int64_t max_len, int64_t prefix_cells) {
    SharedCut c = {};
    const int group = n_head / n_head_kv, block_tokens = block_tokens_of(group, head_dim), sms = device_sms();
    const int64_t units = unit_bound(n_tok, n_seq, n_head_kv, block_tokens);
    const int64_t prefix_units = unit_bound(n_tok, 1, n_head_kv, block_tokens);
    const int64_t prefix_tiles = std::min(prefix_cells, max_len) / kPrefillTile;
    const bool fits = shared_line_fits(n_tok, n_seq, n_head_kv, group, head_dim, max_len, prefix_cells);
    const char* env = std::getenv("KVATTN_PREFILL_CTAS");
    int64_t n = units + prefix_units * (prefix_tiles / kMinShareTiles + 1);
    n = std::max<int64_t>(std::min<int64_t>(n, sms), 1);
    if (env != nullptr && *env != 0 && std::atoi(env) > 0) n = std::min(std::atoi(env), sms);
    c.n_ctas = (int)n;
    c.shares = n > 1 && fits && !(env != nullptr && *env != 0 && std::atoi(env) <= 0);
    // (the parts' room does not go by the lengths, so that a size serves every smaller call)
    const size_t rows = (size_t)sms * 2 * (size_t)prefill_groups(head_dim) * 128;
    const size_t out_rows = 2 * (size_t)n_tok * (size_t)n_head;
    size_t off = kStatusBytes;
    c.join_off = off;
    off = align_up(off + sizeof(uint2), kWsAlign);
    c.note_off = off;
    off = align_up(off + 2 * (size_t)n_tok * (size_t)n_head_kv * sizeof(PrefillNote), kWsAlign);
    c.whole_lse_off = off;
    off = align_up(off + out_rows * 4, kWsAlign);
    c.whole_o_off = off;
    off = align_up(off + out_rows * (size_t)head_dim * 4, kWsAlign);
    c.lse_off = off;
    off = align_up(off + rows * 4, kWsAlign);
    c.o_off = off;
    // (a call that shares no tile is the plain form's, whose notes of cuts can be more than few rows' results)
    c.total = std::max(align_up(off + rows * (size_t)head_dim * 4, kWsAlign),
                       chunk_cut(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len, true).total);
    return c;
}

// What the attention entry points have in common.
enum class Form { plain, window, shared };
int launch_attention(Form form, PrefillParams& p, const void* q, int64_t q_stride, int kv_type, int n_head, int n_head_kv,
                     int head_dim, int64_t rows, float scale, bool shares, int n_ctas, const char* name, void* stream) {
    p.n_head = n_head;
    p.n_head_kv = n_head_kv;
    p.group = n_head / n_head_kv;
    p.group_tokens = 128 / p.group;
    p.block_tokens = p.group_tokens * prefill_groups(head_dim);
    p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    p.single_length = 8;
    if (kv_type == KVATTN_KV_F16 && head_dim == 128) {
        // (64 single tokens behind 8192 shared cells: 52 us at 5, 48 at 4; through a plan 55, 55, 58 at 6)
        if (form == Form::shared)
            p.single_length = p.plan == nullptr ? 4 : 5;
        else if (p.plan == nullptr)
            p.single_length = 5;
    }
    p.shares = shares ? 1 : 0;
    p.out_sectors = aligned(p.out, 32) ? 1 : 0;
    debug_waits(&p.wait_limit_ns, &p.stall_tx);
    if (!encode_prefill_map(&p.tmap_q, q, p.n_tok, n_head, head_dim, q_stride, p.group, p.group_tokens)) return KVATTN_ERR_CUDA;
    // (a window's first tile is brought in parts, by maps with smaller boxes)
    const bool parts = form == Form::window && p.plan == nullptr;
    if (kv_type == KVATTN_KV_F16) {
        auto planes = [&](CUtensorMap* m, const void* x, int64_t stride, int box_rows, int box_planes) {
            return encode_planes_map(m, x, rows, n_head_kv, head_dim, stride, box_rows, box_planes);
        };
        p.use_tma = planes(&p.tmap_k, p.k, p.k_stride, kPrefillTile, 2) && planes(&p.tmap_v, p.v, p.v_stride, kPrefillTile, 2) &&
                    (!parts || (planes(&p.tmap_k32, p.k, p.k_stride, 32, 1) && planes(&p.tmap_v32, p.v, p.v_stride, 32, 1)));
    } else {
        const int kb = kv_type == KVATTN_KV_Q4_0 ? 4 : 8, vb = kv_type == KVATTN_KV_Q8_0 ? 8 : 4;
        auto codes = [&](CUtensorMap* m, const void* x, int bits, int box_rows) {
            return encode_codes_map(m, x, rows, n_head_kv, head_dim * bits / 8, 16 * bits, box_rows);
        };
        p.use_tma = codes(&p.tmap_k, p.k, kb, kPrefillTile) && codes(&p.tmap_v, p.v, vb, kPrefillTile) &&
                    (!parts || (codes(&p.tmap_k32, p.k, kb, 32) && codes(&p.tmap_v32, p.v, vb, 32)));
        p.scl_tma = p.use_tma != 0 && rows <= (int64_t)INT32_MAX &&
                    encode_scale_tensor_map(&p.tmap_ks, p.k_scale, rows, n_head_kv, head_dim, kPrefillTile) &&
                    encode_scale_tensor_map(&p.tmap_vs, p.v_scale, rows, n_head_kv, head_dim, kPrefillTile);
    }
    if (!tma_enabled()) p.use_tma = p.scl_tma = 0;
    if (log_enabled()) {
        char buf[256];
        std::snprintf(buf, sizeof(buf), "%s kv_type=%d n_seq=%d n_tok=%lld n_head=%d/%d head_dim=%d plan=%d shares=%d grid=%d tma=%d",
                      name, kv_type, p.n_seq, (long long)p.n_tok, n_head, n_head_kv, head_dim, p.plan != nullptr, p.shares,
                      n_ctas, p.use_tma);
        log_text(buf);
    }
    const auto launch = form == Form::plain ? launch_prefill : (form == Form::window ? launch_prefill_window : launch_prefill_shared);
    return cuda_status(launch(p, kv_type, head_dim, n_ctas, static_cast<cudaStream_t>(stream), pdl_enabled()));
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

int kvattn_rope_axes(int n_rot, const int32_t* sections, int n_axes, int order, uint8_t* axis) {
    if (n_rot < 2 || n_rot % 2 != 0 || n_axes < 1 || sections == nullptr || axis == nullptr) return KVATTN_ERR_INVALID_ARG;
    if (order != KVATTN_AXES_BLOCKS && order != KVATTN_AXES_CYCLE) return KVATTN_ERR_INVALID_ARG;
    if (n_axes > kMaxAxes) return KVATTN_ERR_UNSUPPORTED;
    int64_t sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 0) return KVATTN_ERR_INVALID_ARG;
        sum += sections[a];
    }
    if (sum != n_rot / 2) return KVATTN_ERR_INVALID_ARG;
    int pair = 0;
    if (order == KVATTN_AXES_BLOCKS) {
        for (int a = 0; a < n_axes; ++a)
            for (int i = 0; i < sections[a]; ++i) axis[pair++] = (uint8_t)a;
    } else {
        for (int i = 0; pair < n_rot / 2; ++i)
            for (int a = 0; a < n_axes; ++a)
                if (i < sections[a]) axis[pair++] = (uint8_t)a;
    }
    return KVATTN_OK;
}

int kvattn_norm_rope(const void* q, int64_t q_stride, int n_head, const void* q_weight, const void* k, int64_t k_stride,
                     int n_head_kv, const void* k_weight, float eps, const int32_t* positions, int64_t pos_stride, int n_axes,
                     const uint8_t* axis, const uint64_t* turns, float gain, int n_rot, int layout, int64_t n_tok, int head_dim,
                     void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
    if (n_tok < 0 || n_head < 0 || n_head_kv < 0 || n_rot < 0 || !std::isfinite(gain) || !(eps >= 0.f) || !std::isfinite(eps))
        return KVATTN_ERR_INVALID_ARG;
    if (layout != KVATTN_ROPE_HALF && layout != KVATTN_ROPE_INTERLEAVED) return KVATTN_ERR_INVALID_ARG;
    if (n_axes < 1) return KVATTN_ERR_INVALID_ARG;
    if (!known_dim(head_dim) || n_rot % 16 != 0 || n_axes > kMaxAxes) return KVATTN_ERR_UNSUPPORTED;
    if (n_rot > head_dim) return KVATTN_ERR_INVALID_ARG;
    if (n_tok > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    if ((n_head == 0 && n_head_kv == 0) || n_tok == 0) return KVATTN_OK;
    if ((int64_t)n_head + n_head_kv > 65536) return KVATTN_ERR_UNSUPPORTED;
    if (n_rot > 0 && (positions == nullptr || !aligned(positions, 4) || turns == nullptr || !aligned(turns, 8)))
        return KVATTN_ERR_INVALID_ARG;
    if (n_rot > 0 && n_axes > 1 && (axis == nullptr || !aligned(axis, 8) || pos_stride < n_tok)) return KVATTN_ERR_INVALID_ARG;
    if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return KVATTN_ERR_INVALID_ARG;
    if (n_head > 0 && !(row_ok(q, q_stride, n_head, head_dim) && row_ok(q_out, q_out_stride, n_head, head_dim)))
        return KVATTN_ERR_INVALID_ARG;
    if (n_head_kv > 0 && !(row_ok(k, k_stride, n_head_kv, head_dim) && row_ok(k_out, k_out_stride, n_head_kv, head_dim)))
        return KVATTN_ERR_INVALID_ARG;
    NormRopeParams p = {};
    p.r.src[0] = static_cast<const __half*>(q);
    p.r.src[1] = static_cast<const __half*>(k);
    p.r.dst[0] = static_cast<__half*>(q_out);
    p.r.dst[1] = static_cast<__half*>(k_out);
    p.r.src_stride[0] = q_stride;
    p.r.src_stride[1] = k_stride;
    p.r.dst_stride[0] = q_out_stride;
    p.r.dst_stride[1] = k_out_stride;
    p.r.n_head[0] = n_head;
    p.r.n_head[1] = n_head_kv;
    p.r.pos = positions;
    p.r.turns = turns;
    p.r.n_tok = n_tok;
    p.r.head_dim = head_dim;
    p.r.n_rot = n_rot;
    p.r.interleaved = layout == KVATTN_ROPE_INTERLEAVED;
    p.r.gain = gain;
    p.weight[0] = n_head > 0 ? static_cast<const __half*>(q_weight) : nullptr;
    p.weight[1] = n_head_kv > 0 ? static_cast<const __half*>(k_weight) : nullptr;
    p.axis = axis;
    p.pos_stride = pos_stride;
    p.n_axes = n_axes;
    p.eps = eps;
    return cuda_status(launch_norm_rope(p, device_sms(), static_cast<cudaStream_t>(stream), pdl_enabled()));
}

int kvattn_step_maps(const int32_t* lens, const int32_t* n_new, int n_seq, int32_t* tables, int64_t table_stride, int block_cells,
                     const int32_t* free_blocks, int64_t n_list, const int32_t* n_free, int64_t n_cells, int64_t n_tok,
                     int32_t* offsets, int32_t* seq_lens, int32_t* positions, int32_t* slots, int32_t* n_free_out,
                     int32_t* cell_plan, int64_t plan_stride, int whole_plan, uint32_t* status, void* stream) {
    if (n_seq < 0 || table_stride < 0 || n_list < 0 || n_cells < 0 || n_tok < 0 || block_cells < 1 ||
        (cell_plan != nullptr && plan_stride < 0))
        return KVATTN_ERR_INVALID_ARG;
    if ((block_cells & (block_cells - 1)) != 0 || block_cells < 4 || block_cells > 65536 || n_seq > kMaxMapSequences ||
        n_cells > INT32_MAX || n_tok > INT32_MAX || n_list > INT32_MAX || (cell_plan != nullptr && plan_stride > INT32_MAX))
        return KVATTN_ERR_UNSUPPORTED;
    if (offsets == nullptr || !aligned(offsets, 4) || !aligned(positions, 4) || (n_tok > 0 && slots == nullptr) ||
        !aligned(slots, 4) || !aligned(cell_plan, 4) || !aligned(status, 4))
        return KVATTN_ERR_INVALID_ARG;
    if (n_seq > 0 && (lens == nullptr || n_new == nullptr || tables == nullptr || seq_lens == nullptr || !aligned(lens, 4) ||
                      !aligned(n_new, 4) || !aligned(tables, 4) || !aligned(seq_lens, 4)))
        return KVATTN_ERR_INVALID_ARG;
    // (blocks are taken: all three; or the tables hold all that is needed: none of them)
    if (free_blocks != nullptr ? n_free == nullptr || n_free_out == nullptr || !aligned(free_blocks, 4) || !aligned(n_free, 4) ||
                                     !aligned(n_free_out, 4)
                               : n_free != nullptr || n_free_out != nullptr)
        return KVATTN_ERR_INVALID_ARG;
    // threads read the lengths and the count while others write theirs
    if (n_seq > 0 && (seq_lens == lens || seq_lens == n_new)) return KVATTN_ERR_INVALID_ARG;
    if (n_free != nullptr && n_free_out == n_free) return KVATTN_ERR_INVALID_ARG;
    StepMapsParams p = {};
    p.lens = lens;
    p.n_new = n_new;
    p.tables = tables;
    p.free_list = free_blocks;
    p.n_free = n_free;
    p.offsets = offsets;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.slots = slots;
    p.n_free_out = n_free_out;
    p.plan = cell_plan;
    p.status = status;
    p.table_stride = table_stride;
    p.plan_stride = plan_stride;
    p.n_list = n_list;
    p.n_cells = n_cells;
    p.n_tok = n_tok;
    p.n_seq = n_seq;
    p.whole = whole_plan != 0;
    while ((1 << p.block_shift) < block_cells) ++p.block_shift;
    p.max_len = std::min<int64_t>(table_stride, INT32_MAX >> p.block_shift) << p.block_shift;
    if (cell_plan != nullptr) p.max_len = std::min(p.max_len, plan_stride);
    return cuda_status(launch_step_maps(p, static_cast<cudaStream_t>(stream), pdl_enabled()));
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

// window 0: none
static int prompt_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const int32_t* offsets, int n_seq, int64_t n_tok, int n_head, int n_head_kv, int head_dim,
                            float scale, int64_t window, int64_t sinks, void* out, float* lse, void* ws, size_t ws_bytes,
                            void* stream) {
    const int st = check_heads(n_tok, n_seq, n_head, n_head_kv, head_dim);
    if (st != KVATTN_OK) return st;
    if (!std::isfinite(scale)) return KVATTN_ERR_INVALID_ARG;
    if (n_tok == 0 || n_seq == 0) return KVATTN_OK;
    if (!row_ok(q, q_stride, n_head, head_dim) || !row_ok(k, k_stride, n_head_kv, head_dim) ||
        !row_ok(v, v_stride, n_head_kv, head_dim) || offsets == nullptr || !aligned(offsets, 4) || out == nullptr ||
        !aligned(out, 16) || !aligned(lse, 4) || ws == nullptr || !aligned(ws, kWsAlign))
        return KVATTN_ERR_INVALID_ARG;
    if (ws_bytes < kStatusBytes) return KVATTN_ERR_WORKSPACE;
    const int64_t units = unit_bound(n_tok, n_seq, n_head_kv, block_tokens_of(n_head / n_head_kv, head_dim));
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
    const Cut c = cut_of(units, 1, head_dim, false);
    // (a window that holds the longest sequence is none)
    const bool windowed = window > 0 && window < n_tok;
    if (windowed) {
        p.window = window;
        p.sinks = std::min(sinks, n_tok);
        p.window_tiles = (int)window_tiles_of(p.window, p.sinks, n_head / n_head_kv, head_dim, false);
    }
    return launch_attention(windowed ? Form::window : Form::plain, p, q, q_stride, KVATTN_KV_F16, n_head, n_head_kv, head_dim, n_tok,
                            scale, c.shares, c.n_ctas, windowed ? "prefill_window" : "prefill", stream);
}

int kvattn_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                   const int32_t* offsets, int n_seq, int64_t n_tok, int n_head, int n_head_kv, int head_dim, float scale,
                   void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    return prompt_attention(q, q_stride, k, k_stride, v, v_stride, offsets, n_seq, n_tok, n_head, n_head_kv, head_dim, scale, 0, 0,
                            out, lse, ws, ws_bytes, stream);
}

int kvattn_prefill_window(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const int32_t* offsets, int n_seq, int64_t n_tok, int n_head, int n_head_kv, int head_dim, float scale,
                          int64_t window, int64_t sinks, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    if (window < 1 || sinks < 0) return KVATTN_ERR_INVALID_ARG;
    return prompt_attention(q, q_stride, k, k_stride, v, v_stride, offsets, n_seq, n_tok, n_head, n_head_kv, head_dim, scale,
                            window, sinks, out, lse, ws, ws_bytes, stream);
}

size_t kvattn_prefill_chunk_workspace_bytes(int64_t n_tok, int n_seq, int n_head, int n_head_kv, int head_dim,
                                            int64_t max_len) {
    if (check_heads(n_tok, n_seq, n_head, n_head_kv, head_dim) != KVATTN_OK || max_len < 0 || max_len > INT32_MAX) return 0;
    return chunk_cut(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len, true).total;
}

size_t kvattn_prefill_chunk_shared_workspace_bytes(int64_t n_tok, int n_seq, int n_head, int n_head_kv, int head_dim,
                                                   int64_t max_len) {
    if (check_heads(n_tok, n_seq, n_head, n_head_kv, head_dim) != KVATTN_OK || max_len < 0 || max_len > INT32_MAX) return 0;
    return shared_cut(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len, max_len).total;
}

// Form::window: window, sinks; Form::shared: prefix_cells.
static int chunk_attention(Form form, const void* q, int64_t q_stride, const int32_t* offsets, int64_t n_tok, const void* k_cache,
                           const void* v_cache, const void* k_scales, const void* v_scales, int kv_type, int64_t n_cells,
                           const int32_t* cell_plan, int64_t plan_stride, const int32_t* seq_lens, int n_seq, int64_t max_len,
                           int n_head, int n_head_kv, int head_dim, float scale, int64_t window, int64_t sinks,
                           int64_t prefix_cells, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
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
    const int group = n_head / n_head_kv;
    const int64_t units = unit_bound(n_tok, n_seq, n_head_kv, block_tokens_of(group, head_dim));
    if (units > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    if (form == Form::window && window >= max_len) form = Form::plain;   // (it holds all that there is)
    const SharedCut sc = form == Form::shared ? shared_cut(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len, prefix_cells) : SharedCut{};
    if (form == Form::shared && ws_bytes < sc.total) return KVATTN_ERR_WORKSPACE;
    if (form == Form::shared && std::min(prefix_cells, max_len) < kPrefillTile) form = Form::plain;   // (no tile is shared)
    PrefillParams p = {};
    char* wsb = static_cast<char*>(ws);
    bool shares;
    int n_ctas;
    if (form == Form::shared) {
        const SharedCut& c = sc;
        if (units + unit_bound(n_tok, 1, n_head_kv, block_tokens_of(group, head_dim)) > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
        shares = c.shares;
        n_ctas = c.n_ctas;
        p.prefix_cells = prefix_cells;
        p.join = reinterpret_cast<uint2*>(wsb + c.join_off);
        p.notes = reinterpret_cast<PrefillNote*>(wsb + c.note_off);
        p.whole_lse = reinterpret_cast<float*>(wsb + c.whole_lse_off);
        p.whole_o = reinterpret_cast<float*>(wsb + c.whole_o_off);
        p.part_lse = reinterpret_cast<float*>(wsb + c.lse_off);
        p.part_o = reinterpret_cast<float*>(wsb + c.o_off);
    } else {
        int64_t tiles = (max_len + kPrefillTile - 1) / kPrefillTile;
        if (form == Form::window) {
            p.window = window;
            p.sinks = std::min(sinks, max_len);
            p.window_tiles = (int)window_tiles_of(p.window, p.sinks, group, head_dim, cell_plan != nullptr);
            tiles = std::min<int64_t>(tiles, p.window_tiles);
        }
        const bool fast_single = kv_type == KVATTN_KV_F16 && head_dim == 128 && cell_plan == nullptr;
        const bool windowed = form == Form::window;
        auto rule = [&](bool merged) { return windowed ? whole_rule(n_tok, n_seq, fast_single, merged, device_sms()) : WholeRule{}; };
        const Cut c = cut_of(units, tiles, head_dim, true, false, rule(false));
        if (!c.forced) p.whole = rule(true);
        if (ws_bytes < c.total) return KVATTN_ERR_WORKSPACE;
        shares = c.shares;
        n_ctas = c.n_ctas;
        p.cuts = reinterpret_cast<PrefillCut*>(wsb + c.cuts_off);
        p.part_lse = reinterpret_cast<float*>(wsb + c.lse_off);
        p.part_o = reinterpret_cast<float*>(wsb + c.o_off);
    }
    p.k = k_cache;
    p.v = v_cache;
    p.k_scale = static_cast<const __half*>(k_scales);
    p.v_scale = static_cast<const __half*>(v_scales);
    p.offsets = offsets;
    p.plan = cell_plan;
    p.seq_lens = seq_lens;
    p.out = static_cast<__half*>(out);
    p.lse = lse;
    p.status = reinterpret_cast<uint32_t*>(wsb);
    p.k_stride = p.v_stride = (int64_t)n_head_kv * head_dim;
    p.n_tok = n_tok;
    p.n_cells = n_cells;
    p.plan_stride = plan_stride;
    p.max_len = max_len;
    p.n_seq = n_seq;
    const char* name = form == Form::plain ? "prefill_chunk" : (form == Form::window ? "prefill_chunk_window" : "prefill_chunk_shared");
    return launch_attention(form, p, q, q_stride, kv_type, n_head, n_head_kv, head_dim, cell_plan != nullptr ? n_cells : n_cells * n_seq,
                            scale, shares, n_ctas, name, stream);
}

int kvattn_prefill_chunk(const void* q, int64_t q_stride, const int32_t* offsets, int64_t n_tok, const void* k_cache,
                         const void* v_cache, const void* k_scales, const void* v_scales, int kv_type, int64_t n_cells,
                         const int32_t* cell_plan, int64_t plan_stride, const int32_t* seq_lens, int n_seq,
                         int64_t max_len, int n_head, int n_head_kv, int head_dim, float scale, void* out, float* lse,
                         void* ws, size_t ws_bytes, void* stream) {
    return chunk_attention(Form::plain, q, q_stride, offsets, n_tok, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells,
                           cell_plan, plan_stride, seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, scale, 0, 0, 0, out, lse,
                           ws, ws_bytes, stream);
}

int kvattn_prefill_chunk_window(const void* q, int64_t q_stride, const int32_t* offsets, int64_t n_tok, const void* k_cache,
                                const void* v_cache, const void* k_scales, const void* v_scales, int kv_type, int64_t n_cells,
                                const int32_t* cell_plan, int64_t plan_stride, const int32_t* seq_lens, int n_seq,
                                int64_t max_len, int n_head, int n_head_kv, int head_dim, float scale, int64_t window,
                                int64_t sinks, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    if (window < 1 || sinks < 0) return KVATTN_ERR_INVALID_ARG;
    return chunk_attention(Form::window, q, q_stride, offsets, n_tok, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells,
                           cell_plan, plan_stride, seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, scale, window, sinks, 0,
                           out, lse, ws, ws_bytes, stream);
}

int kvattn_prefill_chunk_shared(const void* q, int64_t q_stride, const int32_t* offsets, int64_t n_tok, const void* k_cache,
                                const void* v_cache, const void* k_scales, const void* v_scales, int kv_type, int64_t n_cells,
                                const int32_t* cell_plan, int64_t plan_stride, const int32_t* seq_lens, int n_seq,
                                int64_t max_len, int n_head, int n_head_kv, int head_dim, float scale, int64_t prefix_cells,
                                void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    if (prefix_cells < 0) return KVATTN_ERR_INVALID_ARG;
    return chunk_attention(Form::shared, q, q_stride, offsets, n_tok, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells,
                           cell_plan, plan_stride, seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, scale, 0, 0,
                           std::min<int64_t>(prefix_cells, INT32_MAX), out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
