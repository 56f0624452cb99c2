// Prompt-side operators: rotary positions (rope.cu), the cache written in its stored type and
// read back (cache_io.cu), and causal attention of many query tokens per sequence (prefill.cu).
// prompt_api.cu holds their C entry points.
#pragma once

#include "kvattn_internal.cuh"

namespace kvattn {

// ---- rotary positions ----
struct RopeParams {
    const __half* src[2];     // q, k: half [n_tok] rows of n_head[i] x head_dim, token stride[i]
    __half* dst[2];
    int64_t src_stride[2], dst_stride[2];
    int n_head[2];
    const int32_t* pos;       // [n_tok]
    const uint64_t* turns;    // [n_rot / 2]: the angle per position of each pair, in 2^-64 turns
    int64_t n_tok;
    int head_dim, n_rot, interleaved;
    float gain;               // multiplies cosine and sine
};
cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t stream, bool pdl);

// ---- cache rows in their stored type ----
struct CacheIoParams {
    const __half* src[2];     // write: new k, v rows, token stride
    __half* dst[2];           // read: half rows, token stride
    int64_t stride[2];
    void* rows[2];            // the cache's K and V planes
    __half* scales[2];        // null for f16
    const int32_t* slots;     // [n_tok], or null: cell t
    uint32_t* status;         // nullable: KVATTN_DEVICE_BAD_PLAN_ENTRY is or-ed in
    int64_t n_tok, n_cells;
    int n_head_kv, head_dim;
};
cudaError_t launch_cache_write(const CacheIoParams& p, int kv_type, cudaStream_t stream, bool pdl);
cudaError_t launch_cache_read(const CacheIoParams& p, int kv_type, cudaStream_t stream, bool pdl);

// ---- causal attention of packed query tokens ----
struct PrefillCut {          // a work unit that the shares cut (n_parts > 0), noted by the CTA that began it
    int64_t q_tok;           // its first token
    int32_t n_parts, n_tok, g, tiles;
    uint32_t start, end;     // its part of the line
};
struct PrefillParams {
    // use_tma: f16 rows (encode_planes_map), or codes (encode_codes_map), boxes of 128 dims x 128
    // cells
    CUtensorMap tmap_k, tmap_v;
    CUtensorMap tmap_q;       // 3-D {head_dim, heads, tokens}, boxes {64, group, group_tokens}
    const void* k;            // f16: rows k_stride elements apart; quantised: dense planes
    const void* v;
    const __half* k_scale;
    const __half* v_scale;
    const int32_t* offsets;   // [n_seq + 1]
    const int32_t* plan;      // nullable: [n_seq][plan_stride]
    const int32_t* seq_lens;  // null: a sequence's cells are its own tokens
    __half* out;              // [n_tok][n_head][head_dim]
    float* lse;               // nullable: [n_tok][n_head]
    PrefillCut* cuts;         // [CTAs], when shares
    float* part_o;            // [2 CTAs][row groups][128][head_dim], when shares
    float* part_lse;          // [2 CTAs][row groups][128]
    uint32_t* status;
    int64_t k_stride, v_stride;
    int64_t n_tok, n_cells, plan_stride, max_len;
    uint64_t wait_limit_ns;
    uint32_t stall_tx;        // test hook: extra bytes expected on the first slot (never arrive)
    int n_seq, n_head, n_head_kv, group;
    int group_tokens;         // tokens of a row group: floor(128 / group)
    int block_tokens;         // tokens of a unit: two row groups at head_dim 128, one at 256
    int single_length;        // of a tile for one row group in the line of shares, in eighths of one for all
    int shares;               // 1: equal shares of all units' tiles, cut anywhere; 0: whole units
    int use_tma;
    int out_sectors;          // out is 32-byte aligned
    float scale_log2;         // scale * log2(e)
};
constexpr int kPrefillTile = 128;  // cells per tile
inline int prefill_groups(int head_dim) { return head_dim == 128 ? 2 : 1; }
// The attention kernel on n_ctas CTAs (at most one per SM) and, with shares, the merge.
cudaError_t launch_prefill(const PrefillParams& p, int kv_type, int head_dim, int n_ctas, cudaStream_t stream, bool pdl);

// From api.cu: a 3-D map {head_dim, heads, rows} of half rows with boxes {64, box_heads, box_rows}
// and the 128-byte swizzle, SM count, log switch and line, the programmatic-launch switch, the
// limit on waits and its test hook.
bool encode_prefill_map(CUtensorMap* map, const void* base, int64_t rows, int n_head, int head_dim, int64_t row_stride,
                        int box_heads, int box_rows);
// The 4-D map {64, rows, head_dim / 64 planes, KV heads} of half rows, boxes {64, 128, 2, 1} with
// the 128-byte swizzle: 128 cells x 128 dims as two planes in one copy.
bool encode_planes_map(CUtensorMap* map, const void* base, int64_t rows, int n_head_kv, int head_dim, int64_t row_stride);
// The 3-D map {row bytes, KV heads, rows} of a plane of codes, boxes {box_bytes, 1, box_rows}.
bool encode_codes_map(CUtensorMap* map, const void* base, int64_t rows, int n_head_kv, int row_bytes, int box_bytes,
                      int box_rows);
bool tma_enabled();
int device_sms();
bool log_enabled();
void log_text(const char* text);
bool pdl_enabled();
void debug_waits(uint64_t* wait_limit_ns, uint32_t* stall_tx);

}  // namespace kvattn
