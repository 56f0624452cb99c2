// Work units of attention, and the line that equal shares are cut from: the rules that the host bounds
// and the kernel's schedulers and merges compute.  Plain C++ as well as CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

#if defined(__CUDACC__)
#define KVATTN_HD __host__ __device__ __forceinline__
#else
#define KVATTN_HD inline
#endif

namespace kvattn {

constexpr int kPrefillTile = 128;  // cells per tile
constexpr int kUnitCost = 2;       // a unit's fixed cost in tiles

inline int prefill_groups(int head_dim) { return head_dim == 128 ? 2 : 1; }
inline int block_tokens_of(int group, int head_dim) { return 128 / group * prefill_groups(head_dim); }

// Units of all sequences together: at most one part-filled block per sequence.
inline int64_t unit_bound(int64_t n_tok, int n_seq, int n_head_kv, int block_tokens) {
    return std::min((n_tok + block_tokens - 1) / block_tokens + std::max(n_seq - 1, 0), n_tok) * n_head_kv;
}

// The blocks of one sequence and KV head, in eighths of a tile: each a unit's fixed cost, then its tiles
// (by a rule that is linear in the block's number, so that sums have a closed form; the last share of a
// unit takes what is left).
struct Line {
    uint32_t a, step;       // length of block b: a + step b,
    uint32_t blocks, less;  // the last one's less this
    KVATTN_HD uint32_t of(uint32_t b) const { return a + step * b - (b + 1u == blocks ? less : 0u); }
    KVATTN_HD uint32_t upto(uint32_t b) const { return a * b + step * (b * (b - 1u) / 2u) - (b == blocks ? less : 0u); }
};
// A causal block of n tokens ends n / 128 tiles behind the one before it: n / 16 eighths, rounded up.
KVATTN_HD uint32_t line_step(int block_tokens) { return (uint32_t)(block_tokens + 15) / 16u; }

// With a window: when units are dealt out whole.  They take a round of the longest and the others of the
// mean, where shares would take tiles / n; what is lost is weighed against what cut units cost with their
// partials and the merge: base tiles, and up to `more` the more units there are to cut.  Measured, in us
// whole and in shares, of equal units on 152 SMs (units x tiles, tiles lost):
//   single tokens, f16 rows of 128 without a plan (whose tiles are short): 16 x 12 (8.0) 21 17, 64 x 9 (5.2) 17 19,
//     96 x 17 (6.3) 27 30, 512 x 9 (5.7) 57 63, 256 x 33 (10.4) 92 100, 320 x 17 (15) 73 71, 160 x 33 (31) 89 66;
//   single tokens else: 64 x 6 (3.5) 18 20, 128 x 17 (2.7) 38 42, 272 x 17 (3.6) 68 73, 256 x 17 (5.4) 68 67, 240 x
//     17 (7.2) 68 64, through a plan 272 x 19 (4.0) 69 73, 240 x 19 (8.0) 69 64, 352 x 19 (13) 99 88;
//   several tokens: 64 x 9 (5.2) 25 34, 64 x 17 (9.8) 38 41, 256 x 9 (2.8) 49 65, 160 x 17 (16) 72 68, through a plan
//     320 x 11 (9.8) 88 92; 8-bit rows 112 x 33 (8.7) 75 81, 160 x 11 (10.4) 68 63; head_dim 256 8 x 12 (8.0) 34 25,
//     128 x 33 (5.2) 89 116, 240 x 17 (7.2) 96 113, 160 x 17 (16) 92 84.
struct WholeRule {
    uint32_t base, more;   // tiles; base 0: shares
    uint32_t sms;
};
// `units` units of `tiles` tiles together, the longest of them `longest`, and n CTAs for them.
KVATTN_HD bool whole_units(uint32_t units, uint64_t tiles, uint32_t longest, uint32_t n, const WholeRule& r) {
    if (units == 0u) return true;
    const uint32_t before_last = (units - 1u) / n * n;   // units of all rounds but the last
    const uint64_t cost = (uint64_t)r.base * r.sms + (uint64_t)r.more * (units < r.sms ? units : r.sms);
    return (uint64_t)longest * r.sms * units * n <= cost * units * n + (uint64_t)(units - before_last) * tiles * r.sms;
}
// fast_single: f16 rows of 128 without a plan; merged: the merge is launched all the same (2 us for single
// tokens, 4 for several).
inline WholeRule whole_rule(int64_t n_tok, int n_seq, bool fast_single, bool merged, int sms) {
    const uint32_t less = merged ? 1u : 0u;
    if (n_tok > n_seq) return WholeRule{4u - less, 8u, (uint32_t)sms};
    return fast_single ? WholeRule{5u - less, 7u, (uint32_t)sms} : WholeRule{4u - less, 3u, (uint32_t)sms};
}

// Whether the line of a call with a shared prefix stays below 2^31, whatever its sequences' lengths.  Then
// Line's 32 bits hold every part of it, b (b - 1) among them: that is below 2^32 where its half is below
// 2^31.  (Blocks all of one sequence make the longest line: b (b - 1) / 2 of a sum is at least the sum of
// each one's.)
inline bool shared_line_fits(int64_t n_tok, int n_seq, int n_head_kv, int group, int head_dim, int64_t max_len, int64_t prefix_cells) {
    const int64_t most = INT32_MAX;
    const int block_tokens = block_tokens_of(group, head_dim);
    const int64_t own = unit_bound(n_tok, n_seq, 1, block_tokens), prefix = unit_bound(n_tok, 1, 1, block_tokens);
    if ((own + prefix) * n_head_kv > most / (8 * kUnitCost)) return false;   // (and what follows fits 64 bits)
    // (a first block ends in front of its sequence's end, or with its own tokens)
    const int64_t tiles = (std::max<int64_t>(max_len, block_tokens) + kPrefillTile - 1) / kPrefillTile;
    const int64_t prefix_tiles = std::min(prefix_cells, max_len) / kPrefillTile;
    const int64_t length = own * 8 * (kUnitCost + tiles) + (int64_t)line_step(block_tokens) * (own * (own - 1) / 2) +
                           prefix * 8 * (kUnitCost + prefix_tiles);
    return length <= most / n_head_kv;
}

}  // namespace kvattn
