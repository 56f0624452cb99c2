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

// With a window: whether `units` units of `tiles` tiles together, the longest of them `longest`, are dealt
// out whole to n CTAs.  They take a round of the longest and the others of the mean, where shares would
// take tiles / n; what is lost is weighed against what cut units cost with their partials and the merge, in
// tiles (cost; the other side in us, whole units and shares, by tiles lost):
//   single tokens, f16 rows of 128 without a plan: 5.7 57 62, 10.4 92 100, 15.2 73 71, 31 89 66;
//   single tokens else: f16 plan 4.0 69 73, 6.9 79 80, 8.0 69 64, 13 99 88; 8-bit rows 3.6 68 73, 5.4 67 67,
//     7.2 68 64, 10.4 122 113; head_dim 256 5.4 92 99, 7.2 92 94, 8.1 79 74, 16 89 68;
//   several tokens: f16 2.8 49 65, 8.5 47 52, 15.2 106 105, 28 248 230, through a plan 8.0 93 102, 9.8 88 92, 18
//     92 79; 8-bit rows 3.6 45 60, 8.1 73 79, 15.2 119 113, through a plan 8.0 105 114, 9.8 96 102, 10.4 68 63;
//     head_dim 256 5.2 89 116, 8.1 85 91, 16 92 84, through a plan 8.0 119 128, 9.8 108 106.
KVATTN_HD bool whole_units(uint32_t units, uint64_t tiles, uint32_t longest, uint32_t n, uint32_t cost) {
    if (units == 0u) return true;
    const uint32_t before_last = (units - 1u) / n * n;   // units of all rounds but the last
    return (uint64_t)longest * units * n <= (uint64_t)cost * units * n + (uint64_t)(units - before_last) * tiles;
}
// `cost`; fast_single: a tile of one row group takes about half the time of one of both (f16 rows of 128
// without a plan).
inline uint32_t cut_cost(int64_t n_tok, int n_seq, bool fast_single) { return n_tok > n_seq ? 10u : (fast_single ? 13u : 7u); }

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
