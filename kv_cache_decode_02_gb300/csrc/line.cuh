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
