// Attention with a sliding window and first tokens that stay visible: a token with limit lim sees the
// cells c < lim with c < sinks or c >= lim - window.
//
// A block's places are the first cells and, without the gap that no row of it sees, those from its first
// token's window to its last token's end: (sinks + 31 + window + block) / 128 tiles, however long the
// sequence.  What differs from the plain form: where a unit's places lie; a second bound in the masks,
// which are applied in registers (a third of the tiles have one); up to four more tiles at the front
// that only some rows see whole, whose values that are not finite are kept apart like those at the end;
// and a line in which every unit counts as the longest that its sequence and window allow.  Units of equal
// length are often better dealt out whole than cut: the schedulers decide, from the lengths (whole_units in
// line.cuh).
//
// What bounds it: single tokens the bytes of whole tiles and the rounds of units (64 tokens, window 1024
// and 4 first tokens, 32 / 8 heads of 128: 51 us, 74 % of the copy rate for the cells that they see);
// prompts the ends of their short units, about 8000 clocks beside 3300 a tile (8192 tokens through that
// window 138 us, 49 % of cuBLAS bf16; ragged prompts of 16 / 8 heads of 256, window 500 and 130 first
// tokens, 92 us, 31 %).  Bringing only the blocks of 32 cells that a row of the unit sees gained 1 us for
// the single tokens and cost prompts 3 to 10 %.
#include "prefill_kernel.cuh"

namespace kvattn {

cudaError_t launch_prefill_window(const PrefillParams& p, int kv_type, int head_dim, int n_ctas, cudaStream_t stream, bool pdl) {
    return run_prefill<kWindow>(p, kv_type, head_dim, n_ctas, stream, pdl);
}

}  // namespace kvattn
