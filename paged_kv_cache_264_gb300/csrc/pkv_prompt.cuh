// pkv_prompt.cuh -- the work list of prompt attention, shared by its passes (pkv_prompt.cu).
//
// Sequence b has n_b query tokens, the last n_b of its T_b tokens (packed calls: T_b keys of its
// own); query i is at position T_b - n_b + i.  A kv head's group of query heads is served in
// `chunks` of `heads` heads, each a head unit; a row of a unit is one (token, head), token-major.  An item is
// up to 2 * stream_tokens consecutive tokens of one sequence, whose rows form two streams of up to kRowTile, and
// the 128-token tiles that some of its tokens sees.  A unit of work is an item and a head unit; a piece some of its
// tiles, which leaves a partial softmax state per row.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// Tokens that queries at positions first_pos to last_pos see: [lo, hi).
struct PromptSpan {
  int lo, hi;
};
__device__ __forceinline__ PromptSpan prompt_span(const PromptParams& p, int first_pos, int last_pos, int len) {
  return {max(0, first_pos - p.window + 1), p.causal ? min(len, last_pos + 1) : len};
}
// Tiles of a span: [first, first + count).
__device__ __forceinline__ void span_tiles(PromptSpan s, int& first, int& count) {
  first = s.lo / kPromptTile;
  count = s.hi > s.lo ? (s.hi + kPromptTile - 1) / kPromptTile - first : 0;
}

}  // namespace pkv
