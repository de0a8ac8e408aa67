// pkv_prompt.cuh -- the work list of prompt attention, shared by its passes (pkv_prompt.cu).
//
// Sequence b has n_b query tokens, the last n_b of its T_b tokens (packed calls: T_b keys of its
// own); query i is at position T_b - n_b + i.  A kv head's group of query heads is served in
// `chunks` of `heads` heads; a row of a chunk is one (token, head), token-major, and an item is up
// to 2 * kRowTile rows of consecutive tokens of one sequence, in two streams of stream_tokens
// tokens each, with the range of 128-token tiles that some of its rows sees.  Items are the same for every kv head and chunk, so
// the list holds them once and work unit w is item w / units, head unit w % units.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// Tokens that a query at position pos sees: [lo, hi).
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
