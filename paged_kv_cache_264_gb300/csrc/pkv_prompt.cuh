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

struct PromptSeq {
  int row0, n, len, key0;
};
// Sequence b; false where its starts are invalid.  len is 0 where its length is.
__device__ __forceinline__ bool prompt_seq(const PromptParams& p, int b, PromptSeq& s, bool& bad_len) {
  s.row0 = __ldg(p.query_starts + b);
  const int end = __ldg(p.query_starts + b + 1);
  s.n = end - s.row0;
  s.key0 = 0;
  bad_len = false;
  if (s.row0 < 0 || end < s.row0 || end > p.num_tokens) return false;
  if (p.paged) {
    s.len = __ldg(p.context_lens + b);
    if (s.n > 0 && (s.len < s.n || s.len > p.max_context_len)) {
      bad_len = true;
      s.len = 0;
    }
    return true;
  }
  s.key0 = __ldg(p.key_starts + b);
  const int key1 = __ldg(p.key_starts + b + 1);
  s.len = key1 - s.key0;
  return s.key0 >= 0 && key1 >= s.key0 && key1 <= p.num_keys;
}

// Item `index` of sequence b's `count`.
__device__ __forceinline__ PromptItem sequence_item(const PromptParams& p, const PromptSeq& s, int b, int count, int index) {
  const int per = 2 * p.stream_tokens, tok0 = index * per;
  PromptItem x{};
  x.seq = b;
  x.row0 = s.row0 + tok0;
  x.ntok = min(per, s.n - tok0);
  x.pos0 = s.len - s.n + tok0;
  x.len = s.len;
  x.key0 = s.key0;
  x.part = -1;
  x.count = count;
  x.shared = count > 1;
  span_tiles(prompt_span(p, x.pos0, x.pos0 + x.ntok - 1, s.len), x.tile0, x.tiles);
  return x;
}

// A call of up to kDirectSeqs sequences and one unit of work per CTA: this CTA's unit, as a list entry with an int to a
// lane; lane 12 holds whether there is one.  A warp runs it, a lane to a sequence.
__device__ __forceinline__ int direct_entry(const PromptParams& p, int lane) {
  constexpr uint32_t kAll = 0xffffffffu;
  PromptSeq s{};
  bool bad_len = false, ok = true;
  if (lane < p.num_seqs) ok = prompt_seq(p, lane, s, bad_len);
  const int per = 2 * p.stream_tokens, count = ok && lane < p.num_seqs ? (s.n + per - 1) / per : 0;
  ok = __all_sync(kAll, ok);
  if (blockIdx.x == 0) {
    if (!ok && lane == 0) set_error(p.err, kErrQuery);
    if (ok && bad_len) set_error(p.err, kErrContextLen);
  }
  int upto = count;  // items of this sequence and those before it
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kAll, upto, o);
    if (lane >= o) upto += u;
  }
  const int at = int(blockIdx.x) / p.units;
  const uint32_t past = __ballot_sync(kAll, upto > at);
  if (!ok || past == 0) return 0;
  const int b = __ffs(past) - 1;  // the sequence that item `at` belongs to
  const int before = __shfl_sync(kAll, upto - count, b);
  s.row0 = __shfl_sync(kAll, s.row0, b);
  s.n = __shfl_sync(kAll, s.n, b);
  s.len = __shfl_sync(kAll, s.len, b);
  s.key0 = __shfl_sync(kAll, s.key0, b);
  const PromptItem x = sequence_item(p, s, b, __shfl_sync(kAll, count, b), at - before);
  const int v[13] = {x.seq, x.row0, x.ntok, x.pos0, x.len, x.key0, x.tile0, x.tiles, -1, x.shared, int(blockIdx.x) % p.units, 0, 1};
  int mine = 0;
#pragma unroll
  for (int i = 0; i < 13; ++i)
    if (lane == i) mine = v[i];
  return mine;
}

}  // namespace pkv
