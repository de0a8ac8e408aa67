// pkv_prefix.cuh -- the work line of shared-prefix decode attention, shared by its passes.
//
// Group g of the batch is sequences group_starts[g] .. group_starts[g + 1] - 1, whose first
// prefix_lens[g] tokens (whole blocks) are the same.  A group has R = (sequences) * k * (query
// heads per kv head) query rows per kv head, in units of up to 256 rows, and its prefix is cut
// into tiles of 128 tokens.  A unit of more than 128 rows takes a tile at a step, its rows in two
// streams of 128; a unit of up to 128 rows (only a group's last can be) takes two, one per stream.
// All (kv head, unit, step) triples of all groups, in that order, form one line of work, which the
// CTAs of the prefix pass share out in equal contiguous stretches, so that they end together
// whatever the groups' sizes.  Each unit takes places on the line ahead of its steps (unit_cost): what
// loading its queries and writing its partials costs, in steps.  A stretch's steps of one (kv head,
// unit) are a piece; it leaves one partial (running max, sum, accumulator) per row.
//
// Partial rows: CTA c's partial of a unit starts at row (rows of all units before it) + 256 c.
// Going along the line either the unit or the CTA (or both) moves on, by that unit's rows or by
// 256, so no two partials overlap.  A unit of up to 128 rows holds two rows of partials per
// query row, since each stream accumulates its own tiles.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// Query rows of unit u of a group of `rows`.
__host__ __device__ __forceinline__ int unit_rows(int rows, int u) {
  const int left = rows - u * kPrefixRows;
  return left < kPrefixRows ? left : kPrefixRows;
}
// Whether a unit of n rows gives its streams tiles apart, and its steps over `tiles` tiles.
__host__ __device__ __forceinline__ bool tiles_apart(int n) { return n <= kPrefixRows / 2; }
__host__ __device__ __forceinline__ int unit_steps(int n, int tiles) { return tiles_apart(n) ? (tiles + 1) / 2 : tiles; }
// Places ahead of a unit's steps: a piece's start and end, and its rows of partials.  Measured on GB300
// with the same places for every unit (1 / 2 / 4 / 6), whole calls: 16 groups of 1 to 13 sequences
// (MHA) 114.0 / 115.2 / 119.6 / 122.8 us, 2 groups of 96 and 672 rows a kv head (FP8, head_dim 64) 62.7 / 62.0 /
// 59.9 / 62.3; with these 114.5 and 61.8 (56.7 since the states are joined without a merge pass).
// Had the 96 rows' unit one stream, on every tile, it would be 63.7 for 61.8.  Over 36 batches drawn at random
// (1 to 41 groups, all types) a slope of 3 was on average 2.0% above each one's best of 0, 1, 2, 3, 5 and 8; 0
// and 1 were 1.4%, 2 1.5%, 5 3.0%, 8 4.7%.
__host__ __device__ __forceinline__ int unit_cost(int n) {
  return 1 + (tiles_apart(n) ? 2 * n : n) * 3 / kPrefixRows;
}
__host__ __device__ __forceinline__ int unit_line(int n, int tiles) { return unit_cost(n) + unit_steps(n, tiles); }
// Rows of partials that a group of `rows` query rows takes per kv head.
__host__ __device__ __forceinline__ int64_t partial_rows(int rows) {
  const int last = rows <= 0 ? 0 : (rows - 1) % kPrefixRows + 1;
  return int64_t(rows) + (tiles_apart(last) ? last : 0);
}

// a / b for non-negative a and positive b: work lines are short enough for 32 bits as a rule, and a
// 64-bit division is some hundred instructions.
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

struct PrefixGroup {
  int first_seq, rows, units, nblk, tiles;  // units per kv head; blocks and tiles of the prefix
  int64_t w_base, row_base;
};

// Places on the line of one kv head of a group with work, and of the whole group.
__device__ __forceinline__ int64_t head_line(int rows, int units, int tiles) {
  return int64_t(units - 1) * unit_line(kPrefixRows, tiles) + unit_line(unit_rows(rows, units - 1), tiles);
}
__device__ __forceinline__ int64_t group_line(const PrefixParams& p, const PrefixGroup& x) {
  return x.tiles > 0 && x.rows > 0 ? p.kv_heads * head_line(x.rows, x.units, x.tiles) : 0;
}

// The scan of the groups, in scratch shared memory: base[g] = (first place on the line, first
// partial row) of group g.
struct PrefixScan {
  longlong2* base;   // [G + 1]
  longlong2* warp;   // [32]
};
__host__ __device__ constexpr size_t prefix_scan_bytes(int groups) { return (size_t(groups) + 1 + 32) * 16; }

// Sizes of group g; false where its description is invalid.
__device__ __forceinline__ bool prefix_group(const PrefixParams& p, int g, PrefixGroup& x) {
  const int s0 = __ldg(p.group_starts + g), s1 = __ldg(p.group_starts + g + 1), len = __ldg(p.prefix_lens + g);
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= p.num_seqs && len >= 0 && len <= p.max_prefix_len && len % kBlockSize == 0;
  x.first_seq = s0;
  x.rows = ok ? (s1 - s0) * p.num_queries * p.group : 0;
  x.units = (x.rows + kPrefixRows - 1) / kPrefixRows;
  x.nblk = ok ? len / kBlockSize : 0;
  x.tiles = ok ? (len + kPrefixTile - 1) / kPrefixTile : 0;
  return ok;
}

// The scan of up to 32 groups, a lane to a group, by each warp for itself: no barrier, one round
// trip to memory.
constexpr int kFewGroups = 32;
struct PrefixLanes {
  PrefixGroup x;  // lane g's group
};
__device__ __forceinline__ int64_t prefix_scan_few(const PrefixParams& p, PrefixLanes& me) {
  const int lane = threadIdx.x & 31;
  me.x = PrefixGroup{};
  bool ok = true;
  if (lane < p.num_groups) ok = prefix_group(p, lane, me.x);
  const int64_t w = group_line(p, me.x), r = partial_rows(me.x.rows) * p.kv_heads;
  int64_t iw = w, ir = r;
  for (int o = 1; o < p.num_groups; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, iw, o), b = __shfl_up_sync(0xffffffffu, ir, o);
    if (lane >= o) {
      iw += a;
      ir += b;
    }
  }
  me.x.w_base = iw - w;
  me.x.row_base = ir - r;
  const int64_t total = __shfl_sync(0xffffffffu, iw, p.num_groups > 0 ? p.num_groups - 1 : 0);
  return __all_sync(0xffffffffu, ok) ? total : -1;
}
__device__ __forceinline__ PrefixGroup lane_group(const PrefixLanes& me, int g) {
  PrefixGroup x;
  x.first_seq = __shfl_sync(0xffffffffu, me.x.first_seq, g);
  x.rows = __shfl_sync(0xffffffffu, me.x.rows, g);
  x.units = __shfl_sync(0xffffffffu, me.x.units, g);
  x.nblk = __shfl_sync(0xffffffffu, me.x.nblk, g);
  x.tiles = __shfl_sync(0xffffffffu, me.x.tiles, g);
  x.w_base = __shfl_sync(0xffffffffu, me.x.w_base, g);
  x.row_base = __shfl_sync(0xffffffffu, me.x.row_base, g);
  return x;
}

// Fill the scan (all NT threads of the CTA); returns the line's places, or -1 where
// some group is invalid.  Ends with a barrier.
template <int NT>
__device__ __forceinline__ int64_t prefix_scan(const PrefixParams& p, const PrefixScan& sc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.num_groups;
  const int per = (G + NT - 1) / NT;
  const int lo = min(G, tid * per), hi = min(G, lo + per);
  int64_t w = 0, r = 0;
  bool ok = true;
  for (int g = lo; g < hi; ++g) {
    PrefixGroup x;
    ok &= prefix_group(p, g, x);
    w += group_line(p, x);
    r += partial_rows(x.rows) * p.kv_heads;
  }
  int64_t iw = w, ir = r;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, iw, o), b = __shfl_up_sync(0xffffffffu, ir, o);
    if (lane >= o) {
      iw += a;
      ir += b;
    }
  }
  if (lane == 31) sc.warp[warp] = make_longlong2(iw, ir);
  ok = __syncthreads_and(ok);
  int64_t bw = iw - w, br = ir - r, total = 0;
  for (int i = 0; i < NT / 32; ++i) {
    const longlong2 x = sc.warp[i];
    if (i < warp) {
      bw += x.x;
      br += x.y;
    }
    total += x.x;
  }
  for (int g = lo; g < hi; ++g) {
    PrefixGroup x;
    prefix_group(p, g, x);
    sc.base[g] = make_longlong2(bw, br);
    bw += group_line(p, x);
    br += partial_rows(x.rows) * p.kv_heads;
  }
  __syncthreads();
  return ok ? total : -1;
}

// CTAs that take work: no more than the line has places, so that none between a unit's first and
// last tile is without one (its partial would be read unwritten).
__device__ __forceinline__ int stretch_ctas(int64_t total, int grid) { return int(min(total, int64_t(grid))); }
// CTA c's stretch of the line starts here.
__device__ __forceinline__ int64_t stretch_start(int64_t total, int ctas, int c) { return div_pos(total * c, ctas); }
// The CTA whose stretch holds place w: the last one that starts at or before it.
__device__ __forceinline__ int stretch_owner(int64_t total, int ctas, int64_t w) {
  return int(div_pos((w + 1) * ctas - 1, total));
}

// The partial states that the prefix pass leaves for row r (of a group and kv head): rows 256 apart, one
// per CTA that had steps of the row's unit (two where the streams took tiles apart).
struct PrefixParts {
  int count = 0, twice = 0, rows = 0;
  int64_t first = 0;
  PrefixParts() = default;
  __device__ __forceinline__ PrefixParts(const PrefixSeq& d, int kvh, int r, int grid) {
    const int units = (d.rows + kPrefixRows - 1) / kPrefixRows, u = r / kPrefixRows;
    rows = unit_rows(d.rows, u);
    twice = tiles_apart(rows);
    // the places of the unit's steps
    const int64_t w0 = d.w_base + kvh * head_line(d.rows, units, d.tiles) + int64_t(u) * unit_line(kPrefixRows, d.tiles) + unit_cost(rows);
    const int64_t w1 = w0 + unit_steps(rows, d.tiles) - 1;
    const int ctas = stretch_ctas(d.total, grid);
    const int c0 = stretch_owner(d.total, ctas, w0), c1 = stretch_owner(d.total, ctas, w1);
    count = (c1 - c0 + 1) << twice;
    first = d.row_base + int64_t(kvh) * partial_rows(d.rows) + r + int64_t(c0) * kPrefixRows;
  }
  __device__ __forceinline__ int64_t row(int i) const {
    return first + int64_t(i >> twice) * kPrefixRows + (twice && (i & 1) ? rows : 0);
  }
};

// A walk along one CTA's stretch: one (kv head, unit) at a time.
struct PrefixWalk {
  PrefixGroup x;
  int g, kvh, unit;      // group, kv head and unit of the group's rows
  int at;                // place within the unit
  int64_t w, w_end;
};

// A piece as the roles of a CTA see it (tiles == 0: there are no more).
struct PrefixPiece {
  int64_t partial;       // first partial row
  int first_seq, nblk;   // the group's first sequence, the prefix's blocks
  int tile0, tiles;
  int kvh;
  int row0, nrows;       // the unit's query rows within the group
  int again;             // other units read the same tiles
  int pad[2];
};

// The piece at the walk's place, if it has tiles; moves past the unit's part of the stretch.
__device__ __forceinline__ bool walk_piece(const PrefixParams& p, PrefixWalk& k, int cta, PrefixPiece& x) {
  x.row0 = k.unit * kPrefixRows;
  x.nrows = unit_rows(k.x.rows, k.unit);
  const int all = unit_line(x.nrows, k.x.tiles), cost = unit_cost(x.nrows), per = tiles_apart(x.nrows) ? 2 : 1;
  const int len = int(min(int64_t(all - k.at), k.w_end - k.w));
  const int step0 = max(0, k.at - cost), step1 = k.at + len - cost;
  x.tile0 = step0 * per;
  x.tiles = min(k.x.tiles, step1 * per) - x.tile0;
  x.first_seq = k.x.first_seq;
  x.kvh = k.kvh;
  x.again = k.x.units > 1;
  x.nblk = k.x.nblk;
  x.partial = k.x.row_base + int64_t(k.kvh) * partial_rows(k.x.rows) + x.row0 + int64_t(cta) * kPrefixRows;
  k.w += len;
  k.at += len;
  return x.tiles > 0;
}

// This CTA's stretch; false if it has none.
__device__ __forceinline__ bool walk_range(const PrefixParams& p, int64_t total, int cta, PrefixWalk& k) {
  const int ctas = stretch_ctas(total, p.grid);
  if (total <= 0 || cta >= ctas) return false;
  const int64_t at = stretch_start(total, ctas, cta + int(threadIdx.x & 1));  // one division for both
  k.w = __shfl_sync(0xffffffffu, at, 0);
  k.w_end = __shfl_sync(0xffffffffu, at, 1);
  return true;
}
// Its first place, once k.g and k.x are the group that holds it.
__device__ __forceinline__ void walk_first(PrefixWalk& k) {
  const int64_t in_group = k.w - k.x.w_base, head = head_line(k.x.rows, k.x.units, k.x.tiles);
  k.kvh = int(div_pos(in_group, head));
  const int64_t in_head = in_group - k.kvh * head;
  const int all = unit_line(kPrefixRows, k.x.tiles);  // of every unit but the last
  k.unit = k.x.units == 1 ? 0 : min(int(div_pos(in_head, all)), k.x.units - 1);
  k.at = int(in_head - int64_t(k.unit) * all);
}
__device__ __forceinline__ bool walk_begin(const PrefixParams& p, const PrefixScan& sc, int64_t total, int cta,
                                           PrefixWalk& k) {
  if (!walk_range(p, total, cta, k)) return false;
  int lo = 0, hi = p.num_groups;  // the last group that starts at or before w (empty ones share a start)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sc.base[mid].x <= k.w) lo = mid; else hi = mid;
  }
  k.g = lo;
  prefix_group(p, lo, k.x);
  k.x.w_base = sc.base[lo].x;
  k.x.row_base = sc.base[lo].y;
  walk_first(k);
  return true;
}
__device__ __forceinline__ bool walk_begin_few(const PrefixParams& p, const PrefixLanes& me, int64_t total, int cta,
                                               PrefixWalk& k) {
  if (!walk_range(p, total, cta, k)) return false;
  const uint32_t at = __ballot_sync(0xffffffffu, int(threadIdx.x & 31) < p.num_groups && me.x.w_base <= k.w);
  k.g = 31 - __clz(at);
  k.x = lane_group(me, k.g);
  walk_first(k);
  return true;
}

// On to the next unit once this one's part of the stretch is past; false at the stretch's end.
__device__ __forceinline__ bool walk_next(const PrefixParams& p, PrefixWalk& k) {
  if (k.w >= k.w_end) return false;
  k.at = 0;
  if (++k.unit == k.x.units) {
    k.unit = 0;
    if (++k.kvh == p.kv_heads) {
      k.kvh = 0;
      do {  // the next group that has work
        const int64_t w = k.x.w_base + group_line(p, k.x);
        const int64_t rows = k.x.row_base + partial_rows(k.x.rows) * p.kv_heads;
        ++k.g;
        prefix_group(p, k.g, k.x);
        k.x.w_base = w;
        k.x.row_base = rows;
      } while (k.x.units == 0 || k.x.tiles == 0);
    }
  }
  return true;
}

// Row of q and out (in units of head_dim values) of the group's query row r for kv head kvh:
// rows run over the group's sequences, each one's query tokens, each one's heads of the group.
__device__ __forceinline__ int64_t prefix_q_row(const PrefixParams& p, int first_seq, int kvh, int r) {
  const int tok = r / p.group, head = r - tok * p.group;
  return (int64_t(first_seq) * p.num_queries + tok) * p.num_q_heads + int64_t(kvh) * p.group + head;
}

// What the suffix and merge passes need of this CTA's share of the sequences; run by `warps` of
// its warps, this one the `warp`-th of them.  group_of(b, x): the whole warp asks for sequence b's
// group; false where it is in none.
template <typename F>
__device__ __forceinline__ void prefix_describe(const PrefixParams& p, int64_t total, int warp, int warps, F&& group_of) {
  const int lane = threadIdx.x & 31;
  for (int b = blockIdx.x * warps + warp; b < p.num_seqs; b += gridDim.x * warps) {
    const int T = __ldg(p.context_lens + b);
    PrefixSeq d{};
    PrefixGroup x{};
    int len = 0, g = 0;
    if (total >= 0 && p.num_groups > 0 && group_of(b, g, x)) {
      len = __ldg(p.prefix_lens + g);
      d.w_base = x.w_base;
      d.row_base = x.row_base;
      d.tiles = x.tiles;
      d.rows = x.rows;
      d.first_row = (b - x.first_seq) * p.num_queries * p.group;
    }
    d.total = total;
    d.suffix_len = T - len;
    // every query sees the whole prefix, and the table holds the sequence
    if (total < 0 || T < p.num_queries || T - (p.num_queries - 1) < len || T - len > p.max_suffix_len ||
        T > int64_t(p.max_blocks_per_seq) * kBlockSize)
      d.suffix_len = -1;
    const int nblk = d.suffix_len < 0 ? 0 : (d.suffix_len + kBlockSize - 1) / kBlockSize;
    const int32_t* row = p.block_tables + int64_t(b) * p.max_blocks_per_seq + len / kBlockSize;
    int32_t* to = p.suffix_tables + int64_t(b) * p.suffix_blocks;
    for (int j = lane; j < p.suffix_blocks; j += 32) to[j] = j < nblk ? __ldg(row + j) : -1;
    if (lane == 0) {
      p.seqs[b] = d;
      p.suffix_lens[b] = d.suffix_len;
    }
  }
  if (total < 0 && blockIdx.x == 0 && warp == 0 && lane == 0) set_error(p.err, kErrPrefix);
}
__device__ __forceinline__ void prefix_describe_many(const PrefixParams& p, const PrefixScan& sc, int64_t total, int warp,
                                                     int warps) {
  prefix_describe(p, total, warp, warps, [&](int b, int& g, PrefixGroup& x) {
    int lo = 0, hi = p.num_groups;
    while (hi - lo > 1) {  // the last group that starts at or before b
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.group_starts + mid) <= b) lo = mid; else hi = mid;
    }
    if (b < __ldg(p.group_starts + lo) || b >= __ldg(p.group_starts + lo + 1)) return false;
    g = lo;
    prefix_group(p, lo, x);
    x.w_base = sc.base[lo].x;
    x.row_base = sc.base[lo].y;
    return true;
  });
}
__device__ __forceinline__ void prefix_describe_few(const PrefixParams& p, const PrefixLanes& me, int64_t total) {
  prefix_describe(p, total, 0, 1, [&](int b, int& g, PrefixGroup& x) {
    const int first = me.x.first_seq, n = me.x.rows / (p.num_queries * p.group);
    const uint32_t at = __ballot_sync(0xffffffffu, b >= first && b < first + n);
    if (at == 0) return false;
    g = __ffs(at) - 1;
    x = lane_group(me, g);
    return true;
  });
}

}  // namespace pkv
