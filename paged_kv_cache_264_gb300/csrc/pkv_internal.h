// pkv_internal.h -- structures shared by the C-ABI layer and the kernel launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

struct pkv_pool;  // the C ABI's opaque pool descriptor (include/pagedkv.h)

namespace pkv {

constexpr int kBlockSize = 16;                      // tokens per physical block
constexpr uint64_t kWaitTimeoutNs = 2000000000ull;  // bounded waits give up after 2 s
constexpr int kMaxSchedSeqs = 4096;  // largest batch scheduled by the persistent grid
constexpr int kNoWindow = 1 << 30;   // window value meaning "no window" (contexts are shorter)

// Partitions of a sequence's nblk blocks for partition size P (decode kernels, partition
// reduce and host plan alike).  They start at multiples of P, so that an item's slice of the
// block table can be requested before its context length is known, and the last one also
// takes a remainder of at most P / 4 blocks instead of leaving it to an item of its own
// (with its own partial to merge): a partition holds up to partition_cap(P) blocks.
__host__ __device__ constexpr int partition_count(int nblk, int P) {
  return nblk - P / 4 <= P ? 1 : (nblk - P / 4 + P - 1) / P;
}
__host__ __device__ constexpr int partition_cap(int P) { return P + P / 4; }
static_assert(partition_count(64, 64) == 1 && partition_count(80, 64) == 1 && partition_count(81, 64) == 2 &&
                  partition_count(1024, 64) == 16 && partition_count(7, 1) == 7 && partition_count(5, 4) == 1,
              "partition_count");

// Device error word bits (mirror PKV_DEVERR_* of the public header).
constexpr uint32_t kErrBlockId = 0x1u;
constexpr uint32_t kErrContextLen = 0x2u;
constexpr uint32_t kErrSlot = 0x4u;
constexpr uint32_t kErrTimeout = 0x8u;
constexpr uint32_t kErrCapacity = 0x10u;
constexpr uint32_t kErrPosition = 0x20u;
constexpr uint32_t kErrPrefix = 0x40u;

enum class KvType : int { kBf16 = 0, kInt8 = 1, kFp8 = 2 };

struct CacheParams {
  const void* key;              // bf16 [N, Hkv, D]
  const void* value;            // bf16 [N, Hkv, D]
  const int32_t* slot_mapping;  // [N]
  void* k_cache;                // [NB, Hkv, 16, D]
  void* v_cache;
  float* k_scale;               // [NB, Hkv, 16] (int8 only)
  float* v_scale;
  uint32_t* err;
  int64_t num_tokens;
  int64_t num_blocks;
  int kv_heads;
  int head_dim;
};

struct PrefixSeq;

struct DecodeParams {
  const void* q;                // bf16 [B, k, Hq, D]  (k = num_queries)
  const void* k_cache;          // [NB, Hkv, 16, D]
  const void* v_cache;
  const float* k_scale;         // [NB, Hkv, 16] (int8 only)
  const float* v_scale;
  const int32_t* block_tables;  // [B, max_blocks_per_seq]
  const int32_t* context_lens;  // [B]
  void* out;                    // bf16 [B, k, Hq, D]
  float* ws_acc;                // [B, k, Hq, max_parts, D]   (split only)
  float* ws_ml;                 // [B, k, Hq, max_parts, 2]   (split only): running max (log2 units), sum
  uint32_t* err;
  unsigned* sched;              // [2] work ticket and finished-CTA counters (zero between calls)
  int persistent;               // 1: persistent grid taking items from the ticket counter
  int grid;                     // CTAs to launch in persistent mode
  int64_t num_blocks;
  int max_blocks_per_seq;
  int num_seqs;
  int num_q_heads;
  int kv_heads;
  int group;                    // query heads per kv head (num_q_heads / kv_heads), any >= 1
  int group_log2;               // log2(group) when group is a power of two, else -1
  int num_queries;              // k >= 1 query tokens per sequence, the last k positions
  int chunks;                   // column chunks per kv head: group * k columns are served in
                                // chunks of the variant's column slots, one work unit each
  int window;                   // each query sees its last `window` tokens (kNoWindow: all)
  int head_dim;
  int max_context_len;
  int partition_blocks;         // P: blocks per work item
  int max_parts;                // ceil(ceil(max_context_len / 16) / P)
  float scale_log2;             // softmax scale * log2(e)
  int min_len;                  // shortest valid context (num_queries; 0 when another pass
                                // covers the tokens before this call's context)
  int partials;                 // 1: always leave (m, l, acc) in the workspace, never write out
  // For the kernels that join a prefix pass's partial states (pkv_prefix.cuh): its descriptions
  // of the sequences, its states and its CTAs.
  const PrefixSeq* prefix_seqs;
  const float* prefix_acc;
  const float2* prefix_ml;
  int prefix_grid;
};

// Reserving cache slots for new tokens on the device (pkv_slots.cu).
struct SlotParams {
  int32_t* block_tables;        // [B, max_blocks_per_seq], new entries written
  const int32_t* context_lens;  // [B]
  const int32_t* num_new;       // [B]
  const int32_t* free_blocks;   // [num_free] ids in hand-out order
  const int32_t* free_used;     // [1] entries already handed out; NULL: 0
  int32_t* slot_mapping;        // [max_tokens]
  int32_t* positions;           // [max_tokens]
  int32_t* query_starts;        // [B + 1]
  int32_t* new_lens;            // [B], may be context_lens
  int32_t* new_used;            // [1], may be free_used
  uint32_t* err;
  unsigned* counter;            // CTAs that have read their inputs (zero between calls)
  int64_t num_blocks;
  int max_blocks_per_seq;
  int num_seqs;
  int num_free;
  int max_tokens;
};
constexpr int kMaxSlotSeqs = 16384;  // three ints of shared memory per sequence
cudaError_t launch_reserve_slots(const SlotParams& p, cudaStream_t stream);

// Per-head norm, rotation and cache write of new tokens (pkv_rope.cu).
struct RopeParams {
  const void* q;                // bf16 rows of [Hq, D] at token stride q_stride, and so on
  const void* k;
  const void* v;
  const void* q_weight;         // bf16 [D] or NULL: q is not normalised
  const void* k_weight;
  const float* cos_sin;         // [max_position, rot_dim]: cosines, then sines; NULL: no rotation
  const int32_t* positions;     // [N]
  const int32_t* slot_mapping;  // [N]
  void* q_out;                  // bf16 rows of [Hq, D] at token stride out_stride
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  uint32_t* err;
  int64_t q_stride, k_stride, v_stride, out_stride;  // elements
  int64_t num_tokens;
  int64_t num_blocks;
  int num_q_heads;
  int kv_heads;
  int head_dim;
  int rot_dim;
  int max_position;
  int interleaved;
  float eps;
};
cudaError_t launch_norm_rope(const RopeParams& p, KvType kv, cudaStream_t stream);
cudaError_t launch_rope_table(float* out, int64_t max_position, int rot_dim, double base, cudaStream_t stream);

// Decode attention over shared prefixes (pkv_prefix.cu).  The prefix pass writes, besides
// its partials, what the two later passes need: each sequence's descriptor, the length of
// its own tokens and their slice of its block table.
struct PrefixSeq {
  int64_t w_base;     // first place of the sequence's group on the line of work
  int64_t row_base;   // first partial row of the group
  int64_t total;      // places of the whole line
  int suffix_len;     // the sequence's own tokens; -1: its inputs are invalid
  int tiles;          // 128-token tiles of its prefix
  int first_row;      // its first query row among the group's (per kv head)
  int rows;           // the group's query rows per kv head
};
struct PrefixParams {
  const void* q;                // bf16 [B, k, Hq, D]
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* group_starts;  // [G + 1]
  const int32_t* prefix_lens;   // [G]
  void* out;
  PrefixSeq* seqs;              // [B]
  int32_t* suffix_lens;         // [B]
  int32_t* suffix_tables;       // [B, suffix_blocks]
  float* acc;                   // [rows, D] prefix partials
  float2* ml;                   // [rows] running max (log2 units) and sum
  const float* suffix_acc;      // [B, k, Hq, suffix_parts, D]
  const float2* suffix_ml;
  uint32_t* err;
  int64_t num_blocks;
  int max_blocks_per_seq;
  int num_seqs;
  int num_groups;
  int num_q_heads;
  int kv_heads;
  int group;                    // query heads per kv head
  int num_queries;
  int head_dim;
  int max_prefix_len;
  int max_suffix_len;
  int suffix_blocks;            // width of suffix_tables
  int suffix_partition;         // the suffix pass's partition size and most partitions
  int suffix_parts;
  int grid;                     // CTAs of the prefix pass
  float scale_log2;
};
constexpr int kMaxPrefixGroups = 4096;
constexpr int kPrefixTile = 128;     // prefix tokens of one work tile
constexpr int kPrefixRows = 256;     // query rows of one work unit (two 128-row tiles)
cudaError_t launch_prefix(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, KvType kv,
                          cudaStream_t stream);
cudaError_t launch_prefix_quant(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, KvType kv,
                                cudaStream_t stream);
cudaError_t launch_prefix_bf16(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream);
cudaError_t launch_prefix_merge(const PrefixParams& p, cudaStream_t stream);

// Launch a kernel with programmatic stream serialisation (see griddep_wait in
// pkv_device.cuh): its launch may overlap the tail of the previous kernel in the stream.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// Kernel launchers (defined next to their kernels).  Each returns the launch status.
cudaError_t launch_cache_bf16(const CacheParams& p, cudaStream_t stream);
cudaError_t launch_cache_int8(const CacheParams& p, cudaStream_t stream);
cudaError_t launch_cache_fp8(const CacheParams& p, cudaStream_t stream);
cudaError_t launch_copy_blocks(const CacheParams& p, const int32_t* pairs, int n, int elem_bytes,
                               cudaStream_t stream);
// The decode kernels serve, per (sequence, kv head), a tile of query columns: column c is
// query token c / group of head kvh * group + c % group.  `cols` is the column slot count
// of the variant to launch: the smallest built power of two >= group * num_queries, or the
// largest built one, the columns then served in chunks of that many.
cudaError_t launch_decode_bf16(const DecodeParams& p, int cols, cudaStream_t stream);
cudaError_t launch_decode_int8(const DecodeParams& p, int cols, cudaStream_t stream);
cudaError_t launch_decode_fp8(const DecodeParams& p, int cols, cudaStream_t stream);
cudaError_t launch_lse_reduce(const DecodeParams& p, cudaStream_t stream);

// Tensor-core decode (2, 4, 8 or 16 column slots): tk/tv are 2-D tensor maps of the K and
// V pools (rows of head_dim elements, 128-byte boxes of 16 rows, 128-byte swizzle).
bool mma_supported(KvType kv, int head_dim, int cols);
// Ring shape (stages x blocks per stage) index for requested values (0 = default); -1 if
// that shape is not built.
int mma_ring_shape(KvType kv, int head_dim, int stages, int blocks_per_stage);
cudaError_t launch_decode_mma(const DecodeParams& p, const CUtensorMap* tk, const CUtensorMap* tv,
                              KvType kv, int cols, int shape, cudaStream_t stream);
cudaError_t launch_decode_mma_join(const DecodeParams& p, const CUtensorMap* tk, const CUtensorMap* tv, KvType kv, int cols,
                                   cudaStream_t stream);
// gen: the variant with the general masks (several query tokens or a window).
int mma_ctas_per_sm(KvType kv, int head_dim, int cols, int shape, bool gen);
// Whether a tensor-core call takes the general-mask variant: some query has a causal cut
// or a window, or the tile is 16 columns wide (plain decode of a group of more than 8
// heads; the 16-column tiles are built with the general masks only).
inline bool mma_needs_general(int num_queries, int window, int cols) {
  return num_queries > 1 || window != kNoWindow || cols > 8;
}

// The CUDA device a pool was created on (-1 for NULL).
int pool_device(const pkv_pool* pool);

// Resident CTAs per SM of the CUDA-core decode kernel variant (0 if not built).
int decode_ctas_per_sm(KvType kv, int head_dim, int cols);

}  // namespace pkv
