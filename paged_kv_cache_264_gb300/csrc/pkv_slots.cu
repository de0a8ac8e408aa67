// pkv_slots.cu -- reserving cache slots for new tokens on the device: page tables, slot
// mappings and lengths from the lengths alone ("Efficient AI Lecture 13", section
// "PagedAttention / How it works": blocks are allocated on demand and found through a block
// table; the host block manager's append does the same on the host).
//
// Sequence b holds L_b tokens in ceil(L_b / 16) blocks and grows by c_b.  It needs
//     n_b = ceil((L_b + c_b) / 16) - ceil(L_b / 16)
// new blocks and gets entries u + o_b, ..., u + o_b + n_b - 1 of the free list, o the
// exclusive prefix sum of n and u the entries handed out before.  New token i of sequence b
// has position L_b + i and slot table[b][position / 16] * 16 + position % 16.
//
// Every CTA forms both prefix sums (over c and n) itself, in shared memory: that costs two
// loads and a scan per sequence, and saves a second launch or a wait between CTAs.  It then
// fills its share of the tokens, finding a token's sequence by bisection.  Bytes (20 and some per
// sequence, 8 per token) bound nothing here: a call is a launch and three round trips to memory.  Measured
// on GB300, calls back to back in a graph: 8 sequences of one token 4.1 us, 256 4.5, 16384 13.9 (79.9 with
// each thread reading its run of sequences from memory itself), 8 of 8192 tokens 4.1, 64 of 16384 8.7.  The token that
// opens a block writes the block's table entry.  The call is all or nothing: whether it fits
// is known from the sums, before anything is written.
//
// The new lengths may replace the old ones in place, so a CTA reads every length before it
// counts itself as done reading, and the last CTA to do so writes the new ones.
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kSlotThreads = 512;
constexpr int kSlotWarps = kSlotThreads / 32;
constexpr int kPerThread = 4;         // consecutive tokens of one thread
constexpr int kSumLimit = 1 << 30;    // sums saturate here (max_tokens is below it)

// Of values in 0 .. kSumLimit, whose plain sum would pass 2^31 - 1.
__device__ __forceinline__ int sat_add(int a, int b) { return int(min(uint32_t(a) + uint32_t(b), uint32_t(kSumLimit))); }

__global__ void __launch_bounds__(kSlotThreads) reserve_slots_kernel(const SlotParams p) {
  extern __shared__ int smem_slots[];
  int* tok = smem_slots;             // [B + 1] first token of each sequence
  int* blk = tok + p.num_seqs + 1;   // [B + 1] first new block of each sequence
  int* len = blk + p.num_seqs + 1;   // [B] old lengths
  __shared__ int warp_tok[kSlotWarps], warp_blk[kSlotWarps];
  __shared__ int is_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.num_seqs;
  griddep_wait();  // lengths and tables may come from the previous kernel in the stream
  griddep_launch_dependents();

  const int used = p.free_used ? *p.free_used : 0;
  uint32_t bad = 0;
#pragma unroll 4
  for (int b = tid; b < B; b += kSlotThreads) {  // whole lines
    tok[b] = p.num_new[b];
    len[b] = p.context_lens[b];
  }
  __syncthreads();
  const int per = (B + kSlotThreads - 1) / kSlotThreads | 1;  // odd: a warp's sequences lie in 32 banks
  const int lo = min(B, tid * per), hi = min(B, lo + per);
  int st = 0, sb = 0;
  for (int b = lo; b < hi; ++b) {
    int L = len[b], c = tok[b];
    if (L < 0 || c < 0) {
      bad |= kErrContextLen;
      L = c = 0;
    } else if (c > p.max_tokens || (int64_t(L) + c + kBlockSize - 1) / kBlockSize > p.max_blocks_per_seq) {
      bad |= kErrCapacity;
      c = 0;
    }
    // L + c fits: it is at most max_blocks_per_seq * 16, which the host keeps below 2^31
    const int n = c == 0 ? 0 : (L + c + kBlockSize - 1) / kBlockSize - (L + kBlockSize - 1) / kBlockSize;
    tok[b] = c;
    blk[b] = n;
    len[b] = L;
    st = sat_add(st, c);
    sb = sat_add(sb, n);
  }
  // exclusive prefix sums over the threads
  int it = st, ib = sb;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, it, o), y = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      it = sat_add(it, x);
      ib = sat_add(ib, y);
    }
  }
  if (lane == 31) {
    warp_tok[warp] = it;
    warp_blk[warp] = ib;
  }
  int et = __shfl_up_sync(0xffffffffu, it, 1), eb = __shfl_up_sync(0xffffffffu, ib, 1);
  if (lane == 0) et = eb = 0;
  bad = __syncthreads_or(bad & kErrContextLen ? 1 : 0) ? kErrContextLen
        : __syncthreads_or(bad) ? kErrCapacity : 0;
  int total_t = 0, total_b = 0;
#pragma unroll
  for (int w = 0; w < kSlotWarps; ++w) {
    if (w == warp) {
      et = sat_add(et, total_t);
      eb = sat_add(eb, total_b);
    }
    total_t = sat_add(total_t, warp_tok[w]);
    total_b = sat_add(total_b, warp_blk[w]);
  }
  for (int b = lo; b < hi; ++b) {
    const int c = tok[b], n = blk[b];
    tok[b] = et;
    blk[b] = eb;
    et = sat_add(et, c);
    eb = sat_add(eb, n);
  }
  if (tid == 0) {
    tok[B] = total_t;
    blk[B] = total_b;
  }
  if (!bad && (total_t > p.max_tokens || used < 0 || used > p.num_free || total_b > p.num_free - used))
    bad = kErrCapacity;
  if (tid == 0) {
    __threadfence();  // after the barrier above: this CTA has read every length
    is_last = gridDim.x == 1 || atomicAdd(p.counter, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (is_last) {
    for (int b = tid; b < B; b += kSlotThreads) p.new_lens[b] = bad ? p.context_lens[b] : len[b] + (tok[b + 1] - tok[b]);
    if (tid == 0) {
      *p.new_used = bad ? used : used + total_b;
      if (gridDim.x > 1) atomicExch(p.counter, 0u);
      if (bad) set_error(p.err, bad);
    }
  }
  if (blockIdx.x == 0)
    for (int b = tid; b <= B; b += kSlotThreads) p.query_starts[b] = bad ? 0 : tok[b];

  const int ntok = bad ? 0 : total_t;
  const int step = gridDim.x * kSlotThreads * kPerThread;
  for (int i0 = (blockIdx.x * kSlotThreads + tid) * kPerThread; i0 < p.max_tokens; i0 += step) {
    int b = 0, row_slot = -1, last_block = -1;
    if (i0 < ntok) {  // tok[b] <= i0 < tok[b + 1]
      int l = 0, h = B;
      while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (tok[mid] <= i0) l = mid; else h = mid;
      }
      b = l;
    }
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const int i = i0 + e;
      if (i >= p.max_tokens) break;
      int slot = -1, pos = 0;
      if (i < ntok) {
        while (tok[b + 1] <= i) {
          ++b;
          last_block = -1;
        }
        pos = len[b] + i - tok[b];
        const int j = pos / kBlockSize;
        if (j != last_block) {
          const int have = (len[b] + kBlockSize - 1) / kBlockSize;
          int32_t* entry = p.block_tables + int64_t(b) * p.max_blocks_per_seq + j;
          const int id = j < have ? *entry : p.free_blocks[used + blk[b] + j - have];
          if (pos % kBlockSize == 0) *entry = id;
          last_block = j;
          row_slot = -1;
          if (id >= 0 && id < p.num_blocks) row_slot = id * kBlockSize;  // num_blocks * 16 < 2^31
          else set_error(p.err, kErrBlockId);
        }
        if (row_slot >= 0) slot = row_slot + pos % kBlockSize;
      }
      p.slot_mapping[i] = slot;
      p.positions[i] = pos;
    }
  }
}

}  // namespace

cudaError_t launch_reserve_slots(const SlotParams& p, cudaStream_t stream) {
  const size_t smem = (size_t(p.num_seqs) * 3 + 2) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(reserve_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int((size_t(kMaxSlotSeqs) * 3 + 2) * sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  const int64_t need = (int64_t(p.max_tokens) + kSlotThreads * kPerThread - 1) / (kSlotThreads * kPerThread);
  const int grid = int(need < 1 ? 1 : need < 152 ? need : 152);
  return launch_pdl(reserve_slots_kernel, dim3(grid), dim3(kSlotThreads), smem, stream, p);
}

}  // namespace pkv
