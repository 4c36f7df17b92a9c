// Block tables and slot maps of a step, built on the GPU from the requests'
// lengths: the blocks that the step's new tokens need are taken from a free
// list and entered in the tables, and each new token gets its position and its
// cache slot.  What the cache writes and the decodes take as given.
//
//   old_b  = max(0, seq_lens[b] - q_len_b): positions already in the cache
//   tables (one per request, or one per (request, shard) over the shard's local
//   tokens) have ceil(len(old) / bs) entries and get those up to
//   ceil(len(seq) / bs); new entry k, counted over (b, d, column) in order, is
//   free_blocks[free_count - 1 - k].  With a count of the columns that a table
//   holds, from there on instead (after rejected drafts the old tokens end before
//   the blocks do).
//   token i of request b: position p = seq - q_len + i, slot = entry(p) * bs +
//   offset.
//
// Whole numbers only.  A few bytes per request and token, so the time is the
// chain of dependent reads: lengths, free list, tables.  One CTA makes the
// entries (a scan over the tables' needs, 1,024 at a time in shared memory;
// then a thread per new entry finds its table by a search in the scan, so that
// one table's thousand entries are as quick as a thousand tables' one).  Up to
// kFusedTokens tokens follow in the same CTA, behind its own barrier (they find
// their requests in shared memory, where there are not too many); more take a
// second grid whose launch overlaps the first (programmatic dependent
// launch).
//
// One request 4 us, 515 requests' 1,545 rows or 256 requests over eight shards'
// tables 7-8 us, 16,387 tokens over eight shards 4 + 3.5 us (kernel times).
#include "dcp_kernels.h"

namespace dcp {
namespace {

constexpr int kThreads = 1024;
constexpr int kTokenThreads = 256;
constexpr int kFusedTokens = 2048;
constexpr int kKept = 2048;  // requests whose rows and lengths the CTA keeps for its tokens
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int32_t owned(const CacheExtendArgs& a, int32_t L, int32_t d) {
  const int32_t full = a.div_period.d ? fast_div(L, a.div_period) : 0;  // (no divisor: the period is past every length)
  int64_t rem = L - static_cast<int64_t>(full) * a.period - static_cast<int64_t>(d) * a.I;
  rem = rem < 0 ? 0 : (rem > a.I ? a.I : rem);
  return static_cast<int32_t>(static_cast<int64_t>(full) * a.I + rem);
}
// blocks of n tokens
__device__ __forceinline__ int32_t blocks_of(const CacheExtendArgs& a, int32_t n) {
  return n > 0 ? fast_div(n - 1, a.div_bs) + 1 : 0;
}
__device__ __forceinline__ int64_t table_row(const CacheExtendArgs& a, int32_t b, int32_t dd) {
  return (a.local_tables ? dd * a.bt_shard_stride : 0) + static_cast<int64_t>(b) * a.bt_stride;
}

// Position and slot of row t, whose request is b (rows [q0, q1), length seq).
__device__ __forceinline__ void place(const CacheExtendArgs& a, int32_t t, int32_t b, int32_t q0, int32_t q1, int32_t seq) {
  int64_t slot = -1;
  int32_t p = -1;
  if (b >= 0 && seq > 0) {
    const int64_t at = static_cast<int64_t>(seq) - q1 + t;
    if (at >= 0 && at < seq) {
      p = static_cast<int32_t>(at);
      const int32_t run = fast_div(p, a.div_I), turn = fast_div(run, a.div_D);
      const int32_t d = run - turn * a.D;
      if (d >= a.d0 && d < a.d0 + a.Dn) {
        const int32_t j = a.local_tables ? turn * a.I + (p - run * a.I) : p;
        const int32_t col = fast_div(j, a.div_bs);
        if (col < a.bt_width) {
          // (written by this launch or the one before it: no read-only load)
          const int32_t blk = a.block_table[table_row(a, b, d - a.d0) + col];
          if (blk >= 0) slot = static_cast<int64_t>(blk) * a.block_size + (j - col * a.block_size);
        }
      }
    }
  }
  a.positions[t] = p;
  a.slot_mapping[t] = slot;
}

__global__ void __launch_bounds__(kThreads) extend_kernel(CacheExtendArgs a, int fused) {
  __shared__ int32_t start[kThreads + 1];  // first new entry of each of these tables, then their total
  __shared__ int32_t first_col[kThreads];
  __shared__ int32_t warp_sum[kThreads / 32];
  __shared__ int32_t kept_qsl[kKept + 1], kept_seq[kKept];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t tables = static_cast<int64_t>(a.B) * a.S;
  const bool kept = fused && a.B <= kKept;
  if (kept) {
    for (int32_t b = tid; b < a.B; b += kThreads) kept_qsl[b] = __ldg(a.qsl + b), kept_seq[b] = __ldg(a.seq_lens + b);
    if (tid == 0 && a.B > 0) kept_qsl[a.B] = __ldg(a.qsl + a.B);
  }
  int32_t count = *a.free_count;
  count = count < 0 ? 0 : (count > a.num_free ? a.num_free : count);
  uint32_t err = 0;
  int64_t base = 0;  // new entries of the tables before this round's
  for (int64_t i0 = 0; i0 < tables; i0 += kThreads) {
    const int64_t i = i0 + tid;
    int32_t need = 0, c0 = 0;
    int32_t* held = nullptr;
    if (i < tables) {
      const int32_t b = static_cast<int32_t>(a.S == 1 ? i : i / a.S), dd = static_cast<int32_t>(i - static_cast<int64_t>(b) * a.S);
      const int32_t q0 = __ldg(a.qsl + b), q1 = __ldg(a.qsl + b + 1);
      const int32_t seq = max(0, __ldg(a.seq_lens + b));
      if (q1 < q0) err |= DCP_DEVERR_BAD_ROWS;
      if (a.held) {
        held = a.held + static_cast<int64_t>(dd) * a.B + b;
        c0 = max(0, *held);
      } else {
        const int64_t before = static_cast<int64_t>(seq) - max(static_cast<int64_t>(q1) - q0, static_cast<int64_t>(0));
        const int32_t old = before > 0 ? static_cast<int32_t>(before) : 0;
        c0 = blocks_of(a, a.local_tables ? owned(a, old, a.d0 + dd) : old);
      }
      int32_t c1 = blocks_of(a, a.local_tables ? owned(a, seq, a.d0 + dd) : seq);
      if (c1 > a.bt_width) {
        err |= DCP_DEVERR_SEQ_TOO_LONG;
        c1 = a.bt_width;
      }
      need = max(0, c1 - c0);
    }
    int32_t x = need;  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int32_t s = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(kFull, s, o);
        if (lane >= o) s += y;
      }
      warp_sum[lane] = s;
    }
    __syncthreads();
    if (warp > 0) x += warp_sum[warp - 1];
    start[tid] = x - need;
    first_col[tid] = c0;
    if (held && need > 0) {  // as far as the free list reaches
      const int64_t got = static_cast<int64_t>(count) - base - (x - need);
      *held = c0 + (got <= 0 ? 0 : (got < need ? static_cast<int32_t>(got) : need));
    }
    if (tid == kThreads - 1) start[kThreads] = x;
    __syncthreads();
    const int32_t total = start[kThreads];
    for (int32_t k = tid; k < total; k += kThreads) {
      int32_t lo = 0, hi = kThreads;  // the last table whose first new entry is <= k
      while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (start[mid] <= k) lo = mid; else hi = mid;
      }
      const int64_t it = i0 + lo;
      const int32_t b = static_cast<int32_t>(a.S == 1 ? it : it / a.S), dd = static_cast<int32_t>(it - static_cast<int64_t>(b) * a.S);
      const int64_t at = static_cast<int64_t>(count) - 1 - base - k;
      a.block_table[table_row(a, b, dd) + first_col[lo] + (k - start[lo])] = at >= 0 ? __ldg(a.free_blocks + at) : -1;
    }
    base += total;
    __syncthreads();
  }
  if (tid == 0) {
    if (base > count) err |= DCP_DEVERR_NO_BLOCKS;
    *a.free_left = base < count ? static_cast<int32_t>(count - base) : 0;
  }
  if (err && a.dev_error) atomicOr(a.dev_error, static_cast<int32_t>(err));
  if (!fused) return;
  // (the last round's barrier, or none when there are no tables, orders the
  // entries before these reads)
  for (int32_t t = tid; t < a.T; t += kThreads) {
    RequestOfRow q{-1, 0, 0, 0};
    if (!kept) {
      q = request_of_row(a.seq_lens, a.qsl, a.B, t);
    } else if (a.B > 0 && t >= kept_qsl[0] && t < kept_qsl[a.B]) {
      int32_t lo = 0, hi = a.B;  // kept_qsl[lo] <= t < kept_qsl[hi]
      while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (kept_qsl[mid] <= t) lo = mid; else hi = mid;
      }
      q = RequestOfRow{lo, kept_qsl[lo], kept_qsl[lo + 1], kept_seq[lo]};
    }
    place(a, t, q.b, q.q0, q.q1, q.seq);
  }
}

__global__ void __launch_bounds__(kTokenThreads) extend_tokens_kernel(CacheExtendArgs a) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokenThreads + threadIdx.x;
  RequestOfRow q{-1, 0, 0, 0};
  if (t < a.T) q = request_of_row(a.seq_lens, a.qsl, a.B, static_cast<int32_t>(t));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t < a.T) place(a, static_cast<int32_t>(t), q.b, q.q0, q.q1, q.seq);
}

}  // namespace

cudaError_t launch_cache_extend(const CacheExtendArgs& a, cudaStream_t st) {
  const int fused = a.T <= kFusedTokens;
  extend_kernel<<<1, kThreads, 0, st>>>(a, fused);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || fused) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((static_cast<unsigned>(a.T) + kTokenThreads - 1) / kTokenThreads);
  cfg.blockDim = dim3(kTokenThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, extend_tokens_kernel, a);
}

}  // namespace dcp
