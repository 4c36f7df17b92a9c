// Latent-cache read-back: context ranges of a batch of requests gathered from
// the paged cache (either table layout, bf16 or FP8 E4M3) into dense rows, for
// a prefill over a cached prefix, a cache migration or an inspection.
//
//   out[n] = value of position p = seq_starts[b] + n - cu_lens[b],
//            cu_lens[b] <= n < cu_lens[b + 1]
// (code x scale in fp32, rounded once to the output's type; positions that
// belong to shards outside the call's range give zero rows, so that ranks'
// outputs add up to the whole).
//
// A pure copy, bound by DRAM: 1152 (bf16) or 580 (FP8) bytes read and 1152 or
// 2304 written per row.  A warp takes eight consecutive output rows, as 8-
// element units (16 or 8 bytes in, 16 or 32 out): 8 x 72 units are 18 full
// rounds of 32 lanes, nine loads in flight at a time.  Consecutive output rows
// are nearly always the same request's, so its index is searched once per
// warp, 32 ways at a time (two rounds of loads for up to 1,024 requests), and
// lanes 0-7 then walk the block table for one row each.
#include "dcp_kernels.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

namespace dcp {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 8;              // output rows per warp
constexpr int kUnits = kKDim / 8;     // 72 8-element units per row
constexpr int kRounds = kRows * kUnits / 32;
constexpr int kBatch = kRounds / 2;
constexpr unsigned kFull = 0xffffffffu;

// The last request whose cu_lens is <= n (cu[0] <= n < cu[B] given), by the
// whole warp.
__device__ __forceinline__ int32_t request_of(const int32_t* __restrict__ cu, int32_t B, int64_t n, int lane) {
  int32_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) / 32;
    const int64_t at = static_cast<int64_t>(lo) + static_cast<int64_t>(lane + 1) * step;
    const bool le = at < hi && __ldg(cu + at) <= n;
    const int32_t k = __popc(__ballot_sync(kFull, le));
    const int64_t next = static_cast<int64_t>(lo) + static_cast<int64_t>(k + 1) * step;
    lo += k * step;
    hi = next < hi ? static_cast<int32_t>(next) : hi;
  }
  return lo;
}

__device__ __forceinline__ uint32_t widen2(uint32_t codes, float s, float2& f) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  f = __half22float2(*reinterpret_cast<const __half2*>(&h));  // exact
  f.x *= s;
  f.y *= s;
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <bool kFp8, bool kF32>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheReadArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRows;
  if (n0 >= a.N) return;
  const int32_t first = __ldg(a.cu_lens), last = __ldg(a.cu_lens + a.B);
  if (n0 + kRows <= first || n0 >= last) return;  // rows of no request: left as they are
  // lanes 0-7: one output row each; row[l] is its cache row, -1 for a zero
  // row, -2 for a row that is not written
  const int64_t lo_n = n0 > first ? n0 : first;
  const int64_t hi_n = (n0 + kRows < last ? n0 + kRows : last) - 1;
  int32_t b = request_of(a.cu_lens, a.B, lo_n, lane);
  const bool same = __ldg(a.cu_lens + b + 1) > hi_n;
  int64_t row = -2;
  float scale = 0.f;
  const int64_t n = n0 + lane;
  if (lane < kRows && n < a.N && n >= lo_n && n <= hi_n) {
    if (!same) {
      int32_t lo = b, hi = a.B;
      while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (__ldg(a.cu_lens + mid) <= n) lo = mid; else hi = mid;
      }
      b = lo;
    }
    const int64_t p = (a.seq_starts ? __ldg(a.seq_starts + b) : 0) + (n - __ldg(a.cu_lens + b));
    row = -1;
    bool bad = p < 0 || p > 0x7fffffffLL;
    if (!bad) {
      const int32_t pos = static_cast<int32_t>(p);
      const int32_t run = fast_div(pos, a.div_I), turn = fast_div(run, a.div_D);
      const int32_t d = run - turn * a.D;  // the shard that owns the position
      if (d >= a.d0 && d < a.d0 + a.Dn) {
        const int32_t j = a.local_tables ? turn * a.I + (pos - run * a.I) : pos;
        const int32_t col = fast_div(j, a.div_bs);
        if (col < a.bt_width) {
          const int32_t blk = __ldg(a.block_table + (a.local_tables ? (d - a.d0) * a.bt_shard_stride : 0) +
                                    static_cast<int64_t>(b) * a.bt_stride + col);
          if (blk >= 0 && blk < a.num_blocks) {
            row = static_cast<int64_t>(blk) * a.block_size + (j - col * a.block_size);
            if (kFp8) scale = __ldg(a.kv_scale + row);
          } else {
            bad = true;
          }
        } else {
          bad = true;
        }
      }
    }
    if (bad && a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_BAD_BLOCK);
  }
  using InT = typename std::conditional<kFp8, uint2, uint4>::type;
#pragma unroll
  for (int half = 0; half < kRounds / kBatch; ++half) {
    InT v[kBatch];
    int64_t src[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = 32 * (half * kBatch + i) + lane, r = u / kUnits, c = u - r * kUnits;
      src[i] = __shfl_sync(kFull, row, r);
      v[i] = InT{};
      if (src[i] >= 0)
        v[i] = __ldcs(reinterpret_cast<const InT*>(static_cast<const unsigned char*>(a.kv) + src[i] * (kKDim * (kFp8 ? 1 : 2))) + c);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = 32 * (half * kBatch + i) + lane, r = u / kUnits, c = u - r * kUnits;
      const float s = kFp8 ? __shfl_sync(kFull, scale, r) : 0.f;
      float2 f[4];
      uint32_t h[4];
      if constexpr (kFp8) {
        h[0] = widen2(v[i].x, s, f[0]);
        h[1] = widen2(v[i].x >> 16, s, f[1]);
        h[2] = widen2(v[i].y, s, f[2]);
        h[3] = widen2(v[i].y >> 16, s, f[3]);
      } else {
        h[0] = v[i].x, h[1] = v[i].y, h[2] = v[i].z, h[3] = v[i].w;
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = make_float2(__uint_as_float(h[k] << 16), __uint_as_float(h[k] & 0xffff0000u));
      }
      if (src[i] == -2) continue;
      if constexpr (kF32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + (n0 + r) * a.out_stride + 8 * c);
        __stcs(o, make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
        __stcs(o + 1, make_float4(f[2].x, f[2].y, f[3].x, f[3].y));
      } else {
        __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (n0 + r) * a.out_stride + 8 * c),
               make_uint4(h[0], h[1], h[2], h[3]));
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t st) {
  if (a.N <= 0) return cudaSuccess;
  constexpr int kPerCta = kRows * (kThreads / 32);
  const int64_t ctas = (a.N + kPerCta - 1) / kPerCta;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(ctas);
  if (a.kv_scale) {
    if (a.out_f32) cache_read_kernel<true, true><<<grid, kThreads, 0, st>>>(a);
    else cache_read_kernel<true, false><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (a.out_f32) cache_read_kernel<false, true><<<grid, kThreads, 0, st>>>(a);
    else cache_read_kernel<false, false><<<grid, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace dcp
