// The decode step before attention, in one launch: the decode query
// q = [ql_nope | q_pe] (576 bf16 per head) and the write of this step's latent
// rows [kv_c | k_pe] into the paged cache at slot_mapping ("[Kimi-K3] DCP
// support" summary on prhub.com.cn, key snippet "Decode: latent multi-query
// attention": _decode_concat_cache runs before forward_mqa, so the decode
// sees the new tokens).  Byte copies only (bit-exact), in 16-byte units.
//
// One CTA per token: its eight warps copy the token's H query heads (72
// 16-byte units per head: 64 of ql_nope, then 8 of q_pe), and warp 0 also
// copies its cache row when the slot is set.  A negative slot is not written
// (a padding token, or a token another DCP rank owns); a slot past the cache
// is not written either and sets DCP_DEVERR_BAD_BLOCK.
//
// The general form (launch_concat_cache_v2) also writes an FP8 E4M3 cache, and
// may write the cache alone: see its kernel below.
#include "dcp_kernels.h"

#include <cuda_fp8.h>

namespace dcp {
namespace {

constexpr int kThreads = 256;
constexpr int kUnitsNope = kLatent * 2 / 16;  // 64 16-byte units of ql_nope / kv_c
constexpr int kUnitsRope = kRope * 2 / 16;    // 8 of q_pe / k_pe
constexpr int kUnitsRow = kUnitsNope + kUnitsRope;

__device__ __forceinline__ uint4 ld_nc(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

__global__ void __launch_bounds__(kThreads) concat_cache_kernel(ConcatCacheArgs a) {
  const int t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned char* nope = reinterpret_cast<const unsigned char*>(a.ql_nope) + 2 * t * a.ql_nope_stride_tok;
  const unsigned char* pe = reinterpret_cast<const unsigned char*>(a.q_pe) + 2 * t * a.q_pe_stride_tok;
  unsigned char* qo = reinterpret_cast<unsigned char*>(a.q_out) + 2 * t * a.q_out_stride_tok;
  for (int h = warp; h < a.H; h += kThreads / 32) {
    const unsigned char* n = nope + 2 * h * a.ql_nope_stride_head;
    const unsigned char* p = pe + 2 * h * a.q_pe_stride_head;
    uint4* dst = reinterpret_cast<uint4*>(qo + 2 * h * kKDim);
    for (int u = lane; u < kUnitsRow; u += 32) dst[u] = u < kUnitsNope ? ld_nc(n + 16 * u) : ld_nc(p + 16 * (u - kUnitsNope));
  }
  if (warp == 0) {
    const int64_t slot = __ldg(a.slot_mapping + t);
    if (slot >= a.num_slots) {
      if (lane == 0 && a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_BAD_BLOCK);
    } else if (slot >= 0) {
      const unsigned char* c = reinterpret_cast<const unsigned char*>(a.kv_c) + 2 * t * a.kv_c_stride_tok;
      const unsigned char* k = reinterpret_cast<const unsigned char*>(a.k_pe) + 2 * t * a.k_pe_stride_tok;
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(a.kv_cache) + slot * (2 * kKDim));
      for (int u = lane; u < kUnitsRow; u += 32) dst[u] = u < kUnitsNope ? ld_nc(c + 16 * u) : ld_nc(k + 16 * (u - kUnitsNope));
    }
  }
}

// ---------------------------------------------------------------------------
// general form: bf16 or FP8 E4M3 cache, with or without the query
// ---------------------------------------------------------------------------
// The codes of a row x[576] with power-of-two scale s = 2^e, the least with
// max |x| <= 256 s (over the finite x; s = 1 for a row of zeros): code_i is
// x_i / s rounded once to the nearest E4M3 value, ties to even.  x / s only
// moves the exponent, so it is exact before that rounding, as is the decode's
// code x s after it.  A scale that used the format's last octave (448) would
// save no step: a float's relative step does not depend on the scale.
// NaN and infinities become the NaN code.
//
// One warp per cache row (lane: 16-byte units lane, lane + 32 of kv_c and, on
// lanes 0-7, one of k_pe, so that the row is read once and stays in
// registers between the max and the conversion) and one per four query heads
// (288 units: nine full rounds, all nine loads in flight).  No shared memory,
// no barrier: bound by bytes, and for a single token by one round trip to
// memory.
constexpr int kHeadsPerWarp = 4;
constexpr int kThreadsV2 = 128;

// least e with A <= 256 * 2^e for a positive finite A (its fp32 bits): A is
// f 2^k with f in [1, 2), so e = k - 8, one more unless f == 1
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  int k = static_cast<int>(bits >> 23) - 127;
  uint32_t frac = bits & 0x7fffffu;
  if ((bits >> 23) == 0) {  // subnormal: value = frac 2^-149
    const int top = 31 - __clz(static_cast<int>(frac));
    k = top - 149;
    frac ^= 1u << top;
  }
  return k - 8 + (frac != 0 ? 1 : 0);
}
// 2^e for e in [-149, 127]
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(e >= -126 ? static_cast<uint32_t>(e + 127) << 23 : 1u << (e + 149));
}

__device__ __forceinline__ uint32_t abs_max(uint32_t m, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (w[i] << 16) & 0x7fff0000u, hi = w[i] & 0x7fff0000u;  // fp32 bits of |x|
    m = max(m, lo < 0x7f800000u ? lo : 0u);                                  // finite values only
    m = max(m, hi < 0x7f800000u ? hi : 0u);
  }
  return m;
}

// two bf16 (packed) times 2^a 2^b -> two E4M3 codes
__device__ __forceinline__ uint32_t to_codes(uint32_t w, float pa, float pb) {
  float2 f = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  // infinities: to NaN, which converts to the NaN code (the conversion would
  // saturate them)
  if ((w & 0x7f80u) == 0x7f80u) f.x = __uint_as_float(0x7fc00000u);
  if ((w & 0x7f800000u) == 0x7f800000u) f.y = __uint_as_float(0x7fc00000u);
  f.x = f.x * pa * pb;
  f.y = f.y * pa * pb;
  return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 to_codes8(const uint4& v, float pa, float pb) {
  return make_uint2(to_codes(v.x, pa, pb) | to_codes(v.y, pa, pb) << 16,
                    to_codes(v.z, pa, pb) | to_codes(v.w, pa, pb) << 16);
}

template <bool kFp8, bool kQuery>
__global__ void __launch_bounds__(kThreadsV2) concat_cache_v2_kernel(ConcatCacheArgs a, int warps_per_token) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreadsV2 / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = kQuery ? w / warps_per_token : w;
  const int part = kQuery ? static_cast<int>(w - t * warps_per_token) : 0;
  if (t >= a.T) return;
  if (part == 0) {
    // this token's cache row
    const int64_t slot = __ldg(a.slot_mapping + t);
    const uint4* c = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.kv_c) + 2 * t * a.kv_c_stride_tok);
    const uint4* k = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.k_pe) + 2 * t * a.k_pe_stride_tok);
    // (loaded before the slot is known: one round trip in all)
    const uint4 v0 = ld_nc(c + lane), v1 = ld_nc(c + lane + 32);
    const uint4 v2 = lane < kUnitsRope ? ld_nc(k + lane) : make_uint4(0u, 0u, 0u, 0u);
    if (slot >= a.num_slots) {
      if (lane == 0 && a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_BAD_BLOCK);
      return;
    }
    if (slot < 0) return;
    if constexpr (kFp8) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, abs_max(abs_max(abs_max(0u, v0), v1), v2));
      const int e = top != 0 ? scale_exponent(top) : 0;
      // 1 / s as two factors: -e may reach 141, past fp32's largest power
      const float pa = pow2(-e / 2), pb = pow2(-e - (-e / 2));
      uint2* dst = reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.kv_cache) + slot * kKDim);
      dst[lane] = to_codes8(v0, pa, pb);
      dst[lane + 32] = to_codes8(v1, pa, pb);
      if (lane < kUnitsRope) dst[lane + kUnitsNope] = to_codes8(v2, pa, pb);
      if (lane == 0) a.kv_scale[slot] = pow2(e);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.kv_cache) + slot * (2 * kKDim));
      dst[lane] = v0;
      dst[lane + 32] = v1;
      if (lane < kUnitsRope) dst[lane + kUnitsNope] = v2;
    }
    return;
  }
  if constexpr (!kQuery) return;
  const int h0 = (part - 1) * kHeadsPerWarp;
  const int n = min(kHeadsPerWarp, a.H - h0) * kUnitsRow;  // 16-byte units of this warp's heads
  const unsigned char* nope = static_cast<const unsigned char*>(a.ql_nope) + 2 * (t * a.ql_nope_stride_tok + h0 * a.ql_nope_stride_head);
  const unsigned char* pe = static_cast<const unsigned char*>(a.q_pe) + 2 * (t * a.q_pe_stride_tok + h0 * a.q_pe_stride_head);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.q_out) + 2 * (t * a.q_out_stride_tok + static_cast<int64_t>(h0) * kKDim));
  constexpr int kRounds = kHeadsPerWarp * kUnitsRow / 32;
  uint4 v[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int u = 32 * i + lane, h = u / kUnitsRow, c = u - h * kUnitsRow;
    if (u < n)
      v[i] = c < kUnitsNope ? ld_nc(nope + 2 * h * a.ql_nope_stride_head + 16 * c)
                            : ld_nc(pe + 2 * h * a.q_pe_stride_head + 16 * (c - kUnitsNope));
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
    if (32 * i + lane < n) dst[32 * i + lane] = v[i];
}

}  // namespace

cudaError_t launch_concat_cache_v2(const ConcatCacheArgs& a, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  const int per_token = 1 + (a.H + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const int64_t ctas = (static_cast<int64_t>(a.T) * per_token + kThreadsV2 / 32 - 1) / (kThreadsV2 / 32);
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(ctas);
  // (without the query's nine loads a thread takes fewer registers: more rows
  // in flight)
  const auto kernel = a.kv_scale ? (a.H > 0 ? concat_cache_v2_kernel<true, true> : concat_cache_v2_kernel<true, false>)
                                 : (a.H > 0 ? concat_cache_v2_kernel<false, true> : concat_cache_v2_kernel<false, false>);
  kernel<<<grid, kThreadsV2, 0, st>>>(a, per_token);
  return cudaGetLastError();
}

cudaError_t launch_concat_cache(const ConcatCacheArgs& a, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  concat_cache_kernel<<<a.T, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace dcp
