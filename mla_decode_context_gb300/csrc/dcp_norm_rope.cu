// Norm of the latent, rotation of the rope parts by their positions, query
// concat and paged-cache write (bf16 or FP8 E4M3) in one launch: what turns a
// step's projections into the decode's query and cache rows.
//
//   c  = kv_c * rsqrt(mean(kv_c^2) + eps) * norm_weight        (512 dims)
//   rotation by (cos, sin) of the token's position, on 32 pairs of rope dims:
//   (x, y) -> (x cos - y sin, y cos + x sin); pairs are (2i, 2i + 1), or
//   (i, i + 32)
//   cache row = [c | rotated k_pe];  q_out = [ql_nope | rotated q_pe]
//
// All in fp32, rounded once: to bf16, or (FP8 cache) to the code of x / 2^e
// with the row's power-of-two scale (dcp_concat_cache.cu), taken from the fp32
// values.
//
// Few operations a byte, and for one token one round trip to memory, so the work
// is cut into warps without shared memory or barriers: one warp per cache row
// (16 latent values a lane, the rope part on lanes 0-7; the sum of squares and
// the maximum are warp reductions), one per four decode-query heads (eight
// rounds of 16-byte units of ql_nope, and one in which lane = (head, rope
// unit): its angles are loaded once), or one per 16 heads of a chunk's queries
// (rope parts alone, four rounds with the same angles).  A pair that is 32
// dims apart lies four lanes apart.  What bounds it is the latency of two
// dependent trips to memory (position, then angles) under the warps that fit: 56
// registers a thread, 64 with split halves, so nine or eight CTAs, 36 or 32 warps, an
// SM.  256 tokens with 128 heads into an FP8 cache (76 MB read and written): 14 us,
// of which DRAM is busy a third (the output stays in L2); the rope parts of 4,099
// tokens' 128 heads in pieces of 128 bytes (145 MB): 28 us, DRAM 44 % busy; 16,381
// rows alone: 13-14 us, three waves of warps, DRAM 20 % busy.
#include "dcp_kernels.h"

#include <cuda_fp8.h>

namespace dcp {
namespace {

constexpr int kThreads = 128;
constexpr int kUnitsNope = kLatent / 8;  // 64 16-byte units of a latent
constexpr int kUnitsRope = kRope / 8;    // 8
constexpr int kHeadsDecode = 4;          // query heads per warp, with ql_nope
constexpr int kHeadsRope = 16;           // and without
constexpr int kHalf = kRope / 2;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t narrow2(float x, float y) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(narrow2(f[0], f[1]), narrow2(f[2], f[3]), narrow2(f[4], f[5]), narrow2(f[6], f[7]));
}

// Cosines and sines of a rope unit's dims 8 j .. 8 j + 7 (of its four pairs,
// or one per dim).
template <bool kPairs>
struct Angles {
  float c[kPairs ? 4 : 8], s[kPairs ? 4 : 8];
  __device__ __forceinline__ void load(const float* __restrict__ row, int j) {
    constexpr int n = kPairs ? 4 : 8;
    const int i = kPairs ? 4 * j : 8 * (j & 3);
#pragma unroll
    for (int k = 0; k < n; k += 4) {
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row) {
        x = __ldg(reinterpret_cast<const float4*>(row + i + k));
        y = __ldg(reinterpret_cast<const float4*>(row + kHalf + i + k));
      }
      c[k] = x.x, c[k + 1] = x.y, c[k + 2] = x.z, c[k + 3] = x.w;
      s[k] = y.x, s[k + 1] = y.y, s[k + 2] = y.z, s[k + 3] = y.w;
    }
  }
  // by the whole warp: lane ^ 4 holds the other half's dims
  __device__ __forceinline__ void turn(float (&f)[8], int j) const {
    if constexpr (kPairs) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = f[2 * k], y = f[2 * k + 1];
        f[2 * k] = x * c[k] - y * s[k];
        f[2 * k + 1] = y * c[k] + x * s[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float other = __shfl_xor_sync(kFull, f[k], 4);
        f[k] = (j & 4) ? f[k] * c[k] + other * s[k] : f[k] * c[k] - other * s[k];
      }
    }
  }
};

// least e >= -126 with A <= 256 * 2^e, for a positive finite A (its fp32 bits)
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) != 0 ? 1 : 0);
  return e < -126 ? -126 : e;  // (subnormals too)
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ uint32_t finite_max(uint32_t m, const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;
    m = max(m, b < 0x7f800000u ? b : 0u);
  }
  return m;
}
__device__ __forceinline__ float for_code(float x, float inv) {
  // infinities: to NaN, which converts to the NaN code (the conversion would saturate them)
  return (__float_as_uint(x) & 0x7fffffffu) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : x * inv;
}
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(for_code(f[2 * i], inv), for_code(f[2 * i + 1], inv)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// kQuery: 0 none, 1 with ql_nope, 2 rope parts alone
template <bool kFp8, int kQuery, bool kPairs>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeArgs a, int warps_per_token) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = kQuery ? w / warps_per_token : w;
  const int part = kQuery ? static_cast<int>(w - t * warps_per_token) : 0;
  if (t >= a.T) return;
  const int32_t pos = __ldg(a.positions + t);
  const float* angles = pos >= 0 && pos < a.max_pos ? a.cos_sin + static_cast<int64_t>(pos) * kRope : nullptr;
  const int j = lane & 7;
  if (part == 0) {
    const uint4* c = reinterpret_cast<const uint4*>(a.kv_c + t * a.kv_c_stride_tok);
    const uint4* k = reinterpret_cast<const uint4*>(a.k_pe + t * a.k_pe_stride_tok);
    const uint4 v0 = __ldg(c + lane), v1 = __ldg(c + lane + 32);
    const uint4 v2 = lane < kUnitsRope ? __ldg(k + lane) : make_uint4(0u, 0u, 0u, 0u);
    const int64_t slot = __ldg(a.slot_mapping + t);
    uint4 w0{}, w1{};
    if (a.norm_weight) {
      w0 = __ldg(reinterpret_cast<const uint4*>(a.norm_weight) + lane);
      w1 = __ldg(reinterpret_cast<const uint4*>(a.norm_weight) + lane + 32);
    }
    uint32_t err = pos >= a.max_pos ? DCP_DEVERR_BAD_POSITION : 0;
    if (slot >= a.num_slots) err |= DCP_DEVERR_BAD_BLOCK;
    if (err && lane == 0 && a.dev_error) atomicOr(a.dev_error, static_cast<int32_t>(err));
    if (slot < 0 || slot >= a.num_slots) return;
    Angles<kPairs> ang;
    ang.load(angles, j);
    float f0[8], f1[8], f2[8];
    widen8(v0, f0);
    widen8(v1, f1);
    widen8(v2, f2);
    if (a.norm_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f0[i], f0[i], fmaf(f1[i], f1[i], ss));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      const float x = ss * (1.0f / kLatent) + a.eps;
      const float r = 1.0f / sqrtf(x);
      // What the roundings of r and of the product with it left goes into the last
      // product: fewer FP8 codes next to the border take the wrong side (16,381
      // tokens' rows against 64 bits' codes: 3e-5 in 2-norm, 6e-5 without), and the
      // time stays as it was.
      const float xr = x * r;
      float r_lo = 0.5f * r * (fmaf(-xr, r, 1.0f) - fmaf(x, r, -xr) * r);
      if (!(fabsf(r_lo) < r)) r_lo = 0.f;  // (r is 0 or infinity)
      auto normed = [&](float f, float g) {
        const float p = f * r, lo = fmaf(f, r_lo, fmaf(f, r, -p));
        return fmaf(p, g, lo * g);
      };
      float g0[8], g1[8];
      widen8(w0, g0);
      widen8(w1, g1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f0[i] = normed(f0[i], g0[i]);
        f1[i] = normed(f1[i], g1[i]);
      }
    }
    ang.turn(f2, j);
    if constexpr (kFp8) {
      uint32_t top = finite_max(finite_max(0u, f0), f1);
      if (lane < kUnitsRope) top = finite_max(top, f2);
      top = __reduce_max_sync(kFull, top);
      const int e = top != 0 ? scale_exponent(top) : 0;
      const float inv = pow2(-e);
      uint2* dst = reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.kv_cache) + slot * kKDim);
      dst[lane] = codes8(f0, inv);
      dst[lane + 32] = codes8(f1, inv);
      if (lane < kUnitsRope) dst[lane + kUnitsNope] = codes8(f2, inv);
      if (lane == 0) a.kv_scale[slot] = pow2(e);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.kv_cache) + slot * (2 * kKDim));
      dst[lane] = narrow8(f0);
      dst[lane + 32] = narrow8(f1);
      if (lane < kUnitsRope) dst[lane + kUnitsNope] = narrow8(f2);
    }
    return;
  }
  if constexpr (kQuery == 1) {
    const int h0 = (part - 1) * kHeadsDecode;
    const int heads = min(kHeadsDecode, a.H - h0);
    const __nv_bfloat16* nope = a.ql_nope + t * a.ql_nope_stride_tok + h0 * a.ql_nope_stride_head;
    __nv_bfloat16* out = a.q_out + t * a.q_out_stride_tok + h0 * a.q_out_stride_head;
    const int hr = lane >> 3;  // the rope round's head
    uint4 v[2 * kHeadsDecode], r = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 2 * kHeadsDecode; ++i)
      if (i / 2 < heads) v[i] = __ldg(reinterpret_cast<const uint4*>(nope + (i / 2) * a.ql_nope_stride_head) + 32 * (i & 1) + lane);
    if (hr < heads) r = __ldg(reinterpret_cast<const uint4*>(a.q_pe + t * a.q_pe_stride_tok + (h0 + hr) * a.q_pe_stride_head) + j);
    Angles<kPairs> ang;
    ang.load(angles, j);
#pragma unroll
    for (int i = 0; i < 2 * kHeadsDecode; ++i)
      if (i / 2 < heads) *(reinterpret_cast<uint4*>(out + (i / 2) * a.q_out_stride_head) + 32 * (i & 1) + lane) = v[i];
    float f[8];
    widen8(r, f);
    ang.turn(f, j);
    if (hr < heads) *(reinterpret_cast<uint4*>(out + hr * a.q_out_stride_head + kLatent) + j) = narrow8(f);
  }
  if constexpr (kQuery == 2) {
    // (q_out may be q_pe: each unit is read, by its own warp, before it is
    // written; no read-only loads)
    constexpr int kRounds = kHeadsRope / 4;
    const int h0 = (part - 1) * kHeadsRope + (lane >> 3);
    uint4 v[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h0 + 4 * i < a.H)
        v[i] = *(reinterpret_cast<const uint4*>(a.q_pe + t * a.q_pe_stride_tok + (h0 + 4 * i) * a.q_pe_stride_head) + j);
    }
    Angles<kPairs> ang;
    ang.load(angles, j);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      float f[8];
      widen8(v[i], f);
      ang.turn(f, j);
      if (h0 + 4 * i < a.H)
        *(reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride_tok + (h0 + 4 * i) * a.q_out_stride_head) + j) = narrow8(f);
    }
  }
}

template <bool kFp8, int kQuery>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t st) {
  const int heads = kQuery == 1 ? kHeadsDecode : kHeadsRope;
  const int per_token = 1 + (kQuery ? (a.H + heads - 1) / heads : 0);
  const int64_t ctas = (static_cast<int64_t>(a.T) * per_token + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.pairs) norm_rope_kernel<kFp8, kQuery, true><<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(a, per_token);
  else norm_rope_kernel<kFp8, kQuery, false><<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(a, per_token);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  if (a.H == 0) return a.kv_scale ? launch<true, 0>(a, st) : launch<false, 0>(a, st);
  if (a.ql_nope) return a.kv_scale ? launch<true, 1>(a, st) : launch<false, 1>(a, st);
  return a.kv_scale ? launch<true, 2>(a, st) : launch<false, 2>(a, st);
}

}  // namespace dcp
