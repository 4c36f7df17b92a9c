// Chunk attention, second half: causal attention of a chunk's query rows over
// the keys and values that dcp_chunk_expand.cu left as tile images.
//
//   s = scale (q_nope . k_h(p) + q_rope . k_pe(p)),  p < L_r = seq - (q_len - 1 - i)
//   out = sum_p exp(s - lse) v_h(p),  lse = ln sum_p exp(s)
//
// 2 x (192 + 128) operations per (row, token, head): bound by the tensor pipe.
// Unit: 256 rows of one request at one head (cut into pieces along its tokens
// where there are few or uneven units, dcp_chunk_plan.cu), as two MMA tiles of 128
// rows that share each tile of 128 keys and values in shared memory and take turns
// on the tensor pipe: while one's scores go through the softmax, the other's products
// run.  TMEM holds both tiles' scores (128 columns each; the weights P replace
// them as f16) and both outputs (128 columns each): all 512 columns.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax of tile 0, 1 (thread = row = TMEM lane): Q into shared
//                   memory, running maximum and sum, P, the rare rescale of O,
//                   and the output
//   warp 8          MMA issuer: per tile j and group: PV(j - 1), then S(j)
//   warp 9          loads: bulk copies of 16 KB images into a ring of 8 slots (a
//                   tile takes three for K, two for V)
//   warp 10         TMEM allocation
//   warp 11         gate: waits for V(j) and adds its arrival to the softmax's,
//                   so that the issuer has one barrier to wait for (a wait takes
//                   ~200 cycles even when nothing is left to wait for)
// The running maximum moves only when a row's scores grow past it by 2^8, so O is
// rescaled a few times per unit at most.
//
// 2,048 rows on 21,952 tokens at 128 heads: ~2.30 ms, 1.68 PFLOP/s (87 % of the
// measured burst rate, 97 % of the sustained one).  128 tokens take 3,200-3,400
// cycles, 2,560 of them MMAs: a group's chain (S 770, softmax ~1,450, PV 510, and
// ~600 of commits and waits) is that long, and two groups share it.  Setting a unit
// up takes ~5 us, its output ~3.
//
// Roundings: keys (in long requests) and values to f16 once (they are MMA
// operands), P to f16 once, the output once.  Scores, maxima, sums and O are
// fp32.  Queries are f16 exactly: each row is scaled by a power of 2 that makes
// its largest element 1 to 4, and what is left behind lies 2^-25 below that.
#include "dcp_chunk.cuh"

#include <cuda_fp16.h>

#include <cmath>
#include <mutex>
#include <type_traits>

namespace dcp {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kGroup = 128;       // threads of a softmax group
constexpr uint32_t kSlots = 8;         // ring of images
constexpr int kQChunks = 3, kVChunks = 2;  // images of a tile's keys (two more where they have remainders) and values
constexpr int kMaskSlots = 4;     // ring of the tiles' token masks
constexpr int kOffQ = 0;          // two query tiles of 3 images
constexpr int kOffRing = 2 * kQChunks * kImage;
constexpr int kOffMask = kOffRing + kSlots * kImage;  // kMaskSlots x (valid, bad)
constexpr int kOffBars = kOffMask + kMaskSlots * 32;
constexpr float kRescaleLog2 = 8.0f;
// P carries this power of 2: with the 2^8 above, up to 2^14 (f16 ends at 2^16),
// and down to 2^-30 of the largest weight.
constexpr float kLift = 6.0f;
// s c - m in one rounding leaves what m lost by its own: at most 1 up to here, and
// past it more than f16 takes.  (Taking the maximum off before scaling has no
// such end, and cost 7 % of the time.)  A maximum below -kFarthest counts as that: what
// lies there weighs nothing beside any score that may still come, and a row that
// sees no others is NaN.  A piece of a cut unit cannot know: its log-sum-exp is
// kFar, which the join takes for NaN where no piece has more.
constexpr float kFarthest = 33554432.0f;
constexpr float kFar = -3.402823466e38f;  // (the lowest finite number; no log-sum-exp comes near it)

struct Bars {
  uint64_t q_full[2];                  // a group's Q is in shared memory (128)
  uint64_t k_full[2], v_full[2];       // K(j), V(j) are in the ring (barrier j mod 2)
  uint64_t k_free[2], v_free[2];       // both groups are done with them
  uint64_t mask_full[kMaskSlots];
  uint64_t s_full[2];                  // S_g(j) is in TMEM and PV_g(j - 1) complete; last, PV_g of the last tile
  uint64_t p_full[2];                  // P_g(j) is in TMEM and O_g in its scale (4 warps); V(j) is there (gate)
  uint64_t fin;
  uint32_t tmem;
  int32_t live;                        // this CTA has a piece
  int32_t head;                        // of this pass
  int32_t q_exp[2][128];               // row r of group g: its queries are multiplied by 2^-q_exp
  Piece piece;
};
constexpr int kSmemBytes = kOffBars + static_cast<int>(sizeof(Bars)) + 1024;
static_assert(kSmemBytes <= 232448, "exceeds the 227 KB of shared memory per CTA");

// registers per thread: eight softmax warps take what the other four leave
constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * kRegsLaunch, "more than was launched");

constexpr uint32_t kColS = 0, kColO = 256;  // group g: + 128 g

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// CTA `i` of a pass: segments of similar length, within them the heads outermost.
__device__ __forceinline__ bool piece_of(const ChunkArgs& a, int32_t i, Piece& p, int32_t& head) {
  const int32_t at = i / a.heads;
  const int32_t n = *a.num_pieces;
  p = a.pieces[at];  // (whatever it holds past the last one)
  if (at >= n) return false;
  const int32_t in = i - p.seg0 * a.heads;
  head = in / p.seg;
  const int32_t to = p.seg0 + (in - head * p.seg);
  if (to != at) p = a.pieces[to];
  return true;
}

// The rows of this group's tile that exist, and the key tiles of this piece that
// they need.
struct Tile {
  int32_t first, rows;  // row of the request, number of rows
  int32_t tiles;
};
__device__ __forceinline__ Tile tile_of(const Bars& bar, int g) {
  Tile t;
  const int32_t q_len = bar.piece.q1 - bar.piece.q0;
  t.first = bar.piece.block * kChunkRows + 128 * g;
  t.rows = max(0, min(128, q_len - t.first));
  // what the last row sees
  const int64_t end = static_cast<int64_t>(bar.piece.seq) - (q_len - 1) + (t.first + t.rows - 1);
  const int32_t tiles = t.rows > 0 && end > 0 ? static_cast<int32_t>((end + kChunkTile - 1) / kChunkTile) : 0;
  t.tiles = max(0, min(tiles, bar.piece.j1) - bar.piece.j0);
  return t;
}

// The issuing lane's work on tile j for group g: PV(j - 1), then S(j).
struct Issue {
  Bars& bar;
  const uint64_t dq, dring;
  const int32_t n0, n1;
  bool ok;

  // k0: K(j)'s first image; fine: keys have remainders, images 3 and 4 of a tile
  template <int g, bool fine>
  __device__ __forceinline__ void step(int32_t j, uint32_t k0) {
    const int32_t tiles = g ? n1 : n0, n = n0 > n1 ? n0 : n1;
    if (j >= 1 && j - 1 < tiles && ok) {  // O_g += P_g(j - 1) V(j - 1)
      const uint32_t v0 = (k0 - kVChunks) % kSlots, v1 = (v0 + 1) % kSlots;
      ok = mbar_wait(&bar.p_full[g], (j - 1) & 1);
      if (!ok) return;
      tc_fence_after();
      const uint64_t d = dring + ((v0 * kImage) >> 4);
      constexpr uint32_t o = kColO + 128 * g, p = kColS + 128 * g;
      if (v1 == v0 + 1) {
        constexpr uint32_t id = idesc_f16(128, 128, 0, 1);
        mma_ts(o, p, d, id, j > 1);
#pragma unroll
        for (int k = 1; k < 8; ++k) mma_ts(o, p + 8 * k, d + ((2048 * k) >> 4), id, 1);
      } else {  // (64 dims each from the ring's last and first slot)
        constexpr uint32_t id = idesc_f16(128, 64, 0, 1);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          mma_ts(o, p + 8 * k, d + ((2048 * k) >> 4), id, j > 1 || k > 0);
          mma_ts(o + 64, p + 8 * k, dring + ((2048 * k) >> 4), id, j > 1 || k > 0);
        }
      }
      if (j == tiles) mma_commit(&bar.s_full[g]);
    }
    if (g == 1 && j >= 1) mma_commit(&bar.v_free[(j - 1) & 1]);
    if (j < tiles && ok) {  // S_g(j) = Q_g K(j)^T
      if (j == 0) ok = mbar_wait(&bar.q_full[g], 0);
      if (g == 0 || j >= n0) ok = ok && mbar_wait(&bar.k_full[j & 1], (j >> 1) & 1);  // (else group 0 has waited)
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kQChunks; ++c) {
        const uint64_t q = dq + (((g * kQChunks + c) * kImage) >> 4), k = dring + ((((k0 + c) % kSlots) * kImage) >> 4);
        constexpr uint32_t nope = idesc_f16(128, 128, 0, 0), rope = idesc_bf16(128, 128, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_ss(kColS + 128 * g, q + 2 * i, k + 2 * i, c < 2 ? nope : rope, (c | i) != 0);
      }
      if constexpr (fine) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint64_t q = dq + (((g * kQChunks + c) * kImage) >> 4), k = dring + ((((k0 + kQChunks + c) % kSlots) * kImage) >> 4);
          constexpr uint32_t id = idesc_f16(128, 128, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_ss(kColS + 128 * g, q + 2 * i, k + 2 * i, id, 1);
        }
      }
      mma_commit(&bar.s_full[g]);
    }
    if (g == 1 && j < n) mma_commit(&bar.k_free[j & 1]);
  }
};

// Rows of no request: zeros and -inf.
__device__ void pad_rows(const ChunkArgs& a, int64_t r0, int64_t r1, int32_t h) {
  for (int64_t i = threadIdx.x; i < (r1 - r0) * (kVDim / 4); i += kThreads) {
    const int64_t at = ((r0 + i / (kVDim / 4)) * a.H + h) * kVDim + 4 * (i % (kVDim / 4));
    if (a.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(0.f, 0.f, 0.f, 0.f);
    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = make_uint2(0u, 0u);
  }
  for (int64_t r = r0 + threadIdx.x; r < r1; r += kThreads) a.lse[r * a.H + h] = -INFINITY;
}

// Whether a row sees any of a piece's tokens; `left`: those up to its own, from the
// piece's first.  (Rare, and a call: written out in the kernel it cost the softmax's
// loop 2 % of the time.)
__device__ __noinline__ bool sees_any(const uint4* valid, int32_t tiles, int32_t left) {
  for (int32_t j = 0; j < tiles && left > 0; ++j, left -= kChunkTile) {
    const uint4 v = valid[j];
    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
    for (int w = 0; w < 4; ++w)
      if ((left - 32 * w >= 32 ? vw[w] : left > 32 * w ? vw[w] & ((1u << (left - 32 * w)) - 1u) : 0u) != 0u) return true;
  }
  return false;
}

__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bar = *reinterpret_cast<Bars*>(smem + kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  wait_dependency();
  // ---- the piece
  if (warp == 0) {
    Piece p;
    int32_t head;
    const bool live = piece_of(a, static_cast<int32_t>(blockIdx.x), p, head);
    if (lane == 0) {
      bar.live = live;
      if (live) {
        bar.head = head;
        bar.piece = p;
      }
    }
  }
  if (threadIdx.x == 32) {
    for (int g = 0; g < 2; ++g) {
      mbar_init(&bar.q_full[g], kGroup);
      mbar_init(&bar.s_full[g], 1);
      mbar_init(&bar.p_full[g], 5);
      mbar_init(&bar.k_full[g], 1), mbar_init(&bar.v_full[g], 1);
      mbar_init(&bar.k_free[g], 1), mbar_init(&bar.v_free[g], 1);
    }
    for (int i = 0; i < kMaskSlots; ++i) mbar_init(&bar.mask_full[i], 1);
    mbar_init(&bar.fin, 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (!bar.live) return;
  const int32_t hp = bar.head, h = a.h0 + hp;
  if (bar.piece.b < 0) {  // rows before the first request's and from the last one's end on, 256 to a unit
    const int64_t lead = max(0, min(a.qsl[0], a.T)), tail = max(lead, static_cast<int64_t>(min(a.qsl[a.B], a.T)));
    const int64_t n = lead + a.T - tail;
    const int64_t i0 = static_cast<int64_t>(bar.piece.block) * kChunkRows, i1 = min(n, i0 + kChunkRows);
    if (i0 < i1) {
      const int64_t cut = min(max(lead, i0), i1);
      pad_rows(a, i0, cut, h);
      pad_rows(a, cut + tail - lead, i1 + tail - lead, h);
    }
    return;
  }
  if (warp == 10) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = 0;  // (all 512 columns: the allocation starts at the first)
  const int32_t image0 = bar.piece.image;
  const Tile t0 = tile_of(bar, 0), t1 = tile_of(bar, 1);
  const int32_t n0 = t0.tiles, n1 = t1.tiles, n = max(n0, n1);
  const bool fine = bar.piece.lo >= 0;  // keys have remainders
  auto failed = [&]() {
    if (a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_TIMEOUT);
  };

  if (warp < 8) {
    // -------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int g = warp >> 2, quad = warp & 3, row = threadIdx.x & 127;
    const int32_t tiles = g ? n1 : n0, rows = g ? t1.rows : t0.rows, first = g ? t1.first : t0.first;
    const int64_t r = static_cast<int64_t>(bar.piece.q0) + first + row;  // this thread's query row
    unsigned char* qs = smem + kOffQ + g * (kQChunks * kImage);
    // ---- Q: 24 16-byte units a row, eight lanes per 128-byte line
    if (tiles > 0) {
      const int un = lane & 7;
      const int64_t q0 = static_cast<int64_t>(bar.piece.q0) + first;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const int qr = 32 * quad + i + (lane >> 3);
        const uint32_t bytes = qr < rows && q0 + qr < a.T ? 16u : 0u;
        const __nv_bfloat16* src = a.q + (bytes ? (q0 + qr) * a.q_stride_tok : 0) + h * a.q_stride_head + 8 * un;
#pragma unroll
        for (int c = 0; c < kQChunks; ++c) cp_async16_zfill(smem_u32(qs + c * kImage + image_unit(qr, un)), src + 64 * c, bytes);
      }
      cp_async_commit();
      cp_async_wait<0>();
      // to f16 (rope dims: bf16), each row's largest finite element to [1, 4)
#pragma unroll 1
      for (int i = 0; i < 32; i += 4) {
        const int qr = 32 * quad + i + (lane >> 3);
        uint4* at[kQChunks];
        uint4 v[kQChunks];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kQChunks; ++c) {
          at[c] = reinterpret_cast<uint4*>(qs + c * kImage + image_unit(qr, un));
          v[c] = *at[c];
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t x = w[k] & 0x7fffu, y = (w[k] >> 16) & 0x7fffu;
            top = max(top, max(x < 0x7f80u ? x : 0u, y < 0x7f80u ? y : 0u));
          }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // (an exponent of -126 for subnormals, 0 for a row of zeros; 127 as 126,
        // whose power has a reciprocal)
        const int e = top == 0 ? 0 : min(max(static_cast<int>(top >> 7), 1) - 127, 126);
        if (un == 0) bar.q_exp[g][qr] = e;
        const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int c = 0; c < kQChunks; ++c) {
          uint32_t w[4] = {v[c].x ^ a.q_sign, v[c].y ^ a.q_sign, v[c].z ^ a.q_sign, v[c].w ^ a.q_sign};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x = __uint_as_float(w[k] << 16) * f, y = __uint_as_float(w[k] & 0xffff0000u) * f;
            if (c < 2) {
              const __half2 b = __floats2half2_rn(x, y);
              w[k] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
              const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
              w[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
          }
          *at[c] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      fence_proxy_async_smem();
      mbar_arrive(&bar.q_full[g]);
    }
    const int32_t L = static_cast<int32_t>(max(static_cast<int64_t>(0), static_cast<int64_t>(bar.piece.seq) - (bar.piece.q1 - bar.piece.q0 - 1) + first + row));
    const int32_t L_first = __shfl_sync(0xffffffffu, L, 0);  // the least of the warp's
    const uint32_t ts = tmem + (static_cast<uint32_t>(quad) << 21) + kColS + 128u * g;
    const uint32_t to = ts - kColS + kColO;
    float m = -INFINITY, l = 0.f;  // running maximum (log2, scaled) and sum
    bool ok = true, nan_row = false;
    // (never 0, for 0 x -inf would be NaN: the least number, times which any finite
    // score is next to 0)
    const int qe = tiles > 0 ? bar.q_exp[g][row] : 0;
    const float c1 = fmaxf(1.401298464e-45f, a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + qe) << 23));
    const uint64_t c2 = f2_pack(c1, c1);
    for (int32_t j = 0; j < tiles; ++j) {
      ok = mbar_wait_warp(&bar.mask_full[j % kMaskSlots], (j / kMaskSlots) & 1);  // (long there)
      ok = ok && mbar_wait_warp(&bar.s_full[g], j & 1);
      if (!ok) break;
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, reinterpret_cast<uint32_t(&)[32]>(s[32 * c]));
      const uint4* masks = reinterpret_cast<const uint4*>(smem + kOffMask + (j % kMaskSlots) * 32);
      const uint4 valid = masks[0], bad = masks[1];
      tmem_wait_ld();
      const int32_t p0 = (bar.piece.j0 + j) * kChunkTile;
      const bool plain = (valid.x & valid.y & valid.z & valid.w) == 0xffffffffu && (bad.x | bad.y | bad.z | bad.w) == 0u &&
                         p0 + kChunkTile <= L_first;
      if (!plain) {
        const uint32_t vw[4] = {valid.x, valid.y, valid.z, valid.w}, bw[4] = {bad.x, bad.y, bad.z, bad.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int32_t left = L - p0 - 32 * w;
          const uint32_t see = (left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u) & vw[w];
          nan_row = nan_row || (see & bw[w]) != 0u;
#pragma unroll
          for (int k = 0; k < 32; ++k) s[32 * w + k] = (see >> k) & 1u ? s[32 * w + k] : -INFINITY;
        }
      }
      // P and the maximum side by side: the maximum nearly always stays within
      // 2^8 of the running one, and then P is right as it is
      auto weigh = [&](float base) {
        const uint64_t nb = f2_pack(-base, -base);
        uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x, y;
            f2_unpack(f2_fma(f2_pack(s[32 * part + 2 * k], s[32 * part + 2 * k + 1]), c2, nb), x, y);
            x = ex2_approx(x);
            y = ex2_approx(y);
            sum[k & 1] = f2_add(sum[k & 1], f2_pack(x, y));
            const __half2 b = __floats2half2_rn(x, y);
            p[k] = *reinterpret_cast<const uint32_t*>(&b);
          }
          tmem_st16(ts + 16 * part, p);
        }
        float x, y;
        f2_unpack(f2_add(sum[0], sum[1]), x, y);
        return x + y;
      };
      float mx[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = max3(s[k], s[k + 4], s[k + 8]);
#pragma unroll
      for (int i = 12; i < 124; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], s[i + k], s[i + k + 4]);
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[124 + k]);
      const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c1, -kFarthest);
      float add = 0.f;
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {  // (the second where a row has outgrown its maximum)
        add = weigh(m == -INFINITY ? 0.f : m - kLift);
        const bool grow = top > m + kRescaleLog2 || (m == -INFINITY && top > m);
        if (!__any_sync(0xffffffffu, grow)) break;
        const float to_m = grow ? top : m;
        const float f = grow ? ex2_approx(m - to_m) : 1.f;
        m = to_m;
        l *= f;
        if (j > 0) {  // (PV(j - 1) is complete: S(j) came after it)
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(to + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st16(to + 16 * c, o);
          }
        }
      }
      l += add;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[g]);
    }
    // ---- output: O / l through shared memory (Q's, which no MMA reads any more)
    if (tiles > 0 && ok) ok = mbar_wait_warp(&bar.s_full[g], tiles & 1);
    if (!ok) failed();
    tc_fence_after();
    bool far = false;  // sees tokens, and all their scores are below -kFarthest
    if (m <= -kFarthest) far = sees_any(a.valid + bar.piece.image, tiles, L - bar.piece.j0 * kChunkTile);
    const bool cut = bar.piece.pieces > 1;
    if (far && cut && l == l) l = 0.f;  // (some may lie just below)
    if (nan_row || m > kFarthest || (far && !cut)) l = __int_as_float(0x7fc00000);
    const float inv = tiles > 0 && l != 0.f ? 1.0f / l : 0.f;
    const float lse = tiles > 0 && l != 0.f ? (m - kLift + log2f(l)) * kLn2 : far ? kFar : -INFINITY;
    unsigned char* slot = a.partial + (static_cast<int64_t>(hp) * a.slots + bar.piece.slot) * kSlotBytes;  // the unit's first
    unsigned char* own = slot + static_cast<int64_t>(bar.piece.index) * kSlotBytes;
    if (cut) reinterpret_cast<float*>(own)[kChunkRows * kVDim + 128 * g + row] = lse;
    else if (row < rows && r < a.T) a.lse[r * a.H + h] = lse;
    const bool f32 = cut || a.out_f32;
    const int wr = 32 * quad;  // this warp's rows
    const int live = min(32, static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(rows), a.T - static_cast<int64_t>(bar.piece.q0) - first) - wr)));
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {  // 32 dims at a time; a warp's rows are its own
      uint32_t o[32];
      if (tiles > 0) {
        tmem_ld32(to + 32 * c, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = tiles > 0 && l != 0.f ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
      unsigned char* stage = qs + wr * 128;
      const int64_t out0 = (static_cast<int64_t>(bar.piece.q0) + first + wr) * a.H + h;
      const int dim = 32 * c;
      __syncwarp();
      if (f32) {  // 128 bytes a row: eight lanes each
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(stage + image_unit(lane, k)) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int q = 4 * k + (lane >> 3);
          float* dst = cut ? reinterpret_cast<float*>(own) + (128 * g + wr + q) * kVDim
                           : static_cast<float*>(a.out) + (out0 + static_cast<int64_t>(q) * a.H) * kVDim;
          if (q < live) *reinterpret_cast<uint4*>(dst + dim + 4 * (lane & 7)) = *reinterpret_cast<const uint4*>(stage + image_unit(q, lane & 7));
        }
      } else {  // 64 bytes a row: four lanes each
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * e]), __uint_as_float(o[8 * k + 2 * e + 1]));
            w[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(stage + image_unit(lane, k)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int q = 8 * k + (lane >> 2);
          if (q < live)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (out0 + static_cast<int64_t>(q) * a.H) * kVDim + dim + 8 * (lane & 3)) =
                *reinterpret_cast<const uint4*>(stage + image_unit(q, lane & 3));
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
      // -------------------------------------------------- MMAs
      // (one lane, every operand a base plus constants: an issuing thread that
      // computes what its next MMA needs falls behind the tensor pipe)
      if (elected()) {
        const uint64_t dq = smem_desc(smem_u32(smem + kOffQ), 16, 1024, kSwizzle128B);
        // (one descriptor for K and V: the distance of 64-dim images counts for V alone)
        const uint64_t dring = smem_desc(smem_u32(smem + kOffRing), kImage, 1024, kSwizzle128B);
        Issue is{bar, dq, dring, n0, n1, true};
        uint32_t k0 = 0;
        if (!fine) {
          for (int32_t j = 0; j <= n && is.ok; ++j, k0 += kQChunks + kVChunks) {
            is.step<0, false>(j, k0);
            is.step<1, false>(j, k0);
          }
        } else {
          for (int32_t j = 0; j <= n && is.ok; ++j, k0 += kQChunks + 2 + kVChunks) {
            is.step<0, true>(j, k0);
            is.step<1, true>(j, k0);
          }
        }
        if (!is.ok) failed();
        mma_commit(&bar.fin);  // the MMAs are complete before TMEM goes
        mbar_wait(&bar.fin, 0);
      }
      __syncwarp();
    } else if (warp == 9) {
      // -------------------------------------------------- loads
      // (running pointers and slots: a copy whose operands are computed anew
      // takes its thread ~600 cycles)
      if (elected()) {
        const unsigned char* keys = a.keys + (static_cast<int64_t>(hp) * a.tiles + image0) * (2 * kImage);
        const unsigned char* values = a.values + (static_cast<int64_t>(hp) * a.tiles + image0) * (2 * kImage);
        const unsigned char* rope = a.rope + static_cast<int64_t>(image0) * kImage;
        const unsigned char* lo = a.lo_keys + (static_cast<int64_t>(hp) * a.lo_tiles + max(0, bar.piece.lo)) * (2 * kImage);
        const uint4* valid = a.valid + image0;
        const uint4* bad = a.bad + static_cast<int64_t>(hp) * a.tiles + image0;
        unsigned char* ring = smem + kOffRing;
        int32_t nk = 0, nv = 0;  // loaded so far
        bool ok = true;
        auto stream = [&](auto fine_c) {
          constexpr bool kFine = decltype(fine_c)::value;
          constexpr uint32_t kKeyImages = kQChunks + (kFine ? 2 : 0);
          uint32_t slot = 0;
          for (int32_t j = 0; j < n; ++j) {
            // K(j) takes slots of K(j - 2) and V(j - 2), V(j) of K(j - 1); with
            // remainders, K(j) of V(j - 2) and K(j - 1), V(j) of K(j - 1) and V(j - 1)
            const int32_t o = j & 1, before = (j - 1) & 1;
            if (j >= 2) ok = mbar_wait(&bar.v_free[o], ((j >> 1) - 1) & 1);
            if (kFine && j >= 1) ok = ok && mbar_wait(&bar.k_free[before], ((j - 1) >> 1) & 1);
            if (!ok) return;
            mbar_arrive_expect_tx(&bar.k_full[o], kKeyImages * kImage);
            bulk_load(ring + slot * kImage, keys, kImage, &bar.k_full[o]);
            bulk_load(ring + ((slot + 1) % kSlots) * kImage, keys + kImage, kImage, &bar.k_full[o]);
            bulk_load(ring + ((slot + 2) % kSlots) * kImage, rope, kImage, &bar.k_full[o]);
            if constexpr (kFine) {
              bulk_load(ring + ((slot + 3) % kSlots) * kImage, lo, kImage, &bar.k_full[o]);
              bulk_load(ring + ((slot + 4) % kSlots) * kImage, lo + kImage, kImage, &bar.k_full[o]);
              lo += 2 * kImage;
            }
            ++nk;
            uint64_t* mb = &bar.mask_full[j % kMaskSlots];
            unsigned char* dst = smem + kOffMask + (j % kMaskSlots) * 32;
            mbar_arrive_expect_tx(mb, 32);
            bulk_load(dst, valid, 16, mb);
            bulk_load(dst + 16, bad, 16, mb);
            if (j >= 1) ok = mbar_wait(kFine ? &bar.v_free[before] : &bar.k_free[before], ((j - 1) >> 1) & 1);
            if (!ok) return;
            mbar_arrive_expect_tx(&bar.v_full[o], kVChunks * kImage);
            bulk_load(ring + ((slot + kKeyImages) % kSlots) * kImage, values, kImage, &bar.v_full[o]);
            bulk_load(ring + ((slot + kKeyImages + 1) % kSlots) * kImage, values + kImage, kImage, &bar.v_full[o]);
            ++nv;
            slot = (slot + kKeyImages + kVChunks) % kSlots;
            keys += 2 * kImage, values += 2 * kImage, rope += kImage, ++valid, ++bad;
          }
        };
        if (fine) stream(std::true_type{});
        else stream(std::false_type{});
        if (!ok) failed();
        // nothing lands after the CTA is gone
        for (int32_t k = max(0, nk - 2); k < nk; ++k) mbar_wait(&bar.k_full[k & 1], (k >> 1) & 1);
        for (int32_t k = max(0, nv - 2); k < nv; ++k) mbar_wait(&bar.v_full[k & 1], (k >> 1) & 1);
        for (int32_t k = max(0, nk - kMaskSlots); k < nk; ++k) mbar_wait(&bar.mask_full[k % kMaskSlots], (k / kMaskSlots) & 1);
      }
      __syncwarp();
    } else if (warp == 11) {
      // -------------------------------------------------- gate
      if (elected()) {
        bool ok = true;
        for (int32_t j = 0; j < n && ok; ++j) {
          ok = mbar_wait(&bar.v_full[j & 1], (j >> 1) & 1);
          // (an arrival counts for the phase that is open: the one of tile j - 1 must be over)
          if (j < n0) {
            if (j > 0) ok = ok && mbar_wait(&bar.p_full[0], (j - 1) & 1);
            if (ok) mbar_arrive(&bar.p_full[0]);
          }
          if (j < n1) {
            if (j > 0) ok = ok && mbar_wait(&bar.p_full[1], (j - 1) & 1);
            if (ok) mbar_arrive(&bar.p_full[1]);
          }
        }
        if (!ok) failed();
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 10) tmem_dealloc(bar.tmem, 512);
}

// The outputs of units that were cut, from their pieces' (normalised, with their
// log-sum-exps), in the pieces' order.  The grid is the attention's: piece i of n
// takes the i-th of n parts of its unit's rows, a warp per row, eight pieces' rows
// loaded at a time.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ ChunkArgs a) {
  launch_dependents();
  wait_dependency();
  const int lane = threadIdx.x & 31;
  Piece p;
  int32_t hp;
  if (!piece_of(a, static_cast<int32_t>(blockIdx.x), p, hp) || p.b < 0 || p.pieces == 1) return;
  constexpr int kStep = kSlotBytes / 4, kBatch = 8;
  const float* slot = reinterpret_cast<const float*>(a.partial + (static_cast<int64_t>(hp) * a.slots + p.slot) * kSlotBytes);
  const int64_t first = static_cast<int64_t>(a.qsl[p.b]) + static_cast<int64_t>(p.block) * kChunkRows;
  const int64_t end = min(static_cast<int64_t>(a.qsl[p.b + 1]), static_cast<int64_t>(a.T));
  const int32_t rows = static_cast<int32_t>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kChunkRows), end - first)));
  for (int32_t i = rows * p.index / p.pieces + (threadIdx.x >> 5); i < rows * (p.index + 1) / p.pieces; i += kJoinThreads / 32) {
    const float lse = lane < p.pieces ? __ldg(slot + static_cast<int64_t>(lane) * kStep + kChunkRows * kVDim + i) : -INFINITY;
    float top = lse;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // (all -inf: nothing to see; a NaN weighs NaN)
    const float w = lse <= kFar ? 0.f : ex2_approx((lse - top) * kLog2e);
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (top == kFar) sum = __int_as_float(0x7fc00000);  // nothing but far scores
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < p.pieces; k0 += kBatch) {
      float4 v[kBatch];
      float wk[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        wk[k] = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
        if (k0 + k >= p.pieces) wk[k] = 0.f;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        // (a piece without weight may not have written its output)
        if (wk[k] != 0.f) v[k] = __ldg(reinterpret_cast<const float4*>(slot + static_cast<int64_t>(k0 + k) * kStep + i * kVDim) + lane);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        acc.x = fmaf(wk[k], v[k].x, acc.x), acc.y = fmaf(wk[k], v[k].y, acc.y);
        acc.z = fmaf(wk[k], v[k].z, acc.z), acc.w = fmaf(wk[k], v[k].w, acc.w);
      }
    }
    const float inv = sum != 0.f ? 1.0f / sum : 0.f;
    const int32_t h = a.h0 + hp;
    const int64_t at = ((first + i) * a.H + h) * kVDim + 4 * lane;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    if (a.out_f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = acc;
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x, acc.y), y = __floats2bfloat162_rn(acc.z, acc.w);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
    if (lane == 0) a.lse[(first + i) * a.H + h] = sum != 0.f ? top + log2f(sum) * kLn2 : -INFINITY;
  }
}

std::mutex g_mutex;
bool g_ready[64];

cudaError_t set_up() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (dev < 64 && g_ready[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e == cudaSuccess && dev < 64) g_ready[dev] = true;
  return e;
}

}  // namespace

cudaError_t launch_chunk_attention(const ChunkArgs& a, cudaStream_t st) {
  const cudaError_t e = set_up();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(a.max_pieces) * a.heads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t launched = cudaLaunchKernelEx(&cfg, attention_kernel, a);
  if (launched != cudaSuccess || a.slots == 0) return launched;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel, a);
}

}  // namespace dcp
