// Chunk attention, first half: the latents of the requests' contexts, gathered
// from the paged cache, times the up projection's weight.
//
//   keys_h(p) = W_h[0:128] c(p),  values_h(p) = W_h[128:256] c(p)   (c: 512 dims)
//
// A matrix product of tokens x 512 by 512 x 256 per head on the tensor cores:
// 2 x 512 x 256 operations per token and head, 512 bytes out.  Unit of work:
// (two tiles of 128 tokens, head), token-major, in equal shares of a persistent
// grid, so that latents are gathered once per tile (128 KB of a CTA's shared
// memory, all 512 dims) and the weights of head after head stream past them.
// Two CTAs share the weights: one MMA (M = 256, N = 256) reads each CTA's 128
// tokens and half of a head's rows from either's shared memory, so that each
// streams 32 bytes of weights a clock instead of 64.
//
// 24,000 tokens at 128 heads: ~540 us, 1.5 PFLOP/s (77 % of what a library product
// was measured at), 2.9 TB/s of stores.  What bounds it: the weights' loads, 16 KB
// each and four in flight, wait behind the images' stores to DRAM: the tensor pipe is
// busy 64 % of the time (333 us for 12 mixed requests at 16 heads), and without the
// stores an item took 4,105 cycles, its MMAs' 4,096.  A fifth stage, or stores by
// another path, changed nothing.  (A CTA by itself: 851 us.)
//
// Warp roles (512 threads in each CTA of the pair):
//   warps 0-3, 12-15  epilogue of the keys and of the values: accumulator -> f16
//               -> images in shared memory -> bulk stores; thread = token = TMEM
//               lane.  (By four warps for both ~3,400 cycles an item; with plain
//               stores ~4,500, more than its MMAs' 4,096.)
//   warp 4      weights: 16 KB tensor copies (64 latent dims of half a head's rows);
//               both CTAs' complete on CTA 0's barrier, which is what such a copy
//               for a pair of CTAs may do and an untiled one may not
//   warp 5      CTA 0: MMA issuer, two accumulators
//   warp 6      TMEM allocation
//   warps 8-11  gather of the latents (8 lanes per 128-byte line)
// Every wait is bounded (DCP_DEVERR_TIMEOUT).
//
// A value that is not finite would reach query rows that do not see its token
// (0 x NaN in the product with the weights of a tile), so a token with one gets
// a row of zeros and a bit in `bad`: rows that see it become NaN.  A key that is
// not finite, or past f16's largest, is made NaN: an infinite element's score
// could be -inf, which weighs nothing.
#include "dcp_chunk.cuh"

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <mutex>
#include <type_traits>

namespace dcp {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kLoadThreads = 128;
constexpr int kChunks = kLatent / 64;  // 8 chunks of 64 latent dims
constexpr uint32_t kWStages = 4;
constexpr int kWHalf = kWeightStage / 2;  // a CTA's rows of a weight stage
constexpr int kOffA = 0;
constexpr int kOffW = kChunks * kImage;
constexpr int kOffOut = kOffW + kWStages * kWHalf;
constexpr int kOutWarp = 32 * 128;        // an epilogue warp's 32 rows of an image
constexpr int kOffBars = kOffOut + 8 * kOutWarp;

struct Bars {
  uint64_t a_full;            // CTA 0: both CTAs' latents are in shared memory (every loader)
  uint64_t a_free;            // both: the tiles' MMAs are complete
  uint64_t w_full[kWStages];  // CTA 0: both CTAs' halves of a weight stage have landed
  uint64_t w_free[kWStages];  // both
  uint64_t acc_full[2];       // both: an accumulator is complete
  uint64_t acc_free[2];       // CTA 0: both CTAs' epilogues have read it (8 warps each)
  uint64_t fin;               // both: the issuer's MMAs are complete
  uint32_t tmem;
};
constexpr int kSmemBytes = kOffBars + static_cast<int>(sizeof(Bars)) + 1024;
static_assert(kSmemBytes <= 232448, "exceeds the 227 KB of shared memory per CTA");

__device__ __forceinline__ uint32_t widen2(uint32_t codes, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));  // exact
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Cache row of position p of request b, -1 for none (flagged).
__device__ __forceinline__ int64_t cache_row(const ChunkArgs& a, int32_t b, int32_t p) {
  int32_t j = p;
  int64_t table = static_cast<int64_t>(b) * a.bt_stride;
  if (a.local_tables) {
    const int32_t run = fast_div(p, a.div_I), turn = fast_div(run, a.div_D);
    table += (run - turn * a.D) * a.bt_shard_stride;
    j = turn * a.I + (p - run * a.I);
  }
  const int32_t col = fast_div(j, a.div_bs);
  if (col < a.bt_width) {
    const int32_t blk = __ldg(a.block_table + table + col);
    if (blk >= 0 && blk < a.num_blocks) return static_cast<int64_t>(blk) * a.block_size + (j - col * a.block_size);
  }
  if (a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_BAD_BLOCK);
  return -1;
}

// A tile of a request's tokens, and its key remainders (-1: none).  By the whole warp.
struct TileOf {
  int32_t b, index, lo;
};
__device__ __forceinline__ TileOf tile_of(const ChunkArgs& a, int32_t tile) {
  TileOf t;
  t.b = find_range(a.tile_start, a.B, tile);
  t.index = tile - a.tile_start[t.b];
  const int32_t lo = a.lo_start[t.b];
  t.lo = lo >= 0 ? lo + t.index : -1;
  return t;
}

struct Work {
  int32_t i0, i1;  // items [i0, i1): tiles 2 (i / heads) and the next, head i % heads
};
__device__ __forceinline__ Work my_items(const ChunkArgs& a, int32_t tiles) {
  const int64_t n = static_cast<int64_t>((tiles + 1) / 2) * a.heads;
  const int64_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  Work w;
  w.i0 = static_cast<int32_t>(n * pair / pairs);
  w.i1 = static_cast<int32_t>(n * (pair + 1) / pairs);
  return w;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) expand_kernel(const __grid_constant__ ChunkArgs a,
                                                             const __grid_constant__ CUtensorMap weight_map) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bar = *reinterpret_cast<Bars*>(smem + kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    mbar_init(&bar.a_full, 2 * kLoadThreads);
    mbar_init(&bar.a_free, 1);
    for (uint32_t i = 0; i < kWStages; ++i) mbar_init(&bar.w_full[i], 1), mbar_init(&bar.w_free[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bar.acc_full[i], 1), mbar_init(&bar.acc_free[i], 16);
    mbar_init(&bar.fin, 1);
    fence_mbar_init();
  }
  if (warp == 6) {
    tmem_alloc_pair(&bar.tmem, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // (the peer's barriers are set up)
  tc_fence_after();
  const uint32_t tmem = 0;  // (all 512 columns: the allocation starts at the first)
  // While the plan runs: this CTA's share of the weights of the pass, into L2
  // (2,833 us instead of 2,855 for 2,048 rows on 21,952 tokens, 759 instead of 765
  // for 12 mixed requests).
  if (warp == 4 && elected()) {
    const int64_t n = static_cast<int64_t>(a.heads) * (kChunks * kWeightStage / kWHalf);  // of 16 KB
    const unsigned char* w = static_cast<const unsigned char*>(a.weight) + static_cast<int64_t>(a.h0) * (kChunks * kWeightStage);
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) bulk_prefetch(w + i * kWHalf, kWHalf);
  }
  __syncwarp();
  wait_dependency();
  const int32_t tiles = min(a.tile_start[a.B], a.tiles);
  const Work work = my_items(a, tiles);
  auto failed = [&]() {
    if (a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_TIMEOUT);
  };

  if (warp < 4 || warp >= 12) {
    // -------------------------------------------------- epilogue
    const int part = warp >= 12, quad = warp & 3;  // keys or values; the warp's TMEM lanes
    unsigned char* stage = smem + kOffOut + (4 * part + quad) * kOutWarp;
    const uint32_t free0 = map_peer(smem_u32(&bar.acc_free[0]), 0);
    unsigned char* images = part ? a.values : a.keys;
    const uint64_t stream = l2_stream();
    int32_t pair = work.i0 / a.heads, h = work.i0 - pair * a.heads;
    int32_t lo = -1;
    for (int32_t i = work.i0, n = 0; i < work.i1; ++i, ++n) {
      const int acc = n & 1;
      const int32_t tile = 2 * pair + static_cast<int32_t>(rank);
      if (!part && (n == 0 || h == 0)) lo = tile < tiles ? tile_of(a, tile).lo : -1;
      if (!mbar_wait_warp(&bar.acc_full[acc], (n >> 1) & 1)) { failed(); break; }
      tc_fence_after();
      const int64_t slot = static_cast<int64_t>(h) * a.tiles + tile;
      const uint32_t col = tmem + (static_cast<uint32_t>(quad) << 21) + 256u * acc + 128u * part;
      uint32_t v[64];  // 128 dims as f16 pairs
#pragma unroll 1
      for (int turn = 0; turn < 1 + (lo >= 0); ++turn) {  // (keys of short requests: then what their rounding left)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(col + 32 * c, r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float x = __uint_as_float(r[2 * k]), y = __uint_as_float(r[2 * k + 1]);
            __half2 b = __floats2half2_rn(x, y);
            if (turn) {
              const float2 f = __half22float2(b);
              b = __floats2half2_rn(x - f.x, y - f.y);
            }
            v[16 * c + k] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
        if (turn == (lo >= 0)) {
          tc_fence_before();
          __syncwarp();
          // (relaxed: the accumulator has been read, and no write of this warp
          // concerns the issuer; a release waited ~3,000 cycles for them)
          if (lane == 0) mbar_arrive_remote_relaxed(free0 + 8 * acc);
        }
        if (tile >= tiles) continue;  // (the last tile may have no second one)
        if (turn == 0) {
          __half2 zero = __half2half2(__ushort_as_half(0)), sum = zero;  // 0 x (infinity or NaN) is NaN
#pragma unroll
          for (int k = 0; k < 64; ++k) sum = __hfma2(*reinterpret_cast<const __half2*>(&v[k]), zero, sum);
          const bool fin = (*reinterpret_cast<const uint32_t*>(&sum) & 0x7fff7fffu) == 0u;
          if (part) {
            const uint32_t nan_rows = __ballot_sync(0xffffffffu, !fin);
            if (!fin) {
#pragma unroll
              for (int k = 0; k < 64; ++k) v[k] = 0;
            }
            if (lane == 0) reinterpret_cast<uint32_t*>(a.bad + slot)[quad] = nan_rows;
          } else if (!fin) {
            v[0] = 0x7fff7fffu;
          }
        }
        unsigned char* dst = (turn ? a.lo_keys + (static_cast<int64_t>(h) * a.lo_tiles + lo) * (2 * kImage) : images + slot * (2 * kImage)) + quad * kOutWarp;
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // an image's 64 dims
          if (elected()) bulk_wait_read<0>();  // (the last store has read its source)
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(stage + image_unit(lane, u)) =
                make_uint4(v[32 * c + 4 * u], v[32 * c + 4 * u + 1], v[32 * c + 4 * u + 2], v[32 * c + 4 * u + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (elected()) {
            bulk_store_hint(dst + c * kImage, stage, kOutWarp, stream);
            bulk_commit();
          }
        }
      }
      if (++h == a.heads) h = 0, ++pair;
    }
    if (elected()) bulk_wait<0>();
    __syncwarp();
  } else if (warp == 4) {
    // -------------------------------------------------- weights
    // (running slots and phases: with ones computed from a counter a copy took
    // this thread ~600 cycles, and eight of them more than an item's MMAs)
    if (elected()) {
      bool ok = true;
      int32_t h = work.i0 % a.heads;
      uint32_t s = 0, phase = 0, used = 0;
      const uint64_t keep = l2_keep();  // (the images that stream out would push the weights out)
      const uint32_t full = map_peer(smem_u32(&bar.w_full[0]), 0);
      for (int32_t i = work.i0; i < work.i1 && ok; ++i) {
        const int32_t row = (a.h0 + h) * (kChunks * kUp) + static_cast<int32_t>(rank) * (kUp / 2);  // of the packed weight
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          ok = ok && mbar_wait(&bar.w_free[s], phase ^ 1);
          if (ok) {
            if (rank == 0) mbar_arrive_expect_tx(&bar.w_full[s], kWeightStage);
            tma_load_pair(smem + kOffW + s * kWHalf, &weight_map, 0, row + c * kUp, full + 8 * s, keep);
            ++used;
          }
          if (++s == kWStages) s = 0, phase ^= 1;
        }
        h = h + 1 == a.heads ? 0 : h + 1;
      }
      if (!ok) failed();
      // nothing lands after the CTAs are gone (neither goes before the other)
      if (rank == 0)
        for (uint32_t k = used > kWStages ? used - kWStages : 0; k < used; ++k) mbar_wait_cluster(&bar.w_full[k % kWStages], (k / kWStages) & 1);
    }
    __syncwarp();
  } else if (warp == 5) {
    // -------------------------------------------------- MMAs
    // (one lane, every operand a base plus constants: an issuing thread that
    // computes what its next MMA needs falls behind the tensor pipe)
    if (rank == 1) {
      if (elected()) mbar_wait(&bar.fin, 0);
    } else if (elected()) {
      constexpr uint32_t id = idesc_bf16(256, 256, 0, 0);
      const uint64_t da = smem_desc(smem_u32(smem + kOffA), 16, 1024, kSwizzle128B);
      const uint64_t dw = smem_desc(smem_u32(smem + kOffW), 16, 1024, kSwizzle128B);
      uint32_t loads = 0, acc_phase = 1, st = 0, phase = 0;
      int32_t left = 0;  // items of the tile at hand
      bool ok = true;
      int32_t tile_end = (work.i0 / a.heads) * a.heads;  // first item of the next tiles
      // item n of this CTA, into accumulator `acc`
      auto item = [&](auto acc_c, int32_t i) {
        constexpr uint32_t acc = decltype(acc_c)::value;
        if (left == 0) {
          ok = ok && mbar_wait_cluster(&bar.a_full, loads & 1);
          ++loads;
          tile_end += a.heads;
          left = min(tile_end, work.i1) - i;
        }
        ok = ok && mbar_wait_cluster(&bar.acc_free[acc], acc_phase);
        if (!ok) return;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          // (one barrier for both halves: a wait takes ~200 cycles even when
          // nothing is left to wait for)
          ok = ok && mbar_wait_cluster(&bar.w_full[st], phase);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss_pair(256 * acc, da + ((c * kImage) >> 4) + 2 * k, dw + ((st * kWHalf) >> 4) + 2 * k, id, (c | k) != 0);
          mma_commit_pair(&bar.w_free[st]);
          if (++st == kWStages) st = 0, phase ^= 1;
        }
        mma_commit_pair(&bar.acc_full[acc]);
        if (--left == 0) mma_commit_pair(&bar.a_free);
      };
      for (int32_t i = work.i0; i < work.i1 && ok; i += 2, acc_phase ^= 1) {
        item(std::integral_constant<uint32_t, 0>{}, i);
        if (i + 1 < work.i1 && ok) item(std::integral_constant<uint32_t, 1>{}, i + 1);
      }
      if (!ok) failed();
      mma_commit_pair(&bar.fin);  // the MMAs are complete before TMEM goes
      mbar_wait(&bar.fin, 0);
    }
    __syncwarp();
  } else if (warp >= 8) {  // (to 11)
    // -------------------------------------------------- latents
    const int lw = warp - 8;
    int32_t last = -1;
    uint32_t loads = 0;
    for (int32_t i = work.i0; i < work.i1; i = (last + 1) * a.heads) {
      last = i / a.heads;
      const int32_t tile = 2 * last + static_cast<int32_t>(rank);
      // this thread's token (a tile past the last is all zeros)
      int64_t src = -1;
      if (tile < tiles) {
        const TileOf of = tile_of(a, tile);
        const int64_t p = static_cast<int64_t>(of.index) * kChunkTile + 32 * lw + lane;
        if (p < a.seq_lens[of.b]) src = cache_row(a, of.b, static_cast<int32_t>(p));
      }
      const float scale = kFp8 && src >= 0 ? __ldg(a.kv_scale + src) : 0.f;
      // what the heads share is written with the first head
      const bool shared_too = a.h0 == 0 && i == last * a.heads && tile < tiles;
      const uint32_t live = __ballot_sync(0xffffffffu, src >= 0);
      if (shared_too && lane == 0) reinterpret_cast<uint32_t*>(a.valid + tile)[lw] = live;
      if (loads > 0 && !mbar_wait_warp(&bar.a_free, (loads - 1) & 1)) { failed(); break; }
      ++loads;
      const int u = lane & 7;
#pragma unroll 2
      for (int g = 0; g < 8; ++g) {
        const int r = 4 * g + (lane >> 3);
        const int64_t from = __shfl_sync(0xffffffffu, src, r);
        const float s = kFp8 ? __shfl_sync(0xffffffffu, scale, r) : 0.f;
        const uint32_t at = image_unit(32 * lw + r, u);
        uint4 rope = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (kFp8) {
          const uint2* row = reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(a.kv) + from * kKDim) + u;
          uint2 v[kChunks + 1];
#pragma unroll
          for (int c = 0; c <= kChunks; ++c) v[c] = from >= 0 ? __ldg(row + 8 * c) : make_uint2(0u, 0u);
#pragma unroll
          for (int c = 0; c <= kChunks; ++c) {
            const uint4 w = make_uint4(widen2(v[c].x, s), widen2(v[c].x >> 16, s), widen2(v[c].y, s), widen2(v[c].y >> 16, s));
            if (c < kChunks) *reinterpret_cast<uint4*>(smem + kOffA + c * kImage + at) = w;
            else rope = w;
          }
        } else {
          const unsigned char* row = static_cast<const unsigned char*>(a.kv) + (from >= 0 ? from : 0) * (2 * kKDim) + 16 * u;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            cp_async16_zfill(smem_u32(smem + kOffA + c * kImage + at), row + 128 * c, from >= 0 ? 16u : 0u);
          if (shared_too && from >= 0) rope = __ldg(reinterpret_cast<const uint4*>(row + 128 * kChunks));
        }
        if (shared_too) *reinterpret_cast<uint4*>(a.rope + static_cast<int64_t>(tile) * kImage + at) = rope;
      }
      if constexpr (!kFp8) {
        cp_async_commit();
        cp_async_wait<0>();
      }
      fence_proxy_async_smem();
      mbar_arrive_remote(map_peer(smem_u32(&bar.a_full), 0));
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // (neither CTA goes while the other's MMAs or arrivals need it)
  tc_fence_after();
  if (warp == 6) tmem_dealloc_pair(bar.tmem, 512);
}

// packed[h][c] = rows 256 h .. 256 h + 255 of w [H x 256, 512], latent dims
// 64 c .. 64 c + 63, as the MMAs read them
__global__ void __launch_bounds__(256) pack_kernel(const uint4* __restrict__ w, unsigned char* __restrict__ packed, int64_t units) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // 16-byte unit of w
  if (i >= units) return;
  const int64_t row = i >> 6;
  const int u = static_cast<int>(i & 63), r = static_cast<int>(row & (kUp - 1));
  *reinterpret_cast<uint4*>(packed + (row / kUp) * (kChunks * kWeightStage) + (u >> 3) * kWeightStage + image_unit(r, u & 7)) = __ldg(w + i);
}

using Kernel = void (*)(ChunkArgs, CUtensorMap);

cudaLaunchConfig_t pairs_config(int pairs, cudaStream_t st, cudaLaunchAttribute (&attr)[2]) {
  attr[0] = attr[1] = cudaLaunchAttribute{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2u * static_cast<unsigned>(pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Pairs of CTAs that run at once on the current device (looked up once for each
// device and kernel); more would wait for a second turn.
std::mutex g_mutex;
constexpr int kMaxDevices = 64;
int g_pairs[2][kMaxDevices];

cudaError_t resident_pairs(Kernel kernel, bool fp8, int* pairs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (dev < kMaxDevices && g_pairs[fp8][dev] > 0) {
    *pairs = g_pairs[fp8][dev];
    return cudaSuccess;
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pairs_config(1, nullptr, attr);
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (*pairs < 1) return cudaErrorInvalidConfiguration;
  if (dev < kMaxDevices) g_pairs[fp8][dev] = *pairs;
  return cudaSuccess;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The packed weight as rows of 64 latent dims, in boxes of a CTA's 128 rows of a
// stage.  (The driver's entry is looked up once: the library links no libcuda.)
cudaError_t weight_tensor(const void* packed, int32_t H, CUtensorMap* map) {
  static const EncodeTiled encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {64, static_cast<cuuint64_t>(H) * kChunks * kUp}, strides[1] = {128};
  const cuuint32_t box[2] = {64, kUp / 2}, steps[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(packed), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_pack_kv_b(const void* w, int32_t H, void* packed, cudaStream_t st) {
  const int64_t units = static_cast<int64_t>(H) * kUp * (kLatent / 8);
  pack_kernel<<<static_cast<unsigned>((units + 255) / 256), 256, 0, st>>>(static_cast<const uint4*>(w),
                                                                          static_cast<unsigned char*>(packed), units);
  return cudaGetLastError();
}

cudaError_t launch_chunk_expand(const ChunkArgs& a, cudaStream_t st) {
  const bool fp8 = a.kv_scale != nullptr;
  const Kernel kernel = fp8 ? expand_kernel<true> : expand_kernel<false>;
  int pairs = 0;
  cudaError_t e = resident_pairs(kernel, fp8, &pairs);
  if (e != cudaSuccess) return e;
  CUtensorMap weight;
  e = weight_tensor(a.weight, a.H, &weight);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>((a.tiles + 1) / 2) * a.heads;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pairs_config(static_cast<int>(items < pairs ? items : pairs), st, attr);
  return cudaLaunchKernelEx(&cfg, kernel, a, weight);
}

}  // namespace dcp
