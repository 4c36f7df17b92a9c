// Chunk attention, the plan: first images and first blocks of the requests, and
// the pieces of work of the attention in launch order.  One CTA; the lengths are
// on the device only.  A chain of scans and shared-memory searches: 6-8 us for one
// to 12 requests (9-10 in the profiler).
//
// Units are (request, block of 256 rows), the same for every head.  A launch
// takes them longest first, so that the last ones to run are short.  Units of
// similar length (a quarter of an octave) form a segment, in which the heads are
// outermost: the blocks of a request read one head's keys and values at about
// the same time, out of L2.
#include "dcp_chunk.cuh"

namespace dcp {
namespace {

constexpr int kThreads = 1024;
constexpr int kBuckets = 128;  // 4 per octave
constexpr int kKept = 1024;    // requests that are kept in shared memory (more: read back from global memory)
constexpr int kFewUnits = 4;   // an SM could take this many times the units
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

// longest first
__device__ __forceinline__ int bucket_of(int32_t tiles) {
  if (tiles <= 0) return kBuckets - 1;
  const int e = 31 - __clz(tiles);
  const int quarter = e >= 2 ? (tiles >> (e - 2)) & 3 : (tiles << (2 - e)) & 3;
  return kBuckets - 2 - (4 * e + quarter);  // (4 x 30 + 3 at most)
}

// Inclusive scan over the CTA of three numbers a thread.
__device__ __forceinline__ void scan3(int64_t (&x)[3], int64_t (*sums)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, x[k], o);
      if (lane >= o) x[k] += y;
    }
    if (lane == 31) sums[k][warp] = x[k];
  }
  __syncthreads();
  if (warp < 3) {
    int64_t s = sums[warp][lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    sums[warp][lane] = s;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) x[k] += warp > 0 ? sums[k][warp - 1] : 0;
}

// What the CTA looks up of the requests: its own copies, or global memory's.
struct Requests {
  const int32_t *tile_start, *block_start, *lo_start, *qsl, *seq;
};

struct Unit {
  int32_t b, block, tiles;
};
__device__ __forceinline__ Unit unit_of(const ChunkArgs& a, const Requests& r, int32_t u, int32_t blocks) {
  Unit n{-1, u - blocks, 0};
  if (u >= blocks) return n;
  int32_t lo = 0, hi = a.B;  // the last request whose first block is <= u
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (r.block_start[mid] <= u) lo = mid; else hi = mid;
  }
  n.b = lo;
  n.block = u - r.block_start[lo];
  const int64_t q_len = static_cast<int64_t>(r.qsl[lo + 1]) - r.qsl[lo];
  const int64_t rows = min(q_len, static_cast<int64_t>(kChunkRows) * (n.block + 1));  // up to this block's last
  const int64_t seq = max(0, r.seq[lo]);
  const int64_t end = seq - q_len + rows;  // tokens that the last row sees
  const int64_t have = r.tile_start[lo + 1] - r.tile_start[lo];
  if (end > 0 && have >= ceil_div(seq, kChunkTile)) n.tiles = static_cast<int32_t>(ceil_div(end, kChunkTile));
  return n;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ int64_t sums[3][32];
  __shared__ int32_t kept[5][kKept + 1];
  __shared__ int32_t count[kBuckets], first[kBuckets], next[kBuckets];
  __shared__ unsigned long long work;
  __shared__ int32_t slots;
  sm100::launch_dependents();
  const int tid = threadIdx.x;
  for (int i = tid; i < kBuckets; i += kThreads) count[i] = 0;
  if (tid == 0) work = 0, slots = 0;
  // ---- first images and blocks of the requests, and tiles of key remainders
  const bool small = a.B <= kKept;
  const Requests req = small ? Requests{kept[0], kept[1], kept[2], kept[3], kept[4]}
                             : Requests{a.tile_start, a.block_start, a.lo_start, a.qsl, a.seq_lens};
  int64_t base[3] = {0, 0, 0};
  for (int32_t b0 = 0; b0 < a.B; b0 += kThreads) {
    const int32_t b = b0 + tid;
    int64_t x[3] = {0, 0, 0};
    int32_t q0 = 0, q1 = 0, seq = 0;
    if (b < a.B) {
      q0 = __ldg(a.qsl + b), q1 = __ldg(a.qsl + b + 1), seq = __ldg(a.seq_lens + b);
      const bool rows = q0 >= 0 && q1 > q0;
      if ((q1 < q0 || q0 < 0) && a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_BAD_ROWS);
      // (tokens that no row sees are not needed)
      x[0] = rows && seq > 0 ? ceil_div(seq, kChunkTile) : 0;
      x[1] = rows ? ceil_div(static_cast<int64_t>(q1) - q0, kChunkRows) : 0;
      x[2] = seq <= kFineLen ? x[0] : 0;
    }
    const bool some = x[0] > 0;
    const int64_t own = x[2];
    scan3(x, sums);
    if (b < a.B) {
#pragma unroll
      for (int k = 0; k < 3; ++k) x[k] += base[k];
      // ends, cut at what the workspace holds; a request past it sees nothing
      if (x[0] > a.tiles && some && a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_SEQ_TOO_LONG);
      const int32_t tile_end = static_cast<int32_t>(x[0] < a.tiles ? x[0] : a.tiles);
      const int32_t block_end = static_cast<int32_t>(x[1] < 0x7fffffff ? x[1] : 0x7fffffff);
      const int32_t lo = own > 0 && x[2] <= a.lo_tiles ? static_cast<int32_t>(x[2] - own) : -1;
      a.tile_start[b + 1] = tile_end, a.block_start[b + 1] = block_end, a.lo_start[b] = lo;
      if (small) {
        kept[0][b + 1] = tile_end, kept[1][b + 1] = block_end, kept[2][b] = lo, kept[3][b] = q0, kept[4][b] = seq;
        if (b == a.B - 1) kept[3][a.B] = q1;
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) base[k] += sums[k][31];
    __syncthreads();
  }
  if (tid == 0) a.tile_start[0] = a.block_start[0] = kept[0][0] = kept[1][0] = 0;
  __syncthreads();
  // ---- the units: requests' blocks, then the rows of no request
  const int32_t limit = a.max_pieces - (a.slots > 0 ? static_cast<int32_t>(added_pieces(a.sms, a.heads)) : 0);
  const int32_t blocks = min(req.block_start[a.B], limit);
  const int64_t lead = max(0, min(req.qsl[0], a.T)), tail = max(lead, static_cast<int64_t>(min(req.qsl[a.B], a.T)));
  const int32_t units = static_cast<int32_t>(min(static_cast<int64_t>(limit), blocks + ceil_div(lead + a.T - tail, kChunkRows)));
  unsigned long long mine = 0;
  for (int32_t u = tid; u < units; u += kThreads) mine += unit_of(a, req, u, blocks).tiles;
  if (mine) atomicAdd(&work, mine);
  __syncthreads();
  // Pieces of a unit: its share of one piece an SM.  With few units they are
  // rounded down, so that all run at once (16 units of 251 tiles on 152 SMs: 9
  // pieces each, 144 in all; 10 would leave eight pieces for a second turn); with
  // more, which take turns anyway, up.
  const int64_t all = max(static_cast<int64_t>(work) * a.heads, static_cast<int64_t>(1));
  const bool few = static_cast<int64_t>(units) * a.heads * kFewUnits <= a.sms;
  auto cuts = [&](int32_t tiles) {
    if (a.slots == 0) return 1;
    const int64_t share = (static_cast<int64_t>(tiles) * a.sms + (few ? 0 : all - 1)) / all;
    return static_cast<int32_t>(max(static_cast<int64_t>(1), min(share, min(static_cast<int64_t>(kMaxPieces), static_cast<int64_t>(tiles) / kMinPiece))));
  };
  for (int32_t u = tid; u < units; u += kThreads) {
    const int32_t tiles = unit_of(a, req, u, blocks).tiles, c = cuts(tiles);
    atomicAdd(&count[bucket_of((tiles + c - 1) / c)], c);
  }
  __syncthreads();
  if (tid < 32) {  // four buckets a lane
    int32_t c[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = count[4 * tid + i], n += c[i];
    int32_t x = n;
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(kFull, x, o);
      if (tid >= o) x += y;
    }
    x -= n;
#pragma unroll
    for (int i = 0; i < 4; ++i) first[4 * tid + i] = next[4 * tid + i] = x, x += c[i];
    if (tid == 31) *a.num_pieces = x;
  }
  __syncthreads();
  // ---- records.  `next` places a unit's pieces in its bucket; their order there
  // and the slots' do not change results.
  for (int32_t u = tid; u < units; u += kThreads) {
    const Unit n = unit_of(a, req, u, blocks);
    const int32_t c = cuts(n.tiles), bucket = bucket_of((n.tiles + c - 1) / c);
    const int32_t at = atomicAdd(&next[bucket], c);
    const int32_t slot = c > 1 ? atomicAdd(&slots, c) : 0;
    for (int32_t i = 0; i < c && at + i < a.max_pieces; ++i) {
      Piece p{};
      p.b = n.b, p.block = n.block;
      p.q0 = n.b < 0 ? 0 : req.qsl[n.b];
      p.q1 = n.b < 0 ? 0 : req.qsl[n.b + 1];
      p.seq = n.b < 0 ? 0 : max(0, req.seq[n.b]);
      p.j0 = static_cast<int32_t>(static_cast<int64_t>(n.tiles) * i / c);
      p.j1 = static_cast<int32_t>(static_cast<int64_t>(n.tiles) * (i + 1) / c);
      p.image = n.b < 0 ? 0 : req.tile_start[n.b] + p.j0;
      p.lo = n.b < 0 || req.lo_start[n.b] < 0 ? -1 : req.lo_start[n.b] + p.j0;
      p.pieces = c, p.slot = slot, p.index = i;
      p.seg0 = first[bucket], p.seg = count[bucket];
      a.pieces[at + i] = p;
    }
  }
}

}  // namespace

cudaError_t launch_chunk_plan(const ChunkArgs& a, cudaStream_t st) {
  plan_kernel<<<1, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace dcp
