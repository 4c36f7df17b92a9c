// Tensor-core decode of selected tokens for sm_103a: the windowed and tree
// decodes (dcp_select.cuh).
//
// One unit = (group of rows of one request, shard d, split s): up to 128 lanes
// (lane = row x heads, so rows of few heads share their tiles and their MMAs)
// against the tokens of the shard that any of the rows sees, in tiles of 32.
// A unit runs on a cluster of two CTAs with the division of work of the plain
// decode (dcp_decode_tc.cu, which also gives the measurements behind it):
//   score CTA (rank 0)  holds Q in TMEM (288 columns), computes S(j) = Q K(j)^T
//                       into one of four slots, runs the online softmax and
//                       ships P(j) and each lane's running max;
//   value CTA (rank 1)  holds O (all 512 TMEM columns), rescales it when a
//                       running max moves, accumulates O += P(j) V(j) and
//                       writes O / l.
//
// Windows make units short: a 4,096-token window over eight shards is 16
// tiles, while setting a unit up, loading its Q, filling and draining the
// pipeline and writing O took 14 us of a unit's 25 when each unit was its own
// cluster launch.  So clusters are persistent: they walk the list of units,
// and the rings run through the unit borders (a further unit now takes 5-6 us
// besides its tiles; 64 requests x 8 shards on that window: 175 -> 126 us, 101
// now).
//   - A scheduler warp per CTA resolves the next units (rows, spans, the
//     lanes' masks) into a ring of descriptors while the current one runs; it
//     also writes the rows that have nothing to see.
//   - Q of the next unit comes through the score CTA's stage ring as four
//     items (32 lanes x 576 dims, the shape of a KV tile) ahead of its tiles,
//     so it loads while the last tiles of this unit are computed, and moves
//     to TMEM when their S is done.
//   - The next unit's tiles load, are scored and wait as P (four slots) while
//     the value CTA writes this one's O; its first PV waits only until O has
//     been read from TMEM.
// The score CTA's stage sequence counts items (four of Q, then the tiles, per
// unit); everything else counts tiles.  Both counts run through all units, so
// ring slots and parities are those of one long unit.
//
// Lanes may see nothing for many tiles, and sinks may outweigh everything
// after them, so the value CTA keeps O in the scale of the largest running max
// so far and scales a later tile's P down instead of O up (which could
// overflow).  A softmax group moves its max only when a tile's grows past it by
// more than 2^8, so one group may stay below the other for the rest of a unit
// and every second tile be scaled down.  The maxima of a lane are therefore
// whole steps of 2 apart (the first tile's max, or 1, times powers of 2): the
// scaling moves the weights' exponents, and each is rounded to bf16 once.  It
// costs time, not digits (4 trees of 32 rows over 16,000 tokens: 504 us with
// level scores, 591 with one 14 bits above the rest in the fifth tile, 838 with
// scores that rise by 20 bits through the context).
// A weight of 0 does not keep a NaN or an infinity of V out of a product, and a
// token that only some of the rows see may hold one: a non-finite latent shows
// in every lane's score, so the lanes that mask it report it and the value CTA
// clears such values from that tile before PV.  Rows that see the token have a
// NaN weight there and stay NaN, or score it -inf: a weight of 0, with which it
// then counts for nothing, as in the CUDA-core kernel.
//
// What bounds it: the chain of barriers, polls, fences and copies from S to P to
// PV, ~970 cycles a tile (its MMAs alone take ~600; without any KV byte loaded,
// or without the softmax's arithmetic, the time stays), and the way of a unit's
// O out through one SM (26-30 bytes per clock), for which the next unit's PV
// waits ~5,000 cycles (9 % of units of 51 tiles, 30 % of units of 16).  4 trees
// of 32 rows at 128 heads over 8 shards of 12,000-16,384 tokens: 456 us, 58 % of
// the measured bf16 rate; 64 requests x 8 shards on a 4,096-token window: 101
// us, 53 % of the measured bandwidth.  With an FP8 cache a tile takes ~0.75 us,
// the producers' widening.
//
// Roundings: P and, for a bf16 output, O / l once, to bf16 (the MMA's operand
// and the output type); fp8 codes x scale to bf16 (exact for power-of-two
// scales).  Scores, maxima, sums, O and split partials are fp32.
//
// Warp roles (768 threads):
//   warps 0-3   score: softmax group 0 (thread = lane of the unit = TMEM lane;
//                      even tiles)
//               value: max tracking and O rescale; epilogue columns 0-255
//   warps 4-7   score: Q to TMEM; S issuers (warp 4 + b: slot b, tiles j = b mod 4)
//               value: epilogue columns 256-511
//   warps 8-9   score: none
//               value: 8 forwarder (fp8); 9 receive-ring arrivals and the
//                      proxy fence for PV
//   warp 10     both:  TMEM allocation; score: proxy fence of the stage's
//                      rows, forwarder (fp8); value: PV issuer
//   warp 11     both:  scheduler
//   warps 12-19 both:  producers, two groups on alternate items
//   warps 20-23 score: softmax group 1 (odd tiles)
//               value: bf16 cache: receive-ring producers
// Twenty-four warps leave 80 registers a thread, of which softmax and producers
// spill (8 FP8 trees of 16 rows: 150 us with 80 for the producers, 137 with 88),
// so the warps of the issuers and the scheduler hand some of theirs over, a
// group of four warps at a time (Regs).
// Every wait is bounded (a timeout sets DCP_DEVERR_TIMEOUT and ends the
// cluster's work).
#include "dcp_kernels.h"
#include "dcp_select.cuh"
#include "dcp_sm100.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <mutex>

namespace dcp {
namespace {

using namespace sm100;

constexpr int kTile = 32;                        // tokens per tile (MMA N of S, K of PV)
constexpr int kStages = 5;                       // score CTA: stage ring
constexpr int kNch = 9;                          // 64-dim chunks of a latent row
constexpr int kChunkBytes = kTile * 128;         // 32 rows x 64 bf16, 128B-swizzled
constexpr int kStageBytes = kNch * kChunkBytes;  // 36 KB
constexpr int kQItems = 4;                       // stage items of a unit's Q (32 lanes each)
constexpr int kSchedWarp = 11;
constexpr int kProdWarp0 = 12, kProdWarps = 8;   // producer warps: two groups of 4 (alternate items)
constexpr int kGroupThreads = 32 * kProdWarps / 2;
constexpr int kHalfBytes = 4 * kChunkBytes;      // 4 chunks
constexpr int kOwn = 7;                          // value CTA: own ring slots (chunks 4-7)
constexpr int kRecv = 4;                         // value CTA: receive ring slots (chunks 0-3)
// S slots (32 columns) in TMEM, one issuing warp each.  (The plain decode has
// three K-parts of S per tile, so that three warps share its 36 MMAs; behind
// elect_one one warp keeps up, and the parts only cost the softmax their sum:
// 4 trees of 32 rows 510 us, 460 so.)
constexpr int kSBuf = 4;
constexpr int kPSlots = 4;                       // P slots in the value CTA
constexpr int kPBytes = 128 * kTile * 2;         // P tile: 128 rows x 32 bf16, 64B-swizzled
constexpr int kPWarpBytes = kPBytes / 4;         // one softmax warp's 32 rows
// a softmax warp's 32 maxima, then a word (16 bytes in the copy) that says
// whether its lanes met a non-finite score of a token that they do not see
constexpr int kMaxBytes = 128 + 16;
constexpr uint32_t kPTx = kPBytes + 4 * kMaxBytes;  // bytes that fill one P slot
constexpr int kSmWarp1 = kProdWarp0 + kProdWarps;   // score: second softmax group (4 warps)
constexpr int kThreads = 32 * (kSmWarp1 + 4);
// registers a thread of each group of four warps takes (the launch gives 80)
constexpr int kRegsLaunch = 80;
template <bool kFp8>
struct Regs {
  static constexpr int softmax = kFp8 ? 88 : 104, producer = kFp8 ? 88 : 72, issuer = 64, value = 88;
  static constexpr int last = kFp8 ? issuer : producer;  // value CTA's sixth group: idle, or loads the receive ring
  // (more than the launch's would wait forever)
  static_assert(2 * softmax + 2 * producer + 2 * issuer <= 6 * kRegsLaunch, "score CTA: more than was launched");
  static_assert(2 * value + 2 * producer + last + issuer <= 6 * kRegsLaunch, "value CTA: more than was launched");
};
constexpr int kUnits = 3;                        // descriptor ring
constexpr int kFinSlots = 8;                     // value CTA: 1/l of units whose O is not written yet
// P of at most kPSlots later units' tiles can be ahead of a unit's epilogue
static_assert(kFinSlots > kPSlots, "a unit's 1/l must not overwrite one that is still to be read");
constexpr float kRescaleLog2 = 8.0f;  // growth of the running max (a power of 2) that is put up with
constexpr float kWholeSteps = 1048576.0f;  // growths below this are rounded up to whole powers

// TMEM columns
constexpr uint32_t kColQ = 0;    // score: 288 columns of Q, 2 bf16 per column
constexpr uint32_t kColS = 288;  // score: 4 slots x 32 columns of S
constexpr uint32_t kColO = 0;    // value: 512 columns of O
constexpr uint32_t kTmemCols = 512;

// What the roles need to know of a unit.
struct Unit {
  int32_t ntiles;                // < 0: no more units
  int32_t lo, hi;                // its range of the span's index
  int32_t r0, nl;                // first row, lanes in use
  int32_t b, d;                  // request, shard (of D)
  int32_t vs, vb, gap, vlo;      // the rows' span; the least vlo of a row
  int32_t vt;                    // vb under a tree mask, else past everything
  // tiles [plain0, plain1): every row sees every token, and token = index +
  // gap.  All but a few of a long unit's, so what the others need (the span,
  // the rows) is read from here for them and takes no registers.
  int32_t plain0, plain1;
  int32_t c0, c1;                // 128-byte blocks of O's half rows to write (0: lse as well)
  int64_t pair0;                 // (row, head) pair of lane 0 in O_dst / lse_dst
  SelRow row[kMaxGroup];
  uint32_t tree[kMaxGroup][kMaxTree / 32];  // bit t: tree token vb + t
  uint32_t any[kMaxTree / 32];              // their union
};

struct __align__(8) Bars {
  uint64_t kv_loaded[kStages];  // score: this CTA's rows of item g landed (every thread of its producer group)
  // kv_full (score): item g is in its stage: the four producer warps wrote
  // their bytes of the row mask, the forwarder fenced the rows into the async
  // proxy, and (fp8 tiles) the value CTA's 16 KB landed (armed by a producer)
  uint64_t kv_full[kStages];
  // s_done (score): item g's stage is free again: S done
  // (fp8: and chunks 0-3 landed in the value CTA), or Q moved to TMEM.
  // (value, fp8): the same for tiles only
  uint64_t s_done[kStages];
  uint64_t q_gone;            // value (fp8): unit k's Q has left the score CTA's stages (4 remote arrivals)
  uint64_t own_loaded[kOwn];  // value: rows of tile j in own slot j % kOwn
  uint64_t own_free[kOwn];    // value: PV(j) done with own slot j % kOwn
  uint64_t v_full[kRecv];     // value: chunks 0-3 of tile j landed in receive slot j % kRecv
  uint64_t v_free[kRecv];     // both (multicast commit of PV(j)): receive slot j % kRecv may refill
  uint64_t s_full[kSBuf];     // score: S done (commit) + its issuer's arrival
  uint64_t s_free[kSBuf];     // score: the softmax has read the slot (4 warps)
  // score: unit k's Q is in TMEM (four of the S issuers; the others cannot fall
  // two phases behind: the next Q waits for their s_end too)
  uint64_t q_ready;
  uint64_t s_end;             // score: all S of unit k is done (one commit per issuer)
  uint64_t p_full[kPSlots];   // value: P(j) and the maxima of tile j arrived
  uint64_t p_free[kPSlots];   // both (multicast commit of PV(j)); the score CTA waits on it
  uint64_t p_ok[kPSlots];     // value: PV(j) may go (O and P in one scale: 4 warps; V(j) fenced: warp 9)
  uint64_t pv_done[kPSlots];  // value: PV(j) complete
  uint64_t o_final;           // value: unit k's last PV complete
  uint64_t o_free;            // value: unit k's O has been read from TMEM (8 warps)
  uint64_t fin_l[kFinSlots];  // value: 1/l of unit k's lanes arrived
  uint64_t fin[1 + kSBuf];    // each issuing warp's MMAs complete
  uint64_t m_pub[2];          // score: max after unit k's first tile posted (4 warps)
  uint64_t sm_fin;            // score: both softmax groups' l and m of unit k written (8 warps)
  uint64_t ud_full[kUnits], ud_free[kUnits];  // descriptor written / no longer needed (every other warp)
  uint64_t never;             // test hook only: initialised, never arrived on
  int32_t claimed[2];         // score: how many of its items producer group g has claimed a stage for
  int32_t seen[kSBuf];        // score (fp8): tiles up to the last one whose kv_full the issuer of slot b has seen
  uint32_t mask[16];          // score: valid rows of tile j in mask[j % 16]
  uint32_t tmem;
  int32_t abort;
  Unit unit[kUnits];
};

constexpr int kOffStages = 0;                            // score: stage ring
constexpr int kOffOwn = 0;                               // value: own ring
constexpr int kOffRecv = kOwn * kHalfBytes;              // value: receive ring
constexpr int kOffP = kStages * kStageBytes;             // value: P slots; score: P staging
constexpr int kOffMax = kOffP + kPSlots * kPBytes;       // the same for the maxima
constexpr int kOffSm = kOffMax + kPSlots * 4 * kMaxBytes;
constexpr int kSmBytes = (2 + 2 * 4) * 128 * 4;          // score: first tile's max, l and m, of two units
constexpr int kOffFin = kOffSm;                          // value: 1/l per lane, kFinSlots units
constexpr int kOffBars = kOffSm + kSmBytes;
constexpr int kSmemBytes = kOffBars + static_cast<int>(sizeof(Bars)) + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "exceeds the 227 KB of shared memory per CTA");
static_assert(kOffRecv + kRecv * kHalfBytes <= kOffP, "value CTA rings overlap the P slots");
static_assert(kFinSlots * 128 * 4 <= kSmBytes, "the 1/l slots share the score CTA's softmax area");
static_assert(kOffP % 1024 == 0 && kPBytes % 1024 == 0, "P tiles must sit on swizzle-atom boundaries");
static_assert(kRecv <= kPSlots, "a receive ring deeper than the P slots lets p_ok phases mix tiles");
__host__ __device__ constexpr int stage_chunk_off(int st, int c) { return kOffStages + st * kStageBytes + c * kChunkBytes; }

constexpr unsigned kFull = 0xffffffffu;

// (by all warps of a group of four)
template <int kN>
__device__ __forceinline__ void take_regs() {
  if constexpr (kN > kRegsLaunch) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN));
  if constexpr (kN < kRegsLaunch) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN));
}

__device__ __forceinline__ void report(int32_t* dev_error, uint32_t bits) {
  if (dev_error) atomicOr(dev_error, static_cast<int32_t>(bits));
}
__device__ __forceinline__ bool aborted(Bars& bar) { return *reinterpret_cast<volatile int32_t*>(&bar.abort) != 0; }
__device__ __forceinline__ void set_abort(Bars& bar, int32_t* dev_error) {
  report(dev_error, DCP_DEVERR_TIMEOUT);
  atomicExch(&bar.abort, 1);
}
// One lane of the warp, always the same.  MMAs, commits and bulk copies take
// operands that all lanes share; behind this, unlike behind a compare of the
// lane index, they can be kept as such: ~65 cycles per MMA of an issuing warp
// instead of ~120 (4 trees of 32 rows: 548 -> 511 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}
__device__ __forceinline__ bool wait_all(uint64_t* b, uint32_t parity) { return __all_sync(kFull, mbar_wait(b, parity)); }
__device__ __forceinline__ bool wait_all_cluster(uint64_t* b, uint32_t parity) {
  return __all_sync(kFull, mbar_wait_cluster(b, parity));
}

// A warp's place in the ring of unit descriptors.
struct UnitIter {
  int slot = 0;
  uint32_t parity = 0;
  // the next unit, nullptr at the end or when a wait ran out (ok = false)
  __device__ __forceinline__ const Unit* get(Bars& bar, bool& ok) const {
    ok = wait_all(&bar.ud_full[slot], parity);
    if (!ok) return nullptr;
    const Unit* u = &bar.unit[slot];
    return u->ntiles < 0 ? nullptr : u;
  }
  __device__ __forceinline__ void done(Bars& bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.ud_free[slot]);
    if (++slot == kUnits) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// Two FP8 E4M3 codes -> bf16x2 of code x s (s2: s in both halves of a packed
// pair), exact for power-of-two scales.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes, uint64_t s2) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  float lo, hi;
  f2_unpack(f2_mul(f2_pack(f.x, f.y), s2), lo, hi);
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// bits [0, n) of a word
__device__ __forceinline__ uint32_t low_bits(int32_t n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}
// bits [t, t + 32) of a string of kMaxTree bits (zeros outside)
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int32_t t) {
  const int32_t w = t >> 5;
  const uint32_t lo = w >= 0 && w < kMaxTree / 32 ? words[w] : 0u;
  const uint32_t hi = w >= -1 && w < kMaxTree / 32 - 1 ? words[w + 1] : 0u;
  return __funnelshift_r(lo, hi, t & 31);
}

// 32 contiguous bytes of global memory: one store where they are aligned to
// 32, else two.
__device__ __forceinline__ void store32(unsigned char* p, const uint32_t (&w)[8], bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// 4 x 4 transpose of 32-byte sectors over each four lanes: lane t comes with
// the four sectors of its own row and leaves with sector t % 4 of the four rows
// of its lanes (slot i: row t - t % 4 + i), so that four lanes store a row's
// whole 128-byte line.
__device__ __forceinline__ void transpose_sectors(uint32_t (&o)[32], int lane) {
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    const bool up = lane & x;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & x) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t &lo = o[8 * a + i], &hi = o[8 * (a | x) + i];
        const uint32_t got = __shfl_xor_sync(kFull, up ? lo : hi, x);
        if (up) lo = got; else hi = got;
      }
    }
  }
}

// Writes `n` empty rows from `row` on, of one (split, shard): 0 / -inf.  One
// warp of each CTA of the cluster, each writing half of the zeros.
__device__ __forceinline__ void write_empty(const DecodeArgs& a, int32_t s, int32_t dd, int32_t row, int32_t n,
                                            bool score, int lane) {
  if (n <= 0) return;
  const int64_t first = ((static_cast<int64_t>(s) * a.Dn + dd) * a.T + row) * a.H;
  const int64_t pairs = static_cast<int64_t>(n) * a.H;
  const int row_bytes = a.o_bf16 ? 2 * kLatent : 4 * kLatent;
  unsigned char* o = static_cast<unsigned char*>(a.O_dst) + first * row_bytes;
  const bool al32 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
  const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  for (int64_t i = lane + (score ? 32 : 0); i < pairs * (row_bytes / 32); i += 64) store32(o + 32 * i, zero, al32);
  if (score)
    for (int64_t i = lane; i < pairs; i += 32) a.lse_dst[first + i] = -INFINITY;
}

// The descriptor's rows: what each sees of the span, by one warp.
__device__ __forceinline__ void describe_rows(const DecodeArgs& a, const SelRows& R, const SelSpan& S, int32_t d,
                                              int32_t lo, int32_t hi, Unit& U, int lane) {
  const bool tree = a.sel.tree != nullptr;
  // the rows' mask words, two per lane: word w of row i in lane 4 (i % 8) + w,
  // slot i / 8; with the bits of lower words counted
  unsigned long long m[2] = {0ull, 0ull};
  int32_t below[2] = {0, 0}, len[2] = {0, 0};
  const int words = tree ? sel_words(a, R) : 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 8 * e + (lane >> 2), w = lane & 3;
    if (w < words && i < R.n) m[e] = sel_word(a, R, R.i0 + i, w);
  }
  int32_t vlo = 0x7fffffff, from = max(S.vs, 0), to = S.vb;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    int32_t c = __popcll(m[e]), incl = c;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const int32_t v = __shfl_up_sync(kFull, incl, o, 4);
      if ((lane & 3) >= o) incl += v;
    }
    below[e] = incl - c;
    const int i = 8 * e + (lane >> 2);
    len[e] = tree ? sel_prefix(R) + __shfl_sync(kFull, incl, 3, 4) : sel_chain_len(R, R.i0 + i);
    if (i < R.n) {
      const SelRow r = sel_row<true>(a, R, S, R.i0 + i, len[e], d);
      vlo = min(vlo, r.vlo);
      from = max(from, r.vlo);
      to = min(to, r.vend);
      if ((lane & 3) == 0) U.row[i] = r;
    }
  }
  vlo = __reduce_min_sync(kFull, vlo);
  from = __reduce_max_sync(kFull, from);
  to = min(__reduce_min_sync(kFull, to), hi);
  if (lane == 0) {
    U.vlo = vlo;
    U.plain0 = max(from - lo + kTile - 1, 0) / kTile;
    U.plain1 = max(to - lo, 0) / kTile;
  }
  if (!tree) return;
  const int32_t nt = min(S.nv - S.vb, kMaxTree);  // tree tokens of this shard
  const int nw = (nt + 31) / 32;
  for (int w = 0; w < kMaxTree / 32; ++w) {
    const int32_t t = 32 * w + lane;
    const bool in = w < nw && t < nt;
    const int32_t k = in ? sel_position<true>(a, S.token_of(S.vb + t), d) - (R.seq - R.q_len) : 0;
    uint32_t any = 0;
    for (int i = 0; i < R.n; ++i) {
      uint32_t bits = 0;
      if (w < nw) {
        const int from = 4 * (i & 7) + ((k >> 6) & 3), e = i >> 3;
        const unsigned long long word = __shfl_sync(kFull, e ? m[1] : m[0], from);
        const int32_t lower = __shfl_sync(kFull, e ? below[1] : below[0], from);
        const int32_t n = __shfl_sync(kFull, e ? len[1] : len[0], from);
        bool see = in && k >= 0 && k < 64 * words && ((word >> (k & 63)) & 1ull);
        if (a.sel.window > 0) {
          const int32_t rank = sel_prefix(R) + lower + __popcll(word & ((1ull << (k & 63)) - 1ull));
          see = see && (rank < a.sel.sinks || rank >= n - a.sel.window);
        }
        bits = __ballot_sync(kFull, see);
      }
      any |= bits;
      if (lane == 0) U.tree[i][w] = bits;
    }
    if (lane == 0) U.any[w] = any;
  }
}

// -------------------------------------------------------------- producers
// As in the plain decode: warp gw of a group owns rows 8 gw .. 8 gw + 7 of
// an item, four at a time, eight lanes per row (lane x: the x-th 16-byte
// unit of every chunk it loads).  The warp finds the cache rows of four of its
// group's tiles at a time, a lane one row of one tile (resolved by the threads
// that copy, two rows each, the arithmetic took as long as the copies of a
// tile: 4 trees of 32 rows 587 us, 560 so), and fetches their block ids four
// tiles ahead, the first ones of a unit ahead of its Q items.
// (The kind is a value, not a template argument: compiled for one kind, the
// copies of a tile came in one burst per thread, which held up the other
// warps' shared-memory accesses: 0.77 us a tile instead of 0.60.)
enum ProducerKind { kScoreStage, kValueOwn, kValueRecv };
template <bool kFp8>
__device__ __forceinline__ void produce(const DecodeArgs& a, Bars& bar, uint32_t smem_base, int group, int gw,
                                        ProducerKind kind) {
  const bool score = kind == kScoreStage, vrecv = kind == kValueRecv;
  const int lane = threadIdx.x & 31;
  const int x = lane & 7;
  const int row0 = 8 * gw + (lane >> 3), row1 = row0 + 4;
  const int nch = score ? (kFp8 ? 5 : 9) : 4;  // chunks of a tile this CTA loads itself
  const unsigned char* kvb = reinterpret_cast<const unsigned char*>(a.kv);
  const int step = vrecv ? 1 : 2, pre = score ? kQItems : 0;
  uint64_t* slot_free = score ? bar.s_done : (vrecv ? bar.v_free : bar.own_free);
  uint64_t* slot_loaded = score ? bar.kv_loaded : (vrecv ? bar.v_full : bar.own_loaded);
  const int nslots = score ? kStages : (vrecv ? kRecv : kOwn);
  int g = vrecv ? 0 : group;  // this warp's next item in its CTA's sequence
  int base = 0;               // the sequence index of the unit's first item
  int jbase = 0;              // tiles before the unit
  int st = g, round = 0;      // slot and turn of item g
  UnitIter it;
  int32_t other_claimed = 0;  // the other group's claim count as last read (it only grows)
  bool ok = true;
  for (;;) {
    const Unit* U = it.get(bar, ok);
    if (!U) break;
    const int32_t ntiles = U->ntiles, plain0 = U->plain0, plain1 = U->plain1;
    const int32_t l0 = U->lo + U->gap + 8 * gw + (lane & 7);
    const int32_t dI = U->d * a.I, DI = static_cast<int32_t>(a.sel.div_period.d);
    const int32_t* trow = a.block_table + static_cast<int64_t>(U->b) * a.bt_stride +
                          (a.local_tables ? static_cast<int64_t>(U->d - a.d0) * a.bt_shard_stride : 0);
    const int j1 = (g - base) & (step - 1);  // the unit's first tile of this warp
    bool in_n = false;
    int32_t off_n = 0, blk_n = -1;  // row within its block, block id
    // of this lane's row (lane % 8) of the warp's tile n + lane / 8
    auto fetch = [&](int n) {
      const int jj = j1 + (n + (lane >> 3)) * step;
      int32_t tok = l0 + jj * kTile;
      in_n = jj < ntiles;
      if (in_n && (jj < plain0 || jj >= plain1)) {
        // seen by some row of the group?  Then its token of the shard.
        const volatile Unit* V = U;
        const int32_t vs = V->vs, l = tok - V->gap, t = l - V->vb;
        in_n = l < V->hi;
        if (in_n && t >= 0) in_n = t < kMaxTree && ((V->any[t >> 5] >> (t & 31)) & 1u);
        else in_n = in_n && (l < vs || l >= V->vlo);
        if (l < vs) tok = l;
      }
      // the table index: the shard token's position, or (per-shard layout)
      // the local token index itself
      const int32_t lq = fast_div(tok, a.div_I);
      const int32_t pos = in_n ? (a.local_tables ? tok : lq * DI + dI + (tok - lq * a.I)) : 0;
      const int32_t pb = fast_div(pos, a.div_bs);
      off_n = pos - pb * a.block_size;
      blk_n = in_n ? __ldg(trow + pb) : -1;
    };
    // the cache rows of the four tiles that were fetched (-1: not seen)
    int32_t crow_l = -1;
    uint32_t seen_l = 0;
    auto resolve = [&]() {
      const bool there = blk_n >= 0 && blk_n < a.num_blocks;
      crow_l = in_n && there ? blk_n * a.block_size + off_n : -1;
      seen_l = __ballot_sync(kFull, crow_l >= 0);
      if (__any_sync(kFull, in_n && !there) && score && lane == 0) report(a.dev_error, DCP_DEVERR_BAD_BLOCK);
    };
    // tile n: this thread's two rows, and the warp's eight bits of the mask
    int32_t crow[2] = {-1, -1};
    uint32_t m8 = 0;
    auto take = [&](int n) {
      const int from = 8 * (n & 3) + (lane >> 3);
      crow[0] = __shfl_sync(kFull, crow_l, from);
      crow[1] = __shfl_sync(kFull, crow_l, from + 4);
      m8 = (seen_l >> (8 * (n & 3))) & 0xffu;
    };
    // FP8 cache: codes (8 per row and chunk) and row scales of the group's next
    // tile: a tile's are loaded into the registers that the one before leaves
    // as it is converted
    uint2 codes[2][5];
    float rscale[2] = {0.f, 0.f};
    auto load_codes = [&]() {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool valid = crow[e] >= 0;
        const unsigned char* code_row = kvb + static_cast<int64_t>(max(crow[e], 0)) * kKDim + x * 8 + (score ? 0 : 4 * 64);
        rscale[e] = valid ? __ldg(a.kv_scale + crow[e]) : 0.f;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          const int c = i == 4 ? 8 : i;
          if (i < nch) codes[e][i] = valid ? __ldg(reinterpret_cast<const uint2*>(code_row + c * 64)) : make_uint2(0u, 0u);
        }
      }
    };
    int n = 0;  // the warp's tiles of this unit so far
    if (j1 < ntiles) {
      fetch(0);
      if constexpr (kFp8) {
        resolve();
        if (j1 + 4 * step < ntiles) fetch(4);
        take(0);
        load_codes();
      }
    }
    for (; g < base + pre + ntiles; g += step) {
      const int j = g - base - pre;  // tile of the unit, or < 0: a quarter of Q
      // score CTA: the other group has claimed its stage for item g - 5 (so
      // the parity below can only mean that item; see the plain decode)
      if (score && g >= kStages) {
        const int32_t need = ((g - kStages) >> 1) + 1;
        for (uint32_t i = 0; other_claimed < need && i < kWaitLimit; ++i)
          other_claimed = ld_relaxed_shared(&bar.claimed[group ^ 1]);
        ok = __all_sync(kFull, other_claimed >= need);
      }
      if (!ok) break;
      if (!kFp8 && j >= 0) {
        if ((n & 3) == 0) {
          resolve();
          if (j + 4 * step < ntiles) fetch(n + 4);
        }
        take(n);
      }
      const bool ab = aborted(bar);
      ok = wait_all(&slot_free[st], (round & 1) ^ 1);
      if (!ok) break;
      if (score && gw == 0 && lane == 0) st_relaxed_shared(&bar.claimed[group], (g >> 1) + 1);
      if (score) {
        // this warp's 8 rows of the tile's mask, released by its arrival on
        // kv_full; fp8: warp 0 also arms kv_full for the value CTA's 16 KB
        if (lane == 0) {
          if (j >= 0) reinterpret_cast<volatile uint8_t*>(&bar.mask[(jbase + j) & 15])[gw] = static_cast<uint8_t>(m8);
          if (kFp8 && gw == 0 && j >= 0) mbar_arrive_expect_tx(&bar.kv_full[st], kHalfBytes);
          else mbar_arrive(&bar.kv_full[st]);
        }
      }
      if (j < 0) {
        // 32 lanes of Q (zeros past the unit's lanes), laid out as a tile
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = e ? row1 : row0, h = 32 * (g - base) + row;
          const bool live = h < U->nl;
          const int i = live ? fast_div(h, a.sel.div_H) : 0;
          const unsigned char* src = reinterpret_cast<const unsigned char*>(a.q) +
                                     2 * ((U->r0 + i) * a.q_stride_tok + (live ? h - i * a.H : 0) * kKDim) + x * 16;
          const uint32_t dst = smem_base + stage_chunk_off(st, 0) + static_cast<uint32_t>(row * 128 + ((x ^ (row & 7)) << 4));
#pragma unroll
          for (int c = 0; c < kNch; ++c) cp_async16_zfill(dst + c * kChunkBytes, src + c * 128, live ? 16u : 0u);
        }
        cp_async_mbar_arrive_noinc(&slot_loaded[st]);
      } else {
        // (the slot's first chunk and the row's first byte that this CTA loads:
        // what follows is constant offsets)
        const uint32_t slot0 = score ? smem_base + stage_chunk_off(st, 0)
                                     : smem_base + (vrecv ? kOffRecv : kOffOwn) + st * kHalfBytes;
        const int src_off = score || vrecv ? 0 : 4 * 128;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = e ? row1 : row0;
          const unsigned char* src_row = kvb + static_cast<int64_t>(max(crow[e], 0)) * (kKDim * 2) + x * 16 + src_off;
          const uint32_t src_bytes = crow[e] >= 0 ? 16u : 0u;
          const uint32_t dst0 = slot0 + static_cast<uint32_t>(row * 128 + ((x ^ (row & 7)) << 4));
          const uint64_t sc = f2_pack(rscale[e], rscale[e]);
#pragma unroll
          for (int i = 0; i < (kFp8 ? 5 : 9); ++i) {
            if (i >= nch) continue;
            const int c = kFp8 && i == 4 ? 8 : i;  // (the score CTA's fifth FP8 chunk is the rope's)
            const uint32_t dst = dst0 + c * kChunkBytes;
            if constexpr (kFp8) {
              const uint2 w = codes[e][i];
              const uint4 v = make_uint4(e4m3x2_to_bf16x2(w.x, sc), e4m3x2_to_bf16x2(w.x >> 16, sc),
                                         e4m3x2_to_bf16x2(w.y, sc), e4m3x2_to_bf16x2(w.y >> 16, sc));
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                           : "memory");
            } else {
              cp_async16_zfill(dst, src_row + c * 128, src_bytes);
            }
          }
        }
        ++n;
        if (kFp8 && j + step < ntiles) {  // (after the stores: in between, they held the stores up)
          if ((n & 3) == 0) {
            resolve();
            if (j + 5 * step < ntiles) fetch(n + 4);
          }
          take(n);
          load_codes();
        }
        if constexpr (kFp8) mbar_arrive(&slot_loaded[st]);
        else cp_async_mbar_arrive_noinc(&slot_loaded[st]);
      }
      if (__any_sync(kFull, ab)) {
        ok = false;
        break;
      }
      st += step;
      if (st >= nslots) {
        st -= nslots;
        ++round;
      }
    }
    if (!ok) break;
    base += pre + ntiles;
    jbase += ntiles;
    it.done(bar, lane);
  }
  if (!ok) set_abort(bar, a.dev_error);
  cp_async_wait<0>();
}

// kFp8: the cache holds FP8 E4M3 codes (576 bytes a row) with one fp32 scale
// per slot; the producers widen them to bf16 on their way into shared memory.
template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) decode_select_kernel(DecodeArgs a, int32_t units) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // (an offset from the array, not a rounded pointer, keeps the address space
  // known: 32-bit shared-memory accesses instead of 64-bit generic ones)
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars& bar = *reinterpret_cast<Bars*>(smem + kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const bool score = cta == 0;
  const uint32_t peer = cta ^ 1u;

  // ---------------------------------------------------------------- setup
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.kv_loaded[i], kGroupThreads);
      mbar_init(&bar.kv_full[i], 5);  // 4 producer warps of the item's group + the forwarder
      mbar_init(&bar.s_done[i], kFp8 ? 2 : 1);
    }
    for (int i = 0; i < kOwn; ++i) { mbar_init(&bar.own_loaded[i], kGroupThreads); mbar_init(&bar.own_free[i], 1); }
    mbar_init(&bar.q_gone, 4);
    for (int i = 0; i < kRecv; ++i) { mbar_init(&bar.v_full[i], kFp8 ? 1 : kGroupThreads); mbar_init(&bar.v_free[i], 1); }
    for (int i = 0; i < kSBuf; ++i) { mbar_init(&bar.s_full[i], 2); mbar_init(&bar.s_free[i], 4); }
    mbar_init(&bar.q_ready, 4);
    mbar_init(&bar.s_end, kSBuf);
    for (int i = 0; i < kPSlots; ++i) {
      mbar_init(&bar.p_full[i], 1);
      mbar_init(&bar.p_free[i], 1);
      mbar_init(&bar.p_ok[i], 5);
      mbar_init(&bar.pv_done[i], 1);
    }
    mbar_init(&bar.o_final, 1);
    mbar_init(&bar.o_free, 8);
    for (int i = 0; i < kFinSlots; ++i) mbar_init(&bar.fin_l[i], 1);
    for (int i = 0; i < 1 + kSBuf; ++i) mbar_init(&bar.fin[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bar.m_pub[i], 4);
    mbar_init(&bar.sm_fin, 8);
    for (int i = 0; i < kUnits; ++i) { mbar_init(&bar.ud_full[i], 1); mbar_init(&bar.ud_free[i], kThreads / 32 - 1); }
    mbar_init(&bar.never, 1);
    bar.claimed[0] = bar.claimed[1] = 0;
    for (int i = 0; i < kSBuf; ++i) bar.seen[i] = 0;
    bar.abort = 0;
    fence_mbar_init();
    if (!score) {
      for (int i = 0; i < kPSlots; ++i) mbar_arrive_expect_tx(&bar.p_full[i], kPTx);
      if (kFp8)
        for (int i = 0; i < kRecv; ++i) mbar_arrive_expect_tx(&bar.v_full[i], kHalfBytes);
      for (int i = 0; i < kFinSlots; ++i) mbar_arrive_expect_tx(&bar.fin_l[i], 128 * 4);
    }
  }
  if (warp == 10) {
    tmem_alloc(&bar.tmem, kTmemCols);
    tmem_relinquish();
  }
  UnitIter it;
  // The cluster's units, in both CTAs alike: the list is dealt to the clusters
  // in rounds, every other round backwards (it is sorted by length, so that
  // evens out the longer units of the early places).
  int32_t dealt = 0;
  // scheduler: the next unit with something to see goes into descriptor U
  // (rows without are written on the way); false at the end of the list
  auto next_unit = [&](Unit& U) {
    const int32_t clusters = static_cast<int32_t>(gridDim.x >> 1), c = static_cast<int32_t>(blockIdx.x >> 1);
    for (; dealt * clusters < units; ++dealt) {
      const int32_t at = dealt * clusters + ((dealt & 1) ? clusters - 1 - c : c);
      if (at >= units) continue;
      // (units whose output several clusters share are all in the first turn of the deal)
      int32_t u = at, part = 0;
      if (a.unit_order) {
        u = *static_cast<const volatile int32_t*>(a.unit_order + at);
      } else if (a.sel.parts_log2 > 0) {
        const int32_t parts = 1 << a.sel.parts_log2, mine = a.B * a.sel.chunks * a.Dn * a.plan.splits;
        part = at < mine * parts ? at & (parts - 1) : 0;
        u = at < mine * parts ? at >> a.sel.parts_log2 : at - mine * (parts - 1);
      }
      const SelCoords k = sel_coords(a, u);
      const SelUnit su = sel_unit(a, k.b, k.c);
      const int32_t d = a.d0 + k.dd;
      if (su.R.err && lane == 0 && score && part == 0 && k.c == 0 && k.dd == 0 && k.s == 0) report(a.dev_error, su.R.err);
      SelSpan S{0, 0, 0, 0};
      if (su.live) S = sel_span<true>(a, su.R, d);
      const int32_t lo = k.s * a.plan.chunk;
      const int32_t hi = min(S.nv, lo + a.plan.chunk);
      if (part == 0) write_empty(a, k.s, k.dd, su.extra0, su.extra, score, lane);
      if (lo >= hi) {
        if (part == 0) write_empty(a, k.s, k.dd, su.R.r0, su.R.n, score, lane);
        continue;
      }
      if (lane == 0) {
        U.ntiles = (hi - lo + kTile - 1) / kTile;
        U.lo = lo;
        U.hi = hi;
        U.r0 = su.R.r0;
        U.nl = su.R.n * a.H;
        U.b = su.R.b;
        U.d = d;
        U.vs = S.vs;
        U.vb = S.vb;
        U.vt = a.sel.tree ? S.vb : 0x7fffffff;
        U.gap = S.gap;
        const int32_t blocks = a.o_bf16 ? 4 : 8;
        U.c0 = (blocks * part) >> a.sel.parts_log2;
        U.c1 = (blocks * (part + 1)) >> a.sel.parts_log2;
        U.pair0 = ((static_cast<int64_t>(k.s) * a.Dn + k.dd) * a.T + su.R.r0) * a.H;
      }
      describe_rows(a, su.R, S, d, lo, hi, U, lane);
      ++dealt;
      return true;
    }
    return false;
  };
  bool more = false;
  if (warp == kSchedWarp) {  // alongside the set-up
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the order; the inputs are older
    more = next_unit(bar.unit[0]);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // peer's barriers initialised and armed before any remote operation
  tc_fence_after();
  const uint32_t tbase = bar.tmem;
  const uint32_t smem_base = smem_u32(smem);
  int pdone = 0;  // value, warps 0-3: P tiles received

  // (setmaxnreg is one instruction for a whole group of four warps)
  const int group = warp >> 2;
  if (warp >= kProdWarp0 && (warp < kSmWarp1 || (!kFp8 && !score))) {
    take_regs<Regs<kFp8>::producer>();
    produce<kFp8>(a, bar, smem_base, (warp - kProdWarp0) >> 2, warp & 3,
                  score ? kScoreStage : (warp < kSmWarp1 ? kValueOwn : kValueRecv));
  } else if (score && (group == 0 || group == 5)) {
    take_regs<Regs<kFp8>::softmax>();
    // ------------------------------------------------------------- softmax
    // Two groups take alternate tiles, each with its own running max and sum.
    // A unit's second tile starts from its first one's max, so that both
    // groups keep to the same one until it has to grow by more than 2^8; what
    // a group finds later stays its own (the value CTA brings tiles of
    // different maxima together), so results do not depend on timing.  (The
    // plain decode hands the max over at every tile: a barrier and a shared
    // load that queue behind the copies, 530 of a group's 2,700 cycles.)
    const int sg = warp < 4 ? 0 : 1, q4 = warp & 3;
    const int h = q4 * 32 + lane;
    const uint32_t lane_addr = tbase + (static_cast<uint32_t>(q4 * 32) << 16);
    float* m_first = reinterpret_cast<float*>(smem + kOffSm);  // [unit % 2][128]
    // (as of elect_one, the same for the warp)
    const int qu = __shfl_sync(kFull, q4, 0);
    const uint32_t peer_base = map_peer(smem_base, peer), peer_p_full = map_peer(smem_u32(&bar.p_full[0]), peer);
    const float sl2 = a.scale * kLog2e;
    const int sw = (h >> 1) & 3;  // 64-byte swizzle of row h
    const uint32_t p_row = static_cast<uint32_t>((h >> 3) * 512 + (h & 7) * 64);
    bool ok = true;
    // failure-path test hook: a wait that runs out (nothing completes `never`)
    if (a.stall_test && sg == 0) ok = wait_all(&bar.never, 0);
    int j0 = 0;  // tiles before the unit
    for (int k = 0; ok; ++k) {
      const Unit* U = it.get(bar, ok);
      if (!U) break;
      const int32_t ntiles = U->ntiles, plain0 = U->plain0, plain1 = U->plain1;
      float m_used = -INFINITY, l_sum = 0.f;
      for (int j = j0 + ((j0 ^ sg) & 1); ok && j < j0 + ntiles; j += 2) {
        const uint32_t uj = static_cast<uint32_t>(j);
        const uint32_t b = uj % kSBuf, slot = uj % kPSlots, turn = (uj / kPSlots) & 1;
        static_assert(kSBuf == kPSlots, "one turn for both");
        const int i0 = j - j0;
        float m_other = -INFINITY;
        if (i0 == 1) {
          // (no phase of m_pub is skipped: unit k - 2's is over, since every
          // warp has waited for that unit's sm_fin)
          ok = wait_all(&bar.m_pub[k & 1], (k >> 1) & 1);
          if (!ok) break;
          m_other = *reinterpret_cast<volatile float*>(&m_first[(k & 1) * 128 + h]);
        }
        ok = wait_all(&bar.s_full[b], turn);
        if (!ok) break;
        tc_fence_after();
        uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&bar.mask[j & 15]);
        uint32_t sr[32];
        tmem_ld32(lane_addr + kColS + 32 * b, sr);
        // what this lane sees of the tile, while S arrives
        uint32_t hidden = 0;  // loaded for another row of the group only
        if (i0 < plain0 || i0 >= plain1) {
          const volatile Unit* V = U;
          const int32_t v0 = V->lo + i0 * kTile, vt = V->vt;
          const bool live = h < V->nl;
          const int row_i = live ? fast_div(h, a.sel.div_H) : 0;
          uint32_t mine = low_bits(V->row[row_i].vend - v0) & (low_bits(V->vs - v0) | ~low_bits(V->row[row_i].vlo - v0));
          if (v0 + kTile > vt) mine |= bits_at(U->tree[row_i], v0 - vt);
          hidden = live ? mask & ~mine : 0u;
          mask &= live ? mine : 0u;
        }
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.s_free[b]);
        float sc[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) sc[i] = __uint_as_float(sr[i]);
        bool foul = false;
        if (__any_sync(kFull, hidden != 0)) {
#pragma unroll
          for (int i = 0; i < 32; ++i) foul |= ((hidden >> i) & 1u) && !(fabsf(sc[i]) < INFINITY);
          foul = __any_sync(kFull, foul);
        }
        // online softmax in base 2: x = s * scale * log2(e), scaled before the
        // mask and the max so that any finite scale (zero and negative too)
        // keeps masked tokens at -inf; masked tokens get weight 0 by selection
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
#pragma unroll
        for (int i = 0; i < 16; ++i) f2_unpack(f2_mul(f2_pack(sc[2 * i], sc[2 * i + 1]), sl2x2), sc[2 * i], sc[2 * i + 1]);
        if (mask != 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < 32; ++i) sc[i] = (mask >> i) & 1u ? sc[i] : -INFINITY;
        }
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = fmaxf(fmaxf(sc[4 * i], sc[4 * i + 1]), fmaxf(sc[4 * i + 2], sc[4 * i + 3]));
        const float tmax = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                 fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        // the unit's second tile: adopt the first one's max if it is larger
        if (m_other > m_used) {
          if (m_used != -INFINITY) l_sum *= ex2_approx(m_used - m_other);
          m_used = m_other;
        }
        // lazy rescale: the running max only moves when it would grow by more
        // than 2^8, and then by whole steps (from 0 where the first tile set
        // none; the groups share that first max, so all of a lane's are whole
        // steps apart).  Past 2^20, where fp32 has no sixteenth of a step left,
        // it moves to the score itself: what is scaled across that is 0.
        const bool grow = m_used == -INFINITY ? (tmax != -INFINITY) : (tmax > m_used + kRescaleLog2);
        if (grow) {
          const float up = tmax - m_used;
          float m = i0 == 0 ? tmax : ceilf(tmax);
          if (m_used != -INFINITY) {
            m = up < kWholeSteps ? m_used + ceilf(up) : tmax;
            l_sum *= ex2_approx(m_used - m);
          }
          m_used = m;
        }
        if (i0 == 0) {
          m_first[(k & 1) * 128 + h] = m_used;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.m_pub[k & 1]);
        }
        // p = 2^(x - m); masked (-inf) scores give exactly 0, and nothing is
        // live while m is still -inf
        const float nm = m_used == -INFINITY ? 0.f : -m_used;
        const uint64_t nmx2 = f2_pack(nm, nm);
        uint32_t pk[16];
        uint64_t ps[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float e0, e1;
          f2_unpack(f2_add(f2_pack(sc[2 * i], sc[2 * i + 1]), nmx2), e0, e1);
          const float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
          __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);  // P feeds the PV MMA in bf16
          ps[i & 1] = f2_add(ps[i & 1], f2_pack(p0, p1));     // l (hence the LSE) stays fp32
          pk[i] = *reinterpret_cast<uint32_t*>(&pb);
        }
        float q0, q1, q2, q3;
        f2_unpack(ps[0], q0, q1);
        f2_unpack(ps[1], q2, q3);
        l_sum += (q0 + q1) + (q2 + q3);
        // the slot (and this CTA's staging copy of it) is free once PV(j - kPSlots) is done
        ok = wait_all_cluster(&bar.p_free[slot], turn ^ 1);
        if (!ok) break;
        unsigned char* stg = smem + kOffP + slot * kPBytes;
        unsigned char* smx = smem + kOffMax + (4 * slot + q4) * kMaxBytes;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(stg + p_row + ((c ^ sw) << 4)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        *reinterpret_cast<float*>(smx + 4 * lane) = m_used;
        if (lane == 0) *reinterpret_cast<uint32_t*>(smx + 128) = foul ? 1u : 0u;
        fence_proxy_async_smem();
        __syncwarp();
        const int su = __shfl_sync(kFull, slot, 0);
        if (elect_one()) {
          // this warp's 32 rows of P, then its 32 maxima and flag: two bulk copies
          const uint32_t full = peer_p_full + 8 * su;
          const uint32_t rows = kOffP + su * kPBytes + qu * kPWarpBytes, maxima = kOffMax + (4 * su + qu) * kMaxBytes;
          bulk_copy_to_peer(peer_base + rows, smem + rows, kPWarpBytes, full);
          bulk_copy_to_peer(peer_base + maxima, smem + maxima, kMaxBytes, full);
        }
      }
      // both groups' sums meet here (two units' worth of space); group 0
      // finishes the unit.  A group's next arrival waits for this unit's
      // phase, so one that has no tile in a short unit cannot run ahead.
      if (ok && k > 0) ok = wait_all(&bar.sm_fin, (k - 1) & 1);
      if (!ok) break;
      float* fin_sh = m_first + (2 + 4 * (k & 1)) * 128;  // [group][l, m][128]
      fin_sh[(2 * sg) * 128 + h] = l_sum;
      fin_sh[(2 * sg + 1) * 128 + h] = m_used;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.sm_fin);
      if (sg == 0) {
        ok = wait_all(&bar.sm_fin, k & 1) && !__any_sync(kFull, aborted(bar));
        if (!ok) break;
        const float l1 = *reinterpret_cast<volatile float*>(&fin_sh[2 * 128 + h]);
        const float m1 = *reinterpret_cast<volatile float*>(&fin_sh[3 * 128 + h]);
        // O is in the scale of the largest m of any tile
        const float mo = fmaxf(m_used, m1);
        // (a group whose m is -inf has a sum of 0, or of NaN where all it saw
        // were NaN scores, which a maximum passes over: NaN stays)
        const float l = (m_used != -INFINITY ? l_sum * ex2_approx(m_used - mo) : l_sum) +
                        (m1 != -INFINITY ? l1 * ex2_approx(m1 - mo) : l1);
        const bool some = l != 0.f;  // (a NaN weight gives NaN, not an empty row)
        const int fs = k % kFinSlots;
        st_async_peer_b32(map_peer(smem_base + kOffFin + fs * 512 + 4 * h, peer), __float_as_uint(some ? 1.f / l : 0.f),
                          map_peer(smem_u32(&bar.fin_l[fs]), peer));
        if (h < U->nl && U->c0 == 0) a.lse_dst[U->pair0 + h] = some ? (mo + log2f(l)) * kLn2 : -INFINITY;
      }
      j0 += ntiles;
      it.done(bar, lane);
    }
    if (!ok) set_abort(bar, a.dev_error);
  } else if (!score && group < 2) {
    take_regs<Regs<kFp8>::value>();
    const int q4 = warp & 3;
    const int h = q4 * 32 + lane;
    const uint32_t lane_addr = tbase + (static_cast<uint32_t>(q4 * 32) << 16);
    const bool al32 = (reinterpret_cast<uintptr_t>(a.O_dst) & 31u) == 0;
    bool ok = true;
    int j0 = 0;
    for (int k = 0;; ++k) {
      const Unit* U = it.get(bar, ok);
      if (!U) break;
      const int32_t ntiles = U->ntiles;
      if (warp < 4) {
        // --------------------------------------------- max tracking, rescale
        float m_prev = -INFINITY;
        for (int j = j0; j < j0 + ntiles; ++j) {
          const int slot = j % kPSlots;
          ok = wait_all_cluster(&bar.p_full[slot], (j / kPSlots) & 1);
          if (!ok) break;
          // the slot's next fill (tile j + kPSlots) cannot start before PV(j)
          // frees it, and PV(j) waits for this warp's p_ok below
          if (warp == 0 && lane == 0) mbar_arrive_expect_tx(&bar.p_full[slot], kPTx);
          ++pdone;
          const unsigned char* mx = smem + kOffMax + 4 * slot * kMaxBytes;
          const float m_new = *reinterpret_cast<const volatile float*>(mx + q4 * kMaxBytes + 4 * lane);
          const uint32_t foul = *reinterpret_cast<const volatile uint32_t*>(mx + (lane & 3) * kMaxBytes + 128);
          // a tile computed with m = -inf has P = 0 and leaves O as it is
          const bool up = m_new > m_prev && m_prev != -INFINITY;
          // a tile in a smaller max's scale than O's: this lane's 32 weights
          // of P(j) (64 bytes, in any order) come down to O's, by a power of 2
          const bool down = m_new < m_prev && m_new != -INFINITY;
          const bool rare = __any_sync(kFull, foul != 0 || up || down);  // (one vote in the common case)
          if (rare && __any_sync(kFull, foul != 0)) {
            // clear the tile's NaNs and infinities, a quarter per warp (both
            // rings' slots refill only after PV(j), which waits for this
            // warp's p_ok)
            const int vs = j % kRecv, os = j % kOwn;
            ok = wait_all_cluster(&bar.v_full[vs], (j / kRecv) & 1) && wait_all(&bar.own_loaded[os], (j / kOwn) & 1);
            if (!ok) break;
            for (int i = h; i < 2 * kHalfBytes / 16; i += 128) {
              uint4* p = reinterpret_cast<uint4*>(smem + (i < kHalfBytes / 16 ? kOffRecv + vs * kHalfBytes + 16 * i
                                                                             : kOffOwn + os * kHalfBytes + 16 * i - kHalfBytes));
              uint4 y = *p;
              uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                if ((w[n] & 0x7f80u) == 0x7f80u) w[n] &= 0xffff0000u;
                if ((w[n] & 0x7f800000u) == 0x7f800000u) w[n] &= 0x0000ffffu;
              }
              *p = y;
            }
            fence_proxy_async_smem();
          }
          if (rare && __any_sync(kFull, up)) {
            // O holds this unit's PVs up to j - 1: wait for them, then scale
            // this warp's rows
            const int jp = j - 1;
            ok = wait_all(&bar.pv_done[jp % kPSlots], (jp / kPSlots) & 1);
            if (!ok) break;
            tc_fence_after();
            const float alpha = up ? ex2_approx(m_prev - m_new) : 1.f;
            for (int c = 0; c < 16; ++c) {
              uint32_t o[32];
              tmem_ld32(lane_addr + kColO + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(lane_addr + kColO + 32 * c, o);
            }
            tmem_wait_st();
          }
          if (rare && __any_sync(kFull, down)) {
            if (down) {
              const float f = ex2_approx(m_new - m_prev);
              uint4* row = reinterpret_cast<uint4*>(smem + kOffP + slot * kPBytes + (h >> 3) * 512 + (h & 7) * 64);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint4 y = row[i];
                uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  const __nv_bfloat162 z = __floats2bfloat162_rn(__uint_as_float(w[n] << 16) * f,
                                                                 __uint_as_float(w[n] & 0xffff0000u) * f);
                  w[n] = *reinterpret_cast<const uint32_t*>(&z);
                }
                row[i] = y;
              }
            }
            fence_proxy_async_smem();
          }
          if (m_new > m_prev) m_prev = m_new;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_ok[slot]);
        }
        if (!ok) break;
      }
      // ---------------------------------------------------------- epilogue
      // warps 0-3 write value dims [0, 256), warps 4-7 dims [256, 512), each
      // lane its own row in whole 32-byte sectors, straight from TMEM
      const int fs = k % kFinSlots;
      ok = wait_all(&bar.o_final, k & 1) && wait_all_cluster(&bar.fin_l[fs], (k / kFinSlots) & 1) && !__any_sync(kFull, aborted(bar));
      if (!ok) break;
      tc_fence_after();
      const float inv = *reinterpret_cast<const volatile float*>(smem + kOffFin + fs * 512 + 4 * h);
      // blocks of 128 bytes a row (64 bf16 or 32 fp32 columns), transposed
      // over four lanes to whole lines (each lane storing its own row took
      // 4.2 us a bf16 unit and 7.4 us an fp32 one)
      const volatile Unit* V = U;
      const int32_t nl = V->nl, c0 = V->c0, c1 = V->c1;
      const int64_t pair0 = V->pair0;
      const int row_bytes = a.o_bf16 ? 2 * kLatent : 4 * kLatent;
      const uint32_t col0 = tbase + (static_cast<uint32_t>(q4 * 32) << 16) + kColO + 256 * (warp >> 2);
      unsigned char* out = static_cast<unsigned char*>(a.O_dst) + (pair0 + q4 * 32 + (lane & ~3)) * row_bytes +
                           (warp >> 2) * (row_bytes / 2) + 32 * (lane & 3);
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        uint32_t o[32];
        if (a.o_bf16) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            uint32_t x[32];
            tmem_ld32(col0 + 64 * c + 32 * n, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(x[2 * i]) * inv, __uint_as_float(x[2 * i + 1]) * inv);
              o[16 * n + i] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
        } else {
          tmem_ld32(col0 + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
        }
        if (c == c1 - 1) {
          // O is read: the next unit's PV may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.o_free);
        }
        transpose_sectors(o, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) w[n] = o[8 * i + n];
          if (q4 * 32 + (lane & ~3) + i < nl) store32(out + i * row_bytes + 128 * c, w, al32);
        }
        __syncwarp();
      }
      // every warp has passed this unit's 1/l when the next unit's O is being
      // written, long before the slot's next turn
      if (warp == 0 && lane == 0) mbar_arrive_expect_tx(&bar.fin_l[fs], 128 * 4);
      j0 += ntiles;
      it.done(bar, lane);
    }
    if (!ok) set_abort(bar, a.dev_error);
  } else if (group < 3) {
    take_regs<Regs<kFp8>::issuer>();
    if (warp == kSchedWarp) {
      // ------------------------------------------------------------ scheduler
      bool ok = true;
      for (; more; ) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.ud_full[it.slot]);
        if (++it.slot == kUnits) {
          it.slot = 0;
          it.parity ^= 1u;
        }
        ok = wait_all(&bar.ud_free[it.slot], it.parity ^ 1u);
        if (!ok) break;
        more = next_unit(bar.unit[it.slot]);
      }
      if (ok && lane == 0) {
        bar.unit[it.slot].ntiles = -1;
        mbar_arrive(&bar.ud_full[it.slot]);
      }
      if (!ok) set_abort(bar, a.dev_error);
    } else if (score && warp == 10) {
      // ------------------------------------------------- score CTA forwarder
      // fence: once this CTA's rows of item gf have landed, fence them into the
      //   async proxy and arrive on kv_full.
      // copy (fp8): once tile item gc < gf is fenced and the value CTA's receive
      //   slot is free, copy chunks 0-3 (16 KB) into it.
      bool ok = true;
      int gf = 0, gc = 0, jc = 0, base = 0;
      for (;;) {
        const Unit* U = it.get(bar, ok);
        if (!U) break;
        const int end = base + kQItems + U->ntiles;
        uint32_t idle = 0;
        while (ok && gc < end) {
          bool moved = false;
          if (!kFp8) {
            ok = wait_all(&bar.kv_loaded[gf % kStages], (gf / kStages) & 1);
            if (!ok) break;
          }
          if (gf < end && (!kFp8 || __all_sync(kFull, mbar_peek(&bar.kv_loaded[gf % kStages], (gf / kStages) & 1)))) {
            fence_proxy_async_smem();  // the producers' writes -> S and the bulk copy
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.kv_full[gf % kStages]);
            ++gf;
            moved = true;
          }
          if (!kFp8) gc = gf;
          if (kFp8 && gc < gf) {
            if (gc - base < kQItems) {
              ++gc;
              moved = true;
            } else if (__all_sync(kFull, mbar_peek_cluster(&bar.v_free[jc % kRecv], ((jc / kRecv) & 1) ^ 1))) {
              const int st = gc % kStages, rs = jc % kRecv;
              if (lane == 0)
                bulk_copy_to_peer(map_peer(smem_base + kOffRecv + rs * kHalfBytes, peer), smem + stage_chunk_off(st, 0),
                                  kHalfBytes, map_peer(smem_u32(&bar.v_full[rs]), peer));
              __syncwarp();
              ++gc;
              ++jc;
              moved = true;
            }
          }
          idle = moved ? 0u : idle + 1u;
          if (idle > kWaitLimit) ok = false;
        }
        if (!ok) break;
        base = end;
        it.done(bar, lane);
      }
      if (!ok) set_abort(bar, a.dev_error);
    } else if (score && group == 1) {
      // --------------------------------------------- Q to TMEM, S MMA issuers
      // warp 4 + b owns S slot b, for tiles j = b (mod 4)
      const int b = __shfl_sync(kFull, warp - 4, 0);
      const uint32_t id_s = idesc_bf16(128, kTile, 0, 0);
      const uint64_t dk = smem_desc(smem_base + kOffStages, 16, 1024, kSwizzle128B);
      const uint32_t dS = tbase + kColS + 32 * b, qa = tbase + kColQ;
      bool ok = true;
      int32_t other_seen = 0;
      int g0 = 0, j0 = 0;  // items and tiles before the unit
      for (int k = 0;; ++k) {
        const Unit* U = it.get(bar, ok);
        if (!U) break;
        const int ntiles = U->ntiles;
        {
          // item warp - 4 of the unit's Q, once no MMA reads the previous one
          if (k > 0) ok = wait_all(&bar.s_end, (k - 1) & 1);
          const int g = g0 + warp - 4, st = g % kStages;
          ok = ok && wait_all_cluster(&bar.kv_full[st], (g / kStages) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t lane_addr = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
          // (16 columns at a time, the next 16 read before these are stored)
          uint32_t v[2][16];
          auto read = [&](int n, uint32_t (&r)[16]) {  // dims 32 n ..: unit i of a chunk sits at position i ^ (lane & 7)
            const unsigned char* row = smem + stage_chunk_off(st, 0) + (n >> 1) * kChunkBytes + lane * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 y = *reinterpret_cast<const uint4*>(row + (((4 * (n & 1) + i) ^ (lane & 7)) << 4));
              r[4 * i] = y.x; r[4 * i + 1] = y.y; r[4 * i + 2] = y.z; r[4 * i + 3] = y.w;
            }
          };
          read(0, v[0]);
#pragma unroll 1
          for (int n = 0; n < 2 * kNch; n += 2) {
            read(n + 1, v[1]);
            tmem_st16(lane_addr + kColQ + 16 * n, v[0]);
            if (n + 2 < 2 * kNch) read(n + 2, v[0]);
            tmem_st16(lane_addr + kColQ + 16 * n + 16, v[1]);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            // the stage is free: as many arrivals as a tile's
            for (int i = 0; i < (kFp8 ? 2 : 1); ++i) mbar_arrive(&bar.s_done[st]);
            mbar_arrive(&bar.q_ready);
            if (kFp8) mbar_arrive_remote(map_peer(smem_u32(&bar.q_gone), peer));
          }
          __syncwarp();
        }
        ok = wait_all(&bar.q_ready, k & 1);
        tc_fence_after();
        for (int j = j0 + ((b - j0) & (kSBuf - 1)); ok && j < j0 + ntiles; j += kSBuf) {
          const int g = g0 + kQItems + j - j0, st = g % kStages, u = j / kSBuf;
          ok = wait_all(&bar.s_free[b], (u & 1) ^ 1);
          // The stage's previous item has been full, so that the parity below
          // can only mean this one: the forwarder arrives in order, so it has
          // since S(j - 4) was issued; in the fp8 form the value CTA's halves
          // might land out of order, so that tile's issuer says so (a count
          // that only grows, read again only when it falls short).
          if constexpr (kFp8) {
            for (uint32_t i = 0; other_seen < j - kStages + 1 && i < kWaitLimit; ++i)
              other_seen = ld_relaxed_shared(&bar.seen[(j + kSBuf * kStages - kStages) % kSBuf]);
            ok = ok && __all_sync(kFull, other_seen >= j - kStages + 1);
          }
          ok = ok && wait_all_cluster(&bar.kv_full[st], (g / kStages) & 1);
          if (kFp8 && lane == 0) st_relaxed_shared(&bar.seen[b], j + 1);
          if (!ok) break;
          // this arrival passes on (release after the acquire of kv_full)
          // the producers' write of the tile's mask, read after s_full
          if (lane == 0) mbar_arrive(&bar.s_full[b]);
          tc_fence_after();
          const int stu = __shfl_sync(kFull, st, 0);
          if (elect_one()) {
            const uint64_t bd = dk + static_cast<uint64_t>((stu * kStageBytes) >> 4);
#pragma unroll
            for (int c = 0; c < kNch; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_ts(dS, qa + 32 * c + 8 * i, bd + ((c * kChunkBytes) >> 4) + 2 * i, id_s, (c | i) != 0);
            mma_commit(&bar.s_full[b]);
            if (kFp8) mma_commit_mc(&bar.s_done[stu], 0x3);
            else mma_commit(&bar.s_done[stu]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) mma_commit(&bar.s_end);
        g0 += kQItems + ntiles;
        j0 += ntiles;
        it.done(bar, lane);
      }
      if (!ok) set_abort(bar, a.dev_error);
      if (elect_one()) mma_commit(&bar.fin[1 + b]);
      __syncwarp();
      mbar_wait(&bar.fin[1 + b], 0);
    } else if (!score && warp == 10) {
      // -------------------------------------------------------- PV MMA issuer
      const uint32_t id_o = idesc_bf16(128, 256, 0, 1);
      const uint64_t dv = smem_desc(smem_base, kChunkBytes, 1024, kSwizzle128B);
      const uint64_t dp = smem_desc(smem_base + kOffP, 16, 512, kSwizzle64B);
      // p_ok(j) stands for everything PV(j) needs: P(j) arrived and in O's
      // scale (warps 0-3), V(j) landed and fenced (warp 9).  A unit's first PV
      // overwrites O, once the previous unit's has been read.
      bool ok = true;
      int j0 = 0;
      for (int k = 0;; ++k) {
        const Unit* U = it.get(bar, ok);
        if (!U) break;
        const int ntiles = U->ntiles;
        if (k > 0) ok = wait_all(&bar.o_free, (k - 1) & 1);
        for (int j = j0; j < j0 + ntiles && ok; ++j) {
          const int slot = j % kPSlots;
          ok = wait_all(&bar.p_ok[slot], (j / kPSlots) & 1);
          if (!ok) break;
          tc_fence_after();
          const int ju = __shfl_sync(kFull, j, 0);
          if (elect_one()) {
            const int vs = ju % kRecv, os = ju % kOwn, slot = ju % kPSlots;
            const uint64_t sv[2] = {static_cast<uint64_t>((kOffRecv + vs * kHalfBytes) >> 4),
                                    static_cast<uint64_t>((kOffOwn + os * kHalfBytes) >> 4)};
            const uint64_t po = static_cast<uint64_t>((slot * kPBytes) >> 4);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int n = 0; n < 2; ++n)
                mma_ss(tbase + kColO + 256 * n, dp + po + ((32 * i) >> 4), dv + sv[n] + ((2048 * i) >> 4), id_o,
                       (j > j0 || i > 0) ? 1u : 0u);
            mma_commit_mc(&bar.p_free[slot], 0x3);
            mma_commit_mc(&bar.v_free[vs], 0x3);
            mma_commit(&bar.own_free[os]);
            mma_commit(&bar.pv_done[slot]);
            if (j == j0 + ntiles - 1) mma_commit(&bar.o_final);
          }
          __syncwarp();
        }
        if (!ok) break;
        j0 += ntiles;
        it.done(bar, lane);
      }
      if (!ok) set_abort(bar, a.dev_error);
      if (elect_one()) mma_commit(&bar.fin[0]);
      __syncwarp();
      mbar_wait(&bar.fin[0], 0);
    } else if (!score && warp == 9) {
      // ------------------------------------------------- receive-ring arrivals
      bool ok = true;
      int j = 0, g = 0;
      for (;;) {
        const Unit* U = it.get(bar, ok);
        if (!U) break;
        const int end = j + U->ntiles;
        g += kQItems;
        for (; j < end && ok; ++j, ++g) {
          const int st = g % kStages, vs = j % kRecv, os = j % kOwn;
          ok = wait_all_cluster(&bar.v_full[vs], (j / kRecv) & 1);
          if (!ok) break;
          if (kFp8 && lane == 0) {
            mbar_arrive_expect_tx(&bar.v_full[vs], kHalfBytes);
            mbar_arrive(&bar.s_done[st]);
            mbar_arrive_remote_relaxed(map_peer(smem_u32(&bar.s_done[st]), peer));
          }
          ok = wait_all(&bar.own_loaded[os], (j / kOwn) & 1);
          if (!ok) break;
          fence_proxy_async_smem();  // the own (bf16: and receive) slot's rows -> PV
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_ok[j % kPSlots]);
        }
        if (!ok) break;
        it.done(bar, lane);
      }
      if (!ok) set_abort(bar, a.dev_error);
    } else if (kFp8 && !score) {
      // ------------------------------------------------- value CTA forwarder
      // fp8: own slot j % kOwn (chunks 4-7) -> the score CTA's stage of tile j,
      // once item g - 5 has left it.  Of those items the tiles are waited for in
      // order, each once (a stage's next tile needs this copy, so its barrier
      // cannot get ahead); Q's by its own barrier.
      bool ok = true;
      int g = 0, j = 0;          // next item, next tile
      int wg = 0;                // the next item whose release is to be waited for
      uint32_t turn = 0;         // bit st: parity of stage st's tiles so far
      int gp = 0;                // the previous unit's first item
      for (int k = 0;; ++k) {
        const Unit* U = it.get(bar, ok);
        if (!U) break;
        const int ntiles = U->ntiles, g0 = g;
        g += kQItems;
        for (int n = 0; n < ntiles && ok; ++n, ++g, ++j) {
          const int st = g % kStages, os = j % kOwn;
          ok = wait_all(&bar.own_loaded[os], (j / kOwn) & 1);
          // (a unit of one tile waits too: its S, hence the next unit's Q, then
          // comes after this phase, and no phase is skipped)
          if (n == 1 || ntiles == 1) ok = ok && wait_all_cluster(&bar.q_gone, k & 1);
          // (a unit has five items at least: only this one's and the last one's)
          for (; ok && wg <= g - kStages; ++wg) {
            if (wg - (wg < g0 ? gp : g0) < kQItems) continue;
            const int ws = wg % kStages;
            ok = wait_all_cluster(&bar.s_done[ws], (turn >> ws) & 1u);
            turn ^= 1u << ws;
          }
          if (!ok) break;
          fence_proxy_async_smem();
          if (lane == 0)
            bulk_copy_to_peer(map_peer(smem_base + stage_chunk_off(st, 4), peer), smem + kOffOwn + os * kHalfBytes,
                              kHalfBytes, map_peer(smem_u32(&bar.kv_full[st]), peer));
          __syncwarp();
        }
        if (!ok) break;
        gp = g0;
        it.done(bar, lane);
      }
      if (!ok) set_abort(bar, a.dev_error);
    } else {
      // no role in this form: keep the descriptor ring moving
      bool ok = true;
      while (it.get(bar, ok)) it.done(bar, lane);
      if (!ok) set_abort(bar, a.dev_error);
    }
  } else {
    take_regs<Regs<kFp8>::last>();
    // no role in this form: keep the descriptor ring moving
    bool ok = true;
    while (it.get(bar, ok)) it.done(bar, lane);
    if (!ok) set_abort(bar, a.dev_error);
  }

  // ------------------------------------------------------------- teardown
  // the grid that consumes O_dst / lse_dst may start launching now; it waits
  // for this grid's completion before reading them
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  const bool failed = aborted(bar);
  cluster_sync();  // the peer has issued everything it will send here
  if (failed && !score && threadIdx.x == 0) {
    // failed work may have left some of the score CTA's copies in flight into
    // the P slots: give each slot's next phase a short bounded wait
    for (int b = 0; b < kPSlots; ++b) {
      const int received = pdone > b ? (pdone - 1 - b) / kPSlots + 1 : 0;
      mbar_wait_cluster(&bar.p_full[b], received & 1, 1u << 16);
    }
  }
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// Order of the units, longest first: one CTA; keys (a quarter octave of the
// tile count) count into buckets, then a stable scatter in chunks of 1024
// units (rank in the warp by __match_any_sync, warps before this one by their
// bucket counts), so that equal units keep their places and a request's
// groups stay together.
constexpr int kKeys = 128;
__global__ void __launch_bounds__(1024) select_order_kernel(DecodeArgs a, int32_t units, int32_t* order) {
  __shared__ int32_t cnt[kKeys], off[kKeys];
  __shared__ int32_t wcnt[32][kKeys];
  const int t = threadIdx.x, w = t >> 5, lane = t & 31;
  auto key_of = [&](int32_t u) -> int {
    const SelCoords k = sel_coords(a, u);
    const SelUnit U = sel_unit(a, k.b, k.c);
    const int32_t n = U.live ? sel_span<true>(a, U.R, a.d0 + k.dd).nv : 0;
    const int32_t lo = k.s * a.plan.chunk, hi = min(n, lo + a.plan.chunk);
    if (lo >= hi) return 0;
    const uint32_t tiles4 = static_cast<uint32_t>(hi - lo + kTile - 1) / kTile * 4;  // >= 4
    const int e = 31 - __clz(tiles4);
    return 4 * (e - 2) + static_cast<int>((tiles4 >> (e - 2)) & 3u) + 1;  // < 128
  };
  // The decode's blocks may start on the other SMs: they set up and wait.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (t < kKeys) cnt[t] = 0;
  const int mine = t < units ? key_of(t) : -1;  // (the first 1,024 keys are kept)
  __syncthreads();
  if (mine >= 0) atomicAdd(&cnt[mine], 1);
  for (int32_t u = t + 1024; u < units; u += 1024) atomicAdd(&cnt[key_of(u)], 1);
  __syncthreads();
  if (w == 0) {  // off[k]: the units of larger keys; a lane takes 4 keys, the largest first
    int c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += c[i] = cnt[kKeys - 1 - (4 * lane + i)];
    int acc = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(kFull, acc, d);
      if (lane >= d) acc += x;
    }
    acc -= sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      off[kKeys - 1 - (4 * lane + i)] = acc;
      acc += c[i];
    }
  }
  for (int32_t base = 0; base < units; base += 1024) {
    for (int i = t; i < 32 * kKeys; i += 1024) (&wcnt[0][0])[i] = 0;
    __syncthreads();
    const int32_t u = base + t;
    const int k = base == 0 ? mine : u < units ? key_of(u) : -1;
    const unsigned same = __match_any_sync(kFull, k);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (k >= 0 && rank == 0) wcnt[w][k] = __popc(same);
    __syncthreads();
    if (k >= 0) {
      int32_t pos = off[k] + rank;
      for (int v = 0; v < w; ++v) pos += wcnt[v][k];
      order[pos] = u;
    }
    if (base + 1024 < units) {
      __syncthreads();
      if (t < kKeys) {
        int32_t add = 0;
        for (int v = 0; v < 32; ++v) add += wcnt[v][t];
        off[t] += add;
      }
      __syncthreads();
    }
  }
}

cudaLaunchConfig_t launch_config(int clusters, bool ordered, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // (set up alongside the kernel that orders the units)
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ordered ? 2 : 1;
  return cfg;
}

// Per-device one-time set-up: the shared-memory opt-in and the number of
// clusters that fit on the device at once.
constexpr int kMaxDevices = 64;
std::mutex g_setup_mu;
int g_clusters[kMaxDevices] = {};  // 0: not yet set up

}  // namespace

int decode_select_clusters() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return 0; }
  if (dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(g_setup_mu);
  if (g_clusters[dev] > 0) return g_clusters[dev];
  void (*const kernels[])(DecodeArgs, int32_t) = {decode_select_kernel<false>, decode_select_kernel<true>};
  for (auto k : kernels)
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = launch_config(1, false, nullptr, attr);
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, decode_select_kernel<false>, &cfg) != cudaSuccess || clusters <= 0) {
    cudaGetLastError();
    return 0;
  }
  g_clusters[dev] = clusters;
  return clusters;
}

bool decode_select_supported(int32_t H, int64_t cache_rows, int64_t period) {
  return H <= 128 && cache_rows <= 0x7fffffffLL && period <= 0x7fffffffLL;
}

cudaError_t launch_select_order(const DecodeArgs& a, int32_t units, int32_t* order, cudaStream_t st) {
  if (units <= 0) return cudaSuccess;
  select_order_kernel<<<1, 1024, 0, st>>>(a, units, order);
  return cudaGetLastError();
}

cudaError_t launch_decode_select(const DecodeArgs& a, int32_t units, cudaStream_t st) {
  const int resident = decode_select_clusters();
  if (resident <= 0) return cudaErrorInvalidDevice;
  const int32_t parts = 1 << a.sel.parts_log2;
  if (units <= 0 || a.plan.chunk % kTile != 0 || parts > (a.o_bf16 ? 4 : 8)) return cudaErrorInvalidValue;
  if (parts > 1) {
    units += (parts - 1) * a.B * a.sel.chunks * a.Dn * a.plan.splits;
    if (units > resident || a.unit_order) return cudaErrorInvalidValue;
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = launch_config(units < resident ? units : resident, a.unit_order != nullptr, st, attr);
  return a.kv_fp8 ? cudaLaunchKernelEx(&cfg, decode_select_kernel<true>, a, units)
                  : cudaLaunchKernelEx(&cfg, decode_select_kernel<false>, a, units);
}

}  // namespace dcp
