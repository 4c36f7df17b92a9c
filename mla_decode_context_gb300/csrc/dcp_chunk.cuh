// Shared by the kernels of chunk attention: the up projection of the cached
// latents to keys and values (dcp_chunk_expand.cu) and the attention over them
// (dcp_chunk_attention.cu).
//
// Keys and values pass between the two as images of shared-memory tiles: what
// one writes with a bulk store of 16 KB, the other loads with a bulk copy, and
// no tensor map, address arithmetic or padding is left.  An image is 128 tokens
// (of one request, from a multiple of 128) x 64 dims of 16 bits: 128-byte rows,
// whose 16-byte units are permuted by the row's low three bits (the 128-byte
// swizzle of the MMAs' operands).
//
// Keys, values, queries and softmax weights are f16 (rope dims: bf16, as they
// come): 11 significant bits to bf16's 8, at the same rate.  A key's rounding
// shifts its score by ~2e-4 (bf16: ~1.5e-3), and the log-sum-exp by that over the
// root of the number of tokens that carry it.  In requests of up to kFineLen tokens,
// where those are few more often, keys are f16 pairs, the value and its rounding's
// remainder, at 1.4 times the MMAs: 22 bits.  (A row of a longer request that sees
// little but one token has all of that token's 2e-4; its weights come too late to
// choose by.)
#pragma once

#include "dcp_kernels.h"
#include "dcp_sm100.cuh"

namespace dcp {

constexpr int kChunkTile = 128;                  // tokens of an image
constexpr int kChunkRows = 256;                  // query rows of a unit: two MMA tiles of 128
constexpr int kImage = kChunkTile * 128;         // bytes
constexpr int kFineLen = 1024;                   // requests up to this length have key remainders
constexpr int kFineTiles = kFineLen / kChunkTile;
constexpr int kNope = 128, kVDim = 128;          // a head's key dims from the latent, its value dims
constexpr int kUp = kNope + kVDim;               // rows of the up projection's weight per head
constexpr int kWeightStage = kUp * 128;          // packed weight: 256 rows x 64 latent dims

// Byte offset of 16-byte unit u of row r in an image (of any number of rows).
__host__ __device__ constexpr uint32_t image_unit(uint32_t r, uint32_t u) { return r * 128u + ((u ^ (r & 7u)) << 4); }

// A unit's key tiles are cut into pieces where there are too few units for the
// SMs or some are much longer than others: at least kMinPiece tiles each,
// kMaxPieces a unit, about one piece an SM if all units were cut (two: 12 mixed
// requests at 16 heads 751 us instead of 742, 3 x 700 rows at 64 heads 781 instead
// of 777; six: 818 and 917).  A second kernel joins their outputs.
constexpr int kMinPiece = 6, kMaxPieces = 32;
constexpr int kSlotBytes = kChunkRows * (kVDim + 1) * 4;  // a piece's output and log-sum-exps, fp32

struct __align__(16) Piece {
  int32_t b, block;       // request (-1: rows of no request), block of 256 rows
  int32_t q0, q1, seq;    // the request's rows and length
  int32_t image;          // its image of key tile j0
  int32_t j0, j1;         // key tiles
  int32_t pieces, index;  // of the unit, and which of them this is
  int32_t slot;           // the unit's first slot (of a head's)
  int32_t seg0, seg;      // pieces of similar length: the first, and how many
  int32_t lo;             // its key remainders of key tile j0; -1: none
  int32_t unused[2];
};
static_assert(sizeof(Piece) == 64, "four 16-byte units");

struct ChunkArgs {
  const __nv_bfloat16* q;   // [T, H, 192]
  int64_t q_stride_tok, q_stride_head;
  const void* kv;
  const float* kv_scale;    // FP8 cache, else nullptr
  int32_t num_blocks, block_size;
  const int32_t* block_table;
  int32_t bt_width;
  int64_t bt_stride;
  int32_t local_tables;
  int64_t bt_shard_stride;
  int32_t D, I;
  FastDiv div_I, div_D, div_bs;
  const int32_t* seq_lens;
  const int32_t* qsl;
  int32_t B, T, H;
  float scale_log2;         // |scale| log2 e
  uint32_t q_sign;          // 0x80008000 for a negative scale
  const void* weight;       // packed: [H][8][256 rows x 128 bytes]
  void* out;                // [T, H, 128]
  int32_t out_f32;
  float* lse;               // [T, H]
  int32_t* dev_error;
  // workspace
  int32_t tiles;            // most images per head (tokens / 128 + B)
  int32_t* tile_start;      // [B + 1]: first image of a request
  int32_t* block_start;     // [B + 1]: first unit of a request
  int32_t* lo_start;        // [B]: first tile of a request's key remainders; -1: none
  int32_t lo_tiles;         // most tiles of key remainders per head
  unsigned char* rope;      // [tiles] images of the rope dims
  uint4* valid;             // [tiles]: tokens that exist
  unsigned char* keys;      // [heads of a pass][tiles][2 images]
  unsigned char* values;    // the same
  unsigned char* lo_keys;   // [heads of a pass][lo_tiles][2 images]
  uint4* bad;               // [heads of a pass][tiles]: tokens whose value is not finite (their rows are zeros)
  int32_t h0, heads;        // the heads of this pass
  int32_t sms;
  int32_t max_pieces;       // records (T / 256 + B + 2, and what the cuts add)
  Piece* pieces;            // in launch order: long ones first
  int32_t* num_pieces;
  int32_t slots;            // slots of a head of a pass; 0: no cuts
  unsigned char* partial;   // [heads of a pass][slots][kSlotBytes]
};

// The last b with start[b] <= n (start[0] <= n < start[count] given), by the
// whole warp, 32 ways at a time.
__device__ __forceinline__ int32_t find_range(const int32_t* start, int32_t count, int32_t n) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, hi = count;
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) / 32;
    const int64_t at = static_cast<int64_t>(lo) + static_cast<int64_t>(lane + 1) * step;
    const bool le = at < hi && start[at] <= n;
    const int32_t k = __popc(__ballot_sync(0xffffffffu, le));
    const int64_t next = static_cast<int64_t>(lo) + static_cast<int64_t>(k + 1) * step;
    lo += k * step;
    hi = next < hi ? static_cast<int32_t>(next) : hi;
  }
  return lo;
}

// Pieces that cuts may add to the units of `heads` heads.
DCP_HD int64_t added_pieces(int sms, int heads) { return sms / heads + 1; }

cudaError_t launch_pack_kv_b(const void* w, int32_t H, void* packed, cudaStream_t st);
// One pass over heads [h0, h0 + heads); the first also writes what the heads
// share.
cudaError_t launch_chunk_plan(const ChunkArgs& a, cudaStream_t st);
cudaError_t launch_chunk_expand(const ChunkArgs& a, cudaStream_t st);
cudaError_t launch_chunk_attention(const ChunkArgs& a, cudaStream_t st);

}  // namespace dcp
