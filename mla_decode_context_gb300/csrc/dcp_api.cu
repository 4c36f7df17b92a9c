// C ABI of the DCP MLA hot path: host-side validation, the split-KV plan and
// kernel launches.  No allocation, no synchronisation, no global state.
#include "dcp_chunk.cuh"
#include "dcp_kernels.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>

using dcp::DecodeArgs;
using dcp::SplitPlan;

namespace dcp {

namespace {
constexpr int kTargetCtasPerUnit = 2;  // CTAs the decode spends on one (row, shard, split)
constexpr int32_t kMinSplitTokens = 256;
constexpr int32_t kSplitRound = 32;  // split chunks in whole 32-token tiles
constexpr int kMaxSplits = 32;

// CTAs one wave of the decode can hold: the tensor-core kernel's resident
// cluster count x 2 (one CTA per SM), else the SM count, else GB300's 152.
int current_sm_count() {
  const int tc = decode_tc_resident_ctas();
  if (tc > 0) return tc;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    cudaGetLastError();  // clear: no device is not an error for sizing
    return 152;          // GB300
  }
  return sms;
}
}  // namespace

// Most splits a (row, shard) pair with up to `lmax` local tokens may use:
// enough (row, shard, split) units to give every SM work when there are few
// rows (long-context B=1 decode), never splits shorter than kMinSplitTokens.
static int64_t split_cap(int32_t T, int32_t D, int64_t lmax, int sm_count) {
  const int64_t units = static_cast<int64_t>(T) * D * kTargetCtasPerUnit;
  int64_t want = sm_count / units;  // whole waves only
  const int64_t cap_len = (lmax + kMinSplitTokens - 1) / kMinSplitTokens;
  if (want > cap_len) want = cap_len;
  if (want > kMaxSplits) want = kMaxSplits;
  return want < 1 ? 1 : want;
}

// `units` units of at most `lmax` tokens, cut into splits of whole tiles.
static SplitPlan cut(int64_t lmax, int64_t want) {
  SplitPlan p{1, kSplitRound};
  int64_t chunk = (lmax + want - 1) / want;
  chunk = (chunk + kSplitRound - 1) / kSplitRound * kSplitRound;
  p.chunk = static_cast<int32_t>(chunk);
  p.splits = static_cast<int32_t>((lmax + chunk - 1) / chunk);  // <= want
  if (p.splits < 1) p.splits = 1;
  return p;
}
// Clusters that share a unit's output: each computes the unit and writes its
// own columns of it (`most` of them at most).  A cluster writes through one SM,
// at 26-30 bytes per clock (7.4 us for 128 fp32 rows, as long as the rest of a
// short unit), so clusters that would be idle take a part of that.
static int32_t select_parts(int64_t units, int64_t others, int32_t most, int clusters) {
  int32_t parts = 1;
  while (parts < most && 2 * parts * units + others <= clusters) parts *= 2;
  return parts;
}
constexpr int32_t kMostParts = 8, kMostPartsBf16 = 4;  // (128-byte blocks of a warp's half row)

// Splits of the windowed and tree decodes: `units` units of at most `lmax`
// tokens (and `others` for the rows of no request) on `clusters` persistent
// clusters.  A 32-token tile takes kTileUs, a cluster's further unit kUnitUs
// (its last output store and first tiles), the last output store kStoreUs over
// the clusters that share it (twice that for fp32 partials), the merge kMergeUs
// and kPartialUs for each partial written and read; lengths are only known to
// be at most lmax (kFill of it on average).  While all units run at once, the
// time is a unit's; beyond that the work per cluster and half a unit at the
// end.  So few long units are cut until they fill the GPU (one request on a
// 1,028-token window: 31.9 us whole, 21.6 in four), ragged ones until the last
// one no longer shows (trees of 16 requests of up to 16,384 tokens: 271 us
// whole, 163 in two, 200 in eight), and many short ones not at all (64 requests
// x 8 shards x 512 tokens: 103 us, 220 in two).
constexpr double kTileUs = 0.5, kUnitUs = 6.0, kStoreUs = 3.7, kMergeUs = 4.0, kPartialUs = 0.1, kFill = 0.85;
constexpr int64_t kMinSelectSplit = 128;
static int64_t select_splits(int64_t units, int64_t others, int64_t lmax, int clusters) {
  const int64_t most = std::min<int64_t>(kMaxSplits, (lmax + kMinSelectSplit - 1) / kMinSelectSplit);
  int64_t best = 1;
  double least = 0;
  for (int64_t s = 1; s <= most; ++s) {
    const double n = static_cast<double>(units) * s;
    const double unit = kTileUs * ((lmax + s * kSplitRound - 1) / (s * kSplitRound));
    double t = n <= clusters ? unit : n / clusters * (kFill * unit + kUnitUs) + 0.5 * unit;
    t += (s > 1 ? 2 : 1) * kStoreUs / select_parts(units * s, others * s, s > 1 ? kMostParts : kMostPartsBf16, clusters);
    if (s > 1) t += kMergeUs + kPartialUs * n;
    if (s == 1 || t < least) {
      best = s;
      least = t;
    }
  }
  return best;
}

// Split-KV plan: pure function of its arguments (and the SM count).
SplitPlan plan_splits(int32_t T, int32_t D, int32_t I, int32_t d0, int32_t Dn, int32_t max_seq_len, int sm_count) {
  // the first computed shard is the largest of them
  const int32_t lmax = local_len(max_seq_len < 0 ? 0 : max_seq_len, d0, D, I);
  if (lmax <= 0) return SplitPlan{1, kSplitRound};
  return cut(lmax, split_cap(T, Dn, lmax, sm_count));
}

// Tail of the workspace for the units' launch order (one int32 per unit).
size_t order_workspace_bytes(const SplitPlan& p, int32_t T, int32_t D) {
  const size_t units = static_cast<size_t>(p.splits < 1 ? 1 : p.splits) * D * T;
  return (units * sizeof(int32_t) + 255) / 256 * 256;
}

size_t split_workspace_bytes(const SplitPlan& p, int32_t T, int32_t H, int32_t D) {
  if (p.splits <= 1) return 0;
  const size_t pairs = static_cast<size_t>(p.splits) * D * T * H;
  size_t bytes = pairs * kLatent * sizeof(float);
  bytes = (bytes + 255) / 256 * 256;
  bytes += pairs * sizeof(float);
  return (bytes + 255) / 256 * 256;
}

}  // namespace dcp

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

namespace {
// What one dcp_mla_decode_partial call with these sizes does on the current
// device: its split plan, the workspace the split partials need, and which
// kernels it launches.
struct DecodeLaunch {
  dcp::SplitPlan plan;
  size_t need;       // split partials (required when plan.splits > 1)
  size_t obytes;     // launch order of the units (optional tail)
  bool simt;         // CUDA-core kernel instead of the tensor-core one
  bool use_order;    // units start longest first (order kernel launched)
  int64_t units;     // windowed and tree decodes: units of the launch,
  int32_t parts;     // and clusters that share one's output
};

DecodeLaunch decode_launch(int32_t T, int32_t H, int32_t D, int32_t interleave, int32_t d0, int32_t Dn,
                           int32_t max_seq_len, bool have_workspace, size_t workspace_bytes, bool kv_fp8 = false) {
  DecodeLaunch L{};
  const int sms = dcp::current_sm_count();
  L.plan = dcp::plan_splits(T, D, interleave, d0, Dn, max_seq_len, sms);
  L.need = dcp::split_workspace_bytes(L.plan, T, H, Dn);
  L.obytes = dcp::order_workspace_bytes(L.plan, T, Dn);
  dcp::DecodeArgs a{};
  a.H = H;
  a.plan = L.plan;
  a.kv_fp8 = kv_fp8 ? 1 : 0;
  const char* force = std::getenv("DCP_FORCE_SIMT");  // 1: the CUDA-core reference kernel (A/B checks)
  L.simt = (force && force[0] == '1') || !dcp::decode_tc_supported(a);
  const int64_t units = static_cast<int64_t>(T) * Dn * L.plan.splits;
  const int resident = dcp::decode_tc_resident_ctas();  // 0: no device to size against
  L.use_order = !L.simt && resident > 0 && units > resident / 2 && have_workspace &&
                workspace_bytes >= L.need + L.obytes;
  return L;
}

// Clusters of the windowed and tree decodes that run at once (without a device
// to ask: a GB300's).
int select_clusters() {
  const int n = dcp::decode_select_clusters();
  return n > 0 ? n : 72;
}

constexpr int64_t kMostUnits = 0x3fffffff;  // of one launch

size_t order_bytes(int64_t units) { return (static_cast<size_t>(units) * sizeof(int32_t) + 255) / 256 * 256; }

// The windowed and tree decodes.  A unit is a group of rows of one request
// (as many as fit the tensor-core kernel's 128 lanes), one shard and one split
// of what they may see; `lmax` bounds that per shard.
int32_t select_group(int32_t H, int32_t max_q_len) {
  const int32_t fit = H <= 128 ? 128 / H : 1;
  return std::max(1, std::min(std::min(fit, dcp::kMaxGroup), max_q_len));
}

// Most of n consecutive positions that one shard owns.
int64_t most_owned(int64_t n, int32_t D, int32_t I) {
  const int64_t period = static_cast<int64_t>(D) * I;
  return n / period * I + std::min<int64_t>(n % period, I);
}

// Most tokens that a request's rows see together, on any number of shards.
int64_t select_visible(int32_t max_seq_len, int32_t max_q_len, int32_t window, int32_t sinks) {
  return window > 0 ? std::min<int64_t>(max_seq_len, static_cast<int64_t>(window) + sinks + max_q_len) : max_seq_len;
}

DecodeLaunch select_launch(int32_t B, int32_t T, int32_t H, int32_t D, int32_t interleave, int32_t d0, int32_t Dn,
                           int32_t max_seq_len, int32_t max_q_len, int64_t cache_rows, const dcp::SelectArgs& sel,
                           bool o_bf16, bool have_workspace, size_t workspace_bytes) {
  DecodeLaunch L{};
  int64_t lmax = dcp::local_len(max_seq_len, d0, D, interleave);
  if (sel.window > 0)  // the sinks, and a window for each row of the request
    lmax = std::min(lmax, most_owned(sel.sinks, D, interleave) +
                              most_owned(static_cast<int64_t>(sel.window) + max_q_len, D, interleave));
  const int64_t units = static_cast<int64_t>(B) * sel.chunks * Dn, others = static_cast<int64_t>(sel.chunks) * Dn;
  const int64_t visible = select_visible(max_seq_len, max_q_len, sel.window, sel.sinks);
  const int clusters = select_clusters();
  L.plan = dcp::SplitPlan{1, dcp::kSplitRound};
  if (lmax > 0)  // (never more splits than the workspace's size allows for)
    L.plan = dcp::cut(lmax, std::min(dcp::select_splits(units, others, lmax, clusters),
                                     dcp::select_splits(units, others, visible, clusters)));
  L.need = dcp::split_workspace_bytes(L.plan, T, H, Dn);
  L.units = (units + others) * L.plan.splits;  // (others: the rows of no request)
  L.parts = dcp::select_parts(units * L.plan.splits, others * L.plan.splits,
                              o_bf16 && L.plan.splits == 1 ? dcp::kMostPartsBf16 : dcp::kMostParts, clusters);
  L.obytes = order_bytes(L.units);
  const char* force = std::getenv("DCP_FORCE_SIMT");
  L.simt = (force && force[0] == '1') ||
           !dcp::decode_select_supported(H, cache_rows, static_cast<int64_t>(D) * interleave);
  L.use_order = !L.simt && L.units > select_clusters() && have_workspace && workspace_bytes >= L.need + L.obytes;
  return L;
}
}  // namespace

extern "C" {

const char* dcp_status_str(dcp_status_t s) {
  switch (s) {
    case DCP_OK: return "DCP_OK";
    case DCP_ERR_INVALID_ARG: return "DCP_ERR_INVALID_ARG";
    case DCP_ERR_UNSUPPORTED_DTYPE: return "DCP_ERR_UNSUPPORTED_DTYPE";
    case DCP_ERR_MISALIGNED: return "DCP_ERR_MISALIGNED";
    case DCP_ERR_TABLE_TOO_NARROW: return "DCP_ERR_TABLE_TOO_NARROW";
    case DCP_ERR_WORKSPACE_TOO_SMALL: return "DCP_ERR_WORKSPACE_TOO_SMALL";
    case DCP_ERR_CUDA: return "DCP_ERR_CUDA";
    case DCP_ERR_TIMEOUT: return "DCP_ERR_TIMEOUT";
  }
  return "DCP_ERR_UNKNOWN";
}

int dcp_version(void) { return 1; }

int32_t dcp_shard_of(int64_t pos, int32_t D, int32_t interleave) {
  if (D < 1 || interleave < 1 || pos < 0) return -1;
  return dcp::shard_of(pos, D, interleave);
}

int32_t dcp_local_len(int32_t L, int32_t d, int32_t D, int32_t interleave) {
  if (L < 0 || D < 1 || interleave < 1 || d < 0 || d >= D) return -1;
  return dcp::local_len(L, d, D, interleave);
}

size_t dcp_decode_workspace_size(int32_t B, int32_t T, int32_t H, int32_t D, int32_t max_seq_len,
                                 int32_t max_q_len) {
  if (B < 0 || T < 0 || H < 1 || D < 1 || D > DCP_MAX_SHARDS || max_seq_len < 0 || max_q_len < 0)
    return static_cast<size_t>(-1);
  if (B == 0 || T == 0) return 0;
  // Upper bound over every interleave: a shard never owns more than
  // max_seq_len tokens, and the split count never exceeds split_cap(lmax).
  const int sms = dcp::current_sm_count();
  dcp::SplitPlan p{static_cast<int32_t>(dcp::split_cap(T, D, max_seq_len, sms)), 0};
  return dcp::split_workspace_bytes(p, T, H, D) + dcp::order_workspace_bytes(p, T, D);
}

}  // extern "C"

static dcp_status_t decode_partial_impl(const void* q, int64_t q_stride_tok, const void* kv_cache,
                                        dcp_kv_dtype_t kv_dtype, const float* kv_scale,
                                        int32_t num_blocks, int32_t block_size, const int32_t* block_table,
                                        int32_t bt_width, int64_t bt_stride, bool local, int64_t bt_shard_stride,
                                        int32_t d0, int32_t Dn,
                                        const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B,
                                        int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len, int32_t D,
                                        int32_t interleave, float scale, void* O_part, dcp_dtype_t o_dtype,
                                        float* lse_part, void* workspace, size_t workspace_bytes, int32_t* dev_error,
                                        void* stream, const dcp::SelectArgs* select = nullptr) {
  if (B < 0 || T < 0 || H < 1 || H > 1024 || D < 1 || D > DCP_MAX_SHARDS || interleave < 1 ||
      max_seq_len < 0 || max_q_len < 1 || !std::isfinite(scale))
    return DCP_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return DCP_OK;
  if (!q || !kv_cache || !block_table || !seq_lens || !query_start_loc || !O_part || !lse_part)
    return DCP_ERR_INVALID_ARG;
  if ((kv_dtype != DCP_KV_BF16 && kv_dtype != DCP_KV_FP8_E4M3) || (o_dtype != DCP_DTYPE_F32 && o_dtype != DCP_DTYPE_BF16))
    return DCP_ERR_UNSUPPORTED_DTYPE;
  if (kv_dtype == DCP_KV_FP8_E4M3 && !kv_scale) return DCP_ERR_INVALID_ARG;
  if (num_blocks < 1 || block_size < 1 || bt_width < 1 || bt_stride < bt_width ||
      q_stride_tok < static_cast<int64_t>(H) * DCP_KV_DIM)
    return DCP_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(O_part) || (q_stride_tok % 8) != 0)
    return DCP_ERR_MISALIGNED;
  if (d0 < 0 || Dn < 1 || d0 + Dn > D) return DCP_ERR_INVALID_ARG;
  if (local && Dn > 1 && bt_shard_stride < static_cast<int64_t>(B - 1) * bt_stride + bt_width)
    return DCP_ERR_INVALID_ARG;  // shards' tables would overlap
  // a table row covers the longest sequence (global layout) or the largest
  // computed local shard, the first (per-shard layout)
  const int64_t covered = local ? dcp::local_len(max_seq_len, d0, D, interleave) : max_seq_len;
  if ((covered + block_size - 1) / block_size > bt_width) return DCP_ERR_TABLE_TOO_NARROW;

  dcp::SelectArgs sel{};
  if (select) {
    sel = *select;
    sel.on = 1;
    sel.group = select_group(H, max_q_len);
    sel.chunks = (max_q_len - 1) / sel.group + 1;
  }
  // (a workspace that holds no partials may be misaligned; the launch order,
  // int32 words, goes into it at any multiple of 4)
  const bool usable = workspace != nullptr && reinterpret_cast<uintptr_t>(workspace) % alignof(int32_t) == 0;
  const DecodeLaunch launch =
      select ? select_launch(B, T, H, D, interleave, d0, Dn, max_seq_len, max_q_len,
                             static_cast<int64_t>(num_blocks) * block_size, sel, o_dtype == DCP_DTYPE_BF16,
                             usable, workspace_bytes)
             : decode_launch(T, H, D, interleave, d0, Dn, max_seq_len, usable, workspace_bytes,
                             kv_dtype == DCP_KV_FP8_E4M3);
  const dcp::SplitPlan plan = launch.plan;
  const size_t need = launch.need;
  if (select && launch.units > kMostUnits) return DCP_ERR_INVALID_ARG;  // (max_q_len far beyond any step's rows)
  if (need > 0 && (workspace_bytes < need || !workspace)) return DCP_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !aligned16(workspace)) return DCP_ERR_MISALIGNED;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DecodeArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride_tok = q_stride_tok;
  a.kv = kv_cache;
  a.kv_fp8 = kv_dtype == DCP_KV_FP8_E4M3 ? 1 : 0;
  a.kv_scale = kv_scale;
  // (split partials are in the output's dtype; those of the windowed and tree
  // decodes are fp32, so that a bf16 output is rounded once)
  a.o_bf16 = o_dtype == DCP_DTYPE_BF16 && !(select && launch.plan.splits > 1) ? 1 : 0;
  if (select) {
    sel.div_chunks = dcp::make_fastdiv(sel.chunks);
    sel.div_splits = dcp::make_fastdiv(launch.plan.splits);
    sel.div_Dn = dcp::make_fastdiv(Dn);
    sel.div_period = dcp::make_fastdiv(static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(D) * interleave, 0x7fffffff)));
    sel.div_H = dcp::make_fastdiv(H);
  }
  while (select && 1 << sel.parts_log2 < launch.parts) ++sel.parts_log2;
  a.sel = sel;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.block_table = block_table;
  a.bt_width = bt_width;
  a.bt_stride = bt_stride;
  a.local_tables = local ? 1 : 0;
  a.bt_shard_stride = local ? bt_shard_stride : 0;
  a.seq_lens = seq_lens;
  a.qsl = query_start_loc;
  a.B = B; a.T = T; a.H = H;
  a.max_seq_len = max_seq_len; a.max_q_len = max_q_len;
  // a request's verification rows side by side (when the rows split evenly
  // into groups of max_q_len: a permutation of the units either way)
  a.row_group = (max_q_len >= 2 && max_q_len <= 8 && T % max_q_len == 0) ? max_q_len : 1;
  a.D = D; a.I = interleave;
  a.div_I = dcp::make_fastdiv(interleave);
  a.div_bs = dcp::make_fastdiv(block_size);
  a.d0 = d0; a.Dn = Dn;
  a.scale = scale;
  a.plan = plan;
  a.dev_error = dev_error;
  const char* stall = std::getenv("DCP_TEST_STALL_WAIT");  // failure-path test hook (see DecodeArgs)
  a.stall_test = stall && stall[0] == '1';
  void* ws_O = nullptr;
  float* ws_lse = nullptr;
  if (plan.splits > 1) {
    const size_t pairs = static_cast<size_t>(plan.splits) * Dn * T * H;
    ws_O = workspace;  // split partials in the output's dtype (sized for fp32)
    ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      (pairs * DCP_LATENT_DIM * sizeof(float) + 255) / 256 * 256);
    a.O_dst = ws_O;
    a.lse_dst = ws_lse;
  } else {
    a.O_dst = O_part;
    a.lse_dst = lse_part;
  }
  const bool simt = launch.simt;
  a.unit_order = nullptr;
  cudaError_t e = cudaSuccess;
  if (launch.use_order) {
    // more units than clusters that fit at once: start the long ones first
    // (the order lives in the workspace past the split partials; a workspace
    // without room for it keeps index order)
    const int64_t units = select ? launch.units : static_cast<int64_t>(T) * Dn * plan.splits;
    int32_t* order = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + need);
    e = select ? dcp::launch_select_order(a, static_cast<int32_t>(units), order, st)
               : dcp::launch_unit_order(a, static_cast<int32_t>(units), order, st);
    if (e != cudaSuccess) return DCP_ERR_CUDA;
    a.unit_order = order;
  }
  e = simt ? dcp::launch_decode_simt(a, st)
           : (select ? dcp::launch_decode_select(a, static_cast<int32_t>(launch.units), st) : dcp::launch_decode_tc(a, st));
  if (e != cudaSuccess) return DCP_ERR_CUDA;
  if (plan.splits > 1) {
    const int64_t pairs = static_cast<int64_t>(Dn) * T * H;
    e = dcp::launch_lse_merge(ws_O, a.o_bf16 != 0, ws_lse, pairs * DCP_LATENT_DIM, pairs, plan.splits, pairs, H,
                              nullptr, nullptr, 0, /*row_mask=*/false, O_part, o_dtype == DCP_DTYPE_BF16, lse_part, st);
    if (e != cudaSuccess) return DCP_ERR_CUDA;
  }
  return DCP_OK;
}


extern "C" {

dcp_status_t dcp_mla_decode_partial(const void* q, int64_t q_stride_tok, const void* kv_cache,
                                    int32_t num_blocks, int32_t block_size, const int32_t* block_table,
                                    int32_t bt_width, int64_t bt_stride, const int32_t* seq_lens,
                                    const int32_t* query_start_loc, int32_t B, int32_t T, int32_t H,
                                    int32_t max_seq_len, int32_t max_q_len, int32_t D, int32_t interleave,
                                    float scale, float* O_part, float* lse_part, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_error, void* stream) {
  return decode_partial_impl(q, q_stride_tok, kv_cache, DCP_KV_BF16, nullptr, num_blocks, block_size, block_table,
                             bt_width, bt_stride, false, 0, 0, D, seq_lens, query_start_loc, B, T, H, max_seq_len,
                             max_q_len, D, interleave, scale, O_part, DCP_DTYPE_F32, lse_part, workspace,
                             workspace_bytes, dev_error, stream);
}

dcp_status_t dcp_mla_decode_partial_local(const void* q, int64_t q_stride_tok, const void* kv_cache,
                                          int32_t num_blocks, int32_t block_size, const int32_t* block_table,
                                          int32_t bt_width, int64_t bt_stride, int64_t bt_shard_stride,
                                          const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B,
                                          int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len, int32_t D,
                                          int32_t interleave, int32_t shard_begin, int32_t shard_count,
                                          float scale, float* O_part, float* lse_part, void* workspace,
                                          size_t workspace_bytes, int32_t* dev_error, void* stream) {
  return decode_partial_impl(q, q_stride_tok, kv_cache, DCP_KV_BF16, nullptr, num_blocks, block_size, block_table,
                             bt_width, bt_stride, true, bt_shard_stride, shard_begin, shard_count, seq_lens,
                             query_start_loc, B, T, H, max_seq_len, max_q_len, D, interleave, scale, O_part,
                             DCP_DTYPE_F32, lse_part, workspace, workspace_bytes, dev_error, stream);
}

dcp_status_t dcp_mla_decode_partial_v2(const void* q, int64_t q_stride_tok, const void* kv_cache,
                                       dcp_kv_dtype_t kv_dtype, const float* kv_scale, int32_t num_blocks,
                                       int32_t block_size, const int32_t* block_table, int32_t bt_width,
                                       int64_t bt_stride, int32_t per_shard_tables, int64_t bt_shard_stride,
                                       int32_t shard_begin, int32_t shard_count, const int32_t* seq_lens,
                                       const int32_t* query_start_loc, int32_t B, int32_t T, int32_t H,
                                       int32_t max_seq_len, int32_t max_q_len, int32_t D, int32_t interleave,
                                       float scale, void* O_part, dcp_dtype_t o_dtype, float* lse_part,
                                       void* workspace, size_t workspace_bytes, int32_t* dev_error, void* stream) {
  return decode_partial_impl(q, q_stride_tok, kv_cache, kv_dtype, kv_scale, num_blocks, block_size, block_table,
                             bt_width, bt_stride, per_shard_tables != 0, bt_shard_stride, shard_begin, shard_count,
                             seq_lens, query_start_loc, B, T, H, max_seq_len, max_q_len, D, interleave, scale, O_part,
                             o_dtype, lse_part, workspace, workspace_bytes, dev_error, stream);
}

static dcp_status_t select_impl(const dcp::SelectArgs& sel, const void* q, int64_t q_stride_tok, const void* kv_cache,
                                dcp_kv_dtype_t kv_dtype, const float* kv_scale, int32_t num_blocks,
                                int32_t block_size, const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
                                int32_t per_shard_tables, int64_t bt_shard_stride, int32_t shard_begin,
                                int32_t shard_count, const int32_t* seq_lens, const int32_t* query_start_loc,
                                int32_t B, int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len, int32_t D,
                                int32_t interleave, float scale, void* O_part, dcp_dtype_t o_dtype, float* lse_part,
                                void* workspace, size_t workspace_bytes, int32_t* dev_error, void* stream) {
  if (sel.window < 0 || sel.sinks < 0) return DCP_ERR_INVALID_ARG;
  return decode_partial_impl(q, q_stride_tok, kv_cache, kv_dtype, kv_scale, num_blocks, block_size, block_table,
                             bt_width, bt_stride, per_shard_tables != 0, bt_shard_stride, shard_begin, shard_count,
                             seq_lens, query_start_loc, B, T, H, max_seq_len, max_q_len, D, interleave, scale, O_part,
                             o_dtype, lse_part, workspace, workspace_bytes, dev_error, stream, &sel);
}

dcp_status_t dcp_mla_decode_partial_window(
    const void* q, int64_t q_stride_tok, const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
    int32_t num_blocks, int32_t block_size, const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride, int32_t shard_begin, int32_t shard_count,
    const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B, int32_t T, int32_t H, int32_t max_seq_len,
    int32_t max_q_len, int32_t D, int32_t interleave, float scale, int32_t window, int32_t num_sinks, void* O_part,
    dcp_dtype_t o_dtype, float* lse_part, void* workspace, size_t workspace_bytes, int32_t* dev_error, void* stream) {
  dcp::SelectArgs sel{};
  sel.window = window;
  sel.sinks = num_sinks;
  return select_impl(sel, q, q_stride_tok, kv_cache, kv_dtype, kv_scale, num_blocks, block_size, block_table, bt_width,
                     bt_stride, per_shard_tables, bt_shard_stride, shard_begin, shard_count, seq_lens,
                     query_start_loc, B, T, H, max_seq_len, max_q_len, D, interleave, scale, O_part, o_dtype, lse_part,
                     workspace, workspace_bytes, dev_error, stream);
}

dcp_status_t dcp_mla_decode_partial_tree(
    const void* q, int64_t q_stride_tok, const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
    int32_t num_blocks, int32_t block_size, const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride, int32_t shard_begin, int32_t shard_count,
    const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B, int32_t T, int32_t H, int32_t max_seq_len,
    int32_t max_q_len, int32_t D, int32_t interleave, float scale, const uint64_t* tree_mask, int64_t mask_stride,
    int32_t window, int32_t num_sinks, void* O_part, dcp_dtype_t o_dtype, float* lse_part, void* workspace,
    size_t workspace_bytes, int32_t* dev_error, void* stream) {
  if (max_q_len > DCP_MAX_TREE_ROWS) return DCP_ERR_INVALID_ARG;
  if (B > 0 && T > 0) {
    if (!tree_mask || mask_stride < (max_q_len + 63) / 64) return DCP_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(tree_mask) % 8 != 0) return DCP_ERR_MISALIGNED;
  }
  dcp::SelectArgs sel{};
  sel.window = window;
  sel.sinks = num_sinks;
  sel.tree = reinterpret_cast<const unsigned long long*>(tree_mask);
  sel.tree_stride = mask_stride;
  return select_impl(sel, q, q_stride_tok, kv_cache, kv_dtype, kv_scale, num_blocks, block_size, block_table, bt_width,
                     bt_stride, per_shard_tables, bt_shard_stride, shard_begin, shard_count, seq_lens,
                     query_start_loc, B, T, H, max_seq_len, max_q_len, D, interleave, scale, O_part, o_dtype, lse_part,
                     workspace, workspace_bytes, dev_error, stream);
}

size_t dcp_decode_select_workspace_size(int32_t B, int32_t T, int32_t H, int32_t D, int32_t max_seq_len,
                                        int32_t max_q_len, int32_t window, int32_t num_sinks) {
  if (B < 0 || T < 0 || H < 1 || H > 1024 || D < 1 || D > DCP_MAX_SHARDS || max_seq_len < 0 || max_q_len < 1 ||
      window < 0 || num_sinks < 0)
    return static_cast<size_t>(-1);
  if (B == 0 || T == 0) return 0;
  // Over every interleave and number of computed shards: no call cuts its
  // units into more splits than it would if one shard owned everything.
  const int64_t lmax = select_visible(max_seq_len, max_q_len, window, num_sinks);
  const int32_t chunks = (max_q_len - 1) / select_group(H, max_q_len) + 1;
  size_t most = 0;
  for (int64_t Dn = 1; Dn <= D; ++Dn) {
    const int64_t others = Dn * chunks, units = others * B;
    const dcp::SplitPlan p{static_cast<int32_t>(dcp::select_splits(units, others, lmax, select_clusters())), 0};
    if ((units + others) * p.splits > kMostUnits) return static_cast<size_t>(-1);
    most = std::max(most, dcp::split_workspace_bytes(p, T, H, static_cast<int32_t>(Dn)) + order_bytes((units + others) * p.splits));
  }
  return most;
}

int32_t dcp_decode_kernel_launches(int32_t B, int32_t T, int32_t H, int32_t D, int32_t interleave,
                                   int32_t max_seq_len, int32_t max_q_len, size_t workspace_bytes) {
  if (B < 0 || T < 0 || H < 1 || H > 1024 || D < 1 || D > DCP_MAX_SHARDS || interleave < 1 || max_seq_len < 0 ||
      max_q_len < 0)
    return -1;
  if (B == 0 || T == 0) return 0;
  const DecodeLaunch L =
      decode_launch(T, H, D, interleave, 0, D, max_seq_len, workspace_bytes > 0, workspace_bytes);
  return 1 + (L.plan.splits > 1 ? 1 : 0) + (L.use_order ? 1 : 0);
}

static dcp_status_t combine_impl(const void* O_part, dcp_dtype_t part_dtype, const float* lse_part,
                                 const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B, int32_t T,
                                 int32_t H, int32_t D, void* out, dcp_dtype_t out_dtype, float* out_lse,
                                 void* stream) {
  if (B < 0 || T < 0 || H < 1 || D < 1 || D > DCP_MAX_SHARDS) return DCP_ERR_INVALID_ARG;
  if ((out_dtype != DCP_DTYPE_BF16 && out_dtype != DCP_DTYPE_F32) ||
      (part_dtype != DCP_DTYPE_BF16 && part_dtype != DCP_DTYPE_F32))
    return DCP_ERR_UNSUPPORTED_DTYPE;
  if (B == 0 || T == 0) return DCP_OK;
  if (!O_part || !lse_part || !seq_lens || !query_start_loc || !out || !out_lse)
    return DCP_ERR_INVALID_ARG;
  if (!aligned16(O_part) || !aligned16(out)) return DCP_ERR_MISALIGNED;
  const int64_t pairs = static_cast<int64_t>(T) * H;
  // out must not overlap O_part
  const char* ob = static_cast<const char*>(out);
  const char* oe = ob + pairs * DCP_LATENT_DIM * (out_dtype == DCP_DTYPE_BF16 ? 2 : 4);
  const char* pb = static_cast<const char*>(O_part);
  const char* pe = pb + static_cast<int64_t>(D) * pairs * DCP_LATENT_DIM * (part_dtype == DCP_DTYPE_BF16 ? 2 : 4);
  if (ob < pe && pb < oe) return DCP_ERR_INVALID_ARG;
  const cudaError_t e = dcp::launch_lse_merge(O_part, part_dtype == DCP_DTYPE_BF16, lse_part, pairs * DCP_LATENT_DIM,
                                              pairs, D, pairs, H, seq_lens, query_start_loc, B, /*row_mask=*/true,
                                              out, out_dtype == DCP_DTYPE_BF16, out_lse, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DCP_OK : DCP_ERR_CUDA;
}

dcp_status_t dcp_lse_combine(const float* O_part, const float* lse_part, const int32_t* seq_lens,
                             const int32_t* query_start_loc, int32_t B, int32_t T, int32_t H, int32_t D,
                             void* out, dcp_dtype_t out_dtype, float* out_lse, void* stream) {
  return combine_impl(O_part, DCP_DTYPE_F32, lse_part, seq_lens, query_start_loc, B, T, H, D, out, out_dtype, out_lse,
                      stream);
}

dcp_status_t dcp_lse_combine_v2(const void* O_part, dcp_dtype_t part_dtype, const float* lse_part,
                                const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B, int32_t T,
                                int32_t H, int32_t D, void* out, dcp_dtype_t out_dtype, float* out_lse,
                                void* stream) {
  return combine_impl(O_part, part_dtype, lse_part, seq_lens, query_start_loc, B, T, H, D, out, out_dtype, out_lse,
                      stream);
}

dcp_status_t dcp_decode_concat_cache(const void* ql_nope, int64_t ql_nope_stride_tok, int64_t ql_nope_stride_head,
                                     const void* q_pe, int64_t q_pe_stride_tok, int64_t q_pe_stride_head,
                                     const void* kv_c, int64_t kv_c_stride_tok, const void* k_pe,
                                     int64_t k_pe_stride_tok, const int64_t* slot_mapping, int32_t T, int32_t H,
                                     void* q_out, int64_t q_out_stride_tok, void* kv_cache, int64_t num_slots,
                                     int32_t* dev_error, void* stream) {
  if (T < 0 || H < 1 || num_slots < 1) return DCP_ERR_INVALID_ARG;
  if (T == 0) return DCP_OK;
  if (!ql_nope || !q_pe || !kv_c || !k_pe || !slot_mapping || !q_out || !kv_cache) return DCP_ERR_INVALID_ARG;
  if (ql_nope_stride_tok < 0 || ql_nope_stride_head < 0 || q_pe_stride_tok < 0 || q_pe_stride_head < 0 ||
      kv_c_stride_tok < 0 || k_pe_stride_tok < 0 || q_out_stride_tok < static_cast<int64_t>(H) * DCP_KV_DIM)
    return DCP_ERR_INVALID_ARG;
  const int64_t strides[] = {ql_nope_stride_tok, ql_nope_stride_head, q_pe_stride_tok, q_pe_stride_head,
                             kv_c_stride_tok,    k_pe_stride_tok,     q_out_stride_tok};
  for (int64_t st : strides)
    if (st % 8 != 0) return DCP_ERR_MISALIGNED;  // 16-byte units
  if (!aligned16(ql_nope) || !aligned16(q_pe) || !aligned16(kv_c) || !aligned16(k_pe) || !aligned16(q_out) ||
      !aligned16(kv_cache))
    return DCP_ERR_MISALIGNED;
  dcp::ConcatCacheArgs a{};
  a.ql_nope = ql_nope; a.ql_nope_stride_tok = ql_nope_stride_tok; a.ql_nope_stride_head = ql_nope_stride_head;
  a.q_pe = q_pe; a.q_pe_stride_tok = q_pe_stride_tok; a.q_pe_stride_head = q_pe_stride_head;
  a.kv_c = kv_c; a.kv_c_stride_tok = kv_c_stride_tok;
  a.k_pe = k_pe; a.k_pe_stride_tok = k_pe_stride_tok;
  a.slot_mapping = slot_mapping;
  a.T = T; a.H = H;
  a.q_out = q_out; a.q_out_stride_tok = q_out_stride_tok;
  a.kv_cache = kv_cache; a.num_slots = num_slots;
  a.dev_error = dev_error;
  return dcp::launch_concat_cache(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DCP_OK : DCP_ERR_CUDA;
}

dcp_status_t dcp_decode_concat_cache_v2(const void* ql_nope, int64_t ql_nope_stride_tok, int64_t ql_nope_stride_head,
                                        const void* q_pe, int64_t q_pe_stride_tok, int64_t q_pe_stride_head,
                                        const void* kv_c, int64_t kv_c_stride_tok, const void* k_pe,
                                        int64_t k_pe_stride_tok, const int64_t* slot_mapping, int32_t T, int32_t H,
                                        void* q_out, int64_t q_out_stride_tok, void* kv_cache,
                                        dcp_kv_dtype_t kv_dtype, float* kv_scale, int64_t num_slots,
                                        int32_t* dev_error, void* stream) {
  if (T < 0 || H < 0 || num_slots < 1) return DCP_ERR_INVALID_ARG;
  if (kv_dtype != DCP_KV_BF16 && kv_dtype != DCP_KV_FP8_E4M3) return DCP_ERR_UNSUPPORTED_DTYPE;
  if (T == 0) return DCP_OK;
  const bool fp8 = kv_dtype == DCP_KV_FP8_E4M3, query = H > 0;
  if (!kv_c || !k_pe || !slot_mapping || !kv_cache || (fp8 && !kv_scale)) return DCP_ERR_INVALID_ARG;
  if (query ? (!ql_nope || !q_pe || !q_out) : (ql_nope || q_pe || q_out)) return DCP_ERR_INVALID_ARG;
  if (kv_c_stride_tok < 0 || k_pe_stride_tok < 0) return DCP_ERR_INVALID_ARG;
  if (kv_c_stride_tok % 8 != 0 || k_pe_stride_tok % 8 != 0) return DCP_ERR_MISALIGNED;  // 16-byte units
  if (!aligned16(kv_c) || !aligned16(k_pe) || !aligned16(kv_cache) || (fp8 && reinterpret_cast<uintptr_t>(kv_scale) % 4 != 0))
    return DCP_ERR_MISALIGNED;
  if (query) {
    if (ql_nope_stride_tok < 0 || ql_nope_stride_head < 0 || q_pe_stride_tok < 0 || q_pe_stride_head < 0 ||
        q_out_stride_tok < static_cast<int64_t>(H) * DCP_KV_DIM)
      return DCP_ERR_INVALID_ARG;
    const int64_t strides[] = {ql_nope_stride_tok, ql_nope_stride_head, q_pe_stride_tok, q_pe_stride_head,
                               q_out_stride_tok};
    for (int64_t st : strides)
      if (st % 8 != 0) return DCP_ERR_MISALIGNED;
    if (!aligned16(ql_nope) || !aligned16(q_pe) || !aligned16(q_out)) return DCP_ERR_MISALIGNED;
  }
  dcp::ConcatCacheArgs a{};
  a.ql_nope = ql_nope; a.ql_nope_stride_tok = ql_nope_stride_tok; a.ql_nope_stride_head = ql_nope_stride_head;
  a.q_pe = q_pe; a.q_pe_stride_tok = q_pe_stride_tok; a.q_pe_stride_head = q_pe_stride_head;
  a.kv_c = kv_c; a.kv_c_stride_tok = kv_c_stride_tok;
  a.k_pe = k_pe; a.k_pe_stride_tok = k_pe_stride_tok;
  a.slot_mapping = slot_mapping;
  a.T = T; a.H = H;
  a.q_out = q_out; a.q_out_stride_tok = q_out_stride_tok;
  a.kv_cache = kv_cache; a.num_slots = num_slots;
  a.kv_scale = fp8 ? kv_scale : nullptr;
  a.dev_error = dev_error;
  return dcp::launch_concat_cache_v2(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DCP_OK : DCP_ERR_CUDA;
}

dcp_status_t dcp_latent_cache_read(const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
                                   int32_t num_blocks, int32_t block_size, const int32_t* block_table,
                                   int32_t bt_width, int64_t bt_stride, int32_t per_shard_tables,
                                   int64_t bt_shard_stride, int32_t D, int32_t interleave, int32_t shard_begin,
                                   int32_t shard_count, const int32_t* seq_starts, const int32_t* cu_lens, int32_t B,
                                   int64_t N, void* out, dcp_dtype_t out_dtype, int64_t out_stride,
                                   int32_t* dev_error, void* stream) {
  if (B < 0 || N < 0 || D < 1 || D > DCP_MAX_SHARDS || interleave < 1) return DCP_ERR_INVALID_ARG;
  if ((kv_dtype != DCP_KV_BF16 && kv_dtype != DCP_KV_FP8_E4M3) ||
      (out_dtype != DCP_DTYPE_F32 && out_dtype != DCP_DTYPE_BF16))
    return DCP_ERR_UNSUPPORTED_DTYPE;
  if (B == 0 || N == 0) return DCP_OK;
  const bool fp8 = kv_dtype == DCP_KV_FP8_E4M3, f32 = out_dtype == DCP_DTYPE_F32;
  if (!kv_cache || !block_table || !cu_lens || !out || (fp8 && !kv_scale)) return DCP_ERR_INVALID_ARG;
  if (num_blocks < 1 || block_size < 1 || bt_width < 1 || bt_stride < bt_width || out_stride < DCP_KV_DIM)
    return DCP_ERR_INVALID_ARG;
  if (shard_begin < 0 || shard_count < 1 || shard_begin + static_cast<int64_t>(shard_count) > D) return DCP_ERR_INVALID_ARG;
  if (per_shard_tables && shard_count > 1 && bt_shard_stride < static_cast<int64_t>(B - 1) * bt_stride + bt_width)
    return DCP_ERR_INVALID_ARG;  // shards' tables would overlap
  if (!aligned16(kv_cache) || !aligned16(out) || out_stride % (f32 ? 4 : 8) != 0) return DCP_ERR_MISALIGNED;
  dcp::CacheReadArgs a{};
  a.kv = kv_cache;
  a.kv_scale = fp8 ? kv_scale : nullptr;
  a.num_blocks = num_blocks; a.block_size = block_size;
  a.block_table = block_table; a.bt_width = bt_width; a.bt_stride = bt_stride;
  a.local_tables = per_shard_tables ? 1 : 0;
  a.bt_shard_stride = per_shard_tables ? bt_shard_stride : 0;
  a.D = D; a.I = interleave; a.d0 = shard_begin; a.Dn = shard_count;
  a.div_I = dcp::make_fastdiv(interleave);
  a.div_bs = dcp::make_fastdiv(block_size);
  a.div_D = dcp::make_fastdiv(D);
  a.seq_starts = seq_starts; a.cu_lens = cu_lens; a.B = B; a.N = N;
  a.out = out; a.out_stride = out_stride; a.out_f32 = f32 ? 1 : 0;
  a.dev_error = dev_error;
  return dcp::launch_cache_read(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DCP_OK : DCP_ERR_CUDA;
}

dcp_status_t dcp_norm_rope_cache(const void* ql_nope, int64_t ql_nope_stride_tok, int64_t ql_nope_stride_head,
                                 const void* q_pe, int64_t q_pe_stride_tok, int64_t q_pe_stride_head, void* q_out,
                                 int64_t q_out_stride_tok, int64_t q_out_stride_head, const void* kv_c,
                                 int64_t kv_c_stride_tok, const void* k_pe, int64_t k_pe_stride_tok,
                                 const void* norm_weight, float eps, const int32_t* positions, const float* cos_sin,
                                 int32_t max_pos, int32_t interleaved, const int64_t* slot_mapping, int32_t T,
                                 int32_t H, void* kv_cache, dcp_kv_dtype_t kv_dtype, float* kv_scale,
                                 int64_t num_slots, int32_t* dev_error, void* stream) {
  if (T < 0 || H < 0 || num_slots < 1 || max_pos < 1) return DCP_ERR_INVALID_ARG;
  if (kv_dtype != DCP_KV_BF16 && kv_dtype != DCP_KV_FP8_E4M3) return DCP_ERR_UNSUPPORTED_DTYPE;
  if (T == 0) return DCP_OK;
  const bool fp8 = kv_dtype == DCP_KV_FP8_E4M3, query = H > 0;
  if (!kv_c || !k_pe || !slot_mapping || !kv_cache || !positions || !cos_sin || (fp8 && !kv_scale)) return DCP_ERR_INVALID_ARG;
  if (query ? (!q_pe || !q_out) : (ql_nope || q_pe || q_out)) return DCP_ERR_INVALID_ARG;
  if (norm_weight && !(eps >= 0.f && std::isfinite(eps))) return DCP_ERR_INVALID_ARG;
  if (kv_c_stride_tok < 0 || k_pe_stride_tok < 0) return DCP_ERR_INVALID_ARG;
  if (kv_c_stride_tok % 8 != 0 || k_pe_stride_tok % 8 != 0) return DCP_ERR_MISALIGNED;  // 16-byte units
  if (!aligned16(kv_c) || !aligned16(k_pe) || !aligned16(kv_cache) || !aligned16(norm_weight) || !aligned16(cos_sin) ||
      (fp8 && reinterpret_cast<uintptr_t>(kv_scale) % 4 != 0))
    return DCP_ERR_MISALIGNED;
  if (query) {
    if (!ql_nope) ql_nope_stride_tok = ql_nope_stride_head = 0;
    const int64_t width = ql_nope ? DCP_KV_DIM : DCP_ROPE_DIM;
    if (ql_nope_stride_tok < 0 || ql_nope_stride_head < 0 || q_pe_stride_tok < 0 || q_pe_stride_head < 0 ||
        (H > 1 && q_out_stride_head < width) || (T > 1 && q_out_stride_tok < width))
      return DCP_ERR_INVALID_ARG;
    // one (token, head)'s output must not be another's: heads within tokens, or tokens within heads
    if (T > 1 && H > 1 && q_out_stride_tok < (H - 1) * q_out_stride_head + width &&
        q_out_stride_head < (T - 1) * q_out_stride_tok + width)
      return DCP_ERR_INVALID_ARG;
    const int64_t strides[] = {ql_nope_stride_tok, ql_nope_stride_head, q_pe_stride_tok, q_pe_stride_head,
                               q_out_stride_tok, q_out_stride_head};
    for (int64_t st : strides)
      if (st % 8 != 0) return DCP_ERR_MISALIGNED;
    if (!aligned16(ql_nope) || !aligned16(q_pe) || !aligned16(q_out)) return DCP_ERR_MISALIGNED;
  }
  dcp::NormRopeArgs a{};
  a.ql_nope = static_cast<const __nv_bfloat16*>(ql_nope);
  a.ql_nope_stride_tok = ql_nope_stride_tok; a.ql_nope_stride_head = ql_nope_stride_head;
  a.q_pe = static_cast<const __nv_bfloat16*>(q_pe);
  a.q_pe_stride_tok = q_pe_stride_tok; a.q_pe_stride_head = q_pe_stride_head;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.q_out_stride_tok = q_out_stride_tok; a.q_out_stride_head = q_out_stride_head;
  a.kv_c = static_cast<const __nv_bfloat16*>(kv_c); a.kv_c_stride_tok = kv_c_stride_tok;
  a.k_pe = static_cast<const __nv_bfloat16*>(k_pe); a.k_pe_stride_tok = k_pe_stride_tok;
  a.norm_weight = static_cast<const __nv_bfloat16*>(norm_weight);
  a.eps = eps;
  a.positions = positions; a.cos_sin = cos_sin; a.max_pos = max_pos; a.pairs = interleaved != 0;
  a.slot_mapping = slot_mapping;
  a.T = T; a.H = H;
  a.kv_cache = kv_cache; a.kv_scale = fp8 ? kv_scale : nullptr; a.num_slots = num_slots;
  a.dev_error = dev_error;
  return dcp::launch_norm_rope(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DCP_OK : DCP_ERR_CUDA;
}

dcp_status_t dcp_cache_extend_v2(int32_t* block_table, int32_t bt_width, int64_t bt_stride, int32_t per_shard_tables,
                                 int64_t bt_shard_stride, const int32_t* seq_lens, const int32_t* query_start_loc,
                                 int32_t B, int32_t T, int32_t block_size, int32_t D, int32_t interleave,
                                 int32_t shard_begin, int32_t shard_count, const int32_t* free_blocks, int32_t num_free,
                                 const int32_t* free_count, int32_t* free_left, int32_t* held,
                                 int32_t* positions, int64_t* slot_mapping, int32_t* dev_error, void* stream) {
  if (B < 0 || T < 0 || D < 1 || D > DCP_MAX_SHARDS || interleave < 1 || block_size < 1 || num_free < 0)
    return DCP_ERR_INVALID_ARG;
  if (shard_begin < 0 || shard_count < 1 || shard_begin + static_cast<int64_t>(shard_count) > D) return DCP_ERR_INVALID_ARG;
  if (!free_count || !free_left || (num_free > 0 && !free_blocks)) return DCP_ERR_INVALID_ARG;
  if (T > 0 && (!positions || !slot_mapping)) return DCP_ERR_INVALID_ARG;
  if (B > 0) {
    if (!block_table || !seq_lens || !query_start_loc || bt_width < 1 || bt_width > (1 << 20) || bt_stride < bt_width)
      return DCP_ERR_INVALID_ARG;
    if (per_shard_tables && shard_count > 1 && bt_shard_stride < static_cast<int64_t>(B - 1) * bt_stride + bt_width)
      return DCP_ERR_INVALID_ARG;  // shards' tables would overlap
  }
  dcp::CacheExtendArgs a{};
  a.block_table = block_table; a.bt_width = bt_width; a.bt_stride = bt_stride;
  a.local_tables = per_shard_tables ? 1 : 0;
  a.bt_shard_stride = per_shard_tables ? bt_shard_stride : 0;
  a.seq_lens = seq_lens; a.qsl = query_start_loc; a.B = B; a.T = T; a.block_size = block_size;
  a.D = D; a.I = interleave; a.d0 = shard_begin; a.Dn = shard_count;
  a.S = a.local_tables ? shard_count : 1;
  a.period = static_cast<int64_t>(D) * interleave;
  if (a.period <= 0x7fffffff) a.div_period = dcp::make_fastdiv(static_cast<int32_t>(a.period));
  a.div_I = dcp::make_fastdiv(interleave);
  a.div_D = dcp::make_fastdiv(D);
  a.div_bs = dcp::make_fastdiv(block_size);
  a.free_blocks = free_blocks; a.num_free = num_free; a.free_count = free_count; a.free_left = free_left;
  a.held = held;
  a.positions = positions; a.slot_mapping = slot_mapping;
  a.dev_error = dev_error;
  return dcp::launch_cache_extend(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DCP_OK : DCP_ERR_CUDA;
}

dcp_status_t dcp_cache_extend(int32_t* block_table, int32_t bt_width, int64_t bt_stride, int32_t per_shard_tables,
                              int64_t bt_shard_stride, const int32_t* seq_lens, const int32_t* query_start_loc,
                              int32_t B, int32_t T, int32_t block_size, int32_t D, int32_t interleave,
                              int32_t shard_begin, int32_t shard_count, const int32_t* free_blocks, int32_t num_free,
                              const int32_t* free_count, int32_t* free_left, int32_t* positions,
                              int64_t* slot_mapping, int32_t* dev_error, void* stream) {
  return dcp_cache_extend_v2(block_table, bt_width, bt_stride, per_shard_tables, bt_shard_stride, seq_lens,
                             query_start_loc, B, T, block_size, D, interleave, shard_begin, shard_count, free_blocks,
                             num_free, free_count, free_left, nullptr, positions, slot_mapping, dev_error, stream);
}

}  // extern "C"

namespace {

// Workspace of chunk attention: requests' first images and units, the heads'
// shared parts (token masks and rope images), then keys, values and masks of as
// many heads as there is room for.
struct ChunkPlan {
  int64_t tiles, units;                                // images per head, units per head
  size_t starts, pieces, valid, rope;                  // offsets of the parts
  size_t fixed;                                        // bytes of what the heads share
  int64_t lo_tiles;                                    // tiles with key remainders per head
  size_t image_bytes;                                  // bytes of a head's images
  int sms;
};
constexpr size_t kChunkRecommended = size_t{4} << 30;

size_t round256(size_t n) { return (n + 255) & ~size_t{255}; }

bool chunk_plan(int32_t B, int32_t T, int32_t H, int64_t total_len, ChunkPlan* p) {
  if (B < 0 || T < 0 || H < 1 || H > 1024 || total_len < 0 || total_len > (int64_t{1} << 36)) return false;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&p->sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || p->sms <= 0) {
    cudaGetLastError();  // clear: no device is not an error for sizing
    p->sms = 152;        // GB300
  }
  p->tiles = total_len / dcp::kChunkTile + B;
  p->units = T / dcp::kChunkRows + static_cast<int64_t>(B) + 2;
  const int64_t most = p->units + dcp::added_pieces(p->sms, 1);
  if (p->tiles * H > 0x7fffffff || most * H > 0x7fffffff) return false;
  const size_t n = static_cast<size_t>(p->tiles);
  p->starts = 0;
  p->pieces = round256((3 * (static_cast<size_t>(B) + 1) + 1) * 4);
  p->valid = round256(p->pieces + static_cast<size_t>(most) * sizeof(dcp::Piece));
  p->rope = round256(p->valid + n * 16);
  p->fixed = p->rope + n * dcp::kImage;
  p->lo_tiles = std::min<int64_t>(p->tiles, static_cast<int64_t>(B) * dcp::kFineTiles);
  p->image_bytes = n * (4 * dcp::kImage + 16) + static_cast<size_t>(p->lo_tiles) * 2 * dcp::kImage;
  return true;
}

// Slots for the pieces of cut units, per head of a pass of `heads`: twice the
// pieces that the cuts add, and none where no unit is long enough to be cut.
int64_t chunk_slots(const ChunkPlan& p, int32_t heads) {
  if (p.tiles < 2 * dcp::kMinPiece) return 0;
  const int64_t by_units = p.units * std::min<int64_t>(dcp::kMaxPieces, (p.tiles + dcp::kMinPiece - 1) / dcp::kMinPiece);
  return std::min(by_units, 2 * dcp::added_pieces(p.sms, heads));
}
size_t chunk_bytes(const ChunkPlan& p, int32_t heads) {
  const size_t slots = static_cast<size_t>(chunk_slots(p, heads)) * heads;
  return p.fixed + round256(p.image_bytes * heads) + slots * dcp::kSlotBytes;
}

}  // namespace

extern "C" {

size_t dcp_chunk_attention_workspace_size(int32_t B, int32_t T, int32_t H, int64_t total_len) {
  ChunkPlan p{};
  if (!chunk_plan(B, T, H, total_len, &p)) return static_cast<size_t>(-1);
  if (B == 0 || T == 0) return 0;
  size_t heads = p.image_bytes > 0 ? kChunkRecommended / p.image_bytes : 1;
  heads = heads < 1 ? 1 : (heads > static_cast<size_t>(H) ? static_cast<size_t>(H) : heads);
  return chunk_bytes(p, static_cast<int32_t>(heads));
}

dcp_status_t dcp_pack_kv_b(const void* w_kv_b, int32_t H, void* packed, void* stream) {
  if (H < 1 || H > 1024 || !w_kv_b || !packed) return DCP_ERR_INVALID_ARG;
  if (!aligned16(w_kv_b) || !aligned16(packed)) return DCP_ERR_MISALIGNED;
  return dcp::launch_pack_kv_b(w_kv_b, H, packed, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DCP_OK : DCP_ERR_CUDA;
}

dcp_status_t dcp_mla_chunk_attention(const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                                     const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
                                     int32_t num_blocks, int32_t block_size, const int32_t* block_table,
                                     int32_t bt_width, int64_t bt_stride, int32_t per_shard_tables,
                                     int64_t bt_shard_stride, int32_t D, int32_t interleave, const int32_t* seq_lens,
                                     const int32_t* query_start_loc, int32_t B, int32_t T, int32_t H,
                                     int64_t total_len, float scale, const void* packed_kv_b, void* out,
                                     dcp_dtype_t out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                                     int32_t* dev_error, void* stream) {
  ChunkPlan p{};
  if (!chunk_plan(B, T, H, total_len, &p) || D < 1 || D > DCP_MAX_SHARDS || interleave < 1 || !std::isfinite(scale))
    return DCP_ERR_INVALID_ARG;
  if ((kv_dtype != DCP_KV_BF16 && kv_dtype != DCP_KV_FP8_E4M3) ||
      (out_dtype != DCP_DTYPE_F32 && out_dtype != DCP_DTYPE_BF16))
    return DCP_ERR_UNSUPPORTED_DTYPE;
  if (B == 0 || T == 0) return DCP_OK;
  const bool fp8 = kv_dtype == DCP_KV_FP8_E4M3;
  if (!q || !kv_cache || !block_table || !seq_lens || !query_start_loc || !packed_kv_b || !out || !lse || (fp8 && !kv_scale))
    return DCP_ERR_INVALID_ARG;
  if (num_blocks < 1 || block_size < 1 || bt_width < 1 || bt_stride < bt_width || q_stride_tok < 0 || q_stride_head < 0)
    return DCP_ERR_INVALID_ARG;
  if (per_shard_tables && D > 1 && bt_shard_stride < static_cast<int64_t>(B - 1) * bt_stride + bt_width)
    return DCP_ERR_INVALID_ARG;  // shards' tables would overlap
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(packed_kv_b) || !aligned16(out) || !aligned16(workspace) ||
      q_stride_tok % 8 != 0 || q_stride_head % 8 != 0)
    return DCP_ERR_MISALIGNED;
  // heads per pass: as many as fit, in passes of nearly equal size
  int32_t heads = H;
  while (heads > 1 && chunk_bytes(p, heads) > workspace_bytes) {
    const int32_t passes = (H + heads - 1) / heads + 1;
    heads = std::min(heads - 1, (H + passes - 1) / passes);
  }
  if (!workspace || chunk_bytes(p, heads) > workspace_bytes) return DCP_ERR_WORKSPACE_TOO_SMALL;
  dcp::ChunkArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride_tok = q_stride_tok; a.q_stride_head = q_stride_head;
  a.kv = kv_cache; a.kv_scale = fp8 ? kv_scale : nullptr;
  a.num_blocks = num_blocks; a.block_size = block_size;
  a.block_table = block_table; a.bt_width = bt_width; a.bt_stride = bt_stride;
  a.local_tables = per_shard_tables ? 1 : 0;
  a.bt_shard_stride = per_shard_tables ? bt_shard_stride : 0;
  a.D = D; a.I = interleave;
  a.div_I = dcp::make_fastdiv(interleave);
  a.div_D = dcp::make_fastdiv(D);
  a.div_bs = dcp::make_fastdiv(block_size);
  a.seq_lens = seq_lens; a.qsl = query_start_loc; a.B = B; a.T = T; a.H = H;
  a.scale_log2 = std::fabs(scale) * dcp::kLog2e;
  a.q_sign = scale < 0.f ? 0x80008000u : 0u;
  a.weight = packed_kv_b;
  a.out = out; a.out_f32 = out_dtype == DCP_DTYPE_F32; a.lse = lse;
  a.dev_error = dev_error;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.tiles = static_cast<int32_t>(p.tiles);
  a.tile_start = reinterpret_cast<int32_t*>(ws + p.starts);
  a.block_start = a.tile_start + B + 1;
  a.lo_start = a.block_start + B + 1;
  a.num_pieces = a.lo_start + B + 1;
  a.pieces = reinterpret_cast<dcp::Piece*>(ws + p.pieces);
  a.valid = reinterpret_cast<uint4*>(ws + p.valid);
  a.rope = ws + p.rope;
  a.keys = ws + p.fixed;
  a.values = a.keys + static_cast<size_t>(heads) * p.tiles * (2 * dcp::kImage);
  a.lo_keys = a.values + static_cast<size_t>(heads) * p.tiles * (2 * dcp::kImage);
  a.lo_tiles = static_cast<int32_t>(p.lo_tiles);
  a.bad = reinterpret_cast<uint4*>(a.lo_keys + static_cast<size_t>(heads) * p.lo_tiles * (2 * dcp::kImage));
  a.sms = p.sms;
  a.slots = static_cast<int32_t>(chunk_slots(p, heads));
  a.max_pieces = static_cast<int32_t>(p.units + (a.slots > 0 ? dcp::added_pieces(p.sms, heads) : 0));
  a.partial = a.keys + round256(p.image_bytes * heads);
  a.heads = heads;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dcp::launch_chunk_plan(a, st) != cudaSuccess) return DCP_ERR_CUDA;
  for (a.h0 = 0; a.h0 < H; a.h0 += heads) {
    a.heads = std::min(heads, H - a.h0);
    if (dcp::launch_chunk_expand(a, st) != cudaSuccess || dcp::launch_chunk_attention(a, st) != cudaSuccess) return DCP_ERR_CUDA;
  }
  return DCP_OK;
}

}  // extern "C"
