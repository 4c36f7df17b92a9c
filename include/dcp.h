/*
 * dcp.h - C ABI of the GB300 (sm_103a) decode-context-parallel MLA hot path.
 *
 * Decode context parallelism (DCP) splits each request's KV context over D
 * shards; every shard runs absorbed-MLA decode attention over its own tokens
 * and returns a partial output plus its log-sum-exp, and an LSE-weighted
 * combine merges the shards.  On one GPU the D shards are D disjoint token
 * partitions of one paged latent KV cache resident in HBM.
 *
 * Sources (pages on the method):
 *   [PR50484] "[Kimi-K3] DCP support", vllm-project/vllm pull request 50484:
 *             Summary (empty-KV-shard masking of the LSE-weighted reduction),
 *             "CUDA-graph padding follow-up" and the review thread on the
 *             padding-row mask (rows of seq_len == 0 requests).
 *   [PRHUB]   prhub.com.cn summary of the same pull request: implementation
 *             steps 3-4 (interleaved DCP chunking; -inf masking at the source;
 *             exp2 LSE-weighted merge; zero-weight skip at the consumer;
 *             16-byte row alignment), key snippet "Decode: latent multi-query
 *             attention" (forward_mqa returns (latent_out, lse); then
 *             combine(latent_out, lse, seq_lens, query_start_loc)), risk 2
 *             (unsupported dtypes are rejected) and risk 4 (timeouts trap in
 *             the pages' kernel; here they return a status).
 *   [PR565]   "perf(mla): fuse K3 DCP verification queries",
 *             local-inference-lab/vllm pull request 565: Summary (the K=3
 *             verification rows share each KV load) and review follow-up
 *             (block-table width contract; reject a table narrower than the
 *             largest local shard).
 *
 * Conventions shared by every entry point:
 *   - All pointers to arrays are DEVICE pointers to caller-owned memory on the
 *     current CUDA device; the library allocates nothing, keeps no state
 *     between calls, never synchronises, and enqueues its kernels on
 *     `stream` (a cudaStream_t; NULL = legacy default stream).  A call
 *     returns DCP_OK once its kernels are enqueued.
 *   - Arrays are dense row-major unless a stride argument says otherwise.
 *     Strides are in ELEMENTS.
 *   - Host-detectable errors return a status before anything is launched.
 *     Errors only the device can see (a block id outside the cache, a
 *     sequence longer than the declared maximum) never trap: the kernel skips
 *     the offending token and ORs a DCP_DEVERR_* bit into *dev_error when
 *     dev_error is non-NULL.
 *   - Latent geometry is fixed: a KV cache row and a query head row are
 *     DCP_KV_DIM = 576 bf16 values (512 compressed-KV dims followed by 64
 *     rope dims); values are the first DCP_LATENT_DIM = 512 dims.
 *   - LSEs are natural logarithms; -inf marks "no tokens".
 *   - Two environment variables, read on every call and unset in normal use,
 *     change what the decodes run (the windowed and tree ones included):
 *       DCP_FORCE_SIMT=1       the CUDA-core reference kernel instead of the
 *                              tensor-core one (A/B checks);
 *       DCP_TEST_STALL_WAIT=1  test hook for the failure path: one wait of
 *                              the tensor-core kernel runs out on purpose
 *                              (on a barrier nothing completes), so the call
 *                              ends with DCP_DEVERR_TIMEOUT in *dev_error
 *                              after about a second per bounded wait; the
 *                              outputs are undefined.
 */
#ifndef DCP_H_
#define DCP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DCP_LATENT_DIM 512
#define DCP_ROPE_DIM 64
#define DCP_KV_DIM 576
#define DCP_MAX_SHARDS 32
#define DCP_MAX_TREE_ROWS 256 /* rows of a request under a tree mask */
#define DCP_NOPE_DIM 128      /* a head's key dims projected up from the latent (chunk attention) */
#define DCP_VALUE_DIM 128     /* and its value dims */

/* Device-side error bits ORed into *dev_error. */
#define DCP_DEVERR_BAD_BLOCK 1    /* a referenced block id is outside [0, num_blocks) */
#define DCP_DEVERR_SEQ_TOO_LONG 2 /* seq_len > max_seq_len (clamped to max_seq_len) */
#define DCP_DEVERR_BAD_ROWS 4     /* query_start_loc decreasing (chunk attention: or negative), or q_len > max_q_len */
#define DCP_DEVERR_TIMEOUT 8      /* a bounded on-device wait gave up */
#define DCP_DEVERR_NO_BLOCKS 16   /* the free list ran out (dcp_cache_extend) */
#define DCP_DEVERR_BAD_POSITION 32 /* a position past the cos/sin table (dcp_norm_rope_cache) */

typedef enum {
  DCP_OK = 0,
  DCP_ERR_INVALID_ARG = 1,       /* null pointer, negative or inconsistent size */
  DCP_ERR_UNSUPPORTED_DTYPE = 2, /* output dtype not supported [PRHUB, risk 2] */
  DCP_ERR_MISALIGNED = 3,        /* pointer or row stride not 16-byte aligned [PRHUB, step 4] */
  DCP_ERR_TABLE_TOO_NARROW = 4,  /* bt_width < ceil(max_seq_len / block_size) [PR565, review follow-up] */
  DCP_ERR_WORKSPACE_TOO_SMALL = 5,
  DCP_ERR_CUDA = 6,              /* a CUDA runtime/driver call failed (launch, attribute query) */
  DCP_ERR_TIMEOUT = 7            /* reserved for bounded cross-device waits */
} dcp_status_t;

typedef enum { DCP_DTYPE_BF16 = 0, DCP_DTYPE_F32 = 1 } dcp_dtype_t;

/* Latent KV cache formats: bf16 rows, or FP8 E4M3 codes (1 sign, 4 exponent
 * bits with bias 7, 3 mantissa bits; no infinity) with one fp32 scale per
 * cache slot (value = code x scale) ["perf(mla): fuse K3 DCP verification
 * queries", review follow-up: fp8 KV verify plans]. */
typedef enum { DCP_KV_BF16 = 0, DCP_KV_FP8_E4M3 = 1 } dcp_kv_dtype_t;

/* Human-readable name of a status code (static string, never NULL). */
const char* dcp_status_str(dcp_status_t status);

/* Library ABI version (increments when a signature changes). */
int dcp_version(void);

/*
 * Token -> shard mapper (host copy of the device code, for tests).
 * Positions are dealt to the D shards round-robin in runs of `interleave`
 * tokens (cp_kv_cache_interleave_size): shard(pos) = floor(pos / I) mod D
 * [PRHUB, implementation step 3].  Returns -1 if D < 1, I < 1 or pos < 0.
 */
int32_t dcp_shard_of(int64_t pos, int32_t D, int32_t interleave);

/*
 * How many of the first L positions shard d owns:
 *   floor(L / (I D)) * I + clamp(L mod (I D) - d I, 0, I).
 * Returns -1 on invalid arguments (L < 0, d outside [0, D), D < 1, I < 1).
 */
int32_t dcp_local_len(int32_t L, int32_t d, int32_t D, int32_t interleave);

/*
 * Bytes of device workspace dcp_mla_decode_partial should get for these sizes
 * on the CURRENT device (the split-KV plan depends on its SM count): the
 * split partials plus one int32 per work unit for the order in which the
 * units start (long ones first when they do not all fit on the GPU at once).
 * A workspace that covers only the split partials is accepted (units then
 * start in index order); with no split partials it may be NULL.  Returns
 * (size_t)-1 on invalid arguments.
 */
size_t dcp_decode_workspace_size(int32_t B, int32_t T, int32_t H, int32_t D,
                                 int32_t max_seq_len, int32_t max_q_len);

/*
 * Number of kernels one dcp_mla_decode_partial call with these sizes and this
 * workspace size launches on the CURRENT device: the decode, plus the merge of
 * the split partials when the long-context split is used, plus the ordering
 * of the work units when there are more of them than fit on the GPU at once
 * (and the workspace has room for it).  0 when B or T is 0; -1 on invalid
 * arguments.  For callers that count or capture launches; no page has a
 * counterpart.
 */
int32_t dcp_decode_kernel_launches(int32_t B, int32_t T, int32_t H, int32_t D, int32_t interleave,
                                   int32_t max_seq_len, int32_t max_q_len, size_t workspace_bytes);

/*
 * Absorbed-MLA decode attention split over D context shards.
 * [PRHUB, snippet "Decode: latent multi-query attention": forward_mqa(q,
 *  kv_cache, metadata) -> (latent_out, lse) per rank's shard;
 *  PR50484 Summary and PRHUB step 4: empty shards masked to -inf at source;
 *  PR565 Summary: verification rows of one request share each KV load.]
 *
 * For query row r of request b (rows qsl[b] .. qsl[b+1]-1, q_len = their
 * count, i = r - qsl[b]) the row's own context length is
 *   L_r = max(0, seq_lens[b] - (q_len - 1 - i))
 * (the new tokens are already in the cache).  For each shard d and head h:
 *   S = { p < L_r : floor(p / interleave) mod D == d }
 *   s_p = scale * sum_{k<576} q[r,h,k] * kv(p)[k]
 *   lse_part[d,r,h] = ln sum_{p in S} exp(s_p)
 *   O_part[d,r,h,v] = sum_{p in S} exp(s_p - lse_part[d,r,h]) * kv(p)[v],  v < 512
 * where kv(p) is cache row block_table[b, p / block_size] * block_size +
 * p % block_size.  If S is empty, the row is a padding row (seq_lens[b] == 0)
 * or r >= qsl[B]: lse_part = -inf and O_part = 0, and no KV is read.
 *
 *   q               bf16 [T, H, 576]; row r starts at q + r * q_stride_tok
 *                   (q_stride_tok >= H * 576, a multiple of 8).
 *   kv_cache        bf16 [num_blocks, block_size, 576], dense.
 *   block_table     int32 [B, bt_width], row stride bt_stride (>= bt_width);
 *                   only columns < ceil(L_r / block_size) are read.
 *   seq_lens        int32 [B]; 0 marks a CUDA-graph padding request.
 *   query_start_loc int32 [B + 1], non-decreasing, qsl[0] = 0.
 *   B, T            requests and query rows (rows past qsl[B] are padding).
 *   H               heads (1 .. 1024).
 *   max_seq_len     host-known upper bound of seq_lens (sizes the split plan
 *                   and the table-width check).
 *   max_q_len       host-known upper bound of rows per request.
 *   D, interleave   shard count (1 .. 32) and run length (>= 1).
 *   scale           softmax scale (1/sqrt(192) for Kimi-K3).
 *   O_part          fp32 [D, T, H, 512] output.
 *   lse_part        fp32 [D, T, H] output.
 *   workspace       device scratch of >= dcp_decode_workspace_size(...) bytes,
 *                   16-byte aligned; its contents on entry are ignored.
 *   dev_error       optional int32 device word for DCP_DEVERR_* bits.
 *   stream          cudaStream_t.
 *
 * B == 0 or T == 0 returns DCP_OK without launching anything.
 */
dcp_status_t dcp_mla_decode_partial(
    const void* q, int64_t q_stride_tok,
    const void* kv_cache, int32_t num_blocks, int32_t block_size,
    const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len,
    int32_t D, int32_t interleave, float scale,
    float* O_part, float* lse_part,
    void* workspace, size_t workspace_bytes,
    int32_t* dev_error, void* stream);

/*
 * LSE-weighted combine of D shard partials, with empty-shard and padding-row
 * masking [PRHUB step 4 "exp2 LSE weighted merge"; PR50484 "CUDA-graph
 * padding follow-up"].
 *
 * For each row r and head h: a row whose request has seq_lens == 0 (or that
 * lies past qsl[B]) is a padding row: out = 0, out_lse = -inf, nothing else
 * read.  Otherwise E = { d : lse_part[d,r,h] != -inf }; if E is empty the
 * result is 0 / -inf.  Else, with l_d = lse_part[d,r,h] * log2(e) and
 * M = max_{d in E} l_d:
 *   w_d = exp2(l_d - M),  out = sum_E w_d O_part[d,r,h,:] / sum_E w_d,
 *   out_lse = (M + log2 sum_E w_d) / log2(e).
 * O_part[d,r,h,:] is not read for d outside E (it may hold stale data/NaN).
 *
 *   O_part     fp32 [D, T, H, 512], 16-byte aligned.
 *   lse_part   fp32 [D, T, H].
 *   seq_lens, query_start_loc, B, T: as for the decode call.
 *   H, D       heads (>= 1), shards (1 .. 32).
 *   out        [T, H, 512] of out_dtype (BF16: round to nearest even; F32),
 *              16-byte aligned; must not overlap O_part.
 *   out_lse    fp32 [T, H]; may alias lse_part (the shard-0 slice): every
 *              LSE of a (row, head) is read before its out_lse is written.
 *
 * B == 0 or T == 0 returns DCP_OK without launching anything.
 */
dcp_status_t dcp_lse_combine(
    const float* O_part, const float* lse_part,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int32_t D,
    void* out, dcp_dtype_t out_dtype, float* out_lse, void* stream);

/*
 * dcp_mla_decode_partial over per-shard (DCP rank-local) block tables: each
 * shard stores only the tokens it owns, densely and in order, in its own
 * blocks, as each rank's own cache does ["[Kimi-K3] DCP support", Summary:
 * each DCP rank keeps its slice of the context; PR565, review follow-up: the
 * plan's page table must cover the largest local KV shard].  Same
 * arguments, results and errors as dcp_mla_decode_partial, except:
 *
 *   shard_begin, shard_count
 *                   the shards this call computes, [shard_begin, shard_begin +
 *                   shard_count) of D (0 <= shard_begin, 1 <= shard_count,
 *                   shard_begin + shard_count <= D, else DCP_ERR_INVALID_ARG):
 *                   all D when one GPU holds every shard, one per DCP rank
 *                   when each rank holds only its own.  D and interleave
 *                   still define which tokens each shard owns.
 *   O_part, lse_part
 *                   fp32 [shard_count, T, H, 512] and [shard_count, T, H].
 *   block_table     int32 [shard_count, B, bt_width]: shard d's j-th local
 *                   token of request b lives in cache row
 *                   table[d - shard_begin, b, j / block_size] * block_size +
 *                   j % block_size.
 *                   Request rows are bt_stride elements apart (>= bt_width),
 *                   shard tables bt_shard_stride apart (with more than one
 *                   shard >= (B - 1) * bt_stride + bt_width, else
 *                   DCP_ERR_INVALID_ARG).  Only the columns a shard's local
 *                   tokens reach are read.
 *   bt_width        must cover the largest computed local shard, the first:
 *                   ceil(local_len(max_seq_len, shard_begin, D, interleave) /
 *                   block_size) <= bt_width, else DCP_ERR_TABLE_TOO_NARROW.
 *
 * The shard of a token and its local index follow the same interleave rule
 * (dcp_shard_of, dcp_local_len).  The workspace is sized by
 * dcp_decode_workspace_size with its D argument = shard_count.
 */
dcp_status_t dcp_mla_decode_partial_local(
    const void* q, int64_t q_stride_tok,
    const void* kv_cache, int32_t num_blocks, int32_t block_size,
    const int32_t* block_table, int32_t bt_width, int64_t bt_stride, int64_t bt_shard_stride,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len,
    int32_t D, int32_t interleave, int32_t shard_begin, int32_t shard_count, float scale,
    float* O_part, float* lse_part,
    void* workspace, size_t workspace_bytes,
    int32_t* dev_error, void* stream);

/*
 * The general form of the decode: dcp_mla_decode_partial with every option.
 * The fp8 latent cache and bf16 partials are the pages' next step for the
 * hot path (they halve its two byte streams) ["perf(mla): fuse K3 DCP
 * verification queries", review follow-up: fp8 KV verify plans].
 *
 *   kv_dtype        DCP_KV_BF16: kv_cache bf16 [num_blocks, block_size, 576].
 *                   DCP_KV_FP8_E4M3: kv_cache uint8 codes [num_blocks,
 *                   block_size, 576] and kv_scale fp32 [num_blocks,
 *                   block_size] (required, else DCP_ERR_INVALID_ARG); the
 *                   latent value of a slot is code x scale.  Other values:
 *                   DCP_ERR_UNSUPPORTED_DTYPE.  The tensor-core kernel
 *                   (H <= 128) widens each code x scale to bf16 on its way
 *                   into shared memory (the fp32 product, rounded to
 *                   nearest even): exact when the scale is a power of two,
 *                   else one bf16 rounding of each latent value, as a bf16
 *                   cache holds them.  The CUDA-core kernel applies the
 *                   scale in fp32 to the dot products and the PV weights.
 *   per_shard_tables, bt_shard_stride, shard_begin, shard_count
 *                   0: one table row per request ([B, bt_width]); 1:
 *                   per-shard tables as for dcp_mla_decode_partial_local.
 *                   Either way the call computes shards [shard_begin,
 *                   shard_begin + shard_count) of D.
 *   O_part, o_dtype fp32 or bf16 (round to nearest even) [shard_count, T,
 *                   H, 512]; lse_part stays fp32.  With bf16 the split-KV
 *                   partials in the workspace are bf16 too.
 * Everything else as for dcp_mla_decode_partial.
 */
dcp_status_t dcp_mla_decode_partial_v2(
    const void* q, int64_t q_stride_tok,
    const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
    int32_t num_blocks, int32_t block_size,
    const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride, int32_t shard_begin, int32_t shard_count,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len,
    int32_t D, int32_t interleave, float scale,
    void* O_part, dcp_dtype_t o_dtype, float* lse_part,
    void* workspace, size_t workspace_bytes,
    int32_t* dev_error, void* stream);

/*
 * dcp_lse_combine over partials in fp32 or bf16 (part_dtype), e.g. those of
 * dcp_mla_decode_partial_v2 with o_dtype = DCP_DTYPE_BF16.  Everything else
 * as for dcp_lse_combine; an unsupported part_dtype returns
 * DCP_ERR_UNSUPPORTED_DTYPE.
 */
dcp_status_t dcp_lse_combine_v2(
    const void* O_part, dcp_dtype_t part_dtype, const float* lse_part,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int32_t D,
    void* out, dcp_dtype_t out_dtype, float* out_lse, void* stream);

/*
 * The decode step before attention, fused into one launch ["[Kimi-K3] DCP
 * support" summary on prhub.com.cn, key snippet "Decode: latent multi-query
 * attention": _decode_concat_cache builds the decode query and writes this
 * step's latent rows into the paged cache before forward_mqa, so the decode
 * call sees the new tokens (seq_lens count them)].  The optional RoPE of the
 * snippet (rope_positions = None) is not applied: the rope parts are taken as
 * given.
 *
 * For every token t < T and head h < H:
 *   q_out[t, h, 0:512]   = ql_nope[t, h, :]
 *   q_out[t, h, 512:576] = q_pe[t, h, :]
 * and, when 0 <= slot_mapping[t] < num_slots:
 *   kv_cache[slot_mapping[t], 0:512]   = kv_c[t, :]
 *   kv_cache[slot_mapping[t], 512:576] = k_pe[t, :]
 * slot_mapping[t] = block * block_size + offset is the token's cache row.  A
 * negative slot is not written: a padding token, or (with per-rank caches) a
 * token another DCP rank owns.  A slot >= num_slots is not written either and
 * sets DCP_DEVERR_BAD_BLOCK in *dev_error.  Byte copies: bit-exact.
 *
 *   ql_nope      bf16 [T, H, 512]; element (t, h, k) at t * ql_nope_stride_tok +
 *                h * ql_nope_stride_head + k (e.g. the transposed output of the
 *                per-head q_nope x W_UK batched matmul).
 *   q_pe         bf16 [T, H, 64], strides likewise.
 *   kv_c, k_pe   bf16 [T, 512] and [T, 64], rows kv_c_stride_tok /
 *                k_pe_stride_tok apart.
 *   slot_mapping int64 [T], device.
 *   q_out        bf16 [T, H, 576], heads dense, rows q_out_stride_tok apart
 *                (>= H * 576); must not overlap any input.
 *   kv_cache     bf16 [num_slots, 576] (num_blocks * block_size rows); two
 *                tokens must not share a slot.
 * Every pointer is 16-byte aligned and every stride a multiple of 8
 * elements, else DCP_ERR_MISALIGNED.  T == 0 returns DCP_OK without
 * launching anything.
 */
dcp_status_t dcp_decode_concat_cache(
    const void* ql_nope, int64_t ql_nope_stride_tok, int64_t ql_nope_stride_head,
    const void* q_pe, int64_t q_pe_stride_tok, int64_t q_pe_stride_head,
    const void* kv_c, int64_t kv_c_stride_tok,
    const void* k_pe, int64_t k_pe_stride_tok,
    const int64_t* slot_mapping, int32_t T, int32_t H,
    void* q_out, int64_t q_out_stride_tok,
    void* kv_cache, int64_t num_slots,
    int32_t* dev_error, void* stream);

/*
 * dcp_mla_decode_partial without a workspace argument, for callers that
 * cannot allocate device memory (their memory is owned and fully reserved by
 * a host framework, or they are plugins handed only their inputs and
 * outputs).  The pages have no counterpart: it is a packaging of the same
 * decode.
 *
 * Same arguments, results and errors as dcp_mla_decode_partial, except that
 * the split-KV scratch comes from a 24 MiB array inside the library (held on
 * every device that loads it, until the process exits).  A call whose split
 * plan needs more than 24 MiB (dcp_decode_workspace_size) returns
 * DCP_ERR_WORKSPACE_TOO_SMALL without launching; H <= 128 always fits on a
 * GB300.  The first call on a device looks up the array's device address, so
 * make it before capturing a stream on that device.  All calls share the
 * array and it keeps the last call's contents (nothing in it needs to start
 * at zero); calls whose kernels overlap on the GPU race on it, so order them
 * on one stream or with events.  Allocates nothing.
 */
dcp_status_t dcp_mla_decode_partial_noalloc(
    const void* q, int64_t q_stride_tok,
    const void* kv_cache, int32_t num_blocks, int32_t block_size,
    const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len,
    int32_t D, int32_t interleave, float scale,
    float* O_part, float* lse_part,
    int32_t* dev_error, void* stream);

/*
 * The general form of dcp_decode_concat_cache: the latent rows are written
 * into a bf16 or an FP8 E4M3 cache, with the decode query or without it (a
 * prefill's tokens) ["perf(mla): fuse K3 DCP verification queries", review
 * follow-up: fp8 KV verify plans].
 *
 *   kv_dtype     DCP_KV_BF16: kv_cache bf16 [num_slots, 576], kv_scale is not
 *                used.  DCP_KV_FP8_E4M3: kv_cache uint8 codes [num_slots, 576]
 *                and kv_scale fp32 [num_slots] (required, else
 *                DCP_ERR_INVALID_ARG).  Other values: DCP_ERR_UNSUPPORTED_DTYPE.
 *                A written slot gets, from its row x = [kv_c | k_pe],
 *                  scale = 2^e, the least power of two with
 *                          max |x_i| <= 256 * scale (over the finite x_i; 1
 *                          when they are all zero),
 *                  code_i = x_i / scale rounded to the nearest E4M3 value,
 *                          ties to even (x_i / scale is exact); NaN and
 *                          infinities give the NaN code.
 *                Scales that are powers of two make the decode's widening to
 *                bf16 exact.
 *   H            0 writes the cache alone; then ql_nope, q_pe and q_out must
 *                be NULL and their strides are not used.
 * Everything else as for dcp_decode_concat_cache.
 */
dcp_status_t dcp_decode_concat_cache_v2(
    const void* ql_nope, int64_t ql_nope_stride_tok, int64_t ql_nope_stride_head,
    const void* q_pe, int64_t q_pe_stride_tok, int64_t q_pe_stride_head,
    const void* kv_c, int64_t kv_c_stride_tok,
    const void* k_pe, int64_t k_pe_stride_tok,
    const int64_t* slot_mapping, int32_t T, int32_t H,
    void* q_out, int64_t q_out_stride_tok,
    void* kv_cache, dcp_kv_dtype_t kv_dtype, float* kv_scale, int64_t num_slots,
    int32_t* dev_error, void* stream);

/*
 * Reads context ranges of the requests back out of the paged cache, as dense
 * rows: what a prefill over a cached prefix attends to, or what moves to
 * another cache.  (The pages' prefill side gathers its context this way; its
 * form is not on them.)
 *
 * For request b and cu_lens[b] <= n < cu_lens[b + 1], output row n is the
 * latent row of position p = seq_starts[b] + n - cu_lens[b]:
 *   out[n, 0:576] = kv(p)   (bf16 cache: a copy, or widened to fp32;
 *                            fp8 cache: code x scale in fp32, rounded to
 *                            nearest even for a bf16 output)
 * with kv(p) found as in the decode.  Rows of positions that shards outside
 * [shard_begin, shard_begin + shard_count) own are zeros, so that the outputs
 * of DCP ranks add up to the whole.  Output rows before cu_lens[0] or from
 * cu_lens[B] on are left as they are.  A position that has no table column, a
 * negative one, or a block id outside the cache gives a zero row and sets
 * DCP_DEVERR_BAD_BLOCK in *dev_error.
 *
 *   kv_cache, kv_dtype, kv_scale, num_blocks, block_size, block_table,
 *   bt_width, bt_stride, per_shard_tables, bt_shard_stride, D, interleave,
 *   shard_begin, shard_count
 *                as for dcp_mla_decode_partial_v2.
 *   seq_starts   int32 [B], first position of each request's range; NULL: 0.
 *   cu_lens      int32 [B + 1], non-decreasing: output row offsets.
 *   B, N         requests, and rows of `out` (cu_lens[B] <= N; rows past N
 *                are not written).
 *   out          bf16 or fp32 [N, 576], rows out_stride elements apart
 *                (>= 576, whole 16-byte units), 16-byte aligned; must not
 *                overlap the cache.
 * B == 0 or N == 0 returns DCP_OK without launching anything.
 */
dcp_status_t dcp_latent_cache_read(
    const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
    int32_t num_blocks, int32_t block_size,
    const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride,
    int32_t D, int32_t interleave, int32_t shard_begin, int32_t shard_count,
    const int32_t* seq_starts, const int32_t* cu_lens, int32_t B, int64_t N,
    void* out, dcp_dtype_t out_dtype, int64_t out_stride,
    int32_t* dev_error, void* stream);

/*
 * The decode over a sliding window and the first tokens of the context (a
 * window layer whose "sink" tokens stay visible): dcp_mla_decode_partial_v2
 * with, for row i of a request and its own context length
 * L = max(0, seq_len - (q_len - 1 - i)),
 *   S = { p < L : (p < num_sinks or p >= L - window), shard(p) == d }.
 * (The pages decode over the whole context; this form is for models whose
 * layers do not.)
 *
 *   window      last tokens of its context, itself included, that a row sees;
 *               0: all of them (then num_sinks has no effect).
 *   num_sinks   first tokens of the context that it sees besides.
 *               Negative values: DCP_ERR_INVALID_ARG.
 *   max_q_len   rows of a request past max_q_len get -inf / 0 (and set
 *               DCP_DEVERR_BAD_ROWS).  It sizes the launch: pass the step's
 *               largest verification width, not a loose bound.
 *   workspace   >= dcp_decode_select_workspace_size(...) bytes.
 * Only blocks that hold a visible token of some row are read: table entries of
 * blocks that have left every window may hold anything.  Split partials in
 * the workspace are fp32 for every o_dtype.  Everything else as for
 * dcp_mla_decode_partial_v2.
 *
 * Numbers: with H <= 128 (and D * interleave and the cache's rows below 2^31)
 * the tensor cores take each softmax weight rounded to bf16, for an fp32 output
 * too, while their sum and everything else is fp32: an output is off by at most
 * 2^-8 max|v| over the visible values, besides fp32 sums.  A bf16 output is
 * rounded once more, by 2^-8 of itself at most.  An FP8 code times a scale that
 * is no power of two is rounded to bf16 there.  A NaN score gives a NaN lse_part
 * and NaN outputs.
 *
 * Padding: many rows past query_start_loc[B] cost time, since few units of work
 * write them (255 of 256 rows at 128 heads: 647 us; the same rows as requests of
 * no tokens: 62 us).
 */
dcp_status_t dcp_mla_decode_partial_window(
    const void* q, int64_t q_stride_tok,
    const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
    int32_t num_blocks, int32_t block_size,
    const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride, int32_t shard_begin, int32_t shard_count,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len,
    int32_t D, int32_t interleave, float scale,
    int32_t window, int32_t num_sinks,
    void* O_part, dcp_dtype_t o_dtype, float* lse_part,
    void* workspace, size_t workspace_bytes,
    int32_t* dev_error, void* stream);

/*
 * The decode of a tree of drafted tokens (tree-shaped speculation; the pages
 * verify a chain, [PR565] Summary).  A request's q_len rows are its tree
 * tokens: row k sits at position seq_len - q_len + k of the cache (written
 * before the call, like a chain's) and sees the context before the tree, the
 * first seq_len - q_len positions, and those rows k' of its request whose bit
 * is set in its mask row: its ancestors, and itself where its own bit is set.
 *   own sequence of row r, n tokens in order:
 *       p = 0 .. seq_len - q_len - 1, then the set bits k' in increasing order
 *       at positions seq_len - q_len + k' (those >= 0)
 *   S = { the tokens of rank < num_sinks or >= n - window : shard(p) == d }
 * (window 0: all of them).  An empty mask row sees the context alone; a row
 * with nothing to see gives -inf / 0.
 *
 *   tree_mask    uint64 device words, 8-byte aligned: bit k' % 64 of word
 *                tree_mask[r * mask_stride + k' / 64], r the query row (of
 *                all T).  Bits at or past the request's q_len are ignored.
 *                Rows past query_start_loc[B] are not read.
 *   mask_stride  words between rows, >= ceil(max_q_len / 64), else
 *                DCP_ERR_INVALID_ARG.
 *   max_q_len    <= DCP_MAX_TREE_ROWS, else DCP_ERR_INVALID_ARG.
 * Everything else as for dcp_mla_decode_partial_window.
 */
dcp_status_t dcp_mla_decode_partial_tree(
    const void* q, int64_t q_stride_tok,
    const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
    int32_t num_blocks, int32_t block_size,
    const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride, int32_t shard_begin, int32_t shard_count,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int32_t max_seq_len, int32_t max_q_len,
    int32_t D, int32_t interleave, float scale,
    const uint64_t* tree_mask, int64_t mask_stride,
    int32_t window, int32_t num_sinks,
    void* O_part, dcp_dtype_t o_dtype, float* lse_part,
    void* workspace, size_t workspace_bytes,
    int32_t* dev_error, void* stream);

/*
 * Bytes of device workspace the windowed and tree decodes need for these
 * sizes on the CURRENT device: enough for every interleave and for every
 * shard_count up to D.  Returns (size_t)-1 on invalid arguments.
 */
size_t dcp_decode_select_workspace_size(int32_t B, int32_t T, int32_t H, int32_t D,
                                        int32_t max_seq_len, int32_t max_q_len,
                                        int32_t window, int32_t num_sinks);

/*
 * Block tables and slot maps of a step, built on the GPU from the requests'
 * lengths: takes the blocks that the step's new tokens need from a free list,
 * enters them in the requests' tables and gives every query row its position
 * and cache slot.  (The pages take tables and slot_mapping as given; each DCP
 * rank's holds its own tokens, [PRHUB] implementation step 3.)
 *
 * Request b has seq_lens[b] tokens after the step, the last q_len = qsl[b+1] -
 * qsl[b] of them new.  Its table (per_shard_tables: each of its shards' tables,
 * over the shard's local tokens, dcp_local_len) holds the blocks of the others
 * and gets columns [ceil(len(old) / block_size), ceil(len(seq) / block_size)),
 * old = max(0, seq_lens[b] - q_len).  New entry k, counted from 0 over
 * requests, then shards, then columns, is free_blocks[free_count - 1 - k].  All
 * other entries are left as they are.  A request of no tokens takes nothing.
 *   - Out of free blocks: the entries are -1 and DCP_DEVERR_NO_BLOCKS is set.
 *   - Columns at or past bt_width are not taken (DCP_DEVERR_SEQ_TOO_LONG).
 *   - A step after rejected drafts has fewer old tokens than the table has blocks
 *     for: the columns past them are taken anew, and what they held is lost to the
 *     free list unless the caller puts it back.  dcp_cache_extend_v2 counts them.
 * Row i of a request is the token at position p = seq_lens[b] - q_len + i:
 *   positions[r] = p, slot_mapping[r] = entry(p) * block_size + offset(p)
 * slot_mapping -1 where the entry is negative or missing, or a shard outside
 * [shard_begin, shard_begin + shard_count) owns the token; both -1 for rows of
 * no request, of a request of no tokens, and before position 0.
 *
 *   block_table  in/out, as for dcp_mla_decode_partial_v2; a width of 2^20 at
 *                most.
 *   seq_lens, query_start_loc, B, T, D, interleave, shard_begin, shard_count
 *                as for dcp_mla_decode_partial_v2.
 *   free_blocks  int32 [num_free], a stack of block ids; free_count int32 [1],
 *                how many of them are left (clamped to [0, num_free]).  Blocks
 *                of finished requests go back by writing their ids from
 *                free_blocks[count] on and raising the count.
 *   free_left    int32 [1], how many are left afterwards; may be free_count.
 *                Calls that share a free list or tables follow one another (one
 *                stream, or events).
 *   positions    int32 [T]; slot_mapping int64 [T].
 */
dcp_status_t dcp_cache_extend(
    int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride,
    const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B, int32_t T, int32_t block_size,
    int32_t D, int32_t interleave, int32_t shard_begin, int32_t shard_count,
    const int32_t* free_blocks, int32_t num_free, const int32_t* free_count, int32_t* free_left,
    int32_t* positions, int64_t* slot_mapping,
    int32_t* dev_error, void* stream);

/*
 * dcp_cache_extend with a count of the blocks that each table holds, for steps
 * of speculative verification, whose drafts may be rejected, and for a free list
 * that may run out.
 *
 *   held  in/out int32 [B] (per_shard_tables: [shard_count, B]), dense, or NULL
 *         (as dcp_cache_extend): the leading columns of a table that hold a
 *         block; 0 for a new request, whatever its table's row held before.  A
 *         request gets columns [held, ceil(len(seq) / block_size)), and held
 *         becomes that end, or the first column without a block where the free
 *         list ran out (the next step takes that column again).  Where the
 *         tokens need fewer columns, none is taken and held stays: a block that a
 *         rejected draft reached into is used by the next one.  The blocks of a
 *         finished request are its first `held` columns.
 */
dcp_status_t dcp_cache_extend_v2(
    int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride,
    const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B, int32_t T, int32_t block_size,
    int32_t D, int32_t interleave, int32_t shard_begin, int32_t shard_count,
    const int32_t* free_blocks, int32_t num_free, const int32_t* free_count, int32_t* free_left,
    int32_t* held,
    int32_t* positions, int64_t* slot_mapping,
    int32_t* dev_error, void* stream);

/*
 * dcp_decode_concat_cache_v2 from the projections' outputs: the latent's norm
 * and the rotation of the rope parts by their positions in the same launch
 * ([PRHUB], key snippet "Decode: latent multi-query attention":
 * _decode_concat_cache with rope_positions).
 *
 *   c    = kv_c * norm_weight / sqrt(mean(kv_c^2) + eps)   (512 dims; norm_weight
 *          NULL: kv_c as it is)
 *   rot  turns pairs (x, y) of a rope part by its token's angles:
 *          (x cos_i - y sin_i, y cos_i + x sin_i), i < 32; pairs are dims
 *          (2i, 2i + 1) if interleaved, else (i, i + 32).
 *   cache row of slot_mapping[t] = [c | rot(k_pe)], q_out = [ql_nope | rot(q_pe)].
 * Computed in fp32 and rounded once: to bf16 (nearest even), or for an FP8
 * cache to the codes of dcp_decode_concat_cache_v2 (scale 2^e with e >= -126)
 * straight from the fp32 values.  (Squares that overflow fp32 give a norm of
 * infinity: a row of zeros and NaN.)
 *
 *   ql_nope      bf16 [T, H, 512], or NULL: q_out gets the rotated rope parts
 *                alone (a chunk's queries, whose other part stays where it is).
 *   q_pe, q_out  bf16 [T, H, 64] and [T, H, 576] (64 without ql_nope); token and
 *                head strides of any order, outputs not overlapping.  Without
 *                ql_nope q_out may be q_pe itself, with the same strides.
 *   H            0: no query; ql_nope, q_pe and q_out NULL.
 *   positions    int32 [T].  Negative: rope parts are not turned (padding
 *                rows).  max_pos or more: likewise, and
 *                DCP_DEVERR_BAD_POSITION is set.
 *   cos_sin      fp32 [max_pos, 64]: a position's 32 cosines, then its 32 sines.
 * Everything else as for dcp_decode_concat_cache_v2 (16-byte alignment,
 * norm_weight bf16 [512] and cos_sin included).
 */
dcp_status_t dcp_norm_rope_cache(
    const void* ql_nope, int64_t ql_nope_stride_tok, int64_t ql_nope_stride_head,
    const void* q_pe, int64_t q_pe_stride_tok, int64_t q_pe_stride_head,
    void* q_out, int64_t q_out_stride_tok, int64_t q_out_stride_head,
    const void* kv_c, int64_t kv_c_stride_tok,
    const void* k_pe, int64_t k_pe_stride_tok,
    const void* norm_weight, float eps,
    const int32_t* positions, const float* cos_sin, int32_t max_pos, int32_t interleaved,
    const int64_t* slot_mapping, int32_t T, int32_t H,
    void* kv_cache, dcp_kv_dtype_t kv_dtype, float* kv_scale, int64_t num_slots,
    int32_t* dev_error, void* stream);

/*
 * The up projection's weight in the order in which dcp_mla_chunk_attention
 * reads it, laid out once per layer.
 *   w_kv_b  bf16 [H * 256, 512], a head's 128 key rows before its 128 value rows.
 *   packed  the same number of bytes; must not overlap w_kv_b.
 */
dcp_status_t dcp_pack_kv_b(const void* w_kv_b, int32_t H, void* packed, void* stream);

/*
 * Causal attention of chunks of new tokens over the paged latent cache (a
 * prefill over a cached prefix, a prompt's chunks, decoding rows among them),
 * with each head's own keys and values projected up from the latents (the
 * pages' prefill side; the decodes work on the latents themselves and return
 * 512 latent dims).
 *
 * Row i of request b sees L = max(0, seq_lens[b] - (q_len - 1 - i)) tokens, as
 * in dcp_mla_decode_partial (the new tokens are already in the cache):
 *   k_h(p) = [W_h[0:128] c(p) | kv(p)[512:576]],  v_h(p) = W_h[128:256] c(p),
 *   c(p) = kv(p)[0:512],  s_p = scale * sum_{k<192} q[r,h,k] * k_h(p)[k]
 *   lse[r,h] = ln sum_{p<L} exp(s_p),  out[r,h,:] = sum_{p<L} exp(s_p - lse[r,h]) v_h(p)
 * A row with nothing to see, of no request or of a request of no tokens: 0 and
 * -inf.  Whole contexts: per-shard tables hold all D shards.  B == 0 or T == 0
 * returns DCP_OK without launching anything: the caller fills the rows of a step
 * without requests (the Python binding does).
 *
 *   q            bf16 [T, H, 192], 128 dims for W_h's keys, then 64 rope dims
 *                (rotated, dcp_norm_rope_cache); token and head strides in
 *                multiples of 8 elements.
 *   kv_cache .. query_start_loc, B, T, scale
 *                as for dcp_mla_decode_partial_v2 (D and interleave matter for
 *                per-shard tables only).  A token without a table column or with
 *                a block id outside the cache is skipped (DCP_DEVERR_BAD_BLOCK).
 *   H            1 .. 1024.
 *   total_len    host-known bound of the sum of seq_lens (sizes the workspace; a
 *                loose one costs workspace, and passes once that is 4 GiB).
 *                Requests past it see nothing (DCP_DEVERR_SEQ_TOO_LONG).
 *   packed_kv_b  from dcp_pack_kv_b.
 *   out          bf16 (round to nearest even) or fp32 [T, H, 128], dense,
 *                16-byte aligned; lse fp32 [T, H].
 *   workspace    16-byte aligned; its contents on entry are ignored.
 *                dcp_chunk_attention_workspace_size(...) bytes hold what the
 *                heads share (16 KB per 128 tokens), keys and values of as many
 *                heads as fit in 4 GiB (one at least; 64 KB per 128 tokens each)
 *                and the outputs of cut units; the call makes as many passes
 *                over the heads as that takes.  With less, down to one head's
 *                part, it makes more.
 *                Calls that may overlap need one each.
 *
 * Numbers: values, and keys of requests of more than 1,024 tokens, are rounded
 * to f16 once (f16's steps are 2^-24 below 2^-14), and so are the softmax weights
 * (relative to a running maximum).  A key's rounding shifts its score by at most
 * 2^-11 scale sum |q k|, ~2e-4 as a rule, and the log-sum-exp of a row that sees
 * little but that token by as much; of a row whose weight is spread over n tokens,
 * by that over the root of n.  Requests of up to 1,024 tokens keep keys to 22 bits.
 * Queries are f16 after a power of 2 that brings a row's largest element to 1 to 4;
 * everything else is fp32.  An FP8 code times a scale that is no power of two is
 * rounded to bf16.  A NaN score makes the rows that see its token NaN, and no
 * others; so does a projected key or value with an element that is not finite or
 * past f16's largest, 65,504.  (An infinite rope element makes its token's scores
 * what the arithmetic makes them: NaN or +inf, and the row NaN, or -inf, and the
 * token weighs nothing.)  A row whose largest score is past 2.3e7 in magnitude (fp32 keeps
 * no digit behind the point there; -inf too) is NaN; scores that far below the
 * largest weigh nothing.
 *
 * Cost: 640 operations per row, token and head and 262,144 per token and head,
 * against 2,176 per row, token and head of the decodes: below ~170 rows of a
 * request a decode with absorbed queries does less work.
 */
dcp_status_t dcp_mla_chunk_attention(
    const void* q, int64_t q_stride_tok, int64_t q_stride_head,
    const void* kv_cache, dcp_kv_dtype_t kv_dtype, const float* kv_scale,
    int32_t num_blocks, int32_t block_size,
    const int32_t* block_table, int32_t bt_width, int64_t bt_stride,
    int32_t per_shard_tables, int64_t bt_shard_stride, int32_t D, int32_t interleave,
    const int32_t* seq_lens, const int32_t* query_start_loc,
    int32_t B, int32_t T, int32_t H, int64_t total_len, float scale,
    const void* packed_kv_b,
    void* out, dcp_dtype_t out_dtype, float* lse,
    void* workspace, size_t workspace_bytes,
    int32_t* dev_error, void* stream);

/*
 * Bytes of workspace for dcp_mla_chunk_attention; (size_t)-1 on invalid
 * arguments.
 */
size_t dcp_chunk_attention_workspace_size(int32_t B, int32_t T, int32_t H, int64_t total_len);

#ifdef __cplusplus
}
#endif

#endif /* DCP_H_ */
