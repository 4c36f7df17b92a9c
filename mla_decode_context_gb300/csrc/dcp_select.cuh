// Row selection of the windowed and tree decodes: which tokens of a shard the
// rows of a request see.
//
// Row i of a q_len-row request has its own sequence of tokens, in order:
//   chain  the first L_i = seq_len - (q_len - 1 - i) positions;
//   tree   the prefix of P = max(0, seq_len - q_len) positions, then the tree
//          tokens k (position seq_len - q_len + k) whose bit is set in the
//          row's mask.
// Without a window it sees all of them; with one, the first `sinks` and the
// last `window` of them.
//
// The rows of a unit (one row, or a group of rows of one request that share
// their tiles) read the union of what they see, so a unit walks a dense index
// v over the shard's tokens j that any of its rows may see:
//   v in [0, vs)    the sinks below the window, j = v;
//   v in [vs, vb)   the window's stretch of the prefix, j = v + gap;
//   v in [vb, nv)   the tree tokens (tree only; a chain has vb = nv).
// A row then sees v < vb iff v < vend and (v < vs or v >= vlo), and a tree
// token iff its bit says so.  Everything is a shard-local count in closed
// form, so no index list is read or built, and tokens that have left every
// window are never touched (their blocks may be gone).
#pragma once

#include "dcp_kernels.h"

namespace dcp {

// The rows r0 .. r0 + n - 1 (i0, i0 + 1, .. of their request); n == 0: none.
struct SelRows {
  int32_t r0, n, b, i0, q_len, seq;
  uint32_t err;
};

// What the rows may see of shard d, as local counts.
struct SelSpan {
  int32_t vs, vb, nv, gap;
  __device__ __forceinline__ int32_t index_of(int32_t j) const {  // v of the first visible token at or after j
    return j <= vs ? j : max(vs, j - gap);
  }
  __device__ __forceinline__ int32_t token_of(int32_t v) const { return v < vs ? v : v + gap; }
};

// One row's part of the span's prefix.
struct SelRow {
  int32_t vlo, vend;
};

#ifdef __CUDACC__
// local_len and local_to_global with the launch's divisors: 64-bit divisions
// by runtime values took a quarter of a short unit's time (512 units of two
// tiles: 134 us with them, 102 us without).  kFast needs D x I < 2^31 (the
// tensor-core kernel); the CUDA-core kernel takes any.
template <bool kFast>
__device__ __forceinline__ int32_t sel_local_len(const DecodeArgs& a, int32_t L, int32_t d) {
  if constexpr (!kFast) return local_len(L, d, a.D, a.I);
  const int32_t q = fast_div(L, a.sel.div_period);
  const int32_t rem = L - q * static_cast<int32_t>(a.sel.div_period.d) - d * a.I;
  return q * a.I + min(max(rem, 0), a.I);
}
template <bool kFast>
__device__ __forceinline__ int32_t sel_position(const DecodeArgs& a, int32_t j, int32_t d) {
  if constexpr (!kFast) return static_cast<int32_t>(local_to_global(j, d, a.D, a.I));
  const int32_t q = fast_div(j, a.div_I);
  return q * static_cast<int32_t>(a.sel.div_period.d) + d * a.I + (j - q * a.I);
}

__device__ __forceinline__ int32_t sel_prefix(const SelRows& R) { return max(0, R.seq - R.q_len); }

// Own length of chain row i.
__device__ __forceinline__ int32_t sel_chain_len(const SelRows& R, int32_t i) {
  return max(0, R.seq - (R.q_len - 1 - i));
}

template <bool kFast>
__device__ __forceinline__ SelSpan sel_span(const DecodeArgs& a, const SelRows& R, int32_t d) {
  const SelectArgs& s = a.sel;
  const bool tree = s.tree != nullptr;
  // the rows' prefix ends at P; no row's window starts before `start`
  const int32_t P = tree ? sel_prefix(R) : sel_chain_len(R, R.i0 + R.n - 1);
  const int32_t shortest = tree ? P : sel_chain_len(R, R.i0);
  const int32_t start = s.window > 0 ? max(0, shortest - s.window) : 0;
  const int32_t ns = sel_local_len<kFast>(a, min(s.sinks, P), d);
  const int32_t lo = s.window > 0 ? max(ns, sel_local_len<kFast>(a, start, d)) : ns;
  const int32_t nb = sel_local_len<kFast>(a, P, d);
  const int32_t ne = tree ? sel_local_len<kFast>(a, max(0, R.seq), d) : nb;
  return SelSpan{ns, nb - (lo - ns), ne - (lo - ns), lo - ns};
}

// Words of a row's mask that hold its request's rows, and word w with the bits
// past the request's rows, or of positions before the context, dropped.
__device__ __forceinline__ int32_t sel_words(const DecodeArgs& a, const SelRows& R) {
  return (min(R.q_len, a.max_q_len) + 63) / 64;
}
__device__ __forceinline__ unsigned long long sel_word(const DecodeArgs& a, const SelRows& R, int32_t i, int32_t w) {
  unsigned long long m = __ldg(a.sel.tree + static_cast<int64_t>(R.r0 - R.i0 + i) * a.sel.tree_stride + w);
  const int32_t hi = min(R.q_len, a.max_q_len) - 64 * w;  // bits below hi exist
  if (hi < 64) m &= (1ull << max(hi, 0)) - 1ull;
  const int32_t lo = R.q_len - R.seq - 64 * w;            // bits from lo on have a position >= 0
  if (lo > 0) m &= lo < 64 ? ~0ull << lo : 0ull;
  return m;
}

// Own length of tree row i: the prefix and its visible tree tokens.
__device__ __forceinline__ int32_t sel_tree_len(const DecodeArgs& a, const SelRows& R, int32_t i) {
  int32_t n = sel_prefix(R);
  for (int32_t w = 0; w < sel_words(a, R); ++w) n += __popcll(sel_word(a, R, i, w));
  return n;
}

// Row i's part of the prefix; len: its own length (chain or tree).
template <bool kFast>
__device__ __forceinline__ SelRow sel_row(const DecodeArgs& a, const SelRows& R, const SelSpan& S, int32_t i,
                                          int32_t len, int32_t d) {
  const int32_t P = a.sel.tree ? sel_prefix(R) : len;
  SelRow r;
  r.vend = a.sel.tree ? S.vb : S.index_of(sel_local_len<kFast>(a, P, d));
  r.vlo = a.sel.window > 0 ? S.index_of(sel_local_len<kFast>(a, min(max(0, len - a.sel.window), P), d)) : 0;
  return r;
}

// Whether tree row i of own length len sees tree token k.
__device__ __forceinline__ bool sel_tree_bit(const DecodeArgs& a, const SelRows& R, int32_t i, int32_t len, int32_t k) {
  if (k < 0 || k >= min(R.q_len, a.max_q_len)) return false;
  const unsigned long long m = sel_word(a, R, i, k >> 6);
  if (!((m >> (k & 63)) & 1ull)) return false;
  if (a.sel.window <= 0) return true;
  int32_t rank = sel_prefix(R) + __popcll(m & ((1ull << (k & 63)) - 1ull));
  for (int32_t w = 0; w < (k >> 6); ++w) rank += __popcll(sel_word(a, R, i, w));
  return rank < a.sel.sinks || rank >= len - a.sel.window;
}

// The one row r (rows past max_q_len of their request count as padding).
__device__ __forceinline__ SelRows sel_rows_of_row(const DecodeArgs& a, int32_t r) {
  SelRows R{r, 0, -1, 0, 0, 0, 0u};
  const RequestOfRow q = request_of_row(a.seq_lens, a.qsl, a.B, r, a.max_q_len);
  if (q.b < 0) return R;
  R.b = q.b;
  R.i0 = r - q.q0;
  R.q_len = q.q1 - q.q0;
  if (R.q_len > a.max_q_len) R.err |= DCP_DEVERR_BAD_ROWS;
  R.seq = q.seq;
  if (R.seq <= 0) return R;
  if (R.seq > a.max_seq_len) { R.err |= DCP_DEVERR_SEQ_TOO_LONG; R.seq = a.max_seq_len; }
  R.n = R.i0 < a.max_q_len ? 1 : 0;
  return R;
}

// Unit (b, c) of the tensor-core kernel: rows c * group .. of request b, the
// first max_q_len of the request at most.  n rows are written, live says
// whether they see anything at all; `extra` rows from extra0 on have no unit
// of their own and are written as padding (a request's rows past max_q_len by
// its last unit; b == B: the rows of no request, dealt to `chunks` units).
struct SelUnit {
  SelRows R;
  bool live;
  int32_t extra0, extra;
};
__device__ __forceinline__ SelUnit sel_unit(const DecodeArgs& a, int32_t b, int32_t c) {
  SelUnit U{};
  U.R.b = b;
  if (b >= a.B) {
    const int32_t first = min(max(__ldg(a.qsl), 0), a.T), last = min(max(__ldg(a.qsl + a.B), 0), a.T);
    // [0, first) before the first request and [last, T) after the last one,
    // as one list of first + T - last rows, an even share per unit
    const int32_t share = (first + a.T - last + a.sel.chunks - 1) / a.sel.chunks;
    const int32_t x0 = c * share, x1 = min(x0 + share, first + a.T - last);
    // (a share that straddles both parts: its first part here, the rest as rows of R)
    const int32_t h1 = min(x1, first);
    U.R.r0 = x0 < first ? x0 : 0;
    U.R.n = max(0, h1 - x0);
    const int32_t t0 = max(x0, first);
    U.extra0 = last + (t0 - first);
    U.extra = max(0, x1 - t0);
    return U;
  }
  const int32_t q0 = __ldg(a.qsl + b), q1 = __ldg(a.qsl + b + 1), seq = __ldg(a.seq_lens + b);
  SelRows& R = U.R;
  R.q_len = q1 - q0;
  R.i0 = c * a.sel.group;
  R.r0 = q0 + R.i0;
  if (R.q_len < 0 || q0 < 0 || q0 > a.T) {
    R.err |= DCP_DEVERR_BAD_ROWS;
    return U;
  }
  const int32_t rows = min(R.q_len, a.max_q_len);
  R.n = max(0, min(min(a.sel.group, rows - R.i0), a.T - R.r0));
  if (R.q_len > a.max_q_len) {
    R.err |= DCP_DEVERR_BAD_ROWS;
    if (c == a.sel.chunks - 1) {
      U.extra0 = q0 + rows;
      U.extra = max(0, min(q1, a.T) - U.extra0);
    }
  }
  R.seq = seq;
  if (seq > a.max_seq_len) { R.err |= DCP_DEVERR_SEQ_TOO_LONG; R.seq = a.max_seq_len; }
  U.live = seq > 0 && R.n > 0;
  return U;
}

// (request, group, shard - d0, split) of unit u: a request's groups innermost,
// so that they read each tile from L2 at the same time.
struct SelCoords {
  int32_t b, c, dd, s;
};
__device__ __forceinline__ SelCoords sel_coords(const DecodeArgs& a, int32_t u) {
  SelCoords k;
  const int32_t v = fast_div(u, a.sel.div_chunks), w = fast_div(v, a.sel.div_splits);
  k.c = u - v * a.sel.chunks;
  k.s = v - w * a.plan.splits;
  k.b = fast_div(w, a.sel.div_Dn);
  k.dd = w - k.b * a.Dn;
  return k;
}
#endif

}  // namespace dcp
