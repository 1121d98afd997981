// C ABI of the operators around a paged K/V cache (rotary positions, append,
// route-set and positional attention of new tokens): host-side argument checks,
// workspace layout and launch sequences.  Nothing here reads device memory or
// synchronises; every launch goes to the caller's stream.
#include <climits>
#include <cmath>
#include <cstdint>

#include "qsa.h"
#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace {

constexpr int kMaxSel = 16384;
constexpr int kMinPage = 16;
constexpr int kMaxSeqs = 1 << 30;                // the searches over B step past it in 32 bits
constexpr int64_t kMaxLen = int64_t{1} << 30;  // positions that a block table can name
// Heads of a token that the rotation and the append take: their kernels count its 16 units a head, and
// up to 1024 behind them, in 32 bits.
constexpr int64_t kMaxRotaryHeads = (INT32_MAX - 1024) / 16;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

#define QSA_TRY(expr)                           \
  do {                                          \
    cudaError_t e_ = (expr);                    \
    if (e_ != cudaSuccess) return QSA_ERR_CUDA; \
  } while (0)

qsa_status_t check_heads(int64_t T, int H, int G) {
  if (T < 1 || T > (int64_t{1} << 30) || H < 1 || G < 1) return QSA_ERR_INVALID_ARGUMENT;
  if (H % G != 0 || H / G != qsa::kHeadsPerGroup) return QSA_ERR_UNSUPPORTED;
  if (T > INT32_MAX / H) return QSA_ERR_INVALID_ARGUMENT;
  return QSA_OK;
}

qsa_status_t check_cache(int B, int64_t n_pages, int page_size, int64_t max_pages) {
  if (B < 1 || B > kMaxSeqs || n_pages < 1 || page_size < 1 || max_pages < 1) return QSA_ERR_INVALID_ARGUMENT;
  if (page_size < kMinPage || (page_size & (page_size - 1)) != 0) return QSA_ERR_UNSUPPORTED;
  if (n_pages > INT32_MAX / page_size || max_pages > kMaxLen / page_size) return QSA_ERR_INVALID_ARGUMENT;
  return QSA_OK;
}

qsa::CacheView view(const int32_t* table, const int32_t* kv_len, const int32_t* cu_q, int B, int64_t n_pages,
                    int page_size, int64_t max_pages) {
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  return {table, kv_len, cu_q, B, static_cast<int>(max_pages), static_cast<int>(n_pages), shift};
}

// One [T, heads, 256] operand with element strides between tokens and heads (its
// span in bytes fits 63 bits).
qsa_status_t check_rows(const void* p, int64_t ts, int64_t hs, int64_t T, int heads) {
  if (!p || ts < 0 || hs < 0 || ts > (int64_t{1} << 60) / T || hs > (int64_t{1} << 60) / heads)
    return QSA_ERR_INVALID_ARGUMENT;
  if (!aligned(p, 16) || ts % 8 != 0 || hs % 8 != 0) return QSA_ERR_MISALIGNED;
  return QSA_OK;
}
// Output rows: as check_rows, and no two rows share an element; they are either
// the input's own rows or overlap the span of none of them.
qsa_status_t check_out_rows(const void* o, int64_t ots, int64_t ohs, const void* x, int64_t ts, int64_t hs, int64_t T,
                            int heads) {
  const qsa_status_t st = check_rows(o, ots, ohs, T, heads);
  if (st != QSA_OK) return st;
  const int64_t d = qsa::kHeadDim;
  const bool heads_inside = heads == 1 || (ohs >= d && (T == 1 || ots >= (heads - 1) * ohs + d));
  const bool tokens_inside = T == 1 || (ots >= d && (heads == 1 || ohs >= (T - 1) * ots + d));
  if (!heads_inside && !tokens_inside) return QSA_ERR_INVALID_ARGUMENT;
  if (o == x && (T == 1 || ots == ts) && (heads == 1 || ohs == hs)) return QSA_OK;
  const uintptr_t o0 = reinterpret_cast<uintptr_t>(o), x0 = reinterpret_cast<uintptr_t>(x);
  const uintptr_t o1 = o0 + 2 * static_cast<uintptr_t>((T - 1) * ots + (heads - 1) * ohs + d);
  const uintptr_t x1 = x0 + 2 * static_cast<uintptr_t>((T - 1) * ts + (heads - 1) * hs + d);
  return o0 < x1 && x0 < o1 ? QSA_ERR_INVALID_ARGUMENT : QSA_OK;
}

qsa_status_t check_rotary(const double* inv_freq, int rot, float mscale) {
  if (!inv_freq || rot < 1 || !(mscale > 0.f) || !std::isfinite(mscale)) return QSA_ERR_INVALID_ARGUMENT;
  if (rot > qsa::kHeadDim || rot % 16 != 0) return QSA_ERR_UNSUPPORTED;
  return aligned(inv_freq, 8) ? QSA_OK : QSA_ERR_MISALIGNED;
}

#define QSA_CHECK(expr)                     \
  do {                                      \
    const qsa_status_t st_ = (expr);        \
    if (st_ != QSA_OK) return st_;          \
  } while (0)

struct PagedLayout {
  size_t status = 0, row_cnt = 0, row_cols = 0, partial = 0, total = 0;
  int splits = 1;
};
PagedLayout paged_layout(int64_t T, int G, int n_sel) {
  PagedLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  L.splits = qsa::paged_splits(T, G, n_sel);
  L.status = take(4);
  L.row_cnt = take(static_cast<size_t>(T) * 4);
  L.row_cols = take(static_cast<size_t>(T) * n_sel * 4);
  L.partial = take(qsa::paged_partial_bytes(T, G, L.splits));
  L.total = off;
  return L;
}

qsa_status_t check_paged(int64_t T, int H, int G, int n_sel, int page_size, int64_t max_pages) {
  QSA_CHECK(check_heads(T, H, G));
  if (n_sel < 1 || n_sel > kMaxSel || T > INT32_MAX / n_sel) return QSA_ERR_INVALID_ARGUMENT;
  return check_cache(1, 1, page_size, max_pages);
}

template <typename P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<uint8_t*>(ws) + off);
}

}  // namespace

extern "C" {

qsa_status_t qsa_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                      int64_t k_token_stride, int64_t k_head_stride, void* q_out, int64_t q_out_token_stride,
                      int64_t q_out_head_stride, void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                      const int32_t* positions, const double* inv_freq, int64_t T, int H, int G, int rotary_dim,
                      int interleaved, float mscale, int backward, qsa_stream_t stream) {
  if (!positions || T < 1 || T > (int64_t{1} << 30) || H < 1 || G < 0) return QSA_ERR_INVALID_ARGUMENT;
  const int64_t heads = static_cast<int64_t>(H) + G;
  if (T > INT32_MAX / heads || heads > kMaxRotaryHeads) return QSA_ERR_INVALID_ARGUMENT;
  QSA_CHECK(check_rotary(inv_freq, rotary_dim, mscale));
  QSA_CHECK(check_rows(q, q_token_stride, q_head_stride, T, H));
  QSA_CHECK(check_out_rows(q_out, q_out_token_stride, q_out_head_stride, q, q_token_stride, q_head_stride, T, H));
  if (G > 0) {
    QSA_CHECK(check_rows(k, k_token_stride, k_head_stride, T, G));
    QSA_CHECK(check_out_rows(k_out, k_out_token_stride, k_out_head_stride, k, k_token_stride, k_head_stride, T, G));
  }
  if (!aligned(positions, 4)) return QSA_ERR_MISALIGNED;
  QSA_TRY(qsa::launch_rope({q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride},
                           {q_out, q_out_token_stride, q_out_head_stride},
                           {k_out, k_out_token_stride, k_out_head_stride}, positions, inv_freq, T, H, G, rotary_dim,
                           interleaved != 0, mscale, backward != 0, reinterpret_cast<cudaStream_t>(stream)));
  return QSA_OK;
}

qsa_status_t qsa_cache_append(const void* k_new, int64_t k_token_stride, int64_t k_head_stride, const void* v_new,
                              int64_t v_token_stride, int64_t v_head_stride, const void* q, int64_t q_token_stride,
                              int64_t q_head_stride, void* q_out, int64_t q_out_token_stride,
                              int64_t q_out_head_stride, const double* inv_freq, int rotary_dim, int interleaved,
                              float mscale, void* k_pages, void* v_pages, const int32_t* block_table,
                              const int32_t* kv_len, const int32_t* cu_q, int64_t T, int B, int64_t n_pages,
                              int page_size, int64_t max_pages, int H, int G, qsa_stream_t stream) {
  if (!k_pages || !v_pages || k_pages == v_pages || !block_table || !kv_len || !cu_q) return QSA_ERR_INVALID_ARGUMENT;
  QSA_CHECK(check_heads(T, H, G));
  if (H + 2 * static_cast<int64_t>(G) > kMaxRotaryHeads) return QSA_ERR_INVALID_ARGUMENT;
  QSA_CHECK(check_cache(B, n_pages, page_size, max_pages));
  if (inv_freq) QSA_CHECK(check_rotary(inv_freq, rotary_dim, mscale));
  QSA_CHECK(check_rows(k_new, k_token_stride, k_head_stride, T, G));
  QSA_CHECK(check_rows(v_new, v_token_stride, v_head_stride, T, G));
  if (q) {
    if (!inv_freq) return QSA_ERR_INVALID_ARGUMENT;  // q is taken to be rotated
    QSA_CHECK(check_rows(q, q_token_stride, q_head_stride, T, H));
    QSA_CHECK(check_out_rows(q_out, q_out_token_stride, q_out_head_stride, q, q_token_stride, q_head_stride, T, H));
  }
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(block_table, 4) || !aligned(kv_len, 4) ||
      !aligned(cu_q, 4))
    return QSA_ERR_MISALIGNED;
  QSA_TRY(qsa::launch_cache_append({q, q_token_stride, q_head_stride}, {k_new, k_token_stride, k_head_stride},
                                   {v_new, v_token_stride, v_head_stride},
                                   {q_out, q_out_token_stride, q_out_head_stride}, k_pages, v_pages,
                                   view(block_table, kv_len, cu_q, B, n_pages, page_size, max_pages), inv_freq, T,
                                   q ? H : 0, G, inv_freq ? rotary_dim : 0, interleaved != 0, mscale,
                                   reinterpret_cast<cudaStream_t>(stream)));
  return QSA_OK;
}

size_t qsa_paged_forward_workspace_size(int64_t T, int H, int G, int n_sel, int page_size, int64_t max_pages) {
  if (check_paged(T, H, G, n_sel, page_size, max_pages) != QSA_OK) return 0;
  return paged_layout(T, G, n_sel).total;
}

qsa_status_t qsa_paged_forward(const void* q, const void* k_pages, const void* v_pages, const int32_t* routes,
                               const int32_t* block_table, const int32_t* kv_len, const int32_t* cu_q, int64_t T,
                               int B, int64_t n_pages, int page_size, int64_t max_pages, int H, int G, int n_sel,
                               float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                               qsa_stream_t stream) {
  if (!q || !k_pages || !v_pages || !routes || !block_table || !kv_len || !cu_q || !out || !lse || !workspace)
    return QSA_ERR_INVALID_ARGUMENT;
  QSA_CHECK(check_paged(T, H, G, n_sel, page_size, max_pages));
  QSA_CHECK(check_cache(B, n_pages, page_size, max_pages));
  if (!(scale > 0.f) || !std::isfinite(scale)) return QSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(routes, 4) ||
      !aligned(block_table, 4) || !aligned(kv_len, 4) || !aligned(cu_q, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 256))
    return QSA_ERR_MISALIGNED;
  const PagedLayout L = paged_layout(T, G, n_sel);
  if (workspace_bytes < L.total) return QSA_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t* row_cnt = at<int32_t>(workspace, L.row_cnt);
  int32_t* row_cols = at<int32_t>(workspace, L.row_cols);
  QSA_TRY(qsa::launch_paged_rows(routes, view(block_table, kv_len, cu_q, B, n_pages, page_size, max_pages), T, n_sel,
                                 at<int>(workspace, L.status), row_cnt, row_cols, s));
  QSA_TRY(qsa::launch_paged_forward(q, k_pages, v_pages, row_cnt, row_cols, T, G, n_sel, scale, L.splits,
                                    at<void>(workspace, L.partial), out, lse, s));
  return QSA_OK;
}

size_t qsa_paged_causal_workspace_size(int64_t T, int H, int G, int page_size, int64_t max_pages, int window,
                                       int sinks) {
  if (check_heads(T, H, G) != QSA_OK || check_cache(1, 1, page_size, max_pages) != QSA_OK || window < 0 || sinks < 0)
    return 0;
  return 256 + align256(qsa::causal_scratch_bytes());
}

qsa_status_t qsa_paged_causal(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                              const int32_t* kv_len, const int32_t* cu_q, int64_t T, int B, int64_t n_pages,
                              int page_size, int64_t max_pages, int H, int G, int window, int sinks, float scale,
                              void* out, float* lse, void* workspace, size_t workspace_bytes, qsa_stream_t stream) {
  if (!q || !k_pages || !v_pages || !block_table || !kv_len || !cu_q || !out || !lse || !workspace)
    return QSA_ERR_INVALID_ARGUMENT;
  QSA_CHECK(check_heads(T, H, G));
  QSA_CHECK(check_cache(B, n_pages, page_size, max_pages));
  if (window < 0 || sinks < 0 || !(scale > 0.f) || !std::isfinite(scale)) return QSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(kv_len, 4) || !aligned(cu_q, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 256))
    return QSA_ERR_MISALIGNED;
  if (workspace_bytes < qsa_paged_causal_workspace_size(T, H, G, page_size, max_pages, window, sinks))
    return QSA_ERR_WORKSPACE_TOO_SMALL;
  QSA_TRY(qsa::launch_paged_causal(q, k_pages, v_pages,
                                   view(block_table, kv_len, cu_q, B, n_pages, page_size, max_pages), T, G, window,
                                   sinks, scale, at<int>(workspace, 0), at<void>(workspace, 256), out, lse,
                                   reinterpret_cast<cudaStream_t>(stream)));
  return QSA_OK;
}

}  // extern "C"
