// C ABI of the library (declared in include/rfp2.h).  Every entry point checks
// its arguments on the host and returns a status before anything is enqueued;
// no HIP call is made for a rejected call.
#include <cmath>

#include "rfp2.h"
#include "rfp2_internal.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;     // row and token counts
constexpr int64_t kMaxGemvK = 32768;               // staged activations fit LDS
constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;  // pages and cached positions
constexpr int64_t kMaxSortSlots = int64_t(1) << 24;  // routed slots of one sort

bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

rfp2_status from_hip(hipError_t e) {
  return e == hipSuccess ? RFP2_OK : RFP2_E_LAUNCH;
}

bool product_k_ok(int64_t K) {
  return K >= 256 && K % 256 == 0 && K <= kMaxGemvK;
}

// A cache descriptor with everything the kernels index by in range; RFP2_OK and
// the kernels' view of it, or the status to return.
rfp2_status check_cache(const rfp2_kv_cache* c, rfp2::KvView* view) {
  if (!c) return RFP2_E_NULL;
  const bool i8 = c->format == RFP2_KV_I8;
  if (!i8 && c->format != RFP2_KV_F16) return RFP2_E_SHAPE;
  if (!c->k || !c->v || !c->page_table || (i8 && (!c->k_scale || !c->v_scale)))
    return RFP2_E_NULL;
  const int64_t P = c->page_size;
  if (c->kv_heads < 1 || c->kv_heads > 1024 || c->head_dim < 32 || c->head_dim > 256 ||
      c->head_dim % 32 != 0 || P < 8 || P > 4096 || (P & (P - 1)) != 0 || c->pages < 1 ||
      c->pages > kMaxIndex || c->seqs < 1 || c->seqs > (int64_t(1) << 20) || c->max_pages < 1 ||
      c->max_pages > kMaxIndex / P)
    return RFP2_E_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) ||
      (i8 && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))))
    return RFP2_E_ALIGN;
  int shift = 3;
  while ((int64_t(1) << shift) < P) ++shift;
  *view = {c->k, c->v, i8 ? c->k_scale : nullptr, i8 ? c->v_scale : nullptr, c->page_table,
           (int32_t)c->seqs, (int32_t)c->max_pages, (int32_t)c->pages, shift,
           (int32_t)c->kv_heads, (int32_t)c->head_dim};
  return RFP2_OK;
}

// Rows of `need` fp32 values that lie `stride` apart and are read 16 bytes at
// a time.
bool row_stride_ok(int64_t stride, int64_t need) {
  return stride >= need && stride % 4 == 0 && stride <= (int64_t(1) << 40);
}

bool rope_ok(int64_t rot, int64_t D, int style, double mscale) {
  return rot >= 2 && rot <= D && rot % 2 == 0 &&
         (style == RFP2_ROPE_HALF || style == RFP2_ROPE_INTERLEAVED) && std::isfinite(mscale);
}

// The checks that writing and reading T tokens share.
rfp2_status check_kv_rows(const rfp2::KvView& c, const void* k, const void* v, int64_t T,
                          int64_t k_stride, int64_t v_stride, const int32_t* seq,
                          const int32_t* pos, const int32_t* err) {
  if (!k || !v || !seq || !pos) return RFP2_E_NULL;
  const int64_t row = (int64_t)c.heads * c.dim;
  if (T < 1 || T > kMaxRows || !row_stride_ok(k_stride, row) || !row_stride_ok(v_stride, row))
    return RFP2_E_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(seq, 4) || !aligned(pos, 4) ||
      (err && !aligned(err, 4)))
    return RFP2_E_ALIGN;
  return RFP2_OK;
}

}  // namespace

extern "C" {

int rfp2_abi_version(void) { return RFP2_ABI_VERSION; }

const char* rfp2_status_string(int status) {
  switch (status) {
    case RFP2_OK: return "ok";
    case RFP2_E_NULL: return "a required pointer is null";
    case RFP2_E_SHAPE: return "a size is out of range for this call";
    case RFP2_E_ALIGN: return "a pointer is not aligned as this call requires";
    case RFP2_E_LAUNCH: return "the HIP runtime reported an error for the launch";
    default: return "unknown status";
  }
}

rfp2_status rfp2_quantize_acts(const float* a, int64_t M, int64_t K, int8_t* q,
                               float* d, hipStream_t stream) {
  if (!a || !q || !d) return RFP2_E_NULL;
  if (M < 1 || M > kMaxRows || K < 32 || K % 32 != 0 || K > (int64_t(1) << 30))
    return RFP2_E_SHAPE;
  if (!aligned(a, 16) || !aligned(q, 4) || !aligned(d, 4)) return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_quantize_acts(a, M, K, q, d, stream));
}

rfp2_status rfp2_quantize_weights(const float* x, int64_t N, int64_t K,
                                  uint8_t* w, hipStream_t stream) {
  if (!x || !w) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || K < 32 || K % 32 != 0 || K > (int64_t(1) << 30))
    return RFP2_E_SHAPE;
  if (!aligned(x, 4) || !aligned(w, 2)) return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_quantize_weights(x, N, K, nullptr, w, stream));
}

rfp2_status rfp2_quantize_weights_imatrix(const float* x, int64_t N, int64_t K,
                                          const float* importance, uint8_t* w,
                                          hipStream_t stream) {
  if (!x || !importance || !w) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || K < 32 || K % 32 != 0 || K > (int64_t(1) << 30))
    return RFP2_E_SHAPE;
  if (!aligned(x, 4) || !aligned(importance, 4) || !aligned(w, 2)) return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_quantize_weights(x, N, K, importance, w, stream));
}

rfp2_status rfp2_gemv(const uint8_t* w, int64_t N, int64_t K, const int8_t* q,
                      const float* d, int64_t M, float* y, hipStream_t stream) {
  if (!w || !q || !d || !y) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || M < 1 || M > RFP2_GEMV_MAX_M || !product_k_ok(K))
    return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(d, 4) || !aligned(y, 4))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_gemv(w, N, K, q, d, M, y, stream));
}

rfp2_status rfp2_gemm(const uint8_t* w, int64_t N, int64_t K, const int8_t* q,
                      const float* d, int64_t M, float* y, hipStream_t stream) {
  if (!w || !q || !d || !y) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || M < 1 || M > kMaxRows || K < 256 || K % 256 != 0 ||
      K > (int64_t(1) << 24))
    return RFP2_E_SHAPE;
  if (((M + 127) / 128) * ((N + 127) / 128) > (int64_t(1) << 31) - 1)
    return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(d, 4) || !aligned(y, 4))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_gemm(w, N, K, q, d, M, y, stream));
}

rfp2_status rfp2_gemm_f16(const uint8_t* w, int64_t N, int64_t K, const int8_t* q,
                          const float* d, int64_t M, float* y, hipStream_t stream) {
  if (!w || !q || !d || !y) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || M < 1 || M > kMaxRows || K < 256 || K % 256 != 0 ||
      K > (int64_t(1) << 24))
    return RFP2_E_SHAPE;
  if (((M + 127) / 128) * ((N + 127) / 128) > (int64_t(1) << 31) - 1)
    return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(d, 4) || !aligned(y, 4))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_gemm_f16(w, N, K, q, d, M, y, stream));
}

rfp2_status rfp2_moe_gemv(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                          const int32_t* ids, int64_t top_k, const int8_t* q,
                          const float* d, float* y, int32_t* err,
                          hipStream_t stream) {
  if (!w || !ids || !q || !d || !y) return RFP2_E_NULL;
  if (E < 1 || E > kMaxRows || N < 1 || N > kMaxRows || top_k < 1 ||
      top_k > 65535 || !product_k_ok(K))
    return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(d, 4) || !aligned(y, 4) ||
      !aligned(ids, 4) || (err && !aligned(err, 4)))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_moe_gemv(w, E, N, K, ids, top_k, q, d, y, err, stream));
}

rfp2_status rfp2_moe_gemv_tokens(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                 const int32_t* ids, int64_t T, int64_t top_k,
                                 const int8_t* q, const float* d, float* y, int32_t* err,
                                 hipStream_t stream) {
  if (!w || !ids || !q || !d || !y) return RFP2_E_NULL;
  if (E < 1 || E > kMaxRows || N < 1 || N > kMaxRows || T < 1 || T > RFP2_GEMV_MAX_M ||
      top_k < 1 || T * top_k > 64 || !product_k_ok(K))
    return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(d, 4) || !aligned(y, 4) ||
      !aligned(ids, 4) || (err && !aligned(err, 4)))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(
      rfp2::launch_moe_gemv_tokens(w, E, N, K, ids, T, top_k, q, d, y, err, stream));
}

rfp2_status rfp2_moe_sort(const int32_t* ids, int64_t S, int64_t E, int32_t* offsets,
                          int32_t* order, int32_t* err, hipStream_t stream) {
  if (!ids || !offsets || !order) return RFP2_E_NULL;
  if (S < 1 || S > kMaxSortSlots || E < 1 || E > rfp2::kMaxSortExperts) return RFP2_E_SHAPE;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4) ||
      (err && !aligned(err, 4)))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_moe_sort(ids, S, E, 0, offsets, nullptr, order, err, nullptr,
                                        0, stream));
}

size_t rfp2_moe_gemm_workspace_bytes(int64_t E, int64_t T, int64_t top_k) {
  if (E < 1 || E > rfp2::kMaxSortExperts || T < 1 || top_k < 1 || T > kMaxSortSlots ||
      top_k > kMaxSortSlots || T * top_k > kMaxSortSlots)
    return 0;
  return rfp2::moe_gemm_workspace_bytes(E, T * top_k);
}

rfp2_status rfp2_moe_gemm(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                          const int32_t* ids, int64_t T, int64_t top_k, const int8_t* q,
                          const float* d, float* y, int32_t* err, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  if (!w || !ids || !q || !d || !y || !workspace) return RFP2_E_NULL;
  const size_t need = rfp2_moe_gemm_workspace_bytes(E, T, top_k);
  if (need == 0 || N < 1 || N > kMaxRows || K < 256 || K % 256 != 0 ||
      K > (int64_t(1) << 24) || workspace_bytes < need)
    return RFP2_E_SHAPE;
  if (rfp2::moe_gemm_max_grid(E, N, T * top_k) > (int64_t(1) << 31) - 1) return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(d, 4) || !aligned(y, 4) ||
      !aligned(ids, 4) || !aligned(workspace, 256) || (err && !aligned(err, 4)))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_moe_gemm(w, E, N, K, ids, T, top_k, q, d, y, err, workspace,
                                        stream));
}

static_assert(RFP2_MOE_GEMM_NOALLOC_MAX_BYTES == rfp2::kNoallocScratchBytes,
              "the header's limit is the size of the library's scratch array");

rfp2_status rfp2_moe_gemm_noalloc(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                  const int32_t* ids, int64_t T, int64_t top_k,
                                  const int8_t* q, const float* d, float* y, int32_t* err,
                                  hipStream_t stream) {
  if (!w || !ids || !q || !d || !y) return RFP2_E_NULL;
  const size_t need = rfp2_moe_gemm_workspace_bytes(E, T, top_k);
  if (need == 0 || need > RFP2_MOE_GEMM_NOALLOC_MAX_BYTES || N < 1 || N > kMaxRows ||
      K < 256 || K % 256 != 0 || K > (int64_t(1) << 24))
    return RFP2_E_SHAPE;
  if (rfp2::moe_gemm_max_grid(E, N, T * top_k) > (int64_t(1) << 31) - 1) return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(d, 4) || !aligned(y, 4) ||
      !aligned(ids, 4) || (err && !aligned(err, 4)))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(
      rfp2::launch_moe_gemm_noalloc(w, E, N, K, ids, T, top_k, q, d, y, err, stream));
}

rfp2_status rfp2_rope_freqs(int64_t rot, double base, double factor, double orig_len,
                            double low_turns, double high_turns, double* freqs,
                            hipStream_t stream) {
  if (!freqs) return RFP2_E_NULL;
  if (rot < 2 || rot > rfp2::kMaxRopeDim || rot % 2 != 0 || !std::isfinite(base) ||
      !(base > 1.0) || !std::isfinite(factor) || !(factor >= 1.0) || !std::isfinite(orig_len) ||
      !(orig_len >= 0.0))
    return RFP2_E_SHAPE;
  if (orig_len > 0.0 && (!std::isfinite(high_turns) || !(low_turns >= 0.0) ||
                         !(low_turns < high_turns)))
    return RFP2_E_SHAPE;
  if (!aligned(freqs, 8)) return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_rope_freqs(rot, base, factor, orig_len, low_turns, high_turns,
                                          freqs, stream));
}

rfp2_status rfp2_rope(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                      const int32_t* pos, const double* freqs, int64_t rot, int style,
                      double mscale, float* y, int64_t y_stride, hipStream_t stream) {
  if (!x || !pos || !freqs || !y) return RFP2_E_NULL;
  if (T < 1 || T > kMaxRows || H < 1 || D < 4 || D > rfp2::kMaxRopeDim || D % 4 != 0 ||
      H > (int64_t(1) << 24) / D || !row_stride_ok(x_stride, H * D) ||
      !row_stride_ok(y_stride, H * D) || (x == y && x_stride != y_stride) ||
      !rope_ok(rot, D, style, mscale))
    return RFP2_E_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(pos, 4) || !aligned(freqs, 8))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  const rfp2::RopeView rope = {freqs, mscale, (int32_t)rot, style == RFP2_ROPE_INTERLEAVED};
  return from_hip(rfp2::launch_rope(x, T, H, D, x_stride, pos, rope, y, y_stride, stream));
}

rfp2_status rfp2_kv_write(const rfp2_kv_cache* cache, const float* k, const float* v, int64_t T,
                          int64_t k_stride, int64_t v_stride, const int32_t* seq,
                          const int32_t* pos, int32_t* err, hipStream_t stream) {
  rfp2::KvView c;
  rfp2_status st = check_cache(cache, &c);
  if (st == RFP2_OK) st = check_kv_rows(c, k, v, T, k_stride, v_stride, seq, pos, err);
  if (st != RFP2_OK) return st;
  (void)hipGetLastError();
  const rfp2::RopeView none = {nullptr, 1.0, 0, 0};
  return from_hip(rfp2::launch_kv_write(c, cache->format == RFP2_KV_I8, nullptr, k, v, T, 0, 0,
                                        k_stride, v_stride, seq, pos, none, nullptr, 0, err,
                                        stream));
}

rfp2_status rfp2_rope_kv_write(const rfp2_kv_cache* cache, const float* q, const float* k,
                               const float* v, int64_t T, int64_t H, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, const int32_t* seq,
                               const int32_t* pos, const double* freqs, int64_t rot, int style,
                               double mscale, float* q_out, int64_t q_out_stride, int32_t* err,
                               hipStream_t stream) {
  rfp2::KvView c;
  rfp2_status st = check_cache(cache, &c);
  if (st == RFP2_OK) st = check_kv_rows(c, k, v, T, k_stride, v_stride, seq, pos, err);
  if (st != RFP2_OK) return st;
  if (!freqs || (H != 0 && (!q || !q_out))) return RFP2_E_NULL;
  if (H < 0 || H > (int64_t(1) << 24) / c.dim || !rope_ok(rot, c.dim, style, mscale))
    return RFP2_E_SHAPE;
  if (H > 0 && (!row_stride_ok(q_stride, H * c.dim) || !row_stride_ok(q_out_stride, H * c.dim)))
    return RFP2_E_SHAPE;
  if (!aligned(freqs, 8) || !aligned(q, 16) || !aligned(q_out, 16)) return RFP2_E_ALIGN;
  if (H > 0 && (q_out == q || q_out == k || q_out == v)) return RFP2_E_SHAPE;
  (void)hipGetLastError();
  const rfp2::RopeView rope = {freqs, mscale, (int32_t)rot, style == RFP2_ROPE_INTERLEAVED};
  return from_hip(rfp2::launch_kv_write(c, cache->format == RFP2_KV_I8, q, k, v, T, H, q_stride,
                                        k_stride, v_stride, seq, pos, rope, q_out, q_out_stride,
                                        err, stream));
}

rfp2_status rfp2_kv_read(const rfp2_kv_cache* cache, int64_t T, const int32_t* seq,
                         const int32_t* pos, float* k, float* v, int64_t k_stride,
                         int64_t v_stride, int32_t* err, hipStream_t stream) {
  rfp2::KvView c;
  rfp2_status st = check_cache(cache, &c);
  if (st == RFP2_OK) st = check_kv_rows(c, k, v, T, k_stride, v_stride, seq, pos, err);
  if (st != RFP2_OK) return st;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_kv_read(c, cache->format == RFP2_KV_I8, T, seq, pos, k, v,
                                       k_stride, v_stride, err, stream));
}

size_t rfp2_paged_attn_workspace_bytes(const rfp2_kv_cache* cache, int64_t B, int64_t new_tokens,
                                       int64_t H) {
  rfp2::KvView c;
  if (check_cache(cache, &c) != RFP2_OK || B < 1 || B > rfp2::kMaxAttnSeqs || B > c.seqs ||
      new_tokens < 1 || new_tokens > RFP2_ATTN_MAX_NEW || H < 1 || H > 1024 || H % c.heads != 0 ||
      B * cache->max_pages * cache->page_size > (int64_t(1) << 36))
    return 0;
  return rfp2::paged_attn_workspace_bytes(c.heads, c.dim, B, new_tokens, H);
}

rfp2_status rfp2_paged_attn(const rfp2_kv_cache* cache, const float* q, int64_t B,
                            int64_t new_tokens, int64_t H, int64_t q_stride,
                            const int32_t* lens, float scale, int64_t window, float* y,
                            int32_t* err, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  rfp2::KvView c;
  const rfp2_status st = check_cache(cache, &c);
  if (st != RFP2_OK) return st;
  if (!q || !lens || !y || !workspace) return RFP2_E_NULL;
  const size_t need = rfp2_paged_attn_workspace_bytes(cache, B, new_tokens, H);
  if (need == 0 || workspace_bytes < need || !row_stride_ok(q_stride, H * c.dim) || window < 0 ||
      !std::isfinite(scale))
    return RFP2_E_SHAPE;
  if (!aligned(q, 16) || !aligned(y, 16) || !aligned(lens, 4) || !aligned(workspace, 256) ||
      (err && !aligned(err, 4)))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_paged_attn(c, cache->format == RFP2_KV_I8, q, B, new_tokens, H,
                                          q_stride, lens, scale, window, y, err, workspace,
                                          stream));
}

rfp2_status rfp2_read_ceiling(const uint8_t* buf, int64_t bytes, uint32_t magic, uint32_t* out,
                              hipStream_t stream) {
  if (!buf || !out) return RFP2_E_NULL;
  if (bytes < 16 || bytes % 16 != 0) return RFP2_E_SHAPE;
  if (!aligned(buf, 16) || !aligned(out, 4)) return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_read_ceiling(buf, bytes, magic, out, stream));
}

rfp2_status rfp2_quant_gemv(const uint8_t* w, int64_t N, int64_t K, const float* a,
                            int8_t* q, float* d, float* y, hipStream_t stream) {
  if (!w || !a || !q || !d || !y) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || !product_k_ok(K)) return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(a, 16) || !aligned(q, 16) || !aligned(d, 4) ||
      !aligned(y, 4))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_quant_gemv(w, N, K, a, q, d, y, stream));
}

rfp2_status rfp2_quant_moe_gemv(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                const int32_t* ids, int64_t top_k, const float* a,
                                int8_t* q, float* d, float* y, int32_t* err,
                                hipStream_t stream) {
  if (!w || !ids || !a || !q || !d || !y) return RFP2_E_NULL;
  if (E < 1 || E > kMaxRows || N < 1 || N > kMaxRows || top_k < 1 ||
      top_k > 65535 || !product_k_ok(K))
    return RFP2_E_SHAPE;
  if (!aligned(w, 16) || !aligned(a, 16) || !aligned(q, 16) || !aligned(d, 4) ||
      !aligned(y, 4) || !aligned(ids, 4) || (err && !aligned(err, 4)))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(
      rfp2::launch_quant_moe_gemv(w, E, N, K, ids, top_k, a, q, d, y, err, stream));
}

rfp2_status rfp2_debug_decode(const uint8_t* w, int64_t N, int64_t K,
                              int8_t* codes_out, float* scales_out,
                              hipStream_t stream) {
  if (!w || !codes_out || !scales_out) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || K < 32 || K % 32 != 0 || K > (int64_t(1) << 30))
    return RFP2_E_SHAPE;
  if (!aligned(w, 2) || !aligned(codes_out, 4) || !aligned(scales_out, 4))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_debug_decode(w, N, K, codes_out, scales_out, stream));
}

rfp2_status rfp2_debug_half_dots(const uint8_t* w, int64_t N, int64_t K,
                                 const int8_t* q, int64_t M, int32_t* sums_out,
                                 hipStream_t stream) {
  if (!w || !q || !sums_out) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || M < 1 || M > kMaxRows || K < 32 || K % 32 != 0 ||
      K > (int64_t(1) << 30))
    return RFP2_E_SHAPE;
  // M * N * (K / 32) half-sum pairs are indexed in 64 bits: keep it below 2^40
  if (N * (K / 32) > (int64_t(1) << 40) / M) return RFP2_E_SHAPE;
  if (!aligned(w, 2) || !aligned(q, 4) || !aligned(sums_out, 4)) return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_debug_half_dots(w, N, K, q, M, sums_out, stream));
}

rfp2_status rfp2_debug_half_sums_mf(const uint8_t* w, int64_t N, int64_t K,
                                    const int8_t* q, int64_t M, int32_t* sums_out,
                                    hipStream_t stream) {
  if (!w || !q || !sums_out) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || M < 1 || M > kMaxRows || K < 256 || K % 256 != 0 ||
      K > (int64_t(1) << 30))
    return RFP2_E_SHAPE;
  if (N * (K / 32) > (int64_t(1) << 40) / M) return RFP2_E_SHAPE;
  if (!aligned(w, 2) || !aligned(q, 4) || !aligned(sums_out, 4)) return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_debug_half_sums_mf(w, N, K, q, M, sums_out, stream));
}

rfp2_status rfp2_debug_decode_f16(const uint8_t* w, int64_t N, int64_t K, int form,
                                  uint16_t* h_out, hipStream_t stream) {
  if (!w || !h_out) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || K < 32 || K % 32 != 0 || K > (int64_t(1) << 30) ||
      (form != 0 && form != 1))
    return RFP2_E_SHAPE;
  if (!aligned(w, 2) || !aligned(h_out, 2)) return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_debug_decode_f16(w, N, K, form, h_out, stream));
}

rfp2_status rfp2_debug_decode_i8(const uint8_t* w, int64_t N, int64_t K, int8_t* wa_out,
                                 int8_t* wb_out, float* scales_out, hipStream_t stream) {
  if (!w || !wa_out || !wb_out || !scales_out) return RFP2_E_NULL;
  if (N < 1 || N > kMaxRows || K < 32 || K % 32 != 0 || K > (int64_t(1) << 30))
    return RFP2_E_SHAPE;
  if (!aligned(w, 2) || !aligned(wa_out, 4) || !aligned(wb_out, 4) || !aligned(scales_out, 4))
    return RFP2_E_ALIGN;
  (void)hipGetLastError();
  return from_hip(rfp2::launch_debug_decode_i8(w, N, K, wa_out, wb_out, scales_out, stream));
}

}  // extern "C"
