// Launchers behind the C ABI.  Arguments have been validated by the caller
// (rfp2_abi.hip); each launcher only sizes the grid and enqueues kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace rfp2 {

constexpr int64_t kMaxGrid = 1 << 20;   // workgroups per launch (grid-stride beyond)
constexpr int kMaxSortExperts = 2048;   // experts of a grouped (sorted) routed product
constexpr int kReadCeilingGrid = 2048;  // workgroups of the read helper (256 threads each)
constexpr size_t kNoallocScratchBytes = size_t(1) << 20;  // library-owned workspace per GPU
constexpr int kMaxRopeDim = 1024;       // values of a rotated head
constexpr int kMaxAttnSeqs = 1024;      // sequences of one attention call

// A key/value cache as the kernels see it (layouts: rfp2_kv_cache in rfp2.h).
struct KvView {
  void* k;
  void* v;
  float* ks;
  float* vs;
  const int32_t* table;
  int32_t seqs, max_pages, pages;
  int32_t page_shift;                   // page_size == 1 << page_shift
  int32_t heads, dim;
};

// Rotary positions as the kernels see them.
struct RopeView {
  const double* freqs;
  double mscale;
  int32_t rot;                          // 0: nothing is rotated
  int32_t interleaved;
};

hipError_t launch_quantize_acts(const float* a, int64_t M, int64_t K, int8_t* q,
                                float* d, hipStream_t stream);
hipError_t launch_quantize_weights(const float* x, int64_t N, int64_t K,
                                   const float* imp, uint8_t* w, hipStream_t stream);
hipError_t launch_gemv(const uint8_t* w, int64_t N, int64_t K, const int8_t* q,
                       const float* d, int64_t M, float* y, hipStream_t stream);
hipError_t launch_moe_gemv(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                           const int32_t* ids, int64_t top_k, const int8_t* q,
                           const float* d, float* y, int32_t* err,
                           hipStream_t stream);
hipError_t launch_moe_gemv_tokens(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                  const int32_t* ids, int64_t T, int64_t top_k,
                                  const int8_t* q, const float* d, float* y, int32_t* err,
                                  hipStream_t stream);
hipError_t launch_quant_gemv(const uint8_t* w, int64_t N, int64_t K, const float* a,
                             int8_t* q, float* d, float* y, hipStream_t stream);
hipError_t launch_quant_moe_gemv(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                 const int32_t* ids, int64_t top_k, const float* a,
                                 int8_t* q, float* d, float* y, int32_t* err,
                                 hipStream_t stream);
hipError_t launch_gemm(const uint8_t* w, int64_t N, int64_t K, const int8_t* q,
                       const float* d, int64_t M, float* y, hipStream_t stream);
hipError_t launch_gemm_f16(const uint8_t* w, int64_t N, int64_t K, const int8_t* q,
                           const float* d, int64_t M, float* y, hipStream_t stream);
hipError_t launch_moe_sort(const int32_t* ids, int64_t S, int64_t E, int64_t tile_rows,
                           int32_t* offsets, int32_t* tile_start, int32_t* order,
                           int32_t* err, float* y, int64_t N, hipStream_t stream);
int moe_gemm_tile_tokens();
hipError_t launch_moe_gemm_sorted(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                  const int32_t* offsets, const int32_t* tile_start,
                                  const int32_t* order, int64_t S, int64_t top_k,
                                  const int8_t* q, const float* d, float* y,
                                  hipStream_t stream);
size_t moe_gemm_workspace_bytes(int64_t E, int64_t S);
int64_t moe_gemm_max_grid(int64_t E, int64_t N, int64_t S);
hipError_t launch_moe_gemm(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                           const int32_t* ids, int64_t T, int64_t top_k, const int8_t* q,
                           const float* d, float* y, int32_t* err, void* workspace,
                           hipStream_t stream);
hipError_t launch_moe_gemm_noalloc(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                   const int32_t* ids, int64_t T, int64_t top_k,
                                   const int8_t* q, const float* d, float* y, int32_t* err,
                                   hipStream_t stream);
hipError_t launch_rope_freqs(int64_t rot, double base, double factor, double orig_len,
                             double low_turns, double high_turns, double* freqs,
                             hipStream_t stream);
hipError_t launch_rope(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                       const int32_t* pos, const RopeView& rope, float* y, int64_t y_stride,
                       hipStream_t stream);
hipError_t launch_kv_write(const KvView& c, bool i8, const float* q, const float* k,
                           const float* v, int64_t T, int64_t H, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const int32_t* seq,
                           const int32_t* pos, const RopeView& rope, float* q_out,
                           int64_t q_out_stride, int32_t* err, hipStream_t stream);
hipError_t launch_kv_read(const KvView& c, bool i8, int64_t T, const int32_t* seq,
                          const int32_t* pos, float* k, float* v, int64_t k_stride,
                          int64_t v_stride, int32_t* err, hipStream_t stream);
size_t paged_attn_workspace_bytes(int64_t kv_heads, int64_t dim, int64_t B, int64_t new_tokens,
                                  int64_t H);
hipError_t launch_paged_attn(const KvView& c, bool i8, const float* q, int64_t B,
                             int64_t new_tokens, int64_t H, int64_t q_stride,
                             const int32_t* lens, float scale, int64_t window, float* y,
                             int32_t* err, void* workspace, hipStream_t stream);
hipError_t launch_rms_norm(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                           const float* gain, double eps, float* y, int64_t y_stride,
                           hipStream_t stream);
hipError_t launch_add_rms_norm(const float* x, const float* add, int64_t T, int64_t K,
                               int64_t x_stride, int64_t add_stride, const float* gain,
                               double eps, float* h, int64_t h_stride, float* y,
                               int64_t y_stride, int8_t* q, float* d, hipStream_t stream);
hipError_t launch_moe_combine(const float* x, const float* rows, const float* weights, int64_t T,
                              int64_t top_k, int64_t K, int64_t x_stride, const float* gain,
                              double eps, float* h, int64_t h_stride, float* y,
                              int64_t y_stride, int8_t* q, float* d, hipStream_t stream);
hipError_t launch_moe_route(const float* logits, int64_t T, int64_t E, int64_t stride,
                            const float* bias, bool sigmoid, int groups, int group_top,
                            int top_groups, int top_k, bool renorm, double scale, int32_t* ids,
                            float* weights, int32_t* err, hipStream_t stream);
hipError_t launch_quantize_gated_acts(const float* gate, const float* up, int64_t M, int64_t K,
                                      int64_t gate_stride, int64_t up_stride, bool gelu,
                                      int8_t* q, float* d, hipStream_t stream);
hipError_t launch_dequantize_acts(const int8_t* q, const float* d, int64_t M, int64_t K, float* a,
                                  hipStream_t stream);
hipError_t launch_read_ceiling(const uint8_t* buf, int64_t bytes, uint32_t magic, uint32_t* out,
                               hipStream_t stream);
hipError_t launch_debug_decode(const uint8_t* w, int64_t N, int64_t K,
                               int8_t* codes, float* scales, hipStream_t stream);
hipError_t launch_debug_half_dots(const uint8_t* w, int64_t N, int64_t K,
                                  const int8_t* q, int64_t M, int32_t* sums,
                                  hipStream_t stream);
hipError_t launch_debug_half_sums_mf(const uint8_t* w, int64_t N, int64_t K,
                                     const int8_t* q, int64_t M, int32_t* sums,
                                     hipStream_t stream);
hipError_t launch_debug_decode_i8(const uint8_t* w, int64_t N, int64_t K, int8_t* wa,
                                  int8_t* wb, float* scales, hipStream_t stream);
hipError_t launch_debug_decode_f16(const uint8_t* w, int64_t N, int64_t K, int form,
                                   uint16_t* out, hipStream_t stream);

}  // namespace rfp2
