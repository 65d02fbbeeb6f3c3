// Attention of each sequence's newest tokens over the paged key/value cache.
//
//   y = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j - m),
//
// over the visible cached tokens j, in one pass with a running maximum m: when
// m grows, the sums so far are multiplied by exp(m_old - m_new).
#include <hip/hip_fp16.h>

#include "kv_device.h"

namespace rfp2 {

namespace {

constexpr int kThreads = 256;

// One workgroup per query row (sequence, new token, head): 256 tokens at a
// time, one per thread for the scores, one value per thread for the sums.
template <bool I8>
__global__ __launch_bounds__(kThreads) void paged_attn_kernel(
    KvView c, const float* __restrict__ q, int T, int H, int64_t q_stride,
    const int32_t* __restrict__ lens, float scale, int64_t window, float* __restrict__ y,
    int32_t* __restrict__ err) {
  __shared__ float qs[256];
  __shared__ float w[kThreads];
  __shared__ int64_t rows_of[kThreads];
  __shared__ float red[kThreads / 64];
  const int64_t row = blockIdx.x;                  // (b * T + t) * H + h
  const int h = (int)(row % H);
  const int64_t bt = row / H;
  const int t = (int)(bt % T), b = (int)(bt / T);
  const int D = c.dim, kvh = h / (H / c.heads), tid = threadIdx.x;
  const int64_t len = lens[b];
  const int64_t at = len - T + t;                  // this query's position
  float* out = y + row * D;
  if (len > ((int64_t)c.max_pages << c.page_shift)) {
    if (err && tid == 0) *err = 1;
    for (int d = tid; d < D; d += kThreads) out[d] = __builtin_nanf("");
    return;
  }
  for (int d = tid; d < D; d += kThreads) qs[d] = q[bt * q_stride + (int64_t)h * D + d];
  float m = -INFINITY, l = 0.0f, acc = 0.0f;
  const int64_t first = window > 0 && at >= window ? at - window + 1 : 0;
  for (int64_t j0 = first; j0 <= at; j0 += kThreads) {
    const int64_t j = j0 + tid;
    float s = -INFINITY;
    int64_t rows = 0;
    __syncthreads();
    if (j <= at) {
      const int32_t page = kv_page(c, b, (int32_t)j);
      const int r = (int)j & ((1 << c.page_shift) - 1);
      if (page < 0) {
        if (err) *err = 1;
        s = __builtin_nanf("");
      } else {
        rows = kv_rows(c, page, kvh);
        float dot = 0.0f;
        for (int g = 0; g < D / 32; ++g) {
          float part = 0.0f;
          for (int d = 32 * g; d < 32 * g + 32; ++d) {
            const int64_t e = k_at(c, rows, r, d);
            part += qs[d] * (I8 ? (float)static_cast<const int8_t*>(c.k)[e]
                                : __half2float(static_cast<const __half*>(c.k)[e]));
          }
          dot += I8 ? part * c.ks[scale_at(c, rows, r, g)] : part;
        }
        s = dot * scale;
      }
      rows += r;                                   // page rows and row in one number
    }
    rows_of[tid] = rows;
    float mx = s;
    for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
    if ((tid & 63) == 0) red[tid >> 6] = mx;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    w[tid] = j <= at ? expf(s - m_new) : 0.0f;
    __syncthreads();
    const float fix = m == m_new ? 1.0f : expf(m - m_new);
    acc *= fix;
    l *= fix;
    m = m_new;
    const int n = (int)min((int64_t)kThreads, at - j0 + 1);
    for (int i = 0; i < n; ++i) {
      const float p = w[i];
      l += p;
      if (tid < D) {
        const int64_t rr = rows_of[i];
        const int r = (int)(rr & 7);
        const int64_t e = (rr - r) * D + tid * 8 + r;
        acc += p * (I8 ? (float)static_cast<const int8_t*>(c.v)[e] *
                             c.vs[(rr - r) * (D >> 5) + (tid >> 5) * 8 + r]
                       : __half2float(static_cast<const __half*>(c.v)[e]));
      }
    }
  }
  if (tid < D) out[tid] = at < 0 ? 0.0f : acc / l;
}

}  // namespace

size_t paged_attn_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 256; }

hipError_t launch_paged_attn(const KvView& c, bool i8, const float* q, int64_t B,
                             int64_t new_tokens, int64_t H, int64_t q_stride,
                             const int32_t* lens, float scale, int64_t window, float* y,
                             int32_t* err, void* workspace, hipStream_t stream) {
  (void)workspace;
  const auto kernel = i8 ? paged_attn_kernel<true> : paged_attn_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((uint32_t)(B * new_tokens * H)), dim3(kThreads), 0, stream, c,
                     q, (int)new_tokens, (int)H, q_stride, lens, scale, window, y, err);
  return hipGetLastError();
}

}  // namespace rfp2
