// Root-mean-square norms: of heads where they lie, and of whole rows with what is added
// to the residual stream before and the int8 form of the result after.
//
//   h = fl32(x + add)   or   fl32(x + sum_j w_j r_j)
//   y = fl32(h * gain / sqrt(mean(h^2) + eps)),   q, d as rfp2_quantize_acts of y
//
// Sums, the root and the products are fp64, rounded once: a last bit of y may flip a
// code, and so the codes are those of the definition whatever the order of the sums.
// Everything here is bound by the transfer: a value is read once and written once.
#include "acts_device.h"
#include "rfp2_internal.h"

namespace rfp2 {

namespace {

constexpr int kThreads = 256;

// The sum over the wave, in every lane.
__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  return s;
}

// One wave a head of D values: heads [.., 4 * blockIdx.y + wave, ..] of row blockIdx.x.
__global__ __launch_bounds__(kThreads) void rms_norm_kernel(const float* x, int H, int D,
                                                            int64_t x_stride,
                                                            const float* __restrict__ gain,
                                                            double eps, float* y,
                                                            int64_t y_stride) {
  const int lane = threadIdx.x & 63;
  const int h = blockIdx.y * (kThreads / 64) + (threadIdx.x >> 6);
  if (h >= H) return;
  const float* xr = x + blockIdx.x * x_stride + (int64_t)h * D;
  float* yr = y + blockIdx.x * y_stride + (int64_t)h * D;
  double s = 0.0;
  for (int i = lane; i < D; i += 64) s += (double)xr[i] * xr[i];
  const double inv = 1.0 / sqrt(wave_sum(s) / D + eps);
  for (int i = lane; i < D; i += 64) yr[i] = (float)((double)xr[i] * inv * gain[i]);
}

// Where a row comes from and goes to; what is null is not there.
struct NormRows {
  const float* x;          // x + row * x_stride
  const float* add;        // MODE_ADD: add + row * add_stride; MODE_SUM: [top_k][K] a row
  const float* weights;    // MODE_SUM: [top_k] a row
  const float* gain;       // null: no norm
  float* h;
  float* y;
  uint32_t* q;
  float* d;
  int64_t x_stride, add_stride, h_stride, y_stride, K;
  double eps;
  int32_t top_k;
};
enum { MODE_ROW, MODE_ADD, MODE_SUM };

// Values 4 * i .. 4 * i + 3 of row t of the stream.
template <int MODE>
__device__ __forceinline__ void stream4(float (&v)[4], const NormRows& r, int64_t t, int64_t i) {
  if (r.x) load4(v, r.x + t * r.x_stride + 4 * i);
  else v[0] = v[1] = v[2] = v[3] = 0.0f;
  if constexpr (MODE == MODE_ADD) {
    float a[4];
    load4(a, r.add + t * r.add_stride + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += a[e];
  }
  if constexpr (MODE == MODE_SUM) {
    double s[4] = {v[0], v[1], v[2], v[3]};
    for (int j = 0; j < r.top_k; ++j) {
      float a[4];
      const double w = r.weights[t * r.top_k + j];
      load4(a, r.add + (t * r.top_k + j) * r.K + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = fma(w, (double)a[e], s[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)s[e];
  }
}

// One workgroup a row.  A thread reads back only what it wrote itself, so h and y may
// be the rows that were read.
template <int MODE>
__global__ __launch_bounds__(kThreads) void row_norm_kernel(NormRows r, int64_t row0) {
  __shared__ double part[kThreads / 64];
  const int64_t t = row0 + blockIdx.x, quads = r.K >> 2;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < quads; i += kThreads) {
    float v[4];
    stream4<MODE>(v, r, t, i);
    if (r.h) store4<false>(r.h + t * r.h_stride + 4 * i, make_float4(v[0], v[1], v[2], v[3]));
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fma((double)v[e], (double)v[e], s);
  }
  if (!r.gain) return;
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < kThreads / 64; ++w) s += part[w];
  const double inv = 1.0 / sqrt(s / (double)r.K + r.eps);
  for (int64_t i = threadIdx.x; i < quads; i += kThreads) {
    float v[4], g[4];
    if (r.h) load4(v, r.h + t * r.h_stride + 4 * i);
    else stream4<MODE>(v, r, t, i);
    load4(g, r.gain + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)((double)v[e] * inv * (double)g[e]);
    if (r.y) store4<false>(r.y + t * r.y_stride + 4 * i, make_float4(v[0], v[1], v[2], v[3]));
    if (r.q) {
      uint32_t codes;
      const float scale = quantize4(v, codes);
      r.q[t * quads + i] = codes;
      if ((threadIdx.x & 7) == 0) r.d[(t * quads + i) >> 3] = scale;
    }
  }
}

template <int MODE>
hipError_t launch_rows(const NormRows& r, int64_t T, hipStream_t stream) {
  for (int64_t t = 0; t < T; t += kMaxGrid) {
    const int64_t n = std::min(T - t, kMaxGrid);
    hipLaunchKernelGGL(row_norm_kernel<MODE>, dim3((uint32_t)n), dim3(kThreads), 0, stream, r, t);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rms_norm(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                           const float* gain, double eps, float* y, int64_t y_stride,
                           hipStream_t stream) {
  const int64_t per = kThreads / 64, groups = (H + per - 1) / per;
  // a launch holds 2^32 threads at most and 65535 workgroups along y
  const int64_t rows = std::max<int64_t>(1, kMaxGrid / groups);
  for (int64_t t = 0; t < T; t += rows) {
    const int64_t n = std::min(T - t, rows);
    for (int64_t g = 0; g < groups; g += 65535) {
      const int64_t m = std::min<int64_t>(groups - g, 65535), h = g * per;
      hipLaunchKernelGGL(rms_norm_kernel, dim3((uint32_t)n, (uint32_t)m), dim3(kThreads), 0,
                         stream, x + t * x_stride + h * D, (int)(H - h), (int)D, x_stride, gain,
                         eps, y + t * y_stride + h * D, y_stride);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

hipError_t launch_add_rms_norm(const float* x, const float* add, int64_t T, int64_t K,
                               int64_t x_stride, int64_t add_stride, const float* gain,
                               double eps, float* h, int64_t h_stride, float* y,
                               int64_t y_stride, int8_t* q, float* d, hipStream_t stream) {
  const NormRows r = {x, add, nullptr, gain, h, y, reinterpret_cast<uint32_t*>(q), d,
                      x_stride, add_stride, h_stride, y_stride, K, eps, 1};
  return add ? launch_rows<MODE_ADD>(r, T, stream) : launch_rows<MODE_ROW>(r, T, stream);
}

hipError_t launch_moe_combine(const float* x, const float* rows, const float* weights, int64_t T,
                              int64_t top_k, int64_t K, int64_t x_stride, const float* gain,
                              double eps, float* h, int64_t h_stride, float* y,
                              int64_t y_stride, int8_t* q, float* d, hipStream_t stream) {
  const NormRows r = {x, rows, weights, gain, h, y, reinterpret_cast<uint32_t*>(q), d,
                      x_stride, 0, h_stride, y_stride, K, eps, (int32_t)top_k};
  return launch_rows<MODE_SUM>(r, T, stream);
}

}  // namespace rfp2
