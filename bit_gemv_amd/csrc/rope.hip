// Rotary positions: the frequencies of the pairs and the rotation of heads.
#include "rope_device.h"

namespace rfp2 {

namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void rope_freqs_kernel(int n, double rot, double base,
                                                              double factor, double orig_len,
                                                              double low, double high,
                                                              double* __restrict__ freqs) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const double f = pow(base, -2.0 * i / rot);
  double g = 0.0;
  if (orig_len > 0.0) {
    const double turns = orig_len * f * 0.15915494309189533577;
    g = fmin(fmax((turns - low) / (high - low), 0.0), 1.0);
  }
  freqs[i] = (1.0 - g) * (f / factor) + g * f;
}

// One workgroup turns heads [blockIdx.y * per, ...) of token blockIdx.x.  A
// thread owns whole pairs, read before they are written, so x may be y.
__global__ __launch_bounds__(kThreads) void rope_kernel(const float* x, int H, int D,
                                                        int64_t x_stride,
                                                        const int32_t* __restrict__ pos,
                                                        RopeView r, float* y, int64_t y_stride,
                                                        int per) {
  __shared__ double2 table[kMaxRopeDim / 2];
  const int64_t t = blockIdx.x;
  rope_table(table, r, pos[t], threadIdx.x, kThreads);
  __syncthreads();
  const int h0 = blockIdx.y * per, h1 = min(H, h0 + per);
  const float* xr = x + t * x_stride;
  float* yr = y + t * y_stride;
  const int half = r.rot >> 1;
  const int units = half + (D - r.rot);     // pairs, then single values that are copied
  for (int u = threadIdx.x; u < (h1 - h0) * units; u += kThreads) {
    const int h = u / units, i = u - h * units;
    const int64_t base = (int64_t)(h0 + h) * D;
    if (i < half) {
      const int64_t a = base + (r.interleaved ? 2 * i : i);
      const int64_t b = r.interleaved ? a + 1 : a + half;
      const float2 o = rope_turn(xr[a], xr[b], table[i]);
      yr[a] = o.x;
      yr[b] = o.y;
    } else {
      const int64_t a = base + r.rot + (i - half);
      yr[a] = xr[a];
    }
  }
}

}  // namespace

hipError_t launch_rope_freqs(int64_t rot, double base, double factor, double orig_len,
                             double low_turns, double high_turns, double* freqs,
                             hipStream_t stream) {
  const int n = (int)(rot / 2);
  hipLaunchKernelGGL(rope_freqs_kernel, dim3((n + kThreads - 1) / kThreads), dim3(kThreads), 0,
                     stream, n, (double)rot, base, factor, orig_len, low_turns, high_turns,
                     freqs);
  return hipGetLastError();
}

hipError_t launch_rope(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                       const int32_t* pos, const RopeView& rope, float* y, int64_t y_stride,
                       hipStream_t stream) {
  const int per = (int)H;
  hipLaunchKernelGGL(rope_kernel, dim3((uint32_t)T, (uint32_t)((H + per - 1) / per)),
                     dim3(kThreads), 0, stream, x, (int)H, (int)D, x_stride, pos, rope, y,
                     y_stride, per);
  return hipGetLastError();
}

}  // namespace rfp2
