// What lies between two products of a feed-forward part: the gate's activation times the
// other half, as the int8 activations of the next product, and the values that int8
// activations stand for.
//
//   silu:  act(g) = g / (1 + exp(-g))
//   gelu:  act(g) = g / (1 + exp(-2 c (g + 0.044715 g^3))),  c = sqrt(2 / pi)
//          (0.5 g (1 + tanh(z)) = g / (1 + exp(-2 z)))
//
// act(g) * u is computed in fp64 and rounded once, so that the codes are those of the
// definition.  Both are bound by the transfer.
#include "acts_device.h"
#include "rfp2_internal.h"

namespace rfp2 {

namespace {

constexpr int kThreads = 256;

// One workgroup a row.
template <bool GELU>
__global__ __launch_bounds__(kThreads) void gated_acts_kernel(
    const float* __restrict__ gate, const float* __restrict__ up, int64_t row0, int64_t quads,
    int64_t gate_stride, int64_t up_stride, uint32_t* __restrict__ q, float* __restrict__ d) {
  const int64_t t = row0 + blockIdx.x;
  for (int64_t i = threadIdx.x; i < quads; i += kThreads) {
    float g[4], u[4];
    load4(g, gate + t * gate_stride + 4 * i);
    load4(u, up + t * up_stride + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double x = g[e];
      const double z = GELU ? 1.5957691216057308 * (x + 0.044715 * x * x * x) : x;
      u[e] = (float)(x / (1.0 + exp(-z)) * (double)u[e]);
    }
    uint32_t codes;
    const float scale = quantize4(u, codes);
    q[t * quads + i] = codes;
    if ((threadIdx.x & 7) == 0) d[(t * quads + i) >> 3] = scale;
  }
}

__global__ __launch_bounds__(kThreads) void dequantize_acts_kernel(
    const uint32_t* __restrict__ q, const float* __restrict__ d, int64_t quads,
    float* __restrict__ a) {
  for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < quads;
       i += gridDim.x * (int64_t)kThreads) {
    const uint32_t c = q[i];
    const float s = d[i >> 3];
    store4<false>(a + 4 * i, make_float4((int8_t)c * s, (int8_t)(c >> 8) * s,
                                         (int8_t)(c >> 16) * s, (int8_t)(c >> 24) * s));
  }
}

}  // namespace

hipError_t launch_quantize_gated_acts(const float* gate, const float* up, int64_t M, int64_t K,
                                      int64_t gate_stride, int64_t up_stride, bool gelu,
                                      int8_t* q, float* d, hipStream_t stream) {
  const auto kernel = gelu ? gated_acts_kernel<true> : gated_acts_kernel<false>;
  for (int64_t t = 0; t < M; t += kMaxGrid) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)std::min(M - t, kMaxGrid)), dim3(kThreads), 0,
                       stream, gate, up, t, K / 4, gate_stride, up_stride,
                       reinterpret_cast<uint32_t*>(q), d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_dequantize_acts(const int8_t* q, const float* d, int64_t M, int64_t K, float* a,
                                  hipStream_t stream) {
  const int64_t quads = M * (K / 4);
  const int64_t grid = std::min<int64_t>((quads + kThreads - 1) / kThreads, kMaxGrid);
  hipLaunchKernelGGL(dequantize_acts_kernel, dim3((uint32_t)grid), dim3(kThreads), 0, stream,
                     reinterpret_cast<const uint32_t*>(q), d, quads, a);
  return hipGetLastError();
}

}  // namespace rfp2
