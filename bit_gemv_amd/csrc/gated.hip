// What lies between two products of a feed-forward part: the gate's activation times the
// other half, as the int8 activations of the next product, and the values that int8
// activations stand for.
//
//   silu:  act(g) = g / (1 + exp(-g))
//   gelu:  act(g) = g / (1 + exp(-2 c (g + 0.044715 g^3))),  c = sqrt(2 / pi)
//          (0.5 g (1 + tanh(z)) = g / (1 + exp(-2 z)))
//
// act(g) * u is computed in fp64 and rounded once.  It is within 2^-43 (the farthest of 4
// million gates: silu 2^-45.0; gelu 2^-45.1 up to |g| = 8, and 2^-43.1 near g = -20, where the
// rounding of an exponent of 869 counts and 2^-868 is left): one value in 2^18 at most may round to
// the other side, which changes a code only where it lies at the border of two.
// The gate enters the exponential held to +-690 (silu) or +-20 (gelu), where the logistic
// function of a smaller one is below 2^-868 and leaves nothing of any product in fp32, and
// that of a larger one is 1.
//
// 4096 rows of 1536 take 10.7 to 11.6 us (5.1 TB/s); reading and writing their 57 MB takes
// 8.8, and the vector instructions, 41 a value, 7: they hide under the transfer only in
// part.  With the library's exp and divisions it was 14.9 us.
#include "acts_device.h"
#include "rfp2_internal.h"
#include "scores_device.h"

namespace rfp2 {

namespace {

constexpr int kThreads = 256;

// n / d for n < 2^31, by the high word of a product.
struct Divisor {
  uint32_t d, magic, shift;
};
Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return {d, (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1), s};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& v) {
  return (__umulhi(n, v.magic) + n) >> v.shift;
}

template <bool GELU>
__device__ __forceinline__ float gated(float x, float u) {
  const double c = __builtin_amdgcn_fmed3f(x, GELU ? -20.0f : -690.0f, GELU ? 20.0f : 690.0f);
  double s;
  if constexpr (GELU) {
    constexpr double k = -2.0 * 0.79788456080286535588 * kLog2E;
    const double t = c * fma(c * c, 0.044715 * k, k), m = t + kRound;
    s = logistic_parts(m, t - (m - kRound));
  } else {
    s = logistic(c);
  }
  return (float)((double)x * (double)u * s);   // NaN and infinity come through x and u
}

// The rows' pieces of N values one after another, one a thread.
template <bool GELU, int N>
__global__ __launch_bounds__(kThreads) void gated_acts_kernel(
    const float* __restrict__ gate, const float* __restrict__ up, uint32_t total, Divisor pieces,
    int64_t gate_stride, int64_t up_stride, uint32_t* __restrict__ q, float* __restrict__ d) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;                    // a block's lanes together
  const uint32_t t = divide(i, pieces), c = i - t * pieces.d;
  const float* gp = gate + t * gate_stride + N * c;
  const float* up_ = up + t * up_stride + N * c;
  float g[N / 4][4], u[N / 4][4], y[N];
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    load4(g[k], gp + 4 * k);
    load4(u[k], up_ + 4 * k);
  }
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = gated<GELU>(g[e / 4][e % 4], u[e / 4][e % 4]);
  uint32_t codes[N / 4];
  const float scale = quantize_block<N>(y, codes);
  if constexpr (N == 8) reinterpret_cast<uint2*>(q)[i] = make_uint2(codes[0], codes[1]);
  else q[i] = codes[0];
  if (i % (32 / N) == 0) d[i / (32 / N)] = scale;
}

template <bool NT>
__global__ __launch_bounds__(kThreads) void dequantize_acts_kernel(
    const uint32_t* __restrict__ q, const float* __restrict__ d, int64_t quads,
    float* __restrict__ a) {
  constexpr int U = 4;
  const int64_t i0 = blockIdx.x * (int64_t)(U * kThreads) + threadIdx.x;
  uint32_t c[U];
  float s[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int64_t i = i0 + k * kThreads;
    if (i < quads) {
      c[k] = q[i];
      s[k] = d[i >> 3];
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int64_t i = i0 + k * kThreads;
    if (i < quads)
      store4<NT>(a + 4 * i, make_float4((int8_t)c[k] * s[k], (int8_t)(c[k] >> 8) * s[k],
                                        (int8_t)(c[k] >> 16) * s[k], (int8_t)(c[k] >> 24) * s[k]));
  }
}

}  // namespace

hipError_t launch_quantize_gated_acts(const float* gate, const float* up, int64_t M, int64_t K,
                                      int64_t gate_stride, int64_t up_stride, bool gelu,
                                      int8_t* q, float* d, hipStream_t stream) {
  // Eight values a thread share a block's reciprocal and store both words of codes; below
  // 2^21 values a shorter thread is done sooner (4096 rows of 1536: 11.2 us with eight, 12.2
  // with four; 2048: 7.1 and 7.4; 1024: 4.7 and 4.7; 512: 3.0 and 2.9; 8: 2.4 and 2.1).  The two
  // words need 8-byte alignment.
  const int n = M * K >= (1 << 21) && (reinterpret_cast<uintptr_t>(q) & 7) == 0 ? 8 : 4;
  const auto kernel = n == 8 ? (gelu ? gated_acts_kernel<true, 8> : gated_acts_kernel<false, 8>)
                             : (gelu ? gated_acts_kernel<true, 4> : gated_acts_kernel<false, 4>);
  const int64_t pieces = K / n;
  const Divisor by = divisor((uint32_t)pieces);
  // the pieces of a launch are counted in 31 bits
  const int64_t rows = std::min(M, ((int64_t(1) << 31) - 2 * kThreads) / pieces);
  for (int64_t t = 0; t < M; t += rows) {
    const uint32_t total = (uint32_t)(std::min(M - t, rows) * pieces);
    hipLaunchKernelGGL(kernel, dim3((total + kThreads - 1) / kThreads), dim3(kThreads), 0, stream,
                       gate + t * gate_stride, up + t * up_stride, total, by, gate_stride,
                       up_stride, reinterpret_cast<uint32_t*>(q) + t * (K / 4), d + t * (K / 32));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_dequantize_acts(const int8_t* q, const float* d, int64_t M, int64_t K, float* a,
                                  hipStream_t stream) {
  // From 2^23 values on (32 MB, the XCDs' second-level caches together) the output goes past the
  // caches: 4096 rows of 5120 16.8 us so (6.4 TB/s), 22.5 without; 2048 of 4096 7.0 and 8.1; 1024
  // 4.1 and 5.1.  A kernel that reads all of it at once pays for that (with one that scales the
  // values 51.3 and 46.0, 20.2 and 18.4, 11.8 and 11.7), so that smaller ones stay.
  const int64_t quads = M * (K / 4), per = 4 * kThreads, most = per * kMaxGrid;
  const auto kernel =
      quads >= (1 << 21) ? dequantize_acts_kernel<true> : dequantize_acts_kernel<false>;
  for (int64_t i = 0; i < quads; i += most) {
    const int64_t n = std::min(quads - i, most);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((n + per - 1) / per)), dim3(kThreads), 0, stream,
                       reinterpret_cast<const uint32_t*>(q) + i, d + i / 8, n, a + 4 * i);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rfp2
