// Root-mean-square norms: of heads where they lie, and of whole rows with what is added
// to the residual stream before and the int8 form of the result after.
//
//   h = fl32(x + add)   or   fl32(x + sum_j w_j r_j)
//   y = fl32(h * gain / sqrt(mean(h^2) + eps)),   q, d as rfp2_quantize_acts of y
//
// Sums, the root and the products are fp64, rounded once: a last bit of y may flip a
// code, and so the codes are those of the definition whatever the order of the sums.
// Everything here is bound by the transfer, a value read once and written once: 4096 rows
// of 5120 added, normed and quantized take 47 us (275 MB, 5.9 TB/s), 512 tokens of eight
// experts' rows of 4096 15 us (86 MB, 5.7 TB/s); a single row 2.6 us, of which the launch
// is 1.7.
#include "acts_device.h"
#include "rfp2_internal.h"

namespace rfp2 {

namespace {

constexpr int kThreads = 256;

// Norm of heads: G lanes own a head of D values, C times four each; a workgroup takes 256 / G
// heads of row blockIdx.x.
template <int G, int C, bool NT>
__global__ __launch_bounds__(kThreads) void rms_norm_kernel(const float* x, int H, int D,
                                                            int64_t x_stride,
                                                            const float* __restrict__ gain,
                                                            double eps, float* y,
                                                            int64_t y_stride) {
  const int lane = threadIdx.x & (G - 1);
  const int h = blockIdx.y * (kThreads / G) + threadIdx.x / G;
  if (h >= H) return;                        // all of a head's lanes
  const float* xr = x + blockIdx.x * x_stride + (int64_t)h * D;
  float* yr = y + blockIdx.x * y_stride + (int64_t)h * D;
  float v[C][4], g[C][4];
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = 4 * (lane + c * G);
    if (i < D) {
      load4(v[c], xr + i);
      load4(g[c], gain + i);
    } else {
      v[c][0] = v[c][1] = v[c][2] = v[c][3] = 0.0f;
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fma((double)v[c][e], (double)v[c][e], s);
  const double inv = inverse_root(fma(group_sum<G>(s), reciprocal((double)D), eps));
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = 4 * (lane + c * G);
    if (i >= D) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[c][e] = (float)((double)v[c][e] * inv * (double)g[c][e]);
    store4<NT>(yr + i, make_float4(v[c][0], v[c][1], v[c][2], v[c][3]));
  }
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
  int64_t x_stride, add_stride, h_stride, y_stride;
  double eps;
  int32_t K, top_k;
};
// Arguments of 113 bytes and more cost the host 0.7 us a launch (2.9 us up to there, 3.6).
static_assert(sizeof(NormRows) <= 112, "");
enum { MODE_ROW, MODE_ADD, MODE_SUM };
// What goes past the caches: nothing, what is written in fp32, the rows that are read too.
enum { KEEP, STREAM_OUT, STREAM_ALL };

// Values 4 * i .. 4 * i + 3 of row t of the stream.
template <int MODE, bool NT>
__device__ __forceinline__ void stream4(float (&v)[4], const NormRows& r, int64_t t, int i) {
  if (MODE != MODE_SUM || r.x) load4<NT>(v, r.x + t * r.x_stride + 4 * i);
  else v[0] = v[1] = v[2] = v[3] = 0.0f;
  if constexpr (MODE == MODE_ADD) {
    float a[4];
    load4<NT>(a, r.add + t * r.add_stride + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += a[e];
  }
  if constexpr (MODE == MODE_SUM) {
    double s[4] = {v[0], v[1], v[2], v[3]};
    const float* w = r.weights + t * r.top_k;
    const float* a0 = r.add + t * r.top_k * r.K + 4 * i;
#pragma unroll 8
    for (int j = 0; j < r.top_k; ++j) {
      float a[4];
      load4(a, a0 + (int64_t)j * r.K);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = fma((double)w[j], (double)a[e], s[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)s[e];
  }
}

template <bool NT>
__device__ __forceinline__ void put_normed(float (&v)[4], const float (&g)[4], double inv,
                                           const NormRows& r, int64_t t, int i) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)((double)v[e] * inv * (double)g[e]);
  if (r.y) store4<NT>(r.y + t * r.y_stride + 4 * i, make_float4(v[0], v[1], v[2], v[3]));
  if (r.q) {
    const int64_t at = t * (r.K >> 2) + i;
    uint32_t codes;
    const float scale = quantize4(v, codes);
    r.q[at] = codes;
    if ((threadIdx.x & 7) == 0) r.d[at >> 3] = scale;
  }
}

// One workgroup a row; C quads of a thread stay in registers, what a row has beyond
// kMostQuads of them is read again.  A thread reads back only what it wrote itself, so h and y
// may be the rows that were read.  Where rows or outputs go past the caches, what lies beyond
// does so in its last read and its outputs, and not where it is read again (600 rows of 32768,
// added, y and codes: 54.2 us so, 68.6 with the hint the other way round; 300 of 131072: 166
// and 191; with h 70.7 and 73.5).
constexpr int kMostQuads = 4096;
template <int MODE, int THREADS, int C, int PAST>
__global__ __launch_bounds__(THREADS) void row_norm_kernel(NormRows r) {
  constexpr bool BEYOND = THREADS * C == kMostQuads;   // the widest: rows may have more
  __shared__ double part[THREADS / 64];
  const int64_t t = blockIdx.x;
  const int quads = r.K >> 2;
  const double inv_k = reciprocal((double)r.K);
  float v[C][4], g[C][4];
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * THREADS;
    if (i < quads) stream4<MODE, PAST == STREAM_ALL>(v[c], r, t, i);
    else v[c][0] = v[c][1] = v[c][2] = v[c][3] = 0.0f;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * THREADS;
    if (i < quads) load4(g[c], r.gain + 4 * i);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * THREADS;
    if (r.h && i < quads)
      store4<PAST != KEEP>(r.h + t * r.h_stride + 4 * i,
                           make_float4(v[c][0], v[c][1], v[c][2], v[c][3]));
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fma((double)v[c][e], (double)v[c][e], s);
  }
  if constexpr (BEYOND) {
    // two loops: of loads that differ in nothing but the hint the compiler makes one without
    const auto square = [&](const float (&x)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fma((double)x[e], (double)x[e], s);
    };
    if (r.h) {
      for (int i = threadIdx.x + C * THREADS; i < quads; i += THREADS) {
        float x[4];
        stream4<MODE, PAST == STREAM_ALL>(x, r, t, i);
        store4<false>(r.h + t * r.h_stride + 4 * i, make_float4(x[0], x[1], x[2], x[3]));
        square(x);
      }
    } else {
      for (int i = threadIdx.x + C * THREADS; i < quads; i += THREADS) {
        float x[4];
        stream4<MODE, false>(x, r, t, i);
        square(x);
      }
    }
  }
  s = sum_in_last_lane(s);
  if ((threadIdx.x & 63) == 63) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = part[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) s += part[w];
  const double inv = inverse_root(fma(s, inv_k, r.eps));
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * THREADS;
    if (i < quads) put_normed<PAST != KEEP>(v[c], g[c], inv, r, t, i);
  }
  if constexpr (BEYOND) {
    for (int i = threadIdx.x + C * THREADS; i < quads; i += THREADS) {
      float x[4], gx[4];
      if (r.h) load4(x, r.h + t * r.h_stride + 4 * i);
      else stream4<MODE, PAST == STREAM_ALL>(x, r, t, i);
      load4(gx, r.gain + 4 * i);
      put_normed<PAST != KEEP>(x, gx, inv, r, t, i);
    }
  }
}

// The weighted sum alone: quads [blockIdx.y * 256, ...) of a row.  Stores are ordinary at any
// size, since the stream is read next: 2000 rows of 4096 from one expert each take 15.4 us past
// the caches and 16.9 so, but with the norm that reads them 41.7 and 38.1; 512 from eight 13.3
// either way, 21.4 and 21.5 with the norm.
__global__ __launch_bounds__(kThreads) void combine_kernel(NormRows r) {
  const int64_t t = blockIdx.x;
  const int i = blockIdx.y * kThreads + threadIdx.x;
  if (i >= r.K >> 2) return;
  float v[4];
  stream4<MODE_SUM, false>(v, r, t, i);
  store4<false>(r.h + t * r.h_stride + 4 * i, make_float4(v[0], v[1], v[2], v[3]));
}

using RowKernel = void (*)(NormRows);
struct RowChoice {
  RowKernel kernel;
  int threads;
};

// One quad a thread up to 512 threads, then up to three, beyond 6144 values 1024 threads with up
// to four.  One row, in us, with the threads x quads taken here first: 512 values 1.9 with 128x1,
// 2.3 with 64x2; 1024 1.9 with 256x1, 2.4 with 128x2; 2048 2.2 with 512x1, 2.3 with 1024x1, 2.5
// with 256x2; 4096 2.7 with 512x2, 2.8 with 1024x1, 3.6 with 256x4; 5120 3.0 with 512x3 or
// 1024x2; 6144 3.4 with 512x3, 3.3 with 1024x2; 8192 3.9 with 1024x2, 4.1 with 512x4.  1024 rows,
// sums of eight experts: 4096 32.4 with 512x2, 34.1 with 1024x1; 6144 48.9 with 512x3, 50.6 with
// 1024x2 (fewer rows of such sums: 128 of 4096 6.2 and 6.0, 16 4.0 with either).  8000 rows of
// 256 6.1 with one wave, 9.0 with 256 threads.  What is longer than 16384 values stays out of the
// registers (one row of 32768: 10.8; 17.0 with eight quads a thread).
template <int MODE, int PAST>
RowChoice choose_row(int64_t quads) {
  if (quads <= 64) return {row_norm_kernel<MODE, 64, 1, PAST>, 64};
  if (quads <= 128) return {row_norm_kernel<MODE, 128, 1, PAST>, 128};
  if (quads <= 256) return {row_norm_kernel<MODE, 256, 1, PAST>, 256};
  if (quads <= 512) return {row_norm_kernel<MODE, 512, 1, PAST>, 512};
  if (quads <= 1024) return {row_norm_kernel<MODE, 512, 2, PAST>, 512};
  if (quads <= 1536) return {row_norm_kernel<MODE, 512, 3, PAST>, 512};
  if (quads <= 2048) return {row_norm_kernel<MODE, 1024, 2, PAST>, 1024};
  return {row_norm_kernel<MODE, 1024, 4, PAST>, 1024};
}

// The rows from row t on.
NormRows rows_from(NormRows r, int mode, int64_t t) {
  if (r.x) r.x += t * r.x_stride;
  if (mode == MODE_ADD) r.add += t * r.add_stride;
  if (mode == MODE_SUM) {
    r.add += t * r.top_k * r.K;
    r.weights += t * r.top_k;
  }
  if (r.h) r.h += t * r.h_stride;
  if (r.y) r.y += t * r.y_stride;
  if (r.q) {
    r.q += t * (r.K / 4);
    r.d += t * (r.K / 32);
  }
  return r;
}

template <int MODE>
hipError_t launch_rows(const NormRows& r, int64_t T, hipStream_t stream) {
  const int64_t quads = r.K / 4;
  // More than an XCD's 4 MB second-level cache of output goes past the caches (512 rows of 4096:
  // 6.4 us so, 7.2 without; 256: 3.5 and 3.8; 128: 3.2 and 3.3).  Two rows to be added, of 64 MB
  // and more each, are read past them as well (4096 rows of 5120: 46.5 us so, 50.7 without; 3000:
  // 35.8 and 38.5; 2048 rows of 4096: 20.5 and 18.0); a row alone only where it is read twice (600
  // of 32768: 36.8 and 39.9; but 4096 of 4096 19.5 and 16.3, 4096 of 5120 23.1 and 22.9, 8192
  // 43.1 and 43.5); the experts' rows never.
  const int64_t values = T * r.K;
  const bool sum_alone = MODE == MODE_SUM && !r.gain;
  RowChoice c = {};
  if (!sum_alone) {
    if (values < (1 << 20)) c = choose_row<MODE, KEEP>(quads);
    else if (MODE == MODE_SUM || values < (1 << 24)) c = choose_row<MODE, STREAM_OUT>(quads);
    else if constexpr (MODE == MODE_ADD) c = choose_row<MODE, STREAM_ALL>(quads);
    else if constexpr (MODE == MODE_ROW)
      c = quads <= kMostQuads ? choose_row<MODE, STREAM_OUT>(quads)
                              : RowChoice{row_norm_kernel<MODE, 1024, 4, STREAM_ALL>, 1024};
  }
  const int64_t parts = sum_alone ? (quads + kThreads - 1) / kThreads : 1;
  for (int64_t t = 0; t < T; t += kMaxGrid / parts) {
    const int64_t n = std::min(T - t, kMaxGrid / parts);
    const NormRows part = rows_from(r, MODE, t);
    if (sum_alone)
      hipLaunchKernelGGL(combine_kernel, dim3((uint32_t)n, (uint32_t)parts), dim3(kThreads), 0,
                         stream, part);
    else
      hipLaunchKernelGGL(c.kernel, dim3((uint32_t)n), dim3(c.threads), 0, stream, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int G, int C>
hipError_t launch_heads(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                        const float* gain, double eps, float* y, int64_t y_stride,
                        hipStream_t stream) {
  // One head a group of lanes: 2049 rows of 40 heads of 128 take 13.2 us (6.4 TB/s; 14.2
  // before the root was shortened, and 14.7 with four heads), one row 2.0 and 2.9.  Large
  // outputs go past the caches (16.9 us without, at 64 rows no difference).
  const auto kernel =
      T * H * D >= (1 << 20) ? rms_norm_kernel<G, C, true> : rms_norm_kernel<G, C, false>;
  const int64_t per = kThreads / G, parts = std::min<int64_t>((H + per - 1) / per, 65535);
  for (int64_t t = 0; t < T; t += kMaxGrid / parts) {
    const int64_t n = std::min(T - t, kMaxGrid / parts);
    for (int64_t h = 0; h < H; h += parts * per) {   // a launch holds 65535 workgroups along y
      const int64_t m = std::min(parts, (H - h + per - 1) / per);
      hipLaunchKernelGGL(kernel, dim3((uint32_t)n, (uint32_t)m), dim3(kThreads), 0, stream,
                         x + t * x_stride + h * D, (int)(H - h), (int)D, x_stride, gain, eps,
                         y + t * y_stride + h * D, y_stride);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rms_norm(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                           const float* gain, double eps, float* y, int64_t y_stride,
                           hipStream_t stream) {
  const auto launch = D <= 32    ? launch_heads<8, 1>
                      : D <= 64  ? launch_heads<16, 1>
                      : D <= 128 ? launch_heads<32, 1>
                      : D <= 256 ? launch_heads<64, 1>
                      : D <= 512 ? launch_heads<64, 2>
                                 : launch_heads<64, 4>;
  return launch(x, T, H, D, x_stride, gain, eps, y, y_stride, stream);
}

hipError_t launch_add_rms_norm(const float* x, const float* add, int64_t T, int64_t K,
                               int64_t x_stride, int64_t add_stride, const float* gain,
                               double eps, float* h, int64_t h_stride, float* y,
                               int64_t y_stride, int8_t* q, float* d, hipStream_t stream) {
  const NormRows r = {x, add, nullptr, gain, h, y, reinterpret_cast<uint32_t*>(q), d,
                      x_stride, add_stride, h_stride, y_stride, eps, (int32_t)K, 1};
  return add ? launch_rows<MODE_ADD>(r, T, stream) : launch_rows<MODE_ROW>(r, T, stream);
}

hipError_t launch_moe_combine(const float* x, const float* rows, const float* weights, int64_t T,
                              int64_t top_k, int64_t K, int64_t x_stride, const float* gain,
                              double eps, float* h, int64_t h_stride, float* y,
                              int64_t y_stride, int8_t* q, float* d, hipStream_t stream) {
  const NormRows r = {x, rows, weights, gain, h, y, reinterpret_cast<uint32_t*>(q), d,
                      x_stride, 0, h_stride, y_stride, eps, (int32_t)K, (int32_t)top_k};
  return launch_rows<MODE_SUM>(r, T, stream);
}

}  // namespace rfp2
