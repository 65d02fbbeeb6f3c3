// The key/value cache: tokens quantized as they are written (with the rotary
// positions of keys and queries in the same launch), and read back.
#include <hip/hip_fp16.h>

#include "kv_device.h"
#include "rope_device.h"

namespace rfp2 {

namespace {

constexpr int kThreads = 256;

// One workgroup handles heads [blockIdx.y * per, ...) of token blockIdx.x; its
// heads are the token's H query heads, then its key heads, then its value
// heads.  A lane owns four consecutive values of a head, so eight lanes own
// one 32-value block, as in the activation quantizer.
template <bool I8>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(
    KvView c, const float* __restrict__ q, const float* __restrict__ k,
    const float* __restrict__ v, int H, int64_t q_stride, int64_t k_stride, int64_t v_stride,
    const int32_t* __restrict__ seq, const int32_t* __restrict__ pos, RopeView r,
    float* __restrict__ q_out, int64_t q_out_stride, int32_t* __restrict__ err, int per) {
  __shared__ double2 table[128];           // rot <= head_dim <= 256
  const int64_t t = blockIdx.x;
  const int32_t p = pos[t];
  if (r.rot) {
    rope_table(table, r, p, threadIdx.x, kThreads);
    __syncthreads();
  }
  const int32_t page = p < 0 ? -1 : kv_page(c, seq[t], p);
  if (p >= 0 && page < 0 && err && threadIdx.x == 0) *err = 1;
  const int row = p & ((1 << c.page_shift) - 1);
  const int heads = H + 2 * c.heads, D = c.dim, quads = D >> 2;
  const int h0 = blockIdx.y * per, h1 = min(heads, h0 + per);
  const int half = r.rot >> 1;
  for (int u = threadIdx.x; u < (h1 - h0) * quads; u += kThreads) {
    const int h = h0 + u / quads, d = 4 * (u % quads);
    const bool is_q = h < H, is_v = h >= H + c.heads;
    const int kvh = h - H - (is_v ? c.heads : 0);
    const float* src = is_q ? q + t * q_stride + (int64_t)h * D
                            : (is_v ? v + t * v_stride : k + t * k_stride) + (int64_t)kvh * D;
    const float4 x4 = *reinterpret_cast<const float4*>(src + d);
    float x[4] = {x4.x, x4.y, x4.z, x4.w};
    if (!is_v && d < r.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = d + i;
        if (e < r.rot) {
          if (r.interleaved) {
            const float2 o = (i & 1) ? rope_turn(i == 1 ? x4.x : x4.z, i == 1 ? x4.y : x4.w,
                                                 table[e >> 1])
                                     : rope_turn(i == 0 ? x4.x : x4.z, i == 0 ? x4.y : x4.w,
                                                 table[e >> 1]);
            x[i] = (i & 1) ? o.y : o.x;
          } else if (e < half) {
            x[i] = rope_turn(x[i], src[e + half], table[e]).x;
          } else {
            x[i] = rope_turn(src[e - half], x[i], table[e - half]).y;
          }
        }
      }
    }
    if (is_q) {
      *reinterpret_cast<float4*>(q_out + t * q_out_stride + (int64_t)h * D + d) =
          make_float4(x[0], x[1], x[2], x[3]);
      continue;
    }
    const int64_t rows = page < 0 ? 0 : kv_rows(c, page, kvh);
    if constexpr (I8) {
      // code and scale as quantize_acts_kernel computes them
      float amax = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
      int finite = isfinite(x[0]) && isfinite(x[1]) && isfinite(x[2]) && isfinite(x[3]);
#pragma unroll
      for (int off = 4; off >= 1; off >>= 1) {
        amax = fmaxf(amax, __shfl_xor(amax, off, 64));
        finite &= __shfl_xor(finite, off, 64);
      }
      float scale = __fdiv_rn(amax, 127.0f);
      int8_t code[4] = {0, 0, 0, 0};
      if (!finite) {
        scale = __builtin_nanf("");
      } else if (scale != 0.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          code[i] = (int8_t)fminf(fmaxf(roundf(__fdiv_rn(x[i], scale)), -127.0f), 127.0f);
      }
      if (page < 0) continue;
      if (is_v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) static_cast<int8_t*>(c.v)[v_at(c, rows, row, d + i)] = code[i];
      } else {
        *reinterpret_cast<char4*>(static_cast<int8_t*>(c.k) + k_at(c, rows, row, d)) =
            make_char4(code[0], code[1], code[2], code[3]);
      }
      if ((d & 31) == 0) (is_v ? c.vs : c.ks)[scale_at(c, rows, row, d >> 5)] = scale;
    } else {
      if (page < 0) continue;
      const __half o[4] = {__float2half_rn(x[0]), __float2half_rn(x[1]), __float2half_rn(x[2]),
                           __float2half_rn(x[3])};
      if (is_v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) static_cast<__half*>(c.v)[v_at(c, rows, row, d + i)] = o[i];
      } else {
        *reinterpret_cast<uint2*>(static_cast<__half*>(c.k) + k_at(c, rows, row, d)) =
            *reinterpret_cast<const uint2*>(o);
      }
    }
  }
}

// One workgroup reads token blockIdx.x back, keys then values, four values a
// lane.
template <bool I8>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(
    KvView c, const int32_t* __restrict__ seq, const int32_t* __restrict__ pos,
    float* __restrict__ k, float* __restrict__ v, int64_t k_stride, int64_t v_stride,
    int32_t* __restrict__ err) {
  const int64_t t = blockIdx.x;
  const int32_t p = pos[t];
  const int32_t page = p < 0 ? -1 : kv_page(c, seq[t], p);
  if (p >= 0 && page < 0 && err && threadIdx.x == 0) *err = 1;
  const int row = p & ((1 << c.page_shift) - 1);
  const int D = c.dim, quads = D >> 2;
  const float none = p < 0 ? 0.0f : __builtin_nanf("");
  for (int u = threadIdx.x; u < 2 * c.heads * quads; u += kThreads) {
    const bool is_v = u >= c.heads * quads;
    const int w = is_v ? u - c.heads * quads : u;
    const int h = w / quads, d = 4 * (w % quads);
    float x[4] = {none, none, none, none};
    if (page >= 0) {
      const int64_t rows = kv_rows(c, page, h);
      const float s = I8 ? (is_v ? c.vs : c.ks)[scale_at(c, rows, row, d >> 5)] : 1.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = is_v ? v_at(c, rows, row, d + i) : k_at(c, rows, row, d + i);
        const void* from = is_v ? c.v : c.k;
        x[i] = I8 ? (float)static_cast<const int8_t*>(from)[at] * s
                  : __half2float(static_cast<const __half*>(from)[at]);
      }
    }
    float* dst = is_v ? v + t * v_stride : k + t * k_stride;
    *reinterpret_cast<float4*>(dst + (int64_t)h * D + d) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

}  // namespace

hipError_t launch_kv_write(const KvView& c, bool i8, const float* q, const float* k,
                           const float* v, int64_t T, int64_t H, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const int32_t* seq,
                           const int32_t* pos, const RopeView& rope, float* q_out,
                           int64_t q_out_stride, int32_t* err, hipStream_t stream) {
  const int heads = (int)H + 2 * c.heads, per = heads;
  const auto kernel = i8 ? kv_write_kernel<true> : kv_write_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((uint32_t)T, (uint32_t)((heads + per - 1) / per)),
                     dim3(kThreads), 0, stream, c, q, k, v, (int)H, q_stride, k_stride, v_stride,
                     seq, pos, rope, q_out, q_out_stride, err, per);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvView& c, bool i8, int64_t T, const int32_t* seq,
                          const int32_t* pos, float* k, float* v, int64_t k_stride,
                          int64_t v_stride, int32_t* err, hipStream_t stream) {
  const auto kernel = i8 ? kv_read_kernel<true> : kv_read_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((uint32_t)T), dim3(kThreads), 0, stream, c, seq, pos, k, v,
                     k_stride, v_stride, err);
  return hipGetLastError();
}

}  // namespace rfp2
