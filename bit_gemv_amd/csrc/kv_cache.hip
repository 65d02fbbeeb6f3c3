// The key/value cache: tokens quantized as they are written (with the rotary
// positions of keys and queries in the same launch), and read back.
//
// Both directions are bound by the transfer.  A lane owns four consecutive
// values of a head, so eight lanes own one 32-value block, as in the activation
// quantizer.  The cache keeps eight tokens of one value side by side, so a
// workgroup takes eight tokens at once: where they fill one such group of the
// cache (a prompt's tokens do), a lane holds four values of all eight and stores
// or loads 32 (int8) or 64 (half) consecutive bytes; tokens that do not (a decode
// step's belong to different sequences) are stored value by value.  20011 int8
// tokens of 8 heads of 128 are read back in 36 us (5.8 TB/s; 73 us with a token a
// workgroup and ordinary stores); 48 tokens are rotated and written in 4.6 us, where
// the launch and the chain position, page, store are the time.
#include <hip/hip_fp16.h>

#include "kv_device.h"
#include "rope_device.h"

namespace rfp2 {

namespace {

constexpr int kThreads = 256;
// Tokens from which a workgroup takes eight of them: below, one each, a shorter chain in
// more workgroups (write and read-back of 16 query and 8 key/value heads of 128: 700
// tokens 16.6 against 26.6 us, 1500 tokens 26.4 against 29.7; 4001 tokens 69.8 against
// 39.4, where one token a workgroup writes every line of the values in eight pieces).
// Groups follow the call's first token (first_token): of several prompts in one call only
// those that lie in step with it modulo 8 keep the wide stores of the values.  Writing two of
// 2001 tokens takes 29.4 us over halves and 33.0 over codes, one of 4002 takes 26.1 and
// 27.6; four of 1001 take 32.4 and 32.9, four of 1000 take 26.0 and 27.5.
constexpr int64_t kGroupTokens = 2048;
// Tokens of a launch, eight to a workgroup (two more where they do not line up): a launch
// holds 2^32 threads at most, so more tokens take several.
constexpr int64_t kLaunchTokens = 8 * (kMaxGrid - 2);

// Where the tokens of a workgroup lie in the cache.
template <int TG>
struct Places {
  int32_t pos[TG], page[TG], row[TG];    // page -1: not in the cache; pos < 0: padding
  int together;                          // the tokens fill one group of eight
};

// Tokens t0 .. t0 + TG - 1 of the call, as far as they are in [0, T).
template <int TG>
__device__ __forceinline__ void find_places(Places<TG>* s, const KvView& c, int64_t t0, int64_t T,
                                            const int32_t* seq, const int32_t* pos,
                                            int32_t* err) {
  const int i = threadIdx.x;
  if (i < TG) {
    const int64_t t = t0 + i;
    const bool in = t >= 0 && t < T;
    const int32_t p = in ? pos[t] : -1;
    const int32_t page = p < 0 ? -1 : kv_page(c, seq[t], p);
    if (p >= 0 && page < 0 && err) *err = 1;
    const int32_t row = p & ((1 << c.page_shift) - 1);
    s->pos[i] = p;
    s->page[i] = page;
    s->row[i] = row;
    if (TG > 1) {
      const bool fits = page >= 0 && page == __shfl(page, 0, 64) && (row & 7) == i &&
                        (row >> 3) == (__shfl(row, 0, 64) >> 3);
      const uint64_t all = __ballot(fits);
      if (i == 0) s->together = (all & 0xFF) == 0xFF;
    } else {
      s->together = 0;
    }
  }
}

// The first token of workgroup `block`: groups of eight follow the positions of
// the call's first token, so that a prompt that starts inside a group of the
// cache lines up all the same.
template <int TG>
__device__ __forceinline__ int64_t first_token(const int32_t* pos, int64_t block) {
  return TG == 1 ? block : block * TG - (pos[0] & 7);
}

__device__ __forceinline__ uint2 halves4(const float (&x)[4]) {
  union { __half h[4]; uint2 u; } o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.h[i] = __float2half_rn(x[i]);
  return o.u;
}

// The four values x from d on of a head at `src`, turned.
__device__ __forceinline__ void turn4(float (&x)[4], const float* src, int d, const RopeView& r,
                                      const double2* table) {
  const int half = r.rot >> 1;
  if (d >= r.rot) return;
  if (r.interleaved) {
    const double2 c0 = table[d >> 1], c1 = table[min((d >> 1) + 1, half - 1)];
    const float2 a = rope_turn(x[0], x[1], c0), b = rope_turn(x[2], x[3], c1);
    x[0] = a.x;
    x[1] = a.y;
    if (d + 2 < r.rot) {
      x[2] = b.x;
      x[3] = b.y;
    }
  } else if ((half & 3) == 0) {             // the four partners lie together too
    const bool first = d < half;
    const double2* cs = table + (first ? d : d - half);
    float o[4];
    load4(o, src + (first ? d + half : d - half));
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = rope_value(x[i], o[i], cs[i], first);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = d + i;
      const bool first = e < half;
      if (e < r.rot)
        x[i] = rope_value(x[i], src[first ? e + half : e - half], table[first ? e : e - half], first);
    }
  }
}

// Workgroup (x, y): tokens first_token(x) .., heads [y * per, ...) of a token's H
// query heads, then key heads, then value heads.
template <bool I8, int TG>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(
    KvView c, const float* __restrict__ q, const float* __restrict__ k,
    const float* __restrict__ v, int64_t T, int H, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, const int32_t* __restrict__ seq, const int32_t* __restrict__ pos,
    RopeView r, float* __restrict__ q_out, int64_t q_out_stride, int32_t* __restrict__ err,
    int per) {
  __shared__ double2 table[TG][128];       // rot <= head_dim <= 256
  __shared__ Places<TG> s;
  const int tid = threadIdx.x, D = c.dim, quads = D >> 2, half = r.rot >> 1;
  const int64_t t0 = first_token<TG>(pos, blockIdx.x);
  const int heads = H + 2 * c.heads;
  const int h0 = blockIdx.y * per, h1 = min(heads, h0 + per);
  const int hv = H + c.heads;              // the first value head
  find_places<TG>(&s, c, t0, T, seq, pos, err);
  if (TG > 1) __syncthreads();
  if (r.rot && h0 < hv) {
    for (int i = tid; i < TG * half; i += kThreads) {
      const int tt = TG > 1 ? i / half : 0;
      const int64_t t = t0 + tt;
      if (t >= 0 && t < T)
        table[tt][i - tt * half] = rope_entry(r, TG > 1 ? s.pos[tt] : pos[t], i - tt * half);
    }
  }
  __syncthreads();
  const int slots = kThreads / quads, slot = tid / quads, d = 4 * (tid - slot * quads);
  if (slot >= slots) return;
  const bool together = TG > 1 && s.together;

  // query, key and (where tokens lie apart) value heads: one token of one head at a time
  const int last = together ? min(h1, hv) : h1;
  for (int w = slot; w < (last - h0) * TG; w += slots) {
    const int tt = TG > 1 ? w % TG : 0, h = h0 + (TG > 1 ? w / TG : w);
    const int64_t t = t0 + tt;
    if (t < 0 || t >= T) continue;
    const bool is_q = h < H, is_v = h >= hv;
    const int kvh = h - H - (is_v ? c.heads : 0);
    const float* src = is_q ? q + t * q_stride + (int64_t)h * D
                            : (is_v ? v + t * v_stride : k + t * k_stride) + (int64_t)kvh * D;
    float x[4];
    load4(x, src + d);
    if (!is_v && r.rot) turn4(x, src, d, r, table[tt]);
    if (is_q) {
      store4<(TG > 1)>(q_out + t * q_out_stride + (int64_t)h * D + d,
                       make_float4(x[0], x[1], x[2], x[3]));
      continue;
    }
    const int32_t page = s.page[tt], row = s.row[tt];
    const int64_t rows = page < 0 ? 0 : kv_rows(c, page, kvh);
    if constexpr (I8) {
      uint32_t codes;
      const float scale = quantize4(x, codes);
      if (page < 0) continue;
      if (is_v) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          static_cast<int8_t*>(c.v)[v_at(c, rows, row, d + i)] = (int8_t)(codes >> (8 * i));
      } else {
        *reinterpret_cast<uint32_t*>(static_cast<int8_t*>(c.k) + k_at(c, rows, row, d)) = codes;
      }
      if ((d & 31) == 0) (is_v ? c.vs : c.ks)[scale_at(c, rows, row, d >> 5)] = scale;
    } else {
      if (page < 0) continue;
      const uint2 o = halves4(x);
      if (is_v) {
        uint16_t* dst = static_cast<uint16_t*>(c.v);
        dst[v_at(c, rows, row, d)] = (uint16_t)o.x;
        dst[v_at(c, rows, row, d + 1)] = (uint16_t)(o.x >> 16);
        dst[v_at(c, rows, row, d + 2)] = (uint16_t)o.y;
        dst[v_at(c, rows, row, d + 3)] = (uint16_t)(o.y >> 16);
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.k) + k_at(c, rows, row, d)) = o;
      }
    }
  }

  // value heads of eight tokens that lie together
  if constexpr (TG > 1) {
    if (together) {
      for (int h = max(h0, hv) + slot; h < h1; h += slots) {
        const int kvh = h - hv;
        const int64_t rows = kv_rows(c, s.page[0], kvh);
        float x[TG][4];
#pragma unroll
        for (int i = 0; i < TG; ++i) load4(x[i], v + (t0 + i) * v_stride + (int64_t)kvh * D + d);
        if constexpr (I8) {
          uint32_t codes[TG];
          float scale[TG];
#pragma unroll
          for (int i = 0; i < TG; ++i) scale[i] = quantize4(x[i], codes[i]);
          uint32_t out[8];                 // value d + e: tokens 0..3, tokens 4..7
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t u = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) u |= ((codes[4 * w + i] >> (8 * e)) & 0xFFu) << (8 * i);
              out[2 * e + w] = u;
            }
          uint4* dst = reinterpret_cast<uint4*>(static_cast<int8_t*>(c.v) +
                                                v_at(c, rows, s.row[0], d));
          dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
          dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
          if ((d & 31) == 0) {
            float4* ds = reinterpret_cast<float4*>(c.vs + scale_at(c, rows, s.row[0], d >> 5));
            ds[0] = make_float4(scale[0], scale[1], scale[2], scale[3]);
            ds[1] = make_float4(scale[4], scale[5], scale[6], scale[7]);
          }
        } else {
          union { __half h[4][TG]; uint4 u[4]; } o;
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < TG; ++i) o.h[e][i] = __float2half_rn(x[i][e]);
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.v) +
                                                v_at(c, rows, s.row[0], d));
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = o.u[e];
        }
      }
    }
  }
}

__device__ __forceinline__ float4 scaled4(uint32_t codes, float s) {
  return make_float4((float)(int8_t)codes * s, (float)(int8_t)(codes >> 8) * s,
                     (float)(int8_t)(codes >> 16) * s, (float)(int8_t)(codes >> 24) * s);
}

// Workgroup x reads tokens first_token(x) .. back: keys, then values.
template <bool I8, int TG>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(
    KvView c, int64_t T, const int32_t* __restrict__ seq, const int32_t* __restrict__ pos,
    float* __restrict__ k, float* __restrict__ v, int64_t k_stride, int64_t v_stride,
    int32_t* __restrict__ err) {
  __shared__ Places<TG> s;
  const int tid = threadIdx.x, D = c.dim, quads = D >> 2;
  const int64_t t0 = first_token<TG>(pos, blockIdx.x);
  find_places<TG>(&s, c, t0, T, seq, pos, err);
  __syncthreads();
  const int slots = kThreads / quads, slot = tid / quads, d = 4 * (tid - slot * quads);
  if (slot >= slots) return;
  const bool together = TG > 1 && s.together;
  const int last = together ? c.heads : 2 * c.heads;
#pragma unroll 4
  for (int w = slot; w < last * TG; w += slots) {
    const int tt = TG > 1 ? w % TG : 0, hh = TG > 1 ? w / TG : w;
    const int64_t t = t0 + tt;
    if (t < 0 || t >= T) continue;
    const bool is_v = hh >= c.heads;
    const int h = is_v ? hh - c.heads : hh;
    const float none = s.pos[tt] < 0 ? 0.0f : __builtin_nanf("");
    float4 x = make_float4(none, none, none, none);
    if (s.page[tt] >= 0) {
      const int64_t rows = kv_rows(c, s.page[tt], h);
      const int row = s.row[tt];
      if constexpr (I8) {
        const float sc = (is_v ? c.vs : c.ks)[scale_at(c, rows, row, d >> 5)];
        uint32_t codes;
        if (is_v) {
          const uint8_t* p = static_cast<const uint8_t*>(c.v) + v_at(c, rows, row, d);
          codes = p[0] | p[8] << 8 | p[16] << 16 | (uint32_t)p[24] << 24;
        } else {
          codes = *reinterpret_cast<const uint32_t*>(static_cast<const int8_t*>(c.k) +
                                                     k_at(c, rows, row, d));
        }
        x = scaled4(codes, sc);
      } else {
        union { __half h[4]; uint2 u; } o;
        if (is_v) {
          const __half* p = static_cast<const __half*>(c.v) + v_at(c, rows, row, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) o.h[i] = p[8 * i];
        } else {
          o.u = *reinterpret_cast<const uint2*>(static_cast<const __half*>(c.k) +
                                                k_at(c, rows, row, d));
        }
        x = make_float4(__half2float(o.h[0]), __half2float(o.h[1]), __half2float(o.h[2]),
                        __half2float(o.h[3]));
      }
    }
    float* dst = is_v ? v + t * v_stride : k + t * k_stride;
    store4<(TG > 1)>(dst + (int64_t)h * D + d, x);
  }
  if constexpr (TG > 1) {
    if (together) {
      for (int h = slot; h < c.heads; h += slots) {
        const int64_t rows = kv_rows(c, s.page[0], h);
        const int64_t at = v_at(c, rows, s.row[0], d);
        float x[TG][4];
        if constexpr (I8) {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(c.v) + at);
          const float4* ps =
              reinterpret_cast<const float4*>(c.vs + scale_at(c, rows, s.row[0], d >> 5));
          const uint4 a = p[0], b = p[1];
          const float4 s0 = ps[0], s1 = ps[1];
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          const float sc[TG] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < TG; ++i)
              x[i][e] = (float)(int8_t)(w[2 * e + (i >> 2)] >> (8 * (i & 3))) * sc[i];
        } else {
          union { uint4 u[4]; __half h[4][TG]; } o;
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(c.v) + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) o.u[e] = p[e];
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < TG; ++i) x[i][e] = __half2float(o.h[e][i]);
        }
#pragma unroll
        for (int i = 0; i < TG; ++i)
          store4<true>(v + (t0 + i) * v_stride + (int64_t)h * D + d,
                       make_float4(x[i][0], x[i][1], x[i][2], x[i][3]));
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_write(const KvView& c, bool i8, const float* q, const float* k,
                           const float* v, int64_t T, int64_t H, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const int32_t* seq,
                           const int32_t* pos, const RopeView& rope, float* q_out,
                           int64_t q_out_stride, int32_t* err, hipStream_t stream) {
  const bool wide = T >= kGroupTokens;
  const int heads = (int)H + 2 * c.heads;
  // A workgroup takes one pass of its threads over the heads (eight heads of 128
  // values), and computes the angles of its tokens for itself: at 4001 tokens of 32 heads
  // the write and read-back take 41 us, 54 us with half the heads a workgroup and 64 us
  // with all of them (502 workgroups, each a long chain).
  const int per = kThreads / (c.dim / 4);
  const auto kernel = wide ? (i8 ? kv_write_kernel<true, 8> : kv_write_kernel<false, 8>)
                           : (i8 ? kv_write_kernel<true, 1> : kv_write_kernel<false, 1>);
  for (int64_t t = 0; t < T; t += kLaunchTokens) {
    const int64_t n = std::min(T - t, kLaunchTokens), blocks = wide ? n / 8 + 2 : n;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)blocks, (uint32_t)((heads + per - 1) / per)),
                       dim3(kThreads), 0, stream, c, H ? q + t * q_stride : q, k + t * k_stride,
                       v + t * v_stride, n, (int)H, q_stride, k_stride, v_stride, seq + t,
                       pos + t, rope, H ? q_out + t * q_out_stride : q_out, q_out_stride, err,
                       per);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv_read(const KvView& c, bool i8, int64_t T, const int32_t* seq,
                          const int32_t* pos, float* k, float* v, int64_t k_stride,
                          int64_t v_stride, int32_t* err, hipStream_t stream) {
  const bool wide = T >= kGroupTokens;
  const auto kernel = wide ? (i8 ? kv_read_kernel<true, 8> : kv_read_kernel<false, 8>)
                           : (i8 ? kv_read_kernel<true, 1> : kv_read_kernel<false, 1>);
  for (int64_t t = 0; t < T; t += kLaunchTokens) {
    const int64_t n = std::min(T - t, kLaunchTokens);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(wide ? n / 8 + 2 : n)), dim3(kThreads), 0, stream,
                       c, n, seq + t, pos + t, k + t * k_stride, v + t * v_stride, k_stride,
                       v_stride, err);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rfp2
