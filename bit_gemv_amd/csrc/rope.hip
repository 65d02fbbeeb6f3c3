// Rotary positions: the frequencies of the pairs and the rotation of heads.
#include "kv_device.h"
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
// thread owns a unit of a head and takes every head's: four pairs of the half
// style (V4: two 16-byte accesses), two neighbouring pairs of the interleaved one
// (V4: one access), or one pair; past the rotated part, four values (V4) or one
// that are copied.  Its pairs are read before they are written, so x may be y.
template <bool INTER, bool V4, bool NT>
__global__ __launch_bounds__(kThreads) void rope_kernel(const float* x, int H, int D,
                                                        int64_t x_stride,
                                                        const int32_t* __restrict__ pos,
                                                        RopeView r, float* y, int64_t y_stride,
                                                        int per) {
  __shared__ double2 table[kMaxRopeDim / 2];
  constexpr int PAIRS = V4 ? (INTER ? 2 : 4) : 1;     // of a unit
  constexpr int COPY = V4 ? 4 : 1;                    // values of a unit that is copied
  constexpr int BATCH = 4;                            // heads whose values are in flight
  const int64_t t = blockIdx.x;
  const int half = r.rot >> 1, tid = threadIdx.x;
  const int h1 = min(H, ((int)blockIdx.y + 1) * per);
  const int turning = half / PAIRS, units = turning + (D - r.rot) / COPY;
  const float* xr = x + t * x_stride;
  float* yr = y + t * y_stride;
  const int width = min(units, kThreads), slots = kThreads / width, slot = tid / width;
  const int lane = tid - slot * width;
  const int32_t p = pos[t];
  for (int i = tid; i < half; i += kThreads) table[i] = rope_entry(r, p, i);
  __syncthreads();
  if (slot >= slots) return;
  for (int u = lane; u < units; u += width) {
    const bool turns = u < turning;
    const int a = turns ? (INTER ? 2 : 1) * PAIRS * u : r.rot + COPY * (u - turning);
    double2 cs[PAIRS];
    if (turns) {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) cs[i] = table[PAIRS * u + i];
    }
    for (int hb = blockIdx.y * per + slot; hb < h1; hb += BATCH * slots) {
      float4 lo[BATCH], hi[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int h = hb + k * slots;
        if (h >= h1) continue;
        const float* s = xr + (int64_t)h * D + a;
        if constexpr (V4) {
          lo[k] = *reinterpret_cast<const float4*>(s);
          if (!INTER && turns) hi[k] = *reinterpret_cast<const float4*>(s + half);
        } else {
          lo[k].x = s[0];
          if (turns) hi[k].x = s[INTER ? 1 : half];
        }
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int h = hb + k * slots;
        if (h >= h1) continue;
        float* o = yr + (int64_t)h * D + a;
        float4 l = lo[k], g = hi[k];
        if (turns) {
          if constexpr (V4 && INTER) {
            const float2 u0 = rope_turn(l.x, l.y, cs[0]), u1 = rope_turn(l.z, l.w, cs[1]);
            l = make_float4(u0.x, u0.y, u1.x, u1.y);
          } else if constexpr (V4) {
            const float2 u0 = rope_turn(l.x, g.x, cs[0]), u1 = rope_turn(l.y, g.y, cs[1]),
                         u2 = rope_turn(l.z, g.z, cs[2]), u3 = rope_turn(l.w, g.w, cs[3]);
            l = make_float4(u0.x, u1.x, u2.x, u3.x);
            g = make_float4(u0.y, u1.y, u2.y, u3.y);
          } else {
            const float2 u0 = rope_turn(l.x, g.x, cs[0]);
            l.x = u0.x;
            g.x = u0.y;
          }
        }
        if constexpr (V4) {
          store4<NT>(o, l);
          if (!INTER && turns) store4<NT>(o + half, g);
        } else {
          o[0] = l.x;
          if (turns) o[INTER ? 1 : half] = g.x;
        }
      }
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
  // 16-byte accesses where the pairs allow them
  const bool inter = rope.interleaved != 0;
  const bool v4 = rope.rot % (inter ? 4 : 8) == 0;
  const int units = rope.rot / (v4 ? (inter ? 4 : 8) : 2) + ((int)D - rope.rot) / (v4 ? 4 : 1);
  // Many tokens: a workgroup takes all heads of its token (the angles are computed once),
  // and what it writes goes past the caches (4096 tokens of 40 heads of 128: 34.5 us
  // without, 27.1 us so; 700 tokens 7.1 us, 8.2 the other way).  Few tokens: one head a
  // thread, and the next call finds the result in the cache (128 tokens 3.5 us, 3.75).
  const bool many = T >= 512;
  const int per = many ? (int)H : std::max(1, kThreads / std::min(units, kThreads));
  const auto kernel =
      !v4    ? (inter ? rope_kernel<true, false, false> : rope_kernel<false, false, false>)
      : many ? (inter ? rope_kernel<true, true, true> : rope_kernel<false, true, true>)
             : (inter ? rope_kernel<true, true, false> : rope_kernel<false, true, false>);
  // One workgroup a token: a launch holds 2^32 threads at most, so more tokens take several.
  for (int64_t t = 0; t < T; t += kMaxGrid) {
    const int64_t n = std::min(T - t, kMaxGrid);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)n, (uint32_t)((H + per - 1) / per)),
                       dim3(kThreads), 0, stream, x + t * x_stride, (int)H, (int)D, x_stride,
                       pos + t, rope, y + t * y_stride, y_stride, per);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rfp2
