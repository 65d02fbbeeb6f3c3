// Routing: which experts a token goes to and with what weights, from the router's
// logits; the ids are what the routed products take.
//
//   p = softmax(l) or 1 / (1 + exp(-l)),   v = p + bias (v = l without a bias),
//   the best groups of experts (each by the sum of its one or two largest v),
//   the top_k largest v in them (the lower expert first among equals),
//   w = scale * p, divided by the chosen p's sum where asked.
//
// Scores and choices are fp64: which of two experts is larger may hang on the last bit
// of fp32 scores.  A logit of minus infinity masks its expert (v = -inf, p = 0).
#include <cmath>

#include "rfp2_internal.h"

namespace rfp2 {

namespace {

constexpr int kNone = 0x7FFFFFFF;

// One wave a token; v [E] and p [E] in LDS.
__global__ __launch_bounds__(64) void moe_route_kernel(
    const float* __restrict__ logits, int64_t t0, int E, int64_t stride,
    const float* __restrict__ bias, int sigmoid, int groups, int group_top, int top_groups,
    int top_k, int renorm, double scale, int32_t* __restrict__ ids, float* __restrict__ weights,
    int32_t* __restrict__ err) {
  extern __shared__ double smem[];
  double *v = smem, *p = smem + E;
  __shared__ double value[64];
  __shared__ int chosen[64];
  const int lane = threadIdx.x;
  const int64_t t = t0 + blockIdx.x;
  const float* l = logits + t * stride;

  float top = -INFINITY;
  bool bad = false;
  for (int e = lane; e < E; e += 64) {
    const float x = l[e];
    bad = bad || !(x < INFINITY) || (bias && !std::isfinite(bias[e]));
    top = fmaxf(top, x);
  }
  for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if (__any(bad)) {                          // nothing can be said of this token
    if (lane < top_k) {
      ids[t * top_k + lane] = -1;
      weights[t * top_k + lane] = __builtin_nanf("");
    }
    if (lane == 0 && err) *err = 1;
    return;
  }
  double sum = 0.0;
  for (int e = lane; e < E; e += 64) {
    const double x = l[e];
    const double s = x == -INFINITY ? 0.0 : sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top);
    p[e] = s;
    sum += s;
  }
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  const double share = sigmoid || sum == 0.0 ? 1.0 : 1.0 / sum;
  for (int e = lane; e < E; e += 64) {
    p[e] *= share;
    v[e] = l[e] == -INFINITY ? -INFINITY : bias ? p[e] + (double)bias[e] : (double)l[e];
  }
  __syncthreads();
  if (groups > 1) {
    const int per = E / groups;
    if (lane < groups) {
      double a = -INFINITY, b = -INFINITY;   // the two largest
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        b = fmax(b, fmin(a, v[e]));
        a = fmax(a, v[e]);
      }
      value[lane] = group_top == 2 && b != -INFINITY ? a + b : a;
    }
    __syncthreads();
    if (lane < groups) {
      int before = 0;
      for (int g = 0; g < groups; ++g)
        before += value[g] > value[lane] || (value[g] == value[lane] && g < lane);
      if (before >= top_groups)
        for (int e = lane * per; e < (lane + 1) * per; ++e) v[e] = __builtin_nan("");
    }
    __syncthreads();
  }
  for (int j = 0; j < top_k; ++j) {          // NaN: taken, or not to be had
    double best = -INFINITY;
    int at = kNone;
    for (int e = lane; e < E; e += 64)
      if (v[e] > best || (v[e] == best && e < at)) {
        best = v[e];
        at = e;
      }
    for (int o = 32; o >= 1; o >>= 1) {
      const double ob = __shfl_xor(best, o, 64);
      const int oa = __shfl_xor(at, o, 64);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (lane == 0) {
      chosen[j] = at;
      v[at] = __builtin_nan("");
    }
    __syncthreads();
  }
  const int id = lane < top_k ? chosen[lane] : 0;
  double w = lane < top_k ? p[id] : 0.0;
  if (renorm) {
    double total = w;
    for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o, 64);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (lane < top_k) {
    ids[t * top_k + lane] = id;
    weights[t * top_k + lane] = (float)(scale * w);
  }
}

}  // namespace

hipError_t launch_moe_route(const float* logits, int64_t T, int64_t E, int64_t stride,
                            const float* bias, bool sigmoid, int groups, int group_top,
                            int top_groups, int top_k, bool renorm, double scale, int32_t* ids,
                            float* weights, int32_t* err, hipStream_t stream) {
  for (int64_t t = 0; t < T; t += kMaxGrid) {
    hipLaunchKernelGGL(moe_route_kernel, dim3((uint32_t)std::min(T - t, kMaxGrid)), dim3(64),
                       16 * (size_t)E, stream, logits, t, (int)E, stride, bias, sigmoid ? 1 : 0,
                       groups, group_top, top_groups, top_k, renorm ? 1 : 0, scale, ids, weights,
                       err);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rfp2
