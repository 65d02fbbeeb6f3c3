// Routing: which experts a token goes to and with what weights, from the router's
// logits; the ids are what the routed products take.
//
//   p = softmax(l) or 1 / (1 + exp(-l)),   v = p + bias (v = l without a bias),
//   the best groups of experts (each by the sum of its one or two largest v),
//   the top_k largest v in them (the lower expert first among equals),
//   w = scale * p, divided by the chosen p's sum where asked.
//
// Scores and choices are fp64: which of two experts is larger may hang on the last bit
// of fp32 scores.  A logit of minus infinity masks its expert.
//
// One wave a token.  Lane i holds experts i V .. i V + V - 1, sorted once; a choice is a
// maximum over the wave and the lowest lane that holds it, which is the lowest expert, and
// that lane's list moves up.  LDS holds what lies across lanes: groups, and the chosen
// experts' scores.  What is chosen without a bias needs no scores: logits are compared as
// whole numbers, and only the chosen ones' exponentials are taken (all of them where a
// softmax is not divided by the chosen ones' sum).  What bounds it is the chain of choices
// and the launch for few tokens (1 over 128 experts 2.6 us, 1024 over 64 2.5), the vector
// instructions for many (4099 over 256 with a bias 7.2 us, with groups 9.3: reading the
// logits takes 0.7).
#include <cmath>
#include <type_traits>

#include "acts_device.h"
#include "rfp2_internal.h"
#include "scores_device.h"

namespace rfp2 {

namespace {

struct Router {
  const float* logits;
  const float* bias;        // null: none
  int32_t* ids;
  float* weights;
  int32_t* err;
  double scale;
  int64_t stride;
  int32_t T, E, groups, group_top, top_groups, top_k;
  int32_t waves;            // of a workgroup
  int32_t per, shift;       // experts of a group; 2^shift lanes look at it, groups << shift <= 64
  uint32_t group_magic;     // ceil(2^31 / (E / groups))
  bool sigmoid, renorm;
};
// Larger arguments, or blockDim in a kernel, cost the host 0.7 us a launch.
static_assert(sizeof(Router) <= 112, "");

// What experts are compared by, the larger first: a logit's bits, or those of a score with
// its bias, as a whole number in the order of the numbers.  The lowest number's is that of
// minus infinity, a mask (chosen where nothing else is left); below it what is taken or was never
// there.
constexpr uint32_t kGone = 0;
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);        // minus zero is zero
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ float number(uint32_t k) {
  return __uint_as_float(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u));
}
// The largest over the wave.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t larger_of(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, ROWS == 0xF));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = larger_of<0xB1, 0xF>(x);               // neighbours
  x = larger_of<0x4E, 0xF>(x);               // pairs
  x = larger_of<0x141, 0xF>(x);              // the other four of eight
  x = larger_of<0x140, 0xF>(x);              // the other eight of sixteen
  x = larger_of<0x142, 0xA>(x);              // rows 1 and 3: the row before
  x = larger_of<0x143, 0xC>(x);              // rows 2 and 3: the two before
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// The lanes that hold the largest key.  Of 64 bits the upper half decides, and the lower
// where several lanes share it.
__device__ __forceinline__ uint64_t lanes_of_largest(uint32_t k) {
  return __ballot(k == wave_max(k));
}
__device__ __forceinline__ uint64_t lanes_of_largest(uint64_t k) {
  const uint32_t hi = (uint32_t)(k >> 32), lo = (uint32_t)k;
  const bool top = hi == wave_max(hi);
  const uint64_t lanes = __ballot(top);
  if ((lanes & (lanes - 1)) == 0) return lanes;
  const uint32_t most = wave_max(top ? lo : 0u);
  return __ballot(top && lo == most);
}

// Scores before they are divided by the softmax's sum; what exp(-690) is more than counts as
// 0.  Without branches, so that the V chains of one lane run side by side.
template <int V>
__device__ __forceinline__ void scores(double (&p)[V], const float (&x)[V], float top,
                                       bool sigmoid) {
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = logistic(__builtin_amdgcn_fmed3f(x[i], -690.0f, 690.0f));
      p[i] = x[i] >= -690.0f ? p[i] : 0.0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double d = (double)x[i] - (double)top;
      p[i] = exp_f64(fmax(d, -690.0));
      p[i] = d >= -690.0 ? p[i] : 0.0;       // not for NaN: all are minus infinity
    }
  }
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }
template <int CTRL>
__device__ __forceinline__ float other(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double other(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float of_lane(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
__device__ __forceinline__ double of_lane(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// 2^shift lanes look at a group's experts (minus infinity: masked); true for the lanes whose
// group stays.
template <class F>
__device__ __forceinline__ bool group_stays(const F* v, const Router& r) {
  const int lane = threadIdx.x & 63, lanes = 1 << r.shift;
  const int g = lane >> r.shift;
  F a = -INFINITY, b = -INFINITY;            // the two largest
  if (g < r.groups)
    for (int e = lane & (lanes - 1); e < r.per; e += lanes) {
      const F x = v[g * r.per + e];
      b = larger(b, smaller(x, a));
      a = larger(a, x);
    }
  const auto join = [&](F oa, F ob) {
    b = larger(larger(b, ob), smaller(a, oa));
    a = larger(a, oa);
  };
  if (lanes >= 2) join(other<0xB1>(a), other<0xB1>(b));
  if (lanes >= 4) join(other<0x4E>(a), other<0x4E>(b));
  if (lanes >= 8) join(other<0x141>(a), other<0x141>(b));
  if (lanes >= 16) join(other<0x140>(a), other<0x140>(b));
  if (lanes >= 32) join(__shfl_xor(a, 16, 64), __shfl_xor(b, 16, 64));
  if (r.group_top == 2 && b > -INFINITY) a += b;
  int before = 0;
  for (int o = 0; o < r.groups; ++o) {
    const F x = of_lane(a, o << r.shift);
    before += x > a || (x == a && o < g);
  }
  return g < r.groups && before < r.top_groups;
}

// A lane's V keys: its largest, where it was among the V (the first of equals), and how to
// take it away.  Up to eight are sorted once and move up (by neighbours' exchanges, which leave
// equals in their order); more are lists of eight.
template <int V, class K>
struct Held {
  K key[V];
  int at[V];
  __device__ __forceinline__ explicit Held(const K* k) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = k[i];
      at[i] = i;
    }
#pragma unroll
    for (int round = 0; round < V; ++round)
#pragma unroll
      for (int i = round & 1; i + 1 < V; i += 2) {
        const bool swap = key[i + 1] > key[i];
        const K a = key[i], b = key[i + 1];
        const int pa = at[i], pb = at[i + 1];
        key[i] = swap ? b : a;
        key[i + 1] = swap ? a : b;
        at[i] = swap ? pb : pa;
        at[i + 1] = swap ? pa : pb;
      }
  }
  __device__ __forceinline__ K best() const { return key[0]; }
  __device__ __forceinline__ int place() const { return at[0]; }
  __device__ __forceinline__ void take(bool mine) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = mine ? (i + 1 < V ? key[(i + 1) % V] : (K)kGone) : key[i];
      if (i + 1 < V) at[i] = mine ? at[(i + 1) % V] : at[i];
    }
  }
};
template <int N, class K>
struct Lists {
  Held<8, K> list;
  Lists<N - 1, K> rest;
  __device__ __forceinline__ explicit Lists(const K* k) : list(k), rest(k + 8) {}
  __device__ __forceinline__ bool later() const { return rest.best() > list.best(); }
  __device__ __forceinline__ K best() const { return later() ? rest.best() : list.best(); }
  __device__ __forceinline__ int place() const {
    return later() ? 8 + rest.place() : list.place();
  }
  __device__ __forceinline__ void take(bool mine) {
    const bool l = later();
    list.take(mine && !l);
    rest.take(mine && l);
  }
};
template <class K>
struct Lists<1, K> : Held<8, K> {
  using Held<8, K>::Held;
};
template <class K>
struct Held<16, K> : Lists<2, K> {
  using Lists<2, K>::Lists;
};
template <class K>
struct Held<32, K> : Lists<4, K> {
  using Lists<4, K>::Lists;
};

// A wave's LDS operations are done in their order; the compiler has to keep it.
__device__ __forceinline__ void in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int V, bool BIAS>
__global__ __launch_bounds__(256) void moe_route_kernel(Router r) {
  using K = std::conditional_t<BIAS, uint64_t, uint32_t>;
  using F = std::conditional_t<BIAS, double, float>;
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x * r.waves + wave;
  if (t >= r.T) return;                      // waves do not wait for each other
  const float* l = r.logits + t * r.stride;

  float x[V], bias[V];                       // past the last expert: the last, masked
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = l[min(lane * V + i, r.E - 1)];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = r.bias[min(lane * V + i, r.E - 1)];
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad = bad || !(x[i] < INFINITY);
    if constexpr (BIAS) bad = bad || !(fabsf(bias[i]) < INFINITY);
    if (lane * V + i >= r.E) x[i] = -INFINITY;
  }
  if (__any(bad)) {                          // nothing can be said of this token
    if (lane < r.top_k) {
      r.ids[t * r.top_k + lane] = -1;
      r.weights[t * r.top_k + lane] = __builtin_nanf("");
    }
    if (lane == 0 && r.err) *r.err = 1;
    return;
  }

  float top = 0.0f;
  double share = 1.0;
  if (!r.sigmoid) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, ordered(x[i]));
    top = number(wave_max(m));
  }
  double p[V];
  const bool all = BIAS || (!r.sigmoid && !r.renorm);   // scores of all experts, kept in LDS
  double* kept = smem + wave * r.E;
  if (all) {
    scores<V>(p, x, top, r.sigmoid);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i < r.E) kept[lane * V + i] = p[i];
    if (!r.sigmoid) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += p[i];
      sum = group_sum<64>(sum);
      share = sum > 0.0 ? reciprocal(sum) : 0.0;
    }
  }
  F v[V];
  K key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (BIAS) v[i] = x[i] == -INFINITY ? (F)x[i] : p[i] * share + (double)bias[i];
    else v[i] = x[i];
    key[i] = ordered(v[i]);                  // of minus infinity: a mask, below every number's
    if (lane * V + i >= r.E) key[i] = kGone;
  }

  if (r.groups > 1) {
    F* mine = reinterpret_cast<F*>(smem + (all ? r.waves * r.E : 0)) + wave * r.E;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i < r.E) mine[lane * V + i] = v[i];
    in_order();
    const uint64_t stays = __ballot(group_stays(mine, r));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t g = __umulhi(2u * (lane * V + i), r.group_magic);
      if (!((stays >> ((g << r.shift) & 63)) & 1)) key[i] = kGone;
    }
  }

  Held<V, K> held(key);
  int id = 0;                                // lane j: choice j
  for (int j = 0; j < r.top_k; ++j) {
    const int from = __builtin_ctzll(lanes_of_largest(held.best()));
    const int chosen = from * V + __builtin_amdgcn_readlane(held.place(), from);
    if (lane == j) id = chosen;
    held.take(lane == from);
  }

  double w = 0.0;
  if (all) {
    in_order();
    if (lane < r.top_k) w = kept[id] * share;
  } else if (lane < r.top_k) {
    const float mine[1] = {l[id]};
    double s[1];
    scores<1>(s, mine, top, r.sigmoid);
    w = s[0];
  }
  if (r.renorm) {
    double total = group_sum<64>(w);
    // Scores so small that some of them count as 0 (e^-346; those are below e^-690): the
    // exponentials over the largest chosen one's, since there a sigmoid's 1 / (1 + e^l) is 1 within
    // 2^-499 and a softmax's sum is the same for all.
    if (of_lane(total, 0) < 0x1p-500) {      // the wave's lanes together
      const float mine[1] = {lane < r.top_k ? l[id] : -INFINITY};
      double s[1];
      scores<1>(s, mine, number(wave_max(ordered(mine[0]))), false);
      w = s[0];
      total = group_sum<64>(w);
    }
    w = total > 0.0 ? w * reciprocal(total) : 0.0;
  }
  if (lane < r.top_k) {
    r.ids[t * r.top_k + lane] = id;
    r.weights[t * r.top_k + lane] = (float)(r.scale * w);
  }
}

template <int V>
void enqueue(const Router& r, size_t lds, hipStream_t stream) {
  const auto kernel = r.bias ? moe_route_kernel<V, true> : moe_route_kernel<V, false>;
  hipLaunchKernelGGL(kernel, dim3((r.T + r.waves - 1) / r.waves), dim3(64 * r.waves), lds, stream,
                     r);
}

}  // namespace

hipError_t launch_moe_route(const float* logits, int64_t T, int64_t E, int64_t stride,
                            const float* bias, bool sigmoid, int groups, int group_top,
                            int top_groups, int top_k, bool renorm, double scale, int32_t* ids,
                            float* weights, int32_t* err, hipStream_t stream) {
  int shift = 6;
  while (groups << shift > 64) --shift;
  const int32_t per = (int32_t)E / groups;
  // Few tokens: a wave a workgroup, more compute units for them (512 over 512 experts 7.2 us, 9.0
  // with four; over 256 in groups 5.0 and 5.3; over 64 2.5 and 2.4).  Many: four, fewer
  // workgroups to start (8000 over 64 3.9 us, 4.5 with one; over 128 5.6 and 6.0; over 512 in
  // groups 24.9 and 28.4; but 4099 over 256 in groups 9.4 and 9.2, over 512 in groups 17.0 and
  // 15.9).  At 1024 tokens the two are within 5 %.
  const int32_t waves = T >= 1024 && E <= 512 ? 4 : 1;
  // at most 32 KiB: scores, and what groups are compared by
  const int tables = (bias || (!sigmoid && !renorm)) + (groups > 1);
  const size_t lds = (size_t)tables * waves * E * sizeof(double);
  for (int64_t t = 0; t < T; t += kMaxGrid) {
    const Router r = {logits + t * stride, bias, ids + t * top_k, weights + t * top_k, err, scale,
                      stride, (int32_t)std::min(T - t, kMaxGrid), (int32_t)E, groups, group_top,
                      top_groups, top_k, waves, per, shift,
                      (uint32_t)(((int64_t(1) << 31) + per - 1) / per), sigmoid, renorm};
    if (E <= 64) enqueue<1>(r, lds, stream);
    else if (E <= 128) enqueue<2>(r, lds, stream);
    else if (E <= 256) enqueue<4>(r, lds, stream);
    else if (E <= 512) enqueue<8>(r, lds, stream);
    else if (E <= 1024) enqueue<16>(r, lds, stream);
    else enqueue<32>(r, lds, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rfp2
