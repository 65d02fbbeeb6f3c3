// The streaming kernel of the paged attention (see paged_attn.h for the method).
#pragma once

#include "paged_attn.h"

namespace rfp2 {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));

template <int I, int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<I + 1, N>(f);
  }
}

// Lane N of each row of 16 lanes, to the whole row (folds into the consumer).
template <int N>
__device__ __forceinline__ float row_bcast(float x) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + N, 0xF, 0xF, true));
}

// scale * x on its own: the broadcast folds into a multiplication, not into a
// fused multiply-add, which would keep every broadcast scale in a register.
__device__ __forceinline__ float scaled(float scale, float x) {
#pragma clang fp contract(off)
  const float y = scale * x;
  return y;
}

// The number of the lane that a shift or broadcast (CTRL) names, in the given rows of 16
// lanes; 0 in the others and where there is no such lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t from_lane(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}

__device__ __forceinline__ float max_over_groups(float x) {     // lanes l, l^16, l^32, l^48
  x = fmaxf(x, __shfl_xor(x, 16, 64));
  return fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float sum_over_groups(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// Eight int8 codes as halves, exactly: a byte with its sign bit flipped is
// u = code + 128; 0x6400 | u is the half 1024 + u, minus 1152 is the code.
__device__ __forceinline__ half8v halves_of(uint2 x) {
  union { uint32_t w[4]; half2v h[4]; half8v v; } o;
  const uint32_t a = x.x ^ 0x80808080u, b = x.y ^ 0x80808080u;
  o.w[0] = __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u);
  o.w[1] = __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u);
  o.w[2] = __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u);
  o.w[3] = __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u);
  const half2v off = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) o.h[i] = o.h[i] - off;
  return o.v;
}
__device__ __forceinline__ half8v halves_of(uint4 x) {
  union { uint4 u; half8v v; } o;
  o.u = x;
  return o.v;
}

// x = hi + lo, both halves, cut off (not rounded: one packed instruction each);
// what remains is below 2^-20 of x, and below 2^-24 absolutely.
// MEETS_INF: the other operand may be infinite (a half key), where a part of 0 would make
// NaN of a product that is infinite.  So neither part of an x that is not 0 is 0: one that
// would be is the smallest half of x's sign, 2^-24 (2^-37 of the row's largest value).
template <bool MEETS_INF>
__device__ __forceinline__ void split8(const float (&x)[8], half8v& hi, half8v& lo) {
  union { half2v h[4]; half8v v; } a, b;
  auto least = [](float part, float x) {
    if constexpr (!MEETS_INF) return part;
    return x != 0.0f && fabsf(part) < 0x1p-24f ? copysignf(0x1p-24f, x) : part;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = x[2 * i], x1 = x[2 * i + 1];
    a.h[i] = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_pkrtz(least(x0, x0), least(x1, x1)));
    const float l0 = __builtin_fmaf((float)a.h[i].x, -1.0f, x0);
    const float l1 = __builtin_fmaf((float)a.h[i].y, -1.0f, x1);
    b.h[i] = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_pkrtz(least(l0, x0), least(l1, x1)));
  }
  hi = a.v;
  lo = b.v;
}

__device__ __forceinline__ float4v mfma(half8v a, half8v b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Sixteen products of 4 x 1 by 1 x 4 (lane 4 b + i holds row i, or column i, of
// block b); the left operand of all eight blocks of a half of the wave is the one of
// the half's block B.
template <int B>
__device__ __forceinline__ float4v mfma4(float a, float b, float4v c) {
  return __builtin_amdgcn_mfma_f32_4x4x1f32(a, b, c, 3, B, 0);
}

// Value J of eight codes or halves.
template <int J>
__device__ __forceinline__ float value_of(uint2 w) {
  const uint32_t u = J < 4 ? w.x : w.y;
  return (float)((int32_t)(u << (24 - 8 * (J & 3))) >> 24);
}
template <int J>
__device__ __forceinline__ float value_of(uint4 w) {
  return (float)halves_of(w)[J];
}

// Values that one wave alone reads go past the caches (ONCE): 317 -> 306 us at 128 sequences
// of up to 8000 tokens; keys, whose lines two or more loads share, must not (388 us).
template <bool ONCE, class R>
__device__ __forceinline__ R load_values(const R* p) {
  typedef uint32_t vec __attribute__((ext_vector_type(sizeof(R) / 4)));
  if constexpr (!ONCE) return *p;
  union { vec v; R r; } o;
  o.v = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p));
  return o.r;
}

// Lanes 32..63 of a for lanes 0..31 of b.
__device__ __forceinline__ void trade_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

__device__ __forceinline__ float lane_of(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute(4 * lane, __float_as_int(x)));
}

// LDS written by some lanes of a wave, read by others of it: the accesses execute in
// order, the compiler has to keep them so.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The same number, computed here: what a lane derives from it (offsets, masks) is not
// carried in registers from further up.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

constexpr float kLowest = -3.0e38f;        // the running maximum before any score
constexpr float kSlack = 8.0f;             // weights may grow to 2^8 before sums are rescaled

// Q: groups of four query rows of a wave (1 to 4); RW as described in paged_attn.h.
template <bool I8, int NB, int Q, int RW>
__global__ __launch_bounds__(kAttnThreads, attn_waves(I8, NB, Q)) void paged_attn_kernel(
    const AttnArgs a) {
  constexpr int WAVES = kAttnThreads / 64, D = 32 * NB, WT = WAVES / RW, WROWS = 4 * Q, ROWS = WROWS * RW, NW = (NB + 1) / 2;
  constexpr int C = NB / 2;                 // whole chunks of 64 values
  constexpr bool HALF = NB % 2 != 0;        // and a chunk of 32
  constexpr int CA = C + (HALF ? 1 : 0);
  constexpr int ES = I8 ? 1 : 2;
  using Reg = std::conditional_t<I8, uint2, uint4>;   // eight codes or halves
  __shared__ uint32_t cum[kMaxAttnSeqs + 1];
  __shared__ int32_t len_of[kMaxAttnSeqs];
  __shared__ uint32_t wave_sum[WAVES];
  __shared__ float2 wave_ml[WAVES][WROWS];
  __shared__ float weights[WAVES][WROWS][40];
  // The queries, two halves each as the first product takes them; once the tiles are
  // done, the waves' sums.
  __shared__ union Shared {
    half8v queries[RW][NB][2][64];
    float sums[WAVES][WROWS][D + 4];
    __device__ Shared() {}
  } sh;

  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wr = wave % RW, wt = wave / RW;
  const int64_t cap = (int64_t)a.c.max_pages << a.c.page_shift;

  // ---- the line of tiles: cum[b] = length of one item of the sequences before b, its
  // tiles and what starting on it costs (one sequence is cut by tiles alone)
  const uint32_t start = a.B == 1 ? 0 : kAttnItemStart;
  {
    const int tid = threadIdx.x, lane = tid & 63;
    constexpr int EACH = kMaxAttnSeqs / kAttnThreads;   // sequences of a thread
    uint32_t nt[EACH], mine = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int b = EACH * tid + i;
      nt[i] = 0;
      if (b < a.B) {
        const int32_t len = a.lens[b];
        len_of[b] = len;
        if (len > cap) {
          if (a.err && blockIdx.x == 0) *a.err = 1;
        } else if (len > 0) {
          const int lo = a.window > 0 ? max(0, len - a.T - a.window + 1) : 0;
          nt[i] = (uint32_t)(((len - 1) >> 5) + 1 - (lo >> 5)) + start;
        }
      }
      mine += nt[i];
    }
    // sum over the lanes up to this one, inside rows of 16, then over the rows
    uint32_t inc = mine;
    if (a.B > EACH) {
      inc += from_lane<0x111, 0xF>(inc);
      inc += from_lane<0x112, 0xF>(inc);
      inc += from_lane<0x114, 0xF>(inc);
      inc += from_lane<0x118, 0xF>(inc);
      inc += from_lane<0x142, 0xA>(inc);
      inc += from_lane<0x143, 0xC>(inc);
    }
    uint32_t at = inc - mine;
    if (a.B > 64 * EACH) {
      if (lane == 63) wave_sum[wave] = inc;
      __syncthreads();
      for (int w = 0; w < wave; ++w) at += wave_sum[w];
    }
    if (tid == 0) cum[0] = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      at += nt[i];
      if (EACH * tid + i < a.B) cum[EACH * tid + i + 1] = at;
    }
    __syncthreads();
  }
  const int items = a.c.heads * a.row_groups;
  // Shares: equal parts of the line.  One sequence's items are cut alike instead, into as
  // many parts as there are workgroups for, so that no workgroup works on two items.
  const bool alike = a.B == 1 && items <= (int)gridDim.x;
  uint32_t line1 = cum[1];
  int64_t share;
  if (alike) {
    const uint32_t parts = max(1u, min(gridDim.x / (uint32_t)items,
                                       (line1 + kAttnMinTiles - 1) / kAttnMinTiles));
    const uint32_t len1 = max(1u, (line1 + parts - 1) / parts);
    line1 = (line1 + len1 - 1) / len1 * len1;
    share = len1;
  } else {
    share = max((int64_t)kAttnMinTiles,
                divided((int64_t)cum[a.B] * items + gridDim.x - 1, (int64_t)gridDim.x));
  }
  auto line = [&](int i) { return a.B == 1 && i == 1 ? line1 : cum[i]; };
  const int64_t total = (int64_t)line(a.B) * items;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.plan[0] = share;
    for (int b = threadIdx.x; b <= a.B; b += kAttnThreads) a.cum[b] = line(b);
  }
  const int64_t first_unit = blockIdx.x * share;
  const int64_t end_unit = min(total, first_unit + share);

  int b = 0;
  if (first_unit < end_unit) {           // the last b whose line starts at or before first_unit
    int hi = a.B - 1;
    while (b < hi) {
      const int mid = (b + hi + 1) >> 1;
      if ((int64_t)cum[mid] * items <= first_unit) b = mid; else hi = mid - 1;
    }
  }

  for (int64_t unit = first_unit; unit < end_unit;) {
    while (unit >= (int64_t)line(b + 1) * items) ++b;       // sequences without tiles
    const int64_t length = line(b + 1) - cum[b];
    const int64_t in_seq = unit - (int64_t)cum[b] * items;
    const int item = (int)divided(in_seq, length);
    const int64_t from = in_seq - item * length;             // of the item
    const int64_t to = min(length, from + (end_unit - unit));
    const int slot = unit == first_unit && from >= start ? 0 : 1;
    unit += to - from;
    const int nt = (int)((alike ? cum[1] : length) - start);
    const int t0 = (int)max((int64_t)0, from - start), t1 = (int)min((int64_t)nt, to - start);
    if (t0 >= t1) continue;                                  // the share ends before the tiles
    const bool whole = t0 == 0 && t1 == nt;

    const int kvh = item / a.row_groups, rg = item - kvh * a.row_groups;
    const int rows_all = a.T * a.group;
    const int len = __builtin_amdgcn_readfirstlane(len_of[b]);
    const int lo = a.window > 0 ? max(0, len - a.T - a.window + 1) : 0;
    const int tile0 = lo >> 5;
    const int group_lo = lo >> 3, group_hi = (len - 1) >> 3;

    const int lane = here(threadIdx.x) & 63, n = lane & 15, g = lane >> 4;

    // ---- the cache's tiles
    struct Keys {                           // a tile's keys and their scales
      uint4 w[2][I8 ? C + 1 : NB];          // int8: 64 values a load, the half chunk's last
      float s[NW];
    } key;
    struct Values {                         // a tile's values, their scales, no such page
      Reg r[4][C > 0 ? C : 1], h[2];
      float s[NW];
      bool bad;
    } v;

    // the page of token group `grp` (eight tokens), -1 where there is none
    auto page_of = [&](int grp) -> int32_t {
      grp = min(max(grp, group_lo), group_hi);
      return a.c.table[(int64_t)b * a.c.max_pages + ((grp << 3) >> a.c.page_shift)];
    };
    auto is_page = [&](int32_t page) { return page >= 0 && page < a.c.pages; };
    // rows before token group `grp` in the cache, given its page
    auto rows_of = [&](int grp, int32_t page) -> int64_t {
      grp = min(max(grp, group_lo), group_hi);
      return kv_rows(a.c, is_page(page) ? page : 0, kvh) +
             ((grp << 3) & ((1 << a.c.page_shift) - 1));
    };
    const int gk = n >> 2;                  // token group of this lane's key rows
    // the first of a lane's eight values in a block of 32
    auto dim_of = [](int g) { return I8 ? 16 * (g & 1) + 8 * (g >> 1) : 8 * g; };
    auto load_k = [&](int tile, int32_t page, int32_t page_s) {
      const int64_t r = rows_of(4 * tile + gk, page) + (n & 3);
      const char* p = static_cast<const char*>(a.c.k) + r * D * ES + 16 * g;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int k = 0; k < (I8 ? C : NB); ++k)
          key.w[s][k] = *reinterpret_cast<const uint4*>(p + 4 * s * D * ES + 64 * k);
        if constexpr (I8 && HALF) {
          const uint2 h = *reinterpret_cast<const uint2*>(
              p - 16 * g + dim_of(g) + 4 * s * D + 64 * C);
          key.w[s][C].x = h.x;
          key.w[s][C].y = h.y;
        }
      }
      if constexpr (I8) {
        const int64_t rs = rows_of(4 * tile + g, page_s);
#pragma unroll
        for (int w = 0; w < NW; ++w)
          key.s[w] = a.c.ks[rs * NB + 16 * w + (2 * w + 1 < NB ? n : (n & 7))];
      }
    };
    auto load_v = [&](int tile, int32_t page) {
      v.bad = !is_page(page);
      int64_t r[4];                         // the four token groups, the same for all lanes
#pragma unroll
      for (int u = 0; u < 4; ++u)
        r[u] = rows_of(4 * tile + u, __builtin_amdgcn_readlane(page, 16 * u));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const char* p = static_cast<const char*>(a.c.v) + r[u] * D * ES;
#pragma unroll
        for (int k = 0; k < C; ++k)
          v.r[u][k] = load_values<RW == 1>(reinterpret_cast<const Reg*>(p + (lane + 64 * k) * 8 * ES));
      }
      if constexpr (HALF) {                 // lanes 32 .. 63: the same values, two groups on
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const char* p = static_cast<const char*>(a.c.v) + (lane < 32 ? r[u] : r[u + 2]) * D * ES;
          v.h[u] = *reinterpret_cast<const Reg*>(p + ((lane & 31) + 64 * C) * 8 * ES);
        }
      }
      if constexpr (I8) {
        const int64_t rs = g == 0 ? r[0] : g == 1 ? r[1] : g == 2 ? r[2] : r[3];
#pragma unroll
        for (int w = 0; w < NW; ++w)
          v.s[w] = a.c.vs[rs * NB + 16 * w + (2 * w + 1 < NB ? n : (n & 7))];
      }
    };

    int t = wr * WROWS < rows_all - rg * ROWS ? t0 + wt : t1;     // (a wave may have no rows)
    int32_t pk = 0, pv = 0;                 // pages of the next tile's keys and values
    const int last = t < t1 ? t + (t1 - 1 - t) / WT * WT : t;     // this wave's last tile
    auto next_pages = [&](int u) {
      pk = page_of(4 * (tile0 + min(u, last)) + gk);
      pv = page_of(4 * (tile0 + min(u, last)) + g);
    };
    next_pages(t);

    // ---- the query rows: row n of this wave's tile, as two halves, scaled by 2^(14 - ex)
    const int lane_q = here(threadIdx.x) & 63, nq = lane_q & 15, gq = lane_q >> 4;
    const int row = rg * ROWS + wr * WROWS + nq;
    const bool row_ok = nq < WROWS && row < rows_all;
    const int row_t = row_ok ? row / a.group : 0;
    const int row_h = kvh * a.group + (row_ok ? row - row_t * a.group : 0);
    const int row_pos = len - a.T + row_t;                  // this row's position
    float qx[NB][8];
    {
      const float* qp = a.q + ((int64_t)b * a.T + row_t) * a.q_stride + (int64_t)row_h * D + dim_of(gq);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float4 u = row_ok ? *reinterpret_cast<const float4*>(qp + 32 * k)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 v = row_ok ? *reinterpret_cast<const float4*>(qp + 32 * k + 4)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        qx[k][0] = u.x; qx[k][1] = u.y; qx[k][2] = u.z; qx[k][3] = u.w;
        qx[k][4] = v.x; qx[k][5] = v.y; qx[k][6] = v.z; qx[k][7] = v.w;
      }
    }
    if (t < t1) {
      const int32_t pk1 = pk, pv1 = pv;
      next_pages(t + WT);
      load_k(tile0 + t, pk1, pv1);
      load_v(tile0 + t, pv1);
    }
    float c;                                                // score -> base 2, unscaled
    {
      float big = 0.0f;
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(qx[k][i]));
      big = max_over_groups(big);
      // 2^(14 - ex) > 2^13 / big, from the exponent's bits; not for 0, infinity
      const int e = (int)(__float_as_uint(big) >> 23);
      const int ex = e == 0 ? (big > 0.0f ? -100 : 0) : e == 255 ? 0 : max(e - 126, -100);
      const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (k % WT != wt) continue;         // the waves of one row tile hold the same: shared out
#pragma unroll
        for (int i = 0; i < 8; ++i) qx[k][i] *= up;
        half8v hi, lo_;
        split8<!I8>(qx[k], hi, lo_);
        sh.queries[wr][k][0][lane_q] = hi;
        sh.queries[wr][k][1][lane_q] = lo_;
      }
      c = a.scale * 1.44269504088896340736f * __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
    }

    __syncthreads();

    // ---- the stream of tiles
    float4v o[CA][Q];                       // lane: value 64 i + lane of four query rows
#pragma unroll
    for (int i = 0; i < CA; ++i)
#pragma unroll
      for (int q = 0; q < Q; ++q) o[i][q] = float4v{0.f, 0.f, 0.f, 0.f};
    float m = kLowest, l = 0.0f;

    // sum += V^T W of a tile, W in `weights` (transposed through LDS: a lane needs the
    // weights of row lane % 4 for one token, and holds one value of eight tokens)
    auto add_products = [&](float4v (&sum)[CA][Q], auto scaled_by_s, auto&& of) {
      const float* w0 = &weights[wave][lane & 3][(lane >> 2) & 7];
      unrolled<0, 4>([&](auto uc) {
        constexpr int u = uc;
        float w[Q], s[CA];
#pragma unroll
        for (int q = 0; q < Q; ++q) w[q] = w0[(4 * q) * 40 + 8 * u];
#pragma unroll
        for (int k = 0; k < C; ++k)
          s[k] = scaled_by_s ? lane_of(v.s[k], 16 * u + 8 * (lane >> 5) + ((lane >> 2) & 7)) : 1.0f;
        unrolled<0, 8>([&](auto jc) {
          constexpr int j = jc;
#pragma unroll
          for (int k = 0; k < C; ++k) {
            const float x = of(value_of<j>(v.r[u][k]));
#pragma unroll
            for (int q = 0; q < Q; ++q)
              sum[k][q] = mfma4<j>(scaled_by_s ? w[q] * s[k] : w[q], x, sum[k][q]);
          }
        });
      });
      if constexpr (HALF) {
        const float* wh = w0 + 16 * (lane >> 5);
        unrolled<0, 2>([&](auto uc) {
          constexpr int u = uc;
          const float s =
              scaled_by_s ? lane_of(v.s[NW - 1], 16 * (u + 2 * (lane >> 5)) + ((lane >> 2) & 7))
                          : 1.0f;
          float w[Q];
#pragma unroll
          for (int q = 0; q < Q; ++q) w[q] = wh[(4 * q) * 40 + 8 * u] * s;
          unrolled<0, 8>([&](auto jc) {
            constexpr int j = jc;
            const float x = of(value_of<j>(v.h[u]));
#pragma unroll
            for (int q = 0; q < Q; ++q) sum[C][q] = mfma4<j>(w[q], x, sum[C][q]);
          });
        });
      }
    };
    auto put_weights = [&](const float (&p)[8]) {
      wave_fence();
      if (n < WROWS) {
        float4* w = reinterpret_cast<float4*>(&weights[wave][n][8 * g]);
        w[0] = make_float4(p[0], p[1], p[2], p[3]);
        w[1] = make_float4(p[4], p[5], p[6], p[7]);
      }
      wave_fence();
    };

    for (; t < t1; t += WT) {
      const int tile = tile0 + t;
      // scores: x[4 s + i] of token 8 g + 4 s + i
      float x[8];
      {
        const half8v* qp = &sh.queries[wr][0][0][lane];
        const float4v zero = {0.f, 0.f, 0.f, 0.f};
        float4v acc[2] = {zero, zero}, low[2] = {zero, zero};
        unrolled<0, NB>([&](auto kc) {
          constexpr int k = kc;
          const half8v hi = qp[(2 * k) * 64], lo_ = qp[(2 * k + 1) * 64];
          unrolled<0, 2>([&](auto sc) {
            constexpr int s = sc;
            if constexpr (I8) {
              uint4& w = key.w[s][k >> 1];
              // 64 values came as 16 a lane; lanes 0..31 hold the first block's, the others
              // the second's.  Trading halves gives every lane eight of each block.
              if constexpr (k % 2 == 0 && k + 1 < NB) {
                trade_halves(w.x, w.z);
                trade_halves(w.y, w.w);
              }
              const half8v kk = halves_of(k % 2 == 0 ? make_uint2(w.x, w.y) : make_uint2(w.z, w.w));
              const float4v part = mfma(kk, lo_, mfma(kk, hi, zero));
              unrolled<0, 4>([&](auto ic) {
                constexpr int i = ic;
                acc[s][i] += scaled(row_bcast<(k & 1) * 8 + 4 * s + i>(key.s[k >> 1]), part[i]);
              });
            } else {
              const half8v kk = halves_of(key.w[s][k]);
              acc[s] = mfma(kk, hi, acc[s]);
              low[s] = mfma(kk, lo_, low[s]);
            }
          });
        });
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = (acc[j >> 2][j & 3] + low[j >> 2][j & 3]) * c;
          asm volatile("" : "+v"(x[j]));    // not put off until after the loads
        }
      }
      // The next tile's keys are requested as soon as this one's have been used, and its
      // values after this one's: one set of registers each (a second set for the values,
      // requested here too, was slower: 98 against 94 us at five verified tokens, 295
      // against 292 at 128 sequences).  The pages after them come first, since loads
      // return in order.  The last tile requests itself again (out of the cache), because
      // requests that only some iterations make would have to be waited for as if none
      // had been made since.
      const int32_t pk1 = pk, pv1 = pv;
      const int ahead = tile0 + min(t + WT, last);
      next_pages(t + 2 * WT);
      load_k(ahead, pk1, pv1);

      // visibility: only a tile at an end of the sequence or of a window has hidden tokens
      const int pos0 = 32 * tile + 8 * g;
      const bool edge = 32 * tile + 31 > len - a.T ||
                        (a.window > 0 && 32 * tile <= len - 1 - a.window);
      if (v.bad) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_nanf("");
        if (a.err) *a.err = 1;
      }
      // (a token's own score may be minus infinity too: what a row sees goes by positions)
      const int from = a.window > 0 ? row_pos - a.window + 1 : 0;
      auto sees = [&](int j) { return pos0 + j <= row_pos && pos0 + j >= from; };
      if (edge) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!sees(j)) x[j] = -INFINITY;
        if constexpr (I8) {
          // scales of tokens that no row sees may hold anything
#pragma unroll
          for (int w = 0; w < NW; ++w)
            if (pos0 + (n & 7) >= len || pos0 + (n & 7) < lo) v.s[w] = 0.0f;
          // A weight of 0 does not cancel the NaN scale of a token that some rows do
          // not see: it is taken out, and its block is lost to the rows that do see it.
          uint64_t odd[NW], any_odd = 0;
#pragma unroll
          for (int w = 0; w < NW; ++w) any_odd |= odd[w] = __ballot(!(fabsf(v.s[w]) < INFINITY));
          if (any_odd) {
            const int lane_o = here(threadIdx.x) & 63, g_o = lane_o >> 4;
            uint32_t seen = 0, lost = 0;                     // tokens; blocks
#pragma unroll
            for (int j = 0; j < 8; ++j) seen |= (sees(j) ? 1u : 0u) << j;
#pragma unroll
            for (int k = 0; k < NB; ++k)
              if ((uint32_t)(odd[k >> 1] >> (16 * g_o + 8 * (k & 1))) & seen) lost |= 1u << k;
            lost |= __shfl_xor(lost, 16, 64);
            lost |= __shfl_xor(lost, 32, 64);
            unrolled<0, WROWS>([&](auto rc) {
              constexpr int r = rc;
              const uint32_t of_row = __float_as_uint(row_bcast<r>(__uint_as_float(lost)));
#pragma unroll
              for (int k = 0; k < CA; ++k)
                if (of_row >> (2 * k + (k < C ? lane_o >> 5 : 0)) & 1)
                  o[k][r >> 2][r & 3] = __builtin_nanf("");
            });
#pragma unroll
            for (int w = 0; w < NW; ++w)
              if (!(fabsf(v.s[w]) < INFINITY)) v.s[w] = 0.0f;
          }
        }
      }

      // running maximum, with slack so that most tiles leave the sums alone
      float big = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) big = fmaxf(big, x[j]);
      if (__any(big > m + kSlack)) {
        const float m_new = fmaxf(m, max_over_groups(big));
        const float fix = __builtin_amdgcn_exp2f(m - m_new);
        m = m_new;
        l *= fix;
        unrolled<0, WROWS>([&](auto rc) {
          constexpr int r = rc;
          const float f = row_bcast<r>(fix);
#pragma unroll
          for (int k = 0; k < CA; ++k) o[k][r >> 2][r & 3] *= f;
        });
      }
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = __builtin_amdgcn_exp2f(x[j] - m);
        l += p[j];
      }

      if constexpr (!I8) {
        if (edge) {
          // Hidden tokens may hold infinities or NaN, which a weight of 0 does not
          // cancel.  Where a tile holds any, they are taken out, and each row that
          // does see one gets it back: the number of seen infinities of either sign
          // (NaN counts as both) comes from the matrix core.
          bool odd = false;
          auto look = [&](const Reg& r) {
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              odd |= (w[i] & 0x7C00u) == 0x7C00u || (w[i] & 0x7C000000u) == 0x7C000000u;
          };
          auto each = [&](auto&& f) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int k = 0; k < C; ++k) f(v.r[u][k], u, k);
            if constexpr (HALF) {
              f(v.h[0], 0, C);
              f(v.h[1], 1, C);
            }
          };
          each([&](Reg& r, int, int) { look(r); });
          if (__any(odd)) {
            float seen[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) seen[j] = sees(j) ? 1.0f : 0.0f;
            put_weights(seen);
            auto count = [&](float inf, auto&& of) {
              float4v seen_of[CA][Q];
#pragma unroll
              for (int k = 0; k < CA; ++k)
#pragma unroll
                for (int q = 0; q < Q; ++q) seen_of[k][q] = float4v{0.f, 0.f, 0.f, 0.f};
              add_products(seen_of, std::false_type{}, of);
#pragma unroll
              for (int k = 0; k < CA; ++k)
#pragma unroll
                for (int q = 0; q < Q; ++q)
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    if (seen_of[k][q][i] > 0.0f) o[k][q][i] += inf;
            };
            count(INFINITY, [](float f) { return f < INFINITY ? 0.0f : 1.0f; });
            count(-INFINITY, [](float f) { return f > -INFINITY ? 0.0f : 1.0f; });
            each([&](Reg& r, int, int) {
              union { Reg u; half8v h; } b_;
              b_.u = r;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (!(fabsf((float)b_.h[j]) < INFINITY)) b_.h[j] = (_Float16)0.0f;
              r = b_.u;
            });
          }
        }
      }
      put_weights(p);
      add_products(o, std::bool_constant<I8>{}, [](float f) { return f; });
      load_v(ahead, pv1);
    }

    // ---- the waves' sums together, then out: finished, or into this share's slot
    const int tid_ = here(threadIdx.x), lane_ = tid_ & 63, n_ = lane_ & 15;
    l = sum_over_groups(l);
    if (lane_ < WROWS) wave_ml[wave][lane_] = make_float2(m, l);
    __syncthreads();
    float m_all = m;
    if (n_ < WROWS) {
#pragma unroll
      for (int w = 0; w < WT; ++w) m_all = fmaxf(m_all, wave_ml[w * RW + wr][n_].x);
    }
    const float fix = __builtin_amdgcn_exp2f(m - m_all);
    unrolled<0, WROWS>([&](auto rc) {
      constexpr int r = rc;
      const float f = row_bcast<r>(fix);
#pragma unroll
      for (int k = 0; k < C; ++k) sh.sums[wave][r][64 * k + lane_] = o[k][r >> 2][r & 3] * f;
      if constexpr (HALF) {
        const float h = o[C][r >> 2][r & 3] * f;
        const float both = h + __shfl_xor(h, 32, 64);
        if (lane_ < 32) sh.sums[wave][r][64 * C + lane_] = both;
      }
    });
    __syncthreads();
    const int rows_here = min(ROWS, rows_all - rg * ROWS);
    for (int e = tid_; e < rows_here * (D / 4); e += kAttnThreads) {
      const int r = e / (D / 4), d = 4 * (e - r * (D / 4));
      const int tile_r = r / WROWS, rn = r % WROWS;
      float mm = kLowest, ll = 0.0f;
#pragma unroll
      for (int w = 0; w < WT; ++w) mm = fmaxf(mm, wave_ml[w * RW + tile_r][rn].x);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WT; ++w) {
        const float2 ml = wave_ml[w * RW + tile_r][rn];
        ll += ml.y * __builtin_amdgcn_exp2f(ml.x - mm);
        const float4 u = *reinterpret_cast<const float4*>(&sh.sums[w * RW + tile_r][rn][d]);
        s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w;
      }
      const int gr = rg * ROWS + r, gt = gr / a.group;
      if (whole) {
        const float f = 1.0f / ll;
        s.x *= f; s.y *= f; s.z *= f; s.w *= f;
        if (len - a.T + gt < 0) s = make_float4(0.f, 0.f, 0.f, 0.f);   // sees nothing
        const int64_t out = ((int64_t)b * a.T + gt) * a.H + kvh * a.group + (gr - gt * a.group);
        *reinterpret_cast<float4*>(a.y + out * D + d) = s;
      } else {
        const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * a.slot_rows + r;
        *reinterpret_cast<float4*>(a.part + at * D + d) = s;
        if (d == 0) a.ml[at] = make_float2(mm, ll);
      }
    }
    __syncthreads();                                         // sums and wave_ml are used again
  }
}

// The variant goes by the query rows of an item: as few groups of four as hold them, since
// the fp32 products are done for whole groups (four rows in one group instead of four at
// 128 sequences: 330 instead of 400 us); beyond 16 rows two or four waves share a tile's
// rows, twelve each up to 48 (40 rows on four waves of twelve 90 us; before the last
// steps, 94 against 109 on waves of sixteen).
template <bool I8, int NB>
hipError_t launch_attn(const AttnArgs& a, int rows, int grid, hipStream_t stream) {
  const auto kernel = rows <= 4    ? paged_attn_kernel<I8, NB, 1, 1>
                      : rows <= 8  ? paged_attn_kernel<I8, NB, 2, 1>
                      : rows <= 16 ? paged_attn_kernel<I8, NB, 4, 1>
                      : rows <= 32 ? paged_attn_kernel<I8, NB, 4, 2>
                      : rows <= 48 ? paged_attn_kernel<I8, NB, 3, 4>
                                   : paged_attn_kernel<I8, NB, 4, 4>;
  hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(kAttnThreads), 0, stream, a);
  return hipGetLastError();
}

template <int NB>
hipError_t launch_attn_nb(const AttnArgs& a, bool i8, int rows, int grid, hipStream_t stream) {
  return i8 ? launch_attn<true, NB>(a, rows, grid, stream)
            : launch_attn<false, NB>(a, rows, grid, stream);
}

}  // namespace rfp2
