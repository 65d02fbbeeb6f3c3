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
__device__ __forceinline__ void split8(const float (&x)[8], half8v& hi, half8v& lo) {
  union { half2v h[4]; half8v v; } a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a.h[i] = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_pkrtz(x[2 * i], x[2 * i + 1]));
    b.h[i] = __builtin_bit_cast(
        half2v, __builtin_amdgcn_cvt_pkrtz(__builtin_fmaf((float)a.h[i].x, -1.0f, x[2 * i]),
                                           __builtin_fmaf((float)a.h[i].y, -1.0f, x[2 * i + 1])));
  }
  hi = a.v;
  lo = b.v;
}

__device__ __forceinline__ float4v mfma(half8v a, half8v b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float4v mfma4(float a, float b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Byte B of a word as a signed number.
template <int B>
__device__ __forceinline__ float code_of(uint32_t w) {
  return (float)((int32_t)(w << (24 - 8 * B)) >> 24);
}

constexpr float kLowest = -3.0e38f;        // the running maximum before any score
constexpr float kSlack = 8.0f;             // weights may grow to 2^8 before sums are rescaled

template <bool I8, int NB, int RW>
__global__ __launch_bounds__(kAttnThreads, (NB <= 4 ? 2 : 1)) void paged_attn_kernel(
    const AttnArgs a) {
  constexpr int D = 32 * NB, WT = 4 / RW, ROWS = 16 * RW, NW = (NB + 1) / 2;
  constexpr int ES = I8 ? 1 : 2;
  using Kreg = std::conditional_t<I8, uint2, uint4>;
  __shared__ uint32_t cum[kMaxAttnSeqs + 1];
  __shared__ uint32_t wave_sum[4];
  __shared__ float2 wave_ml[4][16];
  __shared__ float sums[4][16][D + 4];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave % RW, wt = wave / RW;
  const int n = lane & 15, g = lane >> 4;
  const int64_t cap = (int64_t)a.c.max_pages << a.c.page_shift;

  // ---- the line of tiles: cum[b] = tiles of one item of sequences before b
  {
    uint32_t nt[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 4 * tid + i;
      nt[i] = 0;
      if (b < a.B) {
        const int64_t len = a.lens[b];
        if (len > cap) {
          if (a.err && blockIdx.x == 0) *a.err = 1;
        } else if (len > 0) {
          const int64_t lo = a.window > 0 ? max((int64_t)0, len - a.T - a.window + 1) : 0;
          nt[i] = (uint32_t)(((len + 31) >> 5) - (lo >> 5));
        }
      }
      mine += nt[i];
    }
    uint32_t inc = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t o = __shfl_up(inc, off, 64);
      if (lane >= off) inc += o;
    }
    if (lane == 63) wave_sum[wave] = inc;
    __syncthreads();
    uint32_t at = inc - mine;
    for (int w = 0; w < wave; ++w) at += wave_sum[w];
    if (tid == 0) cum[0] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at += nt[i];
      if (4 * tid + i < a.B) cum[4 * tid + i + 1] = at;
    }
    __syncthreads();
  }
  const int items = a.c.heads * a.row_groups;
  const int64_t total = (int64_t)cum[a.B] * items;
  const int64_t share =
      max((int64_t)kAttnMinTiles, (total + (int64_t)gridDim.x - 1) / (int64_t)gridDim.x);
  if (blockIdx.x == 0) {
    if (tid == 0) a.plan[0] = share;
    for (int b = tid; b <= a.B; b += kAttnThreads) a.cum[b] = cum[b];
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
    while (unit >= (int64_t)cum[b + 1] * items) ++b;        // sequences without tiles
    const int64_t nt = cum[b + 1] - cum[b];
    const int64_t in_seq = unit - (int64_t)cum[b] * items;
    const int item = (int)(in_seq / nt);
    const int t0 = (int)(in_seq - item * nt);
    const int t1 = (int)min(nt, t0 + (end_unit - unit));
    const bool whole = t0 == 0 && t1 == nt;
    const int slot = unit == first_unit ? 0 : 1;
    unit += t1 - t0;

    const int kvh = item / a.row_groups, rg = item - kvh * a.row_groups;
    const int rows_all = a.T * a.group;
    const int len = a.lens[b];
    const int lo = a.window > 0 ? (int)max((int64_t)0, len - a.T - a.window + 1) : 0;
    const int tile0 = lo >> 5;
    const int group_lo = lo >> 3, group_hi = (len - 1) >> 3;

    // ---- the query rows: row n of this wave's tile, as two halves, scaled by 2^(14 - ex)
    const int row = rg * ROWS + wr * 16 + n;
    const bool row_ok = row < rows_all;
    const int row_t = row_ok ? row / a.group : 0;
    const int row_h = kvh * a.group + (row_ok ? row - row_t * a.group : 0);
    const int row_pos = len - a.T + row_t;                  // this row's position
    half8v qh[NB], ql[NB];
    float c;                                                // score -> base 2, unscaled
    {
      const float* qp = a.q + ((int64_t)b * a.T + row_t) * a.q_stride + (int64_t)row_h * D + 8 * g;
      float x[NB][8], big = 0.0f;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float4 u = row_ok ? *reinterpret_cast<const float4*>(qp + 32 * k)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 v = row_ok ? *reinterpret_cast<const float4*>(qp + 32 * k + 4)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        x[k][0] = u.x; x[k][1] = u.y; x[k][2] = u.z; x[k][3] = u.w;
        x[k][4] = v.x; x[k][5] = v.y; x[k][6] = v.z; x[k][7] = v.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[k][i]));
      }
      big = max_over_groups(big);
      int ex = 0;
      if (big > 0.0f && big < INFINITY) ex = max(ilogbf(big) + 1, -100);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = ldexpf(x[k][i], 14 - ex);
        split8(x[k], qh[k], ql[k]);
      }
      c = ldexpf(a.scale * 1.44269504088896340736f, ex - 14);
    }

    // ---- the stream of tiles
    float4v o[2 * NB];
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) o[i] = float4v{0.f, 0.f, 0.f, 0.f};
    float m = kLowest, l = 0.0f;
    struct Keys {                           // a tile's keys and their scales
      Kreg r[2][NB];
      float s[NW];
    } key;
    struct Values {                         // a tile's values, their scales, no such page
      uint4 r[I8 ? NB : 2 * NB];
      float s[NW];
      bool bad;
    } va, vb;

    // the page of token group `grp` (eight tokens), -1 where there is none
    auto page_of = [&](int grp) -> int32_t {
      grp = min(max(grp, group_lo), group_hi);
      return a.c.table[(int64_t)b * a.c.max_pages + ((grp << 3) >> a.c.page_shift)];
    };
    // rows before token group `grp` in the cache, given its page
    auto rows_of = [&](int grp, int32_t page) -> int64_t {
      grp = min(max(grp, group_lo), group_hi);
      return kv_rows(a.c, page, kvh) + ((grp << 3) & ((1 << a.c.page_shift) - 1));
    };
    const int gk = n >> 2;                  // token group of this lane's key rows
    auto load_k = [&](int tile, int32_t page, int32_t page_s) {
      const bool ok = page >= 0 && page < a.c.pages;
      const int64_t r = rows_of(4 * tile + gk, ok ? page : 0) + (n & 3);
      const char* p = static_cast<const char*>(a.c.k) + (r * D + 8 * g) * ES;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < NB; ++k)
          key.r[s][k] = *reinterpret_cast<const Kreg*>(p + (4 * s * D + 32 * k) * ES);
      if constexpr (I8) {
        const bool oks = page_s >= 0 && page_s < a.c.pages;
        const int64_t rs = rows_of(4 * tile + g, oks ? page_s : 0);
#pragma unroll
        for (int w = 0; w < NW; ++w)
          key.s[w] = a.c.ks[rs * NB + 16 * w + (2 * w + 1 < NB ? n : (n & 7))];
      }
    };
    auto load_v = [&](Values& v, int tile, int32_t page) {
      const bool ok = page >= 0 && page < a.c.pages;
      v.bad = !ok;
      const int64_t r = rows_of(4 * tile + g, ok ? page : 0);
      const char* p = static_cast<const char*>(a.c.v) + r * D * ES + 16 * n;
#pragma unroll
      for (int k = 0; k < (I8 ? NB : 2 * NB); ++k)
        v.r[k] = *reinterpret_cast<const uint4*>(p + 256 * k);
      if constexpr (I8) {
#pragma unroll
        for (int w = 0; w < NW; ++w)
          v.s[w] = a.c.vs[r * NB + 16 * w + (2 * w + 1 < NB ? n : (n & 7))];
      }
    };

    int t = t0 + wt;
    int32_t pk = 0, pv = 0;                 // pages of the next tile's keys and values
    auto next_pages = [&](int u) {
      if (u < t1) {
        pk = page_of(4 * (tile0 + u) + gk);
        pv = page_of(4 * (tile0 + u) + g);
      }
    };
    if (t < t1) {
      next_pages(t);
      load_k(tile0 + t, pk, pv);
      load_v(va, tile0 + t, pv);
      next_pages(t + WT);
    }
    // One tile: its values lie in `v`, the next tile's go to `next`.
    auto step = [&](Values& v, Values& next) {
      const int tile = tile0 + t;
      const bool more = t + WT < t1;
      // scores: s[4 s + i] of token 8 g + 4 s + i
      float x[8];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float4v acc = {0.f, 0.f, 0.f, 0.f};
        if constexpr (I8) {
          unrolled<0, NB>([&](auto kc) {
            constexpr int k = kc;
            const half8v kk = halves_of(key.r[s][k]);
            float4v part = {0.f, 0.f, 0.f, 0.f};
            part = mfma(kk, qh[k], part);
            part = mfma(kk, ql[k], part);
            if (s == 0) {
              unrolled<0, 4>([&](auto ic) {
                constexpr int i = ic;
                acc[i] += scaled(row_bcast<(k & 1) * 8 + i>(key.s[k >> 1]), part[i]);
              });
            } else {
              unrolled<0, 4>([&](auto ic) {
                constexpr int i = ic;
                acc[i] += scaled(row_bcast<(k & 1) * 8 + 4 + i>(key.s[k >> 1]), part[i]);
              });
            }
          });
        } else {
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            acc = mfma(halves_of(key.r[s][k]), qh[k], acc);
            acc = mfma(halves_of(key.r[s][k]), ql[k], acc);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * s + i] = acc[i] * c;
      }
      // the next tile's keys and values are on their way while this one is worked on
      if (more) {
        load_k(tile + WT, pk, pv);
        load_v(next, tile + WT, pv);
        next_pages(t + 2 * WT);
      }

      // visibility: only a tile at an end of the sequence or of a window has hidden tokens
      const int pos0 = 32 * tile + 8 * g;
      const bool edge = 32 * tile + 31 > len - a.T ||
                        (a.window > 0 && 32 * tile <= len - 1 - a.window);
      if (v.bad) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_nanf("");
        if (a.err) *a.err = 1;
      }
      if (edge) {
        const int64_t from = a.window > 0 ? row_pos - a.window + 1 : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (pos0 + j > row_pos || pos0 + j < from) x[j] = -INFINITY;
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
            uint32_t seen = 0, lost = 0;                     // tokens; blocks
#pragma unroll
            for (int j = 0; j < 8; ++j) seen |= (x[j] != -INFINITY ? 1u : 0u) << j;
#pragma unroll
            for (int k = 0; k < NB; ++k)
              if ((uint32_t)(odd[k >> 1] >> (16 * g + 8 * (k & 1))) & seen) lost |= 1u << k;
            lost |= __shfl_xor(lost, 16, 64);
            lost |= __shfl_xor(lost, 32, 64);
#pragma unroll
            for (int k = 0; k < NB; ++k)
              if (lost >> k & 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[2 * k + i / 4][i % 4] = __builtin_nanf("");
              }
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
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= fix;
      }
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = __builtin_amdgcn_exp2f(x[j] - m);
        l += p[j];
      }

      if constexpr (I8) {
        unrolled<0, NB>([&](auto kc) {
          constexpr int k = kc;
          const uint4 c4 = v.r[k];
          unrolled<0, 8>([&](auto jc) {
            constexpr int j = jc;
            const float w = row_bcast<(k & 1) * 8 + j>(v.s[k >> 1]) * p[j];
            o[2 * k] = mfma4(code_of<j & 3>(j < 4 ? c4.x : c4.y), w, o[2 * k]);
            o[2 * k + 1] = mfma4(code_of<j & 3>(j < 4 ? c4.z : c4.w), w, o[2 * k + 1]);
          });
        });
      } else {
        if (edge) {
          // Hidden tokens may hold infinities or NaN, which a weight of 0 does not
          // cancel.  Where a tile holds any, they are taken out, and each row that
          // does see one gets it back: the number of seen infinities of either sign
          // (NaN counts as both) comes from the matrix core.
          bool odd = false;
#pragma unroll
          for (int k = 0; k < 2 * NB; ++k) {
            const uint32_t w[4] = {v.r[k].x, v.r[k].y, v.r[k].z, v.r[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              odd |= (w[i] & 0x7C00u) == 0x7C00u || (w[i] & 0x7C000000u) == 0x7C000000u;
          }
          if (__any(odd)) {
            half8v seen;
#pragma unroll
            for (int j = 0; j < 8; ++j) seen[j] = (_Float16)(x[j] == -INFINITY ? 0.0f : 1.0f);
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) {
              half8v f8 = halves_of(v.r[k]), up, dn;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float f = (float)f8[j];
                up[j] = (_Float16)(f < INFINITY ? 0.0f : 1.0f);
                dn[j] = (_Float16)(f > -INFINITY ? 0.0f : 1.0f);
                if (!(fabsf(f) < INFINITY)) f8[j] = (_Float16)0.0f;
              }
              const float4v zero = {0.f, 0.f, 0.f, 0.f};
              const float4v nu = mfma(up, seen, zero), nd = mfma(dn, seen, zero);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (nu[i] > 0.0f) o[k][i] += INFINITY;
                if (nd[i] > 0.0f) o[k][i] -= INFINITY;
              }
              union { half8v v; uint4 u; } back;
              back.v = f8;
              v.r[k] = back.u;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) {
          const half8v f8 = halves_of(v.r[k]);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[k] = mfma4((float)f8[j], p[j], o[k]);
        }
      }
      t += WT;
    };
    while (t < t1) {
      step(va, vb);
      if (t < t1) step(vb, va);
    }

    // ---- the waves' sums together, then out: finished, or into this share's slot
    l = sum_over_groups(l);
    if (lane < 16) wave_ml[wave][lane] = make_float2(m, l);
    __syncthreads();
    float m_all = m;
#pragma unroll
    for (int w = 0; w < WT; ++w) m_all = fmaxf(m_all, wave_ml[w * RW + wr][n].x);
    const float fix = __builtin_amdgcn_exp2f(m - m_all);
    unrolled<0, 2 * NB>([&](auto kc) {
      constexpr int k = kc;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = I8 ? 32 * (k >> 1) + 2 * (4 * g + i) + (k & 1) : 16 * k + 4 * g + i;
        sums[wave][n][d] = o[k][i] * fix;
      }
    });
    __syncthreads();
    const int rows_here = min(ROWS, rows_all - rg * ROWS);
    for (int e = tid; e < rows_here * (D / 4); e += kAttnThreads) {
      const int r = e / (D / 4), d = 4 * (e - r * (D / 4));
      const int tile_r = r >> 4, rn = r & 15;
      float mm = kLowest, ll = 0.0f;
#pragma unroll
      for (int w = 0; w < WT; ++w) mm = fmaxf(mm, wave_ml[w * RW + tile_r][rn].x);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WT; ++w) {
        const float2 ml = wave_ml[w * RW + tile_r][rn];
        ll += ml.y * __builtin_amdgcn_exp2f(ml.x - mm);
        const float4 u = *reinterpret_cast<const float4*>(&sums[w * RW + tile_r][rn][d]);
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

template <bool I8, int NB>
hipError_t launch_attn(const AttnArgs& a, int rw, int grid, hipStream_t stream) {
  const auto kernel = rw == 1 ? paged_attn_kernel<I8, NB, 1>
                      : rw == 2 ? paged_attn_kernel<I8, NB, 2>
                                : paged_attn_kernel<I8, NB, 4>;
  hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(kAttnThreads), 0, stream, a);
  return hipGetLastError();
}

template <int NB>
hipError_t launch_attn_nb(const AttnArgs& a, bool i8, int rw, int grid, hipStream_t stream) {
  return i8 ? launch_attn<true, NB>(a, rw, grid, stream)
            : launch_attn<false, NB>(a, rw, grid, stream);
}

}  // namespace rfp2
