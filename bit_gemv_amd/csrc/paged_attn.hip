// The paged attention's dispatch and the kernel that joins the shares' sums
// (paged_attn.h holds the method, paged_attn_kernel.h the streaming kernel).
#include "paged_attn.h"

namespace rfp2 {

namespace {

// Query rows of an item: what the kernel variant that launch_attn picks takes at once.
int item_rows(int64_t rows) {
  return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 48 : 64;
}

// Rows up to which the join gives each a workgroup for every 32 values: one sequence of
// 4097 tokens (32 rows) 14.2 us in all against 15.5 with a wave a row, of 131001 tokens
// (64 rows) 77.5 against 80.9; 24 sequences (768 rows) 44.5 against 41.7, 128 sequences
// (4096 rows) 316 against 297.
constexpr int64_t kWideJoinRows = 256;

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t cum, ml, part, bytes;
};

Layout layout(int64_t dim, int64_t B, int64_t rows) {
  const size_t slots = size_t(2) * kAttnGroups * std::min<int64_t>(rows, item_rows(rows));
  Layout l;
  l.cum = 256;
  l.ml = l.cum + round256(4 * (size_t)(B + 1));
  l.part = l.ml + round256(slots * sizeof(float2));
  l.bytes = l.part + round256(slots * (size_t)dim * sizeof(float));
  return l;
}

// Joins the parts of an item that several workgroups worked on: their sums, with the
// weights exp2(m_i - m).  Also writes the rows that no tile belongs to: sequences without
// tokens (zeros) or with an impossible length (NaN).
//
// WIDE: a workgroup for 32 values of one row (a few rows in many parts: one long
// sequence), eight lanes side by side, 32 parts at once.  Otherwise a wave for each row
// (many rows, most of them in one or two parts or none at all to join).
template <bool WIDE>
__global__ __launch_bounds__(kJoinThreads) void paged_attn_join_kernel(const AttnArgs a,
                                                                       int rows_of_item) {
  constexpr int TEAM = WIDE ? kJoinThreads : 64;    // threads of a row (or of 32 values of it)
  __shared__ float red[kJoinThreads / 64];
  __shared__ float4 acc[WIDE ? 4 : 1][8];
  __shared__ float accl[4];
  const int D = a.c.dim, tid = threadIdx.x % TEAM;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int chunks = WIDE ? D >> 5 : 1;
  const uint32_t task = WIDE ? blockIdx.x / chunks : blockIdx.x * 4 + wave;
  const int row = (int)task;                        // (b * T + t) * H + h
  if (row >= a.B * a.T * a.H) return;
  const int bt = row / a.H, h = row - bt * a.H;
  const int b = bt / a.T, t = bt - b * a.T;
  const int quads = WIDE ? 8 : D >> 2;              // lanes that hold a part's values
  const int quad0 = WIDE ? 8 * (int)(blockIdx.x - task * chunks) : 0;
  const int lane = tid % quads, group = tid / quads, groups = TEAM / quads;
  float4* out = reinterpret_cast<float4*>(a.y + (int64_t)row * D) + quad0;
  const int64_t length = a.cum[b + 1] - a.cum[b];   // of an item of this sequence
  const int64_t share = a.plan[0];
  const int len = a.lens[b];
  const int start = a.B == 1 ? 0 : kAttnItemStart;
  if (length == 0) {
    const float v = len > 0 ? __builtin_nanf("") : 0.0f;
    if (tid < quads) out[tid] = make_float4(v, v, v, v);
    return;
  }
  const int kvh = h / a.group;
  const int r = t * a.group + (h - kvh * a.group);
  const int rg = r / rows_of_item;
  const int64_t items = (int64_t)a.c.heads * a.row_groups;
  const int64_t first =
      (int64_t)a.cum[b] * items + (int64_t)(kvh * a.row_groups + rg) * length + start;
  const int64_t w0 = divided(first, share), w1 = divided(first + length - start - 1, share);
  if (w0 == w1) return;                             // written by its one workgroup
  const int parts = (int)(w1 - w0 + 1);
  // part i is slot 0 of workgroup w0 + i, but for a first one that starts inside its share
  const int64_t at0 = (2 * w0 + (first != w0 * share ? 1 : 0)) * a.slot_rows + (r - rg * rows_of_item);
  const int64_t at1 = 2 * w0 * a.slot_rows + (r - rg * rows_of_item);
  auto at = [&](int i) { return i == 0 ? at0 : at1 + (int64_t)(2 * i) * a.slot_rows; };
  float m = -INFINITY;
  for (int i = tid; i < parts; i += TEAM) m = fmaxf(m, a.ml[at(i)].x);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if constexpr (WIDE) {
    if ((tid & 63) == 0) red[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.0f;
  if (group < groups) {
#pragma unroll 4
    for (int i = group; i < parts; i += groups) {
      const int64_t k = at(i);
      const float2 ml = a.ml[k];
      const float4 p = reinterpret_cast<const float4*>(a.part + k * D)[quad0 + lane];
      const float f = __builtin_amdgcn_exp2f(ml.x - m);
      l += f * ml.y;
      s.x += f * p.x; s.y += f * p.y; s.z += f * p.z; s.w += f * p.w;
    }
  }
  // the groups of a wave together: group g's lanes are g * quads further on
  if constexpr (WIDE) {
#pragma unroll
    for (int off = 8; off < 64; off <<= 1) {
      s.x += __shfl_xor(s.x, off, 64); s.y += __shfl_xor(s.y, off, 64);
      s.z += __shfl_xor(s.z, off, 64); s.w += __shfl_xor(s.w, off, 64);
      l += __shfl_xor(l, off, 64);
    }
    if ((tid & 63) < 8) acc[wave][tid & 7] = s;
    if ((tid & 63) == 0) accl[wave] = l;
    __syncthreads();
    if (tid < 8) {
      s = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 p = acc[w][tid];
        s.x += p.x; s.y += p.y; s.z += p.z; s.w += p.w;
        l += accl[w];
      }
    }
  } else {
    const float4 s0 = s;
    const float l0 = l;
    for (int g = 1; g < groups; ++g) {
      const int from = (tid + g * quads) & 63;
      s.x += __shfl(s0.x, from, 64); s.y += __shfl(s0.y, from, 64);
      s.z += __shfl(s0.z, from, 64); s.w += __shfl(s0.w, from, 64);
      l += __shfl(l0, from, 64);
    }
  }
  if (tid < quads) {
    const float f = 1.0f / l;
    const bool none = len - a.T + t < 0;            // a row that sees nothing
    out[lane] = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
  }
}

}  // namespace

size_t paged_attn_workspace_bytes(int64_t kv_heads, int64_t dim, int64_t B, int64_t new_tokens,
                                  int64_t H) {
  return layout(dim, B, new_tokens * (H / kv_heads)).bytes;
}

hipError_t launch_paged_attn(const KvView& c, bool i8, const float* q, int64_t B,
                             int64_t new_tokens, int64_t H, int64_t q_stride,
                             const int32_t* lens, float scale, int64_t window, float* y,
                             int32_t* err, void* workspace, hipStream_t stream) {
  const int64_t group = H / c.heads, rows = new_tokens * group;
  const int ir = item_rows(rows);
  const Layout l = layout(c.dim, B, rows);
  char* ws = static_cast<char*>(workspace);
  AttnArgs a;
  a.c = c;
  a.q = q;
  a.lens = lens;
  a.y = y;
  a.err = err;
  a.q_stride = q_stride;
  // positions are below 2^31, so a window of that size hides nothing
  a.window = window < (int64_t(1) << 31) - 16 ? (int32_t)window : 0;
  a.scale = scale;
  a.B = (int)B;
  a.T = (int)new_tokens;
  a.H = (int)H;
  a.group = (int)group;
  a.row_groups = (int)((rows + ir - 1) / ir);
  a.slot_rows = (int)std::min<int64_t>(rows, ir);
  a.plan = reinterpret_cast<int64_t*>(ws);
  a.cum = reinterpret_cast<uint32_t*>(ws + l.cum);
  a.ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part = reinterpret_cast<float*>(ws + l.part);
  // no more workgroups than shares of the longest lengths the page table allows
  const int64_t tiles = ((((int64_t)c.max_pages << c.page_shift) + 31) / 32 + 1) * B * c.heads *
                        a.row_groups;
  const int nb = c.dim / 32, quads = rows <= 4 ? 1 : rows <= 8 ? 2 : ir == 48 ? 3 : 4;
  const int grid = (int)std::min<int64_t>(kAttnCus * attn_waves(i8, nb, quads),
                                          std::max((tiles + kAttnMinTiles - 1) / kAttnMinTiles,
                                                   (int64_t)c.heads * a.row_groups));
  const auto launch = nb <= 2   ? launch_paged_attn_12
                      : nb <= 4 ? launch_paged_attn_34
                      : nb <= 6 ? launch_paged_attn_56
                                : launch_paged_attn_78;
  hipError_t e = launch(a, i8, nb, (int)std::min<int64_t>(rows, 64), grid, stream);
  if (e != hipSuccess) return e;
  const int64_t out_rows = B * new_tokens * H;
  if (out_rows <= kWideJoinRows)
    hipLaunchKernelGGL(paged_attn_join_kernel<true>, dim3((uint32_t)(out_rows * nb)),
                       dim3(kJoinThreads), 0, stream, a, ir);
  else
    hipLaunchKernelGGL(paged_attn_join_kernel<false>, dim3((uint32_t)((out_rows + 3) / 4)),
                       dim3(kJoinThreads), 0, stream, a, ir);
  return hipGetLastError();
}

}  // namespace rfp2
