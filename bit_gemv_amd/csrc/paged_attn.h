// Attention of each sequence's newest tokens over the paged key/value cache:
//
//   y = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j - m),
//
// in one pass over the visible cached tokens j with a running maximum m: when m
// grows, the sums so far are multiplied by exp(m_old - m_new).  Every cached
// byte is needed once and feeds only the few query rows that share its head, so
// the transfer from memory bounds the kernel; the layout of the work follows
// from keeping it streaming.
//
// Rows.  The new_tokens * H / kv_heads query rows of one (sequence, key/value
// head) are taken together, 16 to a matrix tile; RW tiles (1, 2 or 4) go to
// different waves of a workgroup, 4 / RW waves take every 4/RW-th tile of
// tokens.  Rows past 16 * RW are further items that read the cache again.
//
// Tokens.  A tile is 32 cached tokens.  Scores are S = K q^T with
// v_mfma_f32_16x16x32_f16 (16 tokens x 32 values of a head x 16 rows), the sums
// O^T = V^T P^T with v_mfma_f32_16x16x4_f32 (16 values x 4 tokens x 16 rows).
// Row r of the first product's tile s stands for token 8 (r / 4) + 4 s + r % 4,
// which leaves a lane with the scores of eight consecutive tokens 8g .. 8g+7
// (g = lane / 16) of one query row (lane % 16): just what the second product
// takes as its operand, four tokens 8g + j at a step, so the weights never leave
// their registers.  Its other operand is eight tokens of one value, which the
// cache's layout keeps side by side.
//
// Precision.  Scores, weights and sums are fp32.  The query enters the first
// product as two halves, x = hi + lo (22 bits), scaled by a power of two a row;
// with one half, scores would be off by 2^-12 of sum |q k|, which the exponential
// turns into errors of a thousandth.  int8 codes and halves of the cache are
// exact operands.  A block of 32 values is one instruction long, so a key's scale
// multiplies its block's partial score, and a value's scale the weight.  Weights
// span more powers of two than halves hold (the largest may meet a value of 0),
// so the second product is fp32: 64 instructions of 32 clocks a tile of 128
// values, 16 bytes of an int8 cache a clock and compute unit against the 9 that
// memory delivers.
//
// Split over the length.  The tiles of all (sequence, head) items form one line,
// cut into equal shares, one a workgroup: a long sequence is spread over all
// workgroups, short ones are packed, whatever the lengths, which only the GPU
// knows.  A share starts and ends inside an item at most once each: two slots of
// unfinished sums a workgroup in the workspace, which a second kernel joins;
// items inside one share are written out directly.
#pragma once

#include <hip/hip_fp16.h>

#include <type_traits>

#include "kv_device.h"

namespace rfp2 {

constexpr int kAttnThreads = 256;
constexpr int kJoinThreads = 256;
constexpr int kAttnCus = 256;             // compute units that shares are made for
constexpr int kAttnGroups = 3 * kAttnCus; // workgroups (shares) of a launch at most
constexpr int kAttnItemStart = 8;         // tiles in whose time a workgroup starts on an item
constexpr int kAttnMinTiles = 4;          // tiles of a share at least

// Waves a SIMD that a variant's registers allow without spilling (as the compiler
// reported them; nb: blocks of 32 values of a head, q: groups of four query rows).
constexpr int attn_waves(bool i8, int nb, int q) {
  if (i8) return nb <= 4 || (nb <= 6 && q == 1) ? 3 : nb <= 7 || q <= 2 ? 2 : 1;
  return nb <= 4 ? (q == 1 ? 3 : 2) : (nb <= 6 && q <= 2) || q == 1 ? 2 : 1;
}

// a / b for a >= 0, b > 0: by way of a reciprocal while the numbers are small (the full
// division is a long chain of instructions that every workgroup waits for).
__device__ __forceinline__ int64_t divided(int64_t a, int64_t b) {
  if ((a | b) < (int64_t(1) << 22)) {
    const int x = (int)a, y = (int)b;
    int q = (int)((float)x * __builtin_amdgcn_rcpf((float)y));    // off by one at most
    const int rest = x - q * y;
    q += rest >= y ? 1 : rest < 0 ? -1 : 0;
    return q;
  }
  return a / b;
}

struct AttnArgs {
  KvView c;
  const float* q;
  const int32_t* lens;
  float* y;
  int32_t* err;
  int64_t q_stride;
  int32_t window;                         // 0: none
  float scale;
  int32_t B, T, H;
  int32_t group;                          // query heads to a key/value head
  int32_t row_groups;                     // items a key/value head: ceil(T * group / (16 RW))
  int32_t slot_rows;                      // rows of a slot of the workspace
  // workspace
  int64_t* plan;                          // [0] tiles a share
  uint32_t* cum;                          // [B + 1] length of one item of the sequences before
  float2* ml;                             // [groups][2][slot_rows] maximum (base 2) and sum
  float* part;                            // [groups][2][slot_rows][D] sums
};

hipError_t launch_paged_attn_12(const AttnArgs& a, bool i8, int nb, int rows, int grid,
                                hipStream_t stream);
hipError_t launch_paged_attn_34(const AttnArgs& a, bool i8, int nb, int rows, int grid,
                                hipStream_t stream);
hipError_t launch_paged_attn_56(const AttnArgs& a, bool i8, int nb, int rows, int grid,
                                hipStream_t stream);
hipError_t launch_paged_attn_78(const AttnArgs& a, bool i8, int nb, int rows, int grid,
                                hipStream_t stream);

}  // namespace rfp2
