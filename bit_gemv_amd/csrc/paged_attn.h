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
// head) are taken together: up to 16 a wave, in Q groups of four, and RW waves of a
// workgroup (1, 2 or 4) take different rows of the same tokens.  The 4 / RW waves
// that share their rows take every 4/RW-th tile of tokens.  Rows past 4 Q RW (64 at
// most) are further items that read the cache again.
//
// Tokens.  A tile is 32 cached tokens.  Scores are S = K q^T with
// v_mfma_f32_16x16x32_f16 (16 tokens x 32 values of a head x 16 rows); the sums
// O = W V with v_mfma_f32_4x4x1_f32, sixteen products of 4 rows x 1 token x 4
// values at once.  Row r of the first product's tile s stands for token
// 8 (r / 4) + 4 s + r % 4, which gives a lane the scores of eight consecutive tokens
// 8g .. 8g+7 (g = lane / 16) of one query row (lane % 16).  The weights change
// lanes through LDS (2 KB a wave at most); a lane of the second product holds one
// value of eight tokens, which the cache's layout keeps side by side, so neither
// product moves cached data between lanes (int8 keys trade halves once, to be
// loaded 16 bytes at a time).
//
// Precision.  Scores, weights and sums are fp32.  The query enters the first
// product as two halves, x = hi + lo (22 bits), scaled by a power of two a row;
// with one half, scores would be off by 2^-12 of sum |q k|, which the exponential
// turns into errors of a thousandth.  int8 codes and halves of the cache are
// exact operands.  A block of 32 values is one instruction long, so a key's scale
// multiplies its block's partial score, and a value's scale the weight.  Weights
// span more powers of two than halves hold (the largest may meet a value of 0),
// so the second product is fp32.  The 4 x 4 form makes that affordable: it does
// no work for rows that do not exist (with 16-row fp32 products the same kernel
// took 400 us where it takes 330, at 128 sequences of up to 8000 tokens and four
// rows a head).
//
// Split over the length.  The tiles of all (sequence, head) items form one line,
// each item with a few tiles' worth in front for what starting on it costs, cut
// into equal shares, one a workgroup: a long sequence is spread over all
// workgroups, short ones are packed, whatever the lengths, which only the GPU
// knows.  A share starts and ends inside an item at most once each: two slots of
// unfinished sums a workgroup in the workspace, which a second kernel joins;
// items inside one share are written out directly.
//
// What it reaches (MI355X; a plain read of 1 GiB runs at 6.44 TB/s): 128 sequences
// of 3000 to 8000 tokens, 32 query and 8 key/value heads of 128, int8 cache, 1.63 GB:
// 284 us, 5.7 TB/s, with 1.02 times the bytes read from memory that it cannot do
// without; one of 131001 tokens, 64 query heads: 67 us, 4.5 TB/s (start and join are
// about 12 us of it).  At 40 query rows a head (five new tokens, halves) it takes 90 us
// where the transfer alone would take 29, and nothing is busy throughout: the matrix
// cores 37 % of the clocks, the vector pipes 36 %.  They take turns: two waves a SIMD,
// and a wave's products wait for its own conversions of the values to fp32 (64 a lane and
// tile at heads of 128), its weights' way through LDS and the tile's loads.
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

// Waves a SIMD, of those that a variant's registers allow without spilling (nb: blocks of
// 32 values of a head, q: groups of four query rows).  More waves are also more shares to
// start and to join, and pay only where they hide much: codes in heads of up to 128 gain
// from the third (128 sequences 294 against 295 us, 32 sequences of 64 values 75 against
// 78), halves lose (32 + 8 heads of 128, 4 sequences of 2000 to 6000 tokens: 25.8 us with
// three, 23.4 with two; 32 sequences: 105 and 102).  A third wave for codes in heads of 256 (64
// sequences: 70 us -> 83) and a second for 256 halves and eight rows (55 -> 58) lose too.
constexpr int attn_waves(bool i8, int nb, int q) {
  if (i8) return nb <= 4 || (nb <= 6 && q == 1) ? 3 : nb <= 7 || q <= 2 ? 2 : 1;
  return nb <= 4 || (nb <= 6 && q <= 2) || q == 1 ? 2 : 1;
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
