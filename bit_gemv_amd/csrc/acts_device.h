// Rows of fp32 values four to a lane, and their int8 form: what the kernels that write
// activations share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rfp2 {

__device__ __forceinline__ void load4(float (&x)[4], const float* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

// Sixteen bytes to memory that nobody reads soon: past the caches (NT), which a large
// output would only sweep.  Read-back of 20011 tokens of 8 heads of 128: 53.2 us with
// ordinary stores, 34.6 us so.
template <bool NT>
__device__ __forceinline__ void store4(float* p, float4 x) {
  typedef float vec4 __attribute__((ext_vector_type(4)));
  const vec4 v = {x.x, x.y, x.z, x.w};
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<vec4*>(p));
  else *reinterpret_cast<vec4*>(p) = v;
}

// Code and scale as quantize_acts_kernel computes them, of four of the eight lanes' 32
// values.  Magnitudes are compared as integers, where infinities and NaN are the largest.
__device__ __forceinline__ float quantize4(const float (&x)[4], uint32_t& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  // over the eight lanes: neighbours, pairs, then the other four in reverse
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x141, 0xF, 0xF, true));
  const bool finite = top < 0x7F800000u;
  const float scale =
      finite ? __fdiv_rn(__uint_as_float(top), 127.0f) : __builtin_nanf("");
  codes = 0;
  if (finite && scale != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float r = fminf(fmaxf(roundf(__fdiv_rn(x[i], scale)), -127.0f), 127.0f);
      codes |= ((uint32_t)(int32_t)r & 0xFFu) << (8 * i);
    }
  }
  return scale;
}

}  // namespace rfp2
