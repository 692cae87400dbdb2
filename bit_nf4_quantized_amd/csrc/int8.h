// int8 values of blocks of 64, as the blockwise Int8 codec writes them, from 8
// values per lane, 8 neighbouring lanes holding a block. The codec leaves values
// that are not finite unspecified; here a block that holds an infinity or NaN
// has that as its absmax and codes 0, so that all its values are NaN (a NaN left
// out of the maximum would be kept as a finite value, and the backward pass from
// kept values would not show it).
#pragma once

#include "common.h"

namespace qlora {

// The codes of four values: rint(RN32(v c)), |v c| <= 127 (1 + 2^-23), as the low
// byte of RN32(v c) + 1.5 2^23 (whose unit in the last place is 1: the sum rounds
// to nearest even).
__device__ __forceinline__ uint32_t int8_codes(const float* v, float c) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(v[i] * c + 12582912.0f);
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// `at`: index of the lane's first value. The maxima keep a NaN (v_maximum3_f32).
__device__ __forceinline__ void store_int8(const float* v, int8_t* codes, float* absmax, int64_t at) {
  float m = __builtin_fabsf(v[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) m = __builtin_elementwise_maximum(m, __builtin_fabsf(v[e]));
  m = __builtin_elementwise_maximum(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0xB1, 0xF, 0xF, false)));   // quad_perm 1,0,3,2
  m = __builtin_elementwise_maximum(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0x4E, 0xF, 0xF, false)));   // quad_perm 2,3,0,1
  m = __builtin_elementwise_maximum(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0x141, 0xF, 0xF, false)));  // row_half_mirror
  const bool finite = m < __builtin_inff();
  const float c = m < 0x1p-120f ? 0.0f : 127.0f / m;
  *reinterpret_cast<u32x2_t*>(codes + at) = finite ? u32x2_t{int8_codes(v, c), int8_codes(v + 4, c)} : u32x2_t{0u, 0u};
  if ((threadIdx.x & 7) == 0) absmax[at >> 6] = m;
}

}  // namespace qlora
