// An fp32 value as the sum of three bf16 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace lce {

// x = p[0] + p[1] + p[2], each exactly a bf16 value: p[0] the nearest to x, p[1] the nearest to the
// rest, p[2] what is left (8 + 8 + 8 bits hold the 24 of x; exact unless the rest falls below
// bf16's smallest subnormal, 2^-133).  Where the nearest bf16 is inf but x is not, p[0] is x cut off
// to 8 bits.  An inf or NaN is p[0] alone.
__device__ __forceinline__ void split_bf16(float x, float (&p)[3]) {
  p[0] = __bfloat162float(__float2bfloat16_rn(x));
  const bool finite = (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
  if (finite && (__float_as_uint(p[0]) & 0x7f800000u) == 0x7f800000u)
    p[0] = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  const float r = finite ? x - p[0] : 0.f;
  p[1] = __bfloat162float(__float2bfloat16_rn(r));
  p[2] = __bfloat162float(__float2bfloat16_rn(r - p[1]));
}

}  // namespace lce
