// Device helpers of the microscaled 4-bit float kernels.
#pragma once

#include "moe_common.h"

namespace bitffn {

// The 8 values of a 32-bit word of codes (value j in bits 4j..4j+3), scaled by
// the scale byte s.  v_cvt_scalef32_pk_f32_fp4 reads its scale operand's exponent
// field alone: 2^(field - 127) also where a float with that field would be zero
// or subnormal, and NaN where it would be infinite, which is the byte's meaning.
__device__ __forceinline__ void mx_values8(uint32_t c, uint32_t s, float (&f)[8]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const float scale = __builtin_bit_cast(float, s << 23);
  const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
  const f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
  const f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
  const f2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  f[4] = d.x, f[5] = d.y, f[6] = e.x, f[7] = e.y;
}

}  // namespace bitffn
