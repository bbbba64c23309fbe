// mx_widen.cuh -- E4M3 codes and their E8M0 scales as bf16 values, for the
// tensor-core kernels over MXFP8 pools.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace pkv {

// Eight E4M3 codes (two words) times 2^(s - 127), as eight bf16 values in a
// uint4, with integer operations and packed bf16 multiplies only.  A code
// s.eeee.mmm placed as bf16 bits s at 15 and eeeemmm at 10..4 reads as the
// E4M3 value times 2^-120 -- normal codes with exponent field e, subnormal
// codes as the bf16 subnormal m/8 2^-126, zero as zero -- so multiplying by
// 2^(s - 7) gives the scaled value: exact, as the product keeps at most four
// significant bits (values below bf16's smallest subnormal aside).  2^(s-7)
// can pass bf16's range (s > 134), so it is applied as 2^a (a <= 127), then,
// in the warps that need it, 2^(s - 7 - a).
__device__ __forceinline__ uint32_t place2(uint32_t pair) {  // bytes in halves -> bf16x2 bits
  // s.eeee.mmm -> s at 15, eeeemmm at 10..4: pair * 16 + sign * 240 (no carries)
  return (pair & 0x00800080u) * 240u + (pair << 4);
}

__device__ __forceinline__ uint4 widen8(uint2 w, __nv_bfloat162 s1, __nv_bfloat162 s2, bool big) {
  uint32_t out[4];
  const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = place2(__byte_perm(ws[i], 0u, 0x4140u));  // bytes 0, 1
    const uint32_t hi = place2(__byte_perm(ws[i], 0u, 0x4342u));  // bytes 2, 3
    __nv_bfloat162 vlo = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&lo), s1);
    __nv_bfloat162 vhi = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&hi), s1);
    if (big) {
      vlo = __hmul2(vlo, s2);
      vhi = __hmul2(vhi, s2);
    }
    out[2 * i] = *reinterpret_cast<const uint32_t*>(&vlo);
    out[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&vhi);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The two bf16x2 factors for scale byte g of the word sc: 2^a with a =
// min(s - 7, 127), and 2^(s - 7 - a) = 2^max(s - 134, 0).  (Byte g picked by
// a permute, as g varies with the thread.)
__device__ __forceinline__ void scale_factors(uint32_t sc, int g, __nv_bfloat162& s1,
                                              __nv_bfloat162& s2) {
  const uint32_t s = __byte_perm(sc, 0u, 0x4440u | (uint32_t)g);
  const uint32_t m = s < 134u ? s : 134u;
  const uint32_t w1 = m * 0x00800080u + 0x3C003C00u;               // exponent field m + 120
  const uint32_t w2 = (s - m) * 0x00800080u + 0x3F803F80u;         // exponent field s - m + 127
  s1 = *reinterpret_cast<const __nv_bfloat162*>(&w1);
  s2 = *reinterpret_cast<const __nv_bfloat162*>(&w2);
}

}  // namespace pkv
