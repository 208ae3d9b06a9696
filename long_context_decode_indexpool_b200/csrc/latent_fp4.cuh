// The 4-bit latent cache's format, on the device.
//
// A 512-wide latent row is 16 groups of 32 dims.  A value is an E2M1 code
// (sign, two exponent bits with bias 1, one fraction bit: 0, 0.5, 1, 1.5, 2,
// 3, 4, 6) times 2^e, e the exponent of its group, stored as the byte e + 127.
// With nat_g the smallest integer such that max |x_g| <= 6 * 2^nat_g (minus
// infinity for a group of zeros),
//     E   = max_g nat_g, clamped to [-50, 50],
//     e_g = nat_g, clamped to [E - 15, E].
// The first clamp bounds the exponents two rows can differ by (100), which
// the attention's fp32 statistics hold; the second makes a row exact in fp16
// once 2^E is taken out (its smallest step is then 2^-16), so the attention
// can run on fp16 tensor-core operands without rounding the cache again.  A
// value below half a step of its group is stored as zero, one above 6 * 2^50
// as 6 * 2^50.  A group that holds a NaN has the byte 255 and reads back as
// NaN; it does not count in E.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include "spx_internal.h"

namespace spx {

constexpr int kFp4Groups = kLatent / 32;     // scale bytes per row
constexpr int kFp4CodeBytes = kLatent / 2;   // code bytes per row
constexpr int kFp4MaxExp = 50;
constexpr int kFp4Spread = 15;
constexpr int kFp4NanByte = 255;

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float fp4_scale(uint32_t byte) {
  const uint32_t bits = byte == 0 ? 0x00400000u : (byte == kFp4NanByte ? 0x7FC00000u : byte << 23);
  return __uint_as_float(bits);
}

// The two values of a code byte (low half first).
__device__ __forceinline__ __half2 fp4x2_to_half2(uint32_t byte) {
  const __half2_raw h =
      __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte & 0xFFu), __NV_E2M1);
  return *reinterpret_cast<const __half2*>(&h);
}

// The eight values of four code bytes, two to a register.
__device__ __forceinline__ void fp4x8_to_half2x4(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}

}  // namespace spx
