// lora_q4.h -- host checks and device helpers shared by the 4-bit operators
// (internal; not part of the ABI).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lora_sgmv.h"
#include "lora_device.h"

namespace lora {

constexpr int kQ4Panel = 128;     // columns of a panel: 64 bytes and 4 exponents of every row
constexpr int kQ4RowBytes = 64;
constexpr int32_t kQ4Most = 0x7ffff000;  // rows and width: places past the end stay below 2^31
constexpr uint32_t kQ4NoNumber = 255;  // exponent of a block that holds NaN or an infinity

inline int64_t q4_panels(int64_t width) { return (width + kQ4Panel - 1) / kQ4Panel; }

// Checks one 4-bit matrix argument (host fields only); returns LORA_OK or the
// error it has set.
int check_q4(const lora_q4_t* q, const char* name);

// Biased exponent of a block from the largest magnitude's bits: the smallest
// e >= 1 with m <= 6 * 2^(e - 127). 6 = 1.5 * 2^2, so e is m's own exponent
// field less 2, and one more where the fraction is above 0.5. The bits of
// infinities and NaN are the largest of all: their block gets 255.
__device__ __forceinline__ uint32_t q4_exponent(uint32_t bits) {
  const int e = (int)(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return bits >= 0x7f800000u ? kQ4NoNumber : (uint32_t)(e < 1 ? 1 : e);
}

// Eight floats, divided by their block's scale, as eight e2m1 codes (element i
// in bits 4i), ties to even. The division is a product with the scale's
// reciprocal 2^(127 - e), exact for every e that a finite block can have.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&f)[8], float inv) {
  uint32_t v = 0;
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[0] * inv, f[1] * inv, 1.f, 0);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[2] * inv, f[3] * inv, 1.f, 1);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[4] * inv, f[5] * inv, 1.f, 2);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[6] * inv, f[7] * inv, 1.f, 3);
  return v;
}
// 2^(127 - e); a block without a number has the code 0 throughout.
__device__ __forceinline__ float q4_inverse(uint32_t e) {
  return e == kQ4NoNumber ? 0.f : __builtin_bit_cast(float, (254u - e) << 23);
}

// The same codes restored to bf16 (two significant bits times a power of two).
__device__ __forceinline__ u32x4 restore_e2m1(uint32_t q, uint32_t e) {
  const float s = __builtin_bit_cast(float, e << 23);
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  return e == kQ4NoNumber ? u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u} : v;
}

// Largest magnitude (as bits) of 8 bf16, for the exponent above.
__device__ __forceinline__ uint32_t abs_bits8(u32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) m = max(max(m, (v[q] << 16) & 0x7fffffffu), v[q] & 0x7fff0000u);
  return m;
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
// Largest over the 4 lanes that hold one block of 32 columns, in each of them.
__device__ __forceinline__ uint32_t max_over_4(uint32_t m) {
  m = max(m, dpp_move<0xB1>(m));  // quad_perm 1,0,3,2
  return max(m, dpp_move<0x4E>(m));  // quad_perm 2,3,0,1
}
// The four blocks' exponents (one value per quad of a 16-lane row) as the
// panel's dword, in the row's first lane.
__device__ __forceinline__ uint32_t gather_exps(uint32_t e) {
  return e | dpp_move<0x104>(e) << 8 | dpp_move<0x108>(e) << 16 | dpp_move<0x10C>(e) << 24;  // row_shl 4, 8, 12
}

}  // namespace lora
