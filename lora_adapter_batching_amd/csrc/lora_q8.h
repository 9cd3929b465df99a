// lora_q8.h -- host checks and device helpers shared by the 8-bit operators
// (internal; not part of the ABI).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lora_sgmv.h"
#include "lora_device.h"

namespace lora {

constexpr int kQ8Block = 128;  // columns that share one scale

inline int64_t q8_blocks(int64_t width) { return (width + kQ8Block - 1) / kQ8Block; }

// Checks one 8-bit matrix argument (host fields only); returns LORA_OK or the
// error it has set.
int check_q8(const lora_q8_t* q, const char* name, int block_rows);

// 16-byte alignment, stride and width of bf16 rows (the rules of every entry).
int check_bf16_rows(const void* p, int64_t ld, int64_t width, const char* name);

// 2^(e - 127) of a biased exponent 1 .. 254.
__device__ __forceinline__ float q8_scale(uint32_t e) { return __builtin_bit_cast(float, e << 23); }

// Smallest biased exponent e >= 1 with m <= 448 * 2^(e - 127), for the
// largest finite magnitude m of a block. 448 = 1.75 * 2^8, so e is m's own
// exponent field less 8, and one more where the fraction is above 0.75.
// Subnormal m (exponent field 0) and m = 0 end at the lower clamp; the largest
// finite m (field 254) gives 247.
__device__ __forceinline__ uint32_t q8_exponent(float m) {
  const uint32_t b = __builtin_bit_cast(uint32_t, m);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e);
}

// Magnitude of f as far as it is finite (NaN and infinities count as 0, so
// that one of them does not take its whole block with it).
__device__ __forceinline__ float finite_abs(float f) {
  const float a = __builtin_fabsf(f);
  return a <= 3.40282347e38f ? a : 0.f;
}

// Four floats to four e4m3 bytes, already divided by their scale (magnitudes
// up to 448, so nothing saturates), ties to even; NaN and infinities (which
// e4m3 lacks) become NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const float inf = __builtin_inff();
  a = __builtin_fabsf(a) == inf ? __builtin_nanf("") : a;
  b = __builtin_fabsf(b) == inf ? __builtin_nanf("") : b;
  c = __builtin_fabsf(c) == inf ? __builtin_nanf("") : c;
  d = __builtin_fabsf(d) == inf ? __builtin_nanf("") : d;
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// Largest value over the 16 lanes of a DPP row, in every one of them.
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true);
  return __builtin_fmaxf(v, __builtin_bit_cast(float, o));
}
__device__ __forceinline__ float max_over_16(float m) {
  m = dpp_max<0xB1>(m);       // quad_perm 1,0,3,2
  m = dpp_max<0x4E>(m);       // quad_perm 2,3,0,1
  m = dpp_max<0x141>(m);      // row_half_mirror
  return dpp_max<0x140>(m);   // row_mirror
}

}  // namespace lora
