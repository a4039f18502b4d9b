// MXFP8 blocks on the device: 32 consecutive columns share one scale 2^e (byte e + 127; 255:
// the block holds a NaN or an infinity, and every value reads as NaN), a value is an e4m3
// byte. With a the block's largest magnitude, e = max(floor(log2 a) - 8, -127), so that
// a / 2^e lies in [256, 512), and a value's code is x / 2^e rounded to the nearest e4m3 number,
// ties to the even code, magnitudes over 448 to 448 (OCP Microscaling Formats).
#pragma once

#include "sd_rows.h"

namespace sdv {
namespace {

// The largest of the value over a block's four neighbouring threads.
__device__ __forceinline__ uint32_t block_top(uint32_t top) {
  top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true));   // lane ^ 1
  return max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true));  // lane ^ 2
}

// Scale byte of a block from the fp32 bits of its largest magnitude.
__device__ __forceinline__ int mx8_scale(uint32_t top) {
  const int field = (int)(top >> 23);          // floor(log2) + 127 of a normal number
  return field == 255 ? 255 : max(field - 8, 0);
}

// Eight values as e4m3 under a scale byte other than 255. The hardware's conversion divides by
// the scale (an exponent alone: byte 0 is 2^-127) and rounds as above, but gives NaN over 464:
// magnitudes are held to 448 scales first, an fp32 number under every byte that a block has.
__device__ __forceinline__ u32x2 mx8_codes(const f32x4 &lo, const f32x4 &hi, int byte) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float((uint32_t)byte << 23);
  const float most = __uint_as_float((uint32_t)(byte + 8) << 23 | 0x600000u);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __builtin_amdgcn_fmed3f(lo[i], -most, most);
    v[4 + i] = __builtin_amdgcn_fmed3f(hi[i], -most, most);
  }
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s16x2 p = {0, 0};
    p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, v[4 * i], v[4 * i + 1], scale, 0);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, v[4 * i + 2], v[4 * i + 3], scale, 1);
    w[i] = __builtin_bit_cast(uint32_t, p);
  }
  return w;
}

// The eight values of two code words; exact in fp32 but past its largest and smallest numbers.
__device__ __forceinline__ void mx8_values(const u32x2 &w, int byte, f32x4 &lo, f32x4 &hi) {
  const float scale = __uint_as_float((uint32_t)byte << 23);
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], scale, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], scale, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], scale, 0);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], scale, 1);
  lo = f32x4{a[0], a[1], b[0], b[1]};
  hi = f32x4{c[0], c[1], d[0], d[1]};
  if (byte == 255) lo = hi = f32x4{1.f, 1.f, 1.f, 1.f} * __uint_as_float(0x7fc00000u);
}

}  // namespace
}  // namespace sdv
