// Microscaled 4-bit floating point (MXFP4): quantisation, the values back, and logits of
// hidden rows under an MXFP4 LM head (gfx950).
//
// A block of 32 consecutive columns of a row shares one scale 2^e, stored as the byte
// e + 127 (255: the block holds a NaN or an infinity, and every value reads as NaN); each
// value is a 4-bit float (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3,
// 4, 6). With a the block's largest magnitude, e = floor(log2 a) - 2, so that a / 2^e lies
// in [4, 8), and a value's code is x / 2^e rounded to the nearest of those, ties to the
// even code, magnitudes over 6 to 6 (OCP Microscaling Formats, the conversion it gives).
//
// Rows are stored padded to a multiple of 128 columns (one matrix instruction's depth):
// codes [rows][kp / 2] bytes, column 2 i in the low half of byte i, scales [rows][kp / 32]
// bytes; padding is code 0 under scale byte 0, which adds nothing to any product.
#include "sd_launch.h"

namespace sdv {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Eight consecutive values of a row as fp32, 0 past `left` of them. vec: 16-byte loads allowed.
__device__ inline void load8(const void *x, int32_t type, int64_t at, int left, bool vec, float (&v)[8]) {
  if (type == SD_F32) {
    const float *p = reinterpret_cast<const float *>(x) + at;
    if (vec && left >= 8) {
      const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.f;
    }
  } else {
    const uint16_t *p = reinterpret_cast<const uint16_t *>(x) + at;
    uint16_t h[8];
    if (vec && left >= 8) {
      *reinterpret_cast<u32x4 *>(h) = *reinterpret_cast<const u32x4 *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = i < left ? p[i] : (uint16_t)0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = type == SD_BF16 ? bf16_to_f32(h[i]) : (float)__builtin_bit_cast(_Float16, h[i]);
  }
}

// Code of x / 2^e (y = |x| / 2^e): the borders between neighbouring magnitudes lie midway,
// and a value on a border goes to the even code.
__device__ inline uint32_t e2m1(float x, float y) {
  uint32_t c = (y > 0.25f) + (y >= 0.75f) + (y > 1.25f) + (y >= 1.75f) + (y > 2.5f) + (y >= 3.5f) + (y > 5.f);
  return c | ((__float_as_uint(x) >> 31) << 3);
}

struct MxArgs {
  const void *x;
  int32_t type;
  int64_t rows, stride;    // elements from row to row
  int d, kp;
  bool vec;
  uint8_t *codes, *scales;
};

// Eight columns a thread, four neighbouring threads a block: its largest magnitude comes
// from two lane exchanges.
__global__ __launch_bounds__(256) void k_mx_quantize(MxArgs a) {
  const int per = a.kp / 8;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = t / per;
  if (row >= a.rows) return;      // whole groups of four threads: per is a multiple of 16
  const int c = (int)(t - row * per);
  float v[8];
  const int left = a.d - 8 * c;
  if (left > 0) {
    load8(a.x, a.type, row * a.stride + 8 * c, left, a.vec, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
  // As integers the magnitudes order like the values, NaN and infinity on top.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2));
  const int field = (int)(top >> 23);            // floor(log2) + 127 of a normal number
  const bool bad = field == 255;
  const int e = max(field - 127 - 2, -127);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) word |= e2m1(v[i], ldexpf(fabsf(v[i]), -e)) << (4 * i);
  if (bad) word = 0;
  *reinterpret_cast<uint32_t *>(a.codes + row * (a.kp / 2) + 4 * c) = word;
  // Padding keeps scale byte 0.
  if ((c & 3) == 0) a.scales[row * (a.kp / 32) + c / 4] = bad ? 255 : (left > 0 ? (uint8_t)(e + 127) : 0);
}

__device__ inline float e2m1_value(uint32_t c) {
  // Magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 in halves: 0 1 2 3 4 6 8 12.
  const uint32_t h = (0xc8643210u >> (4 * (c & 7))) & 15u;
  const float m = 0.5f * (float)h;
  return (c & 8) ? -m : m;
}

__device__ inline uint16_t f32_to_bf16(float x) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((b >> 16) | 0x40);
  return (uint16_t)((b + 0x7fffu + ((b >> 16) & 1u)) >> 16);
}

__device__ inline uint16_t pack16(float x, int32_t type) {
  return type == SD_BF16 ? f32_to_bf16(x) : __builtin_bit_cast(uint16_t, (_Float16)x);
}

// x[row][8 c ..] from the codes, eight columns a thread; x is written to column d - 1.
__global__ __launch_bounds__(256) void k_mx_dequantize(MxArgs a, void *x) {
  const int per = (a.d + 7) / 8;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = t / per;
  if (row >= a.rows) return;
  const int c = (int)(t - row * per), left = a.d - 8 * c;
  const uint32_t word = *reinterpret_cast<const uint32_t *>(a.codes + row * (a.kp / 2) + 4 * c);
  const int s = a.scales[row * (a.kp / 32) + c / 4];
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = s == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(e2m1_value((word >> (4 * i)) & 15u), s - 127);
  }
  const int64_t at = row * a.stride + 8 * c;
  if (a.type == SD_F32) {
    float *p = reinterpret_cast<float *>(x) + at;
    if (a.vec && left >= 8) {
      *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) if (i < left) p[i] = v[i];
    }
  } else {
    uint16_t *p = reinterpret_cast<uint16_t *>(x) + at;
    uint16_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = pack16(v[i], a.type);
    if (a.vec && left >= 8) {
      *reinterpret_cast<u32x4 *>(p) = *reinterpret_cast<u32x4 *>(h);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) if (i < left) p[i] = h[i];
    }
  }
}

// ------------------------------------------------------------------ product
struct MxGemmArgs {
  const uint8_t *hc, *hs;   // hidden codes [M][kp/2] and scales [M][kp/32]
  const uint8_t *wc, *ws;   // LM head codes [V][kp/2] and scales [V][kp/32]
  int M, V, kp;
  void *out;
  int32_t type;
  int64_t ld;               // elements from row to row
  bool vec;                 // four-element stores allowed
};

// D += A B^T over 128 columns of MXFP4: lane l holds row l % 16 of each operand at columns
// 32 (l / 16) .. + 31 (16 bytes, one scale), and of D the column l % 16 at rows
// 4 (l / 16) .. + 3. The LM-head fragment is operand A, so a lane's four results are
// consecutive vocabulary ids of one hidden row.
__device__ inline f32x4 mfma_mx(const u32x4 &a, int sa, const u32x4 &b, int sb, f32x4 c) {
  const i32x8 aa = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aa, bb, c, 4, 4, 0, sa, 0, sb);
}

__device__ inline void store4(const MxGemmArgs &a, int m, int v, const f32x4 &z) {
  const int64_t at = m * a.ld + v;
  if (a.type == SD_F32) {
    float *p = reinterpret_cast<float *>(a.out) + at;
    if (a.vec && v + 4 <= a.V) {
      *reinterpret_cast<f32x4 *>(p) = z;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) if (v + i < a.V) p[i] = z[i];
    }
  } else {
    uint16_t *p = reinterpret_cast<uint16_t *>(a.out) + at;
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack16(z[i], a.type);
    if (a.vec && v + 4 <= a.V) {
      *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(h);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) if (v + i < a.V) p[i] = h[i];
    }
  }
}

// One 16 x 16 tile a wave.
__global__ __launch_bounds__(256) void k_mx_gemm(MxGemmArgs a) {
  const int lane = threadIdx.x & 63, row = lane & 15, blk = lane >> 4;
  const int v0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 16, m0 = blockIdx.y * 16;
  if (v0 >= a.V) return;
  const int v = min(v0 + row, a.V - 1), m = min(m0 + row, a.M - 1);
  const uint8_t *wc = a.wc + (size_t)v * (a.kp / 2), *ws = a.ws + (size_t)v * (a.kp / 32);
  const uint8_t *hc = a.hc + (size_t)m * (a.kp / 2), *hs = a.hs + (size_t)m * (a.kp / 32);
  f32x4 z = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < a.kp / 32; k += 4) {
    const u32x4 w = *reinterpret_cast<const u32x4 *>(wc + 16 * (k + blk));
    const u32x4 h = *reinterpret_cast<const u32x4 *>(hc + 16 * (k + blk));
    z = mfma_mx(w, ws[k + blk], h, hs[k + blk], z);
  }
  if (m0 + row < a.M) store4(a, m0 + row, v0 + 4 * blk, z);
}

int64_t blocks_of(int64_t threads) { return (threads + 255) / 256; }

}  // namespace

hipError_t launch_mx_quantize(const void *x, int32_t type, int64_t rows, int d, int64_t stride,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const int size = type == SD_F32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (stride * size) % 16 == 0;
  const MxArgs a{x, type, rows, stride, d, mx_padded(d), vec, codes, scales};
  hipLaunchKernelGGL(k_mx_quantize, dim3((unsigned)blocks_of(rows * (a.kp / 8))), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int d,
                                void *x, int32_t type, int64_t stride, hipStream_t stream) {
  const int size = type == SD_F32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (stride * size) % 16 == 0;
  const MxArgs a{nullptr, type, rows, stride, d, mx_padded(d), vec, const_cast<uint8_t *>(codes),
                 const_cast<uint8_t *>(scales)};
  hipLaunchKernelGGL(k_mx_dequantize, dim3((unsigned)blocks_of(rows * ((d + 7) / 8))), dim3(256), 0,
                     stream, a, x);
  return hipGetLastError();
}

hipError_t launch_mx_logits(const void *hidden, int32_t hidden_type, int M, int d, int64_t stride,
                            const uint8_t *w_codes, const uint8_t *w_scales, int V, void *logits,
                            int32_t type, int64_t ld, void *workspace, hipStream_t stream) {
  size_t co, so;
  mx_logits_workspace_layout(M, d, &co, &so);
  uint8_t *w = reinterpret_cast<uint8_t *>(workspace);
  hipError_t e = launch_mx_quantize(hidden, hidden_type, M, d, stride, w + co, w + so, stream);
  if (e != hipSuccess) return e;
  const int size = type == SD_F32 ? 4 : 2;
  const bool vec = reinterpret_cast<uintptr_t>(logits) % (4 * size) == 0 && (ld * size) % (4 * size) == 0;
  const MxGemmArgs a{w + co, w + so, w_codes, w_scales, M, V, mx_padded(d), logits, type, ld, vec};
  hipLaunchKernelGGL(k_mx_gemm, dim3((V + 63) / 64, (M + 15) / 16), dim3(256), 0, stream, a);
  return hipGetLastError();
}

size_t mx_logits_workspace_layout(int M, int d, size_t *codes, size_t *scales) {
  const size_t kp = mx_padded(d), c = sizeof(WsHeader);
  const size_t s = align_up(c + (size_t)M * (kp / 2), 256);
  if (codes) *codes = c;
  if (scales) *scales = s;
  return align_up(s + (size_t)M * (kp / 32), 256);
}

}  // namespace sdv
