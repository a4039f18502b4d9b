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
//
// The product reads both operands tiled: a tile is 64 rows by 128 columns. Its codes are four
// fragments of 16 rows (1 KB each), a fragment's 16 bytes for lane l being row l % 16 at
// columns 32 (l / 16) .. + 31, so a wave loads a fragment as one contiguous KB in the very
// order the matrix instruction takes it, from memory as from LDS without bank conflicts. Its
// scales are one 32-bit word a lane, byte i the scale of row 16 i + l % 16 at block l / 16:
// four fragments share the word, and the instruction's operand selects the byte.
//   codes  [ceil(rows / 64)][kp / 128][4][64 lanes][16 bytes], then
//   scales [ceil(rows / 64)][kp / 128][64 lanes][4 bytes]
#include <utility>

#include "sd_launch.h"

#define LDSP __attribute__((address_space(3)))
#define GLBP __attribute__((address_space(1)))

namespace sdv {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight consecutive values of a row as they are stored, 0 past `left` of them. vec: 16-byte
// loads allowed.
template <int T> struct Raw8 { u32x4 w; };
template <> struct Raw8<SD_F32> { f32x4 a, b; };

template <int T>
__device__ __forceinline__ Raw8<T> load8(const void *x, int64_t at, int left, bool vec) {
  Raw8<T> r;
  if constexpr (T == SD_F32) {
    const float *p = reinterpret_cast<const float *>(x) + at;
    if (vec && left >= 8) {
      r.a = *reinterpret_cast<const f32x4 *>(p);
      r.b = *reinterpret_cast<const f32x4 *>(p + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) { r.a[i] = i < left ? p[i] : 0.f; r.b[i] = 4 + i < left ? p[4 + i] : 0.f; }
    }
  } else {
    const uint16_t *p = reinterpret_cast<const uint16_t *>(x) + at;
    if (vec && left >= 8) {
      r.w = *reinterpret_cast<const u32x4 *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r.w[i] = (2 * i < left ? p[2 * i] : 0u) | (2 * i + 1 < left ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  }
  return r;
}

// The bits as fp32 of the largest of the eight magnitudes; as integers magnitudes order like
// the values, infinity and NaN on top.
template <int T>
__device__ __forceinline__ uint32_t top8(const Raw8<T> &r) {
  if constexpr (T == SD_F32) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      top = max(top, max(__float_as_uint(r.a[i]) & 0x7fffffffu, __float_as_uint(r.b[i]) & 0x7fffffffu));
    return top;
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(r.w[i] & 0x7fffu, (r.w[i] >> 16) & 0x7fffu));
    if (T == SD_BF16) return top << 16;
    return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)top));
  }
}

// By value: a bit cast of a vector's element itself would take the first one.
template <class P>
__device__ __forceinline__ P pair(uint32_t w) { return __builtin_bit_cast(P, w); }

// The eight codes, by the hardware's conversions: x / scale rounded to nearest, ties to the
// even code, magnitudes over 6 to 6, for every scale from 2^-127 on and with denormals (each
// 16-bit pattern and its scales tried against the rule, fp32 at the patterns around ties).
template <int T>
__device__ __forceinline__ uint32_t codes8(const Raw8<T> &r, float scale) {
  uint32_t w = 0;
  if constexpr (T == SD_F32) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r.a[0], r.a[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r.a[2], r.a[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r.b[0], r.b[1], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r.b[2], r.b[3], scale, 3);
  } else if constexpr (T == SD_BF16) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair<bf16x2>(r.w[0]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair<bf16x2>(r.w[1]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair<bf16x2>(r.w[2]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair<bf16x2>(r.w[3]), scale, 3);
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, pair<f16x2>(r.w[0]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, pair<f16x2>(r.w[1]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, pair<f16x2>(r.w[2]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, pair<f16x2>(r.w[3]), scale, 3);
  }
  return w;
}

struct MxArgs {
  const void *x;
  int32_t type;
  int64_t rows, stride;    // elements from row to row
  int d, kp;
  bool vec;
  uint8_t *codes, *scales;
};

// Scale byte (e + 127) of a block from its four threads' magnitudes, 255 for one that is not
// finite; an all-zero block has 0, padding among them. word: the thread's eight codes.
template <int T>
__device__ __forceinline__ int quantize_block(const Raw8<T> &r, uint32_t &word) {
  uint32_t top = top8<T>(r);
  top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true));   // lane ^ 1
  top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true));   // lane ^ 2
  const int field = (int)(top >> 23);          // floor(log2) + 127 of a normal number
  const int byte = max(field - 2, 0);
  word = field == 255 ? 0u : codes8<T>(r, __uint_as_float((uint32_t)byte << 23));
  return field == 255 ? 255 : byte;
}

// Row and column group of item n: base (row, c) of the workgroup's first item, `per` a row.
struct Item { int64_t row; int c; };
__device__ __forceinline__ Item item_at(int64_t row0, int c0, int n, int per) {
  const unsigned at = c0 + n, q = at / (unsigned)per;
  return {row0 + q, (int)(at - q * per)};
}

// An item is eight columns; four neighbouring threads hold a block, whose largest magnitude
// comes from two lane exchanges. A thread takes U items 256 apart, its loads issued together.
// Bound by memory: 129280 x 7168 bf16 in 447 us (2.35 GB, 5.2 TB/s; 847 us with codes formed
// by comparisons and a 64-bit division a thread), back in 390 us (6.0 TB/s).
template <int T, int U>
__global__ __launch_bounds__(256) void k_mx_quantize(MxArgs a) {
  const int per = a.kp / 8;       // a multiple of 16: a block's items are all in or all out
  const int64_t base = (int64_t)blockIdx.x * 256 * U, row0 = base / per;
  const int c0 = (int)(base - row0 * per);
  Item it[U];
  Raw8<T> r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    it[u] = item_at(row0, c0, threadIdx.x + 256 * u, per);
    const int left = it[u].row < a.rows ? a.d - 8 * it[u].c : 0;
    r[u] = Raw8<T>{};
    if (left > 0) r[u] = load8<T>(a.x, it[u].row * a.stride + 8 * it[u].c, left, a.vec);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t word;
    const int byte = quantize_block<T>(r[u], word);
    const int64_t row = it[u].row;
    const int c = it[u].c;
    if (row >= a.rows) continue;
    *reinterpret_cast<uint32_t *>(a.codes + row * (a.kp / 2) + 4 * c) = word;
    if ((c & 3) == 0) a.scales[row * (a.kp / 32) + c / 4] = (uint8_t)byte;
  }
}

// Rows quantised straight into tiles, one workgroup a tile: a wave takes 16 rows, four threads
// a block, and its four blocks in turn, so that each store of the wave is a whole quarter of
// its fragment. Rows past the last are left: their products are not stored.
template <int T>
__global__ __launch_bounds__(256) void k_mx_quantize_tiles(MxArgs a) {
  const int steps = a.kp / 128, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tile = blockIdx.x;
  const int64_t group = tile / steps;
  const int step = (int)(tile - group * steps), row16 = lane >> 2;
  const int64_t row = 64 * group + 16 * wave + row16;
  Raw8<T> r[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = 128 * step + 32 * u + 8 * (lane & 3), left = row < a.rows ? a.d - c : 0;
    r[u] = Raw8<T>{};
    if (left > 0) r[u] = load8<T>(a.x, row * a.stride + c, left, a.vec);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t word;
    const int byte = quantize_block<T>(r[u], word);
    if (row >= a.rows) continue;
    *reinterpret_cast<uint32_t *>(a.codes + tile * 4096 + wave * 1024 + (16 * u + row16) * 16 + (lane & 3) * 4) = word;
    if ((lane & 3) == 0) a.scales[tile * 256 + (16 * u + row16) * 4 + wave] = (uint8_t)byte;
  }
}

// The tiled form of codes and scales stored by row: one workgroup a tile, thread t moves the
// 16 bytes of fragment t / 64's lane t % 64; rows past the last are zero.
__global__ __launch_bounds__(256) void k_mx_tile(const uint8_t *codes, const uint8_t *scales, int V, int kp,
                                                 uint8_t *out_codes, uint8_t *out_scales) {
  const int steps = kp / 128, t = threadIdx.x, lane = t & 63;
  const int64_t tile = blockIdx.x;
  const int group = (int)(tile / steps), step = (int)(tile - (int64_t)group * steps);
  const int64_t row = 64 * (int64_t)group + 16 * (t >> 6) + (lane & 15);
  const int blk = 4 * step + (lane >> 4);
  u32x4 w = {0u, 0u, 0u, 0u};
  uint8_t s = 0;
  if (row < V) {
    w = *reinterpret_cast<const u32x4 *>(codes + row * (kp / 2) + 16 * blk);
    s = scales[row * (kp / 32) + blk];
  }
  *reinterpret_cast<u32x4 *>(out_codes + tile * 4096 + t * 16) = w;
  out_scales[tile * 256 + lane * 4 + (t >> 6)] = s;
}

// Rounded to nearest even, by the hardware's conversions.
__device__ inline u32x2 pack4(const f32x4 &z, int32_t type) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  return type == SD_BF16 ? __builtin_bit_cast(u32x2, __builtin_convertvector(z, bf16x4))
                         : __builtin_bit_cast(u32x2, __builtin_convertvector(z, f16x4));
}

// x[row][8 c ..] from the codes; x is written to column d - 1. Items as in k_mx_quantize.
// The hardware's conversion gives the fp32 value of code and scale exactly (each pair tried).
template <int T, int U>
__global__ __launch_bounds__(256) void k_mx_dequantize(MxArgs a, void *x) {
  const int per = (a.d + 7) / 8;
  const int64_t base = (int64_t)blockIdx.x * 256 * U, row0 = base / per;
  const int c0 = (int)(base - row0 * per);
  Item it[U];
  uint32_t word[U];
  int s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    it[u] = item_at(row0, c0, threadIdx.x + 256 * u, per);
    if (it[u].row < a.rows) {
      word[u] = *reinterpret_cast<const uint32_t *>(a.codes + it[u].row * (a.kp / 2) + 4 * it[u].c);
      s[u] = a.scales[it[u].row * (a.kp / 32) + it[u].c / 4];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (it[u].row >= a.rows) continue;
    const float scale = __uint_as_float((uint32_t)s[u] << 23);
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[u], scale, 0);
    const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[u], scale, 1);
    const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[u], scale, 2);
    const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word[u], scale, 3);
    f32x4 lo = {p0[0], p0[1], p1[0], p1[1]}, hi = {p2[0], p2[1], p3[0], p3[1]};
    if (s[u] == 255) lo = hi = f32x4{1.f, 1.f, 1.f, 1.f} * __uint_as_float(0x7fc00000u);
    const int64_t at = it[u].row * a.stride + 8 * it[u].c;
    const int left = a.d - 8 * it[u].c;
    if constexpr (T == SD_F32) {
      float *p = reinterpret_cast<float *>(x) + at;
      if (a.vec && left >= 8) {
        *reinterpret_cast<f32x4 *>(p) = lo;
        *reinterpret_cast<f32x4 *>(p + 4) = hi;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) if (i < left) p[i] = i < 4 ? lo[i] : hi[i - 4];
      }
    } else {
      uint16_t *p = reinterpret_cast<uint16_t *>(x) + at;
      const u32x2 a2 = pack4(lo, T), b2 = pack4(hi, T);
      const u32x4 h = {a2[0], a2[1], b2[0], b2[1]};
      if (a.vec && left >= 8) {
        *reinterpret_cast<u32x4 *>(p) = h;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) if (i < left) p[i] = (uint16_t)(h[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

// ------------------------------------------------------------------ product
struct MxGemmArgs {
  const uint8_t *hc, *hs;   // hidden rows, tiled
  const uint8_t *wc, *ws;   // LM head, tiled
  int M, V, steps;          // steps: 128-column steps
  void *out;
  int32_t type;
  int64_t ld;               // elements from row to row
  bool vec, wide;           // four-element and 16-byte stores allowed
};

// D += A B^T over 128 columns of MXFP4: lane l holds row l % 16 of each operand at columns
// 32 (l / 16) .. + 31 (16 bytes), of D the column l % 16 at rows 4 (l / 16) .. + 3. sa and sb
// hold four scales, one a byte; byte SA and SB apply. The LM-head fragment is operand A, so
// a lane's four results are consecutive vocabulary ids of one hidden row.
template <int SA, int SB>
__device__ inline f32x4 mfma_mx(const u32x4 &a, int sa, const u32x4 &b, int sb, f32x4 c) {
  const i32x8 aa = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aa, bb, c, 4, 4, SA, sa, SB, sb);
}

// The byte selectors are immediates: a call per (id fragment, row fragment) pair.
template <int SA>
__device__ inline f32x4 mfma_mx_b(int sel_b, const u32x4 &a, int sa, const u32x4 &b, int sb, f32x4 c) {
  return sel_b == 0 ? mfma_mx<SA, 0>(a, sa, b, sb, c) : mfma_mx<SA, 1>(a, sa, b, sb, c);
}

__device__ inline f32x4 mfma_mx_sel(int sel_a, int sel_b, const u32x4 &a, int sa, const u32x4 &b, int sb, f32x4 c) {
  switch (sel_a) {
    case 0: return mfma_mx_b<0>(sel_b, a, sa, b, sb, c);
    case 1: return mfma_mx_b<1>(sel_b, a, sa, b, sb, c);
    case 2: return mfma_mx_b<2>(sel_b, a, sa, b, sb, c);
    default: return mfma_mx_b<3>(sel_b, a, sa, b, sb, c);
  }
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
    const u32x2 h = pack4(z, a.type);
    if (a.vec && v + 4 <= a.V) {
      *reinterpret_cast<u32x2 *>(p) = h;
    } else {
      const uint32_t w[2] = {h[0], h[1]};
#pragma unroll
      for (int i = 0; i < 4; ++i) if (v + i < a.V) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  }
}

// ---------------------------------------------------------- few hidden rows
// Up to 16 MT rows, MT at most 2: the LM head's bytes bound the call. One workgroup per 64 ids; its four
// waves take the 128-column steps in turn (wave w steps w, w + 4, ..), so a workgroup reads
// one contiguous 17 KB run a round, straight into registers: each weight is used by one wave
// only, so LDS would add a copy and share nothing. The hidden fragments are read by every
// workgroup and come from L2: at 64 rows as many bytes as weights, and slower than a tile
// through LDS (129280 x 7168: 108 against 91 us; at 32 rows 86 against 89). The waves'
// partial sums meet in LDS in wave order. 129280 x 7168 under 16 rows: 64 us where the head
// is partly in the memory-side cache (repeated calls), 78 us = 6.3 TB/s from memory.
template <int MT>
__global__ __launch_bounds__(256) void k_mx_skinny(MxGemmArgs a) {
  static_assert(MT <= 2, "selectors of two row fragments");
  constexpr int D = 3;                 // steps a wave has in flight
  constexpr int LDR = 68;              // floats from row to row in LDS: rows start on other banks
  __shared__ float red[4][16 * MT * LDR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t g = blockIdx.x;
  const u32x4 *wc = reinterpret_cast<const u32x4 *>(a.wc + g * a.steps * 4096) + lane;
  const int *ws = reinterpret_cast<const int *>(a.ws + g * a.steps * 256) + lane;
  const u32x4 *hc = reinterpret_cast<const u32x4 *>(a.hc) + lane;
  const int *hs = reinterpret_cast<const int *>(a.hs) + lane;
  f32x4 acc[4][MT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 w[D][4], h[D][MT];
  int sw[D], sh[D];
  auto load = [&](int s, int d) {
    const int64_t k = min(s, a.steps - 1);      // past the end: the last step again, unused
#pragma unroll
    for (int i = 0; i < 4; ++i) w[d][i] = __builtin_nontemporal_load(wc + k * 256 + i * 64);
    sw[d] = __builtin_nontemporal_load(ws + k * 64);
#pragma unroll
    for (int m = 0; m < MT; ++m) h[d][m] = hc[k * 256 + m * 64];
    sh[d] = hs[k * 64];
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(wave + 4 * d, d);
  for (int s = wave; s < a.steps; s += 4 * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (s + 4 * d < a.steps) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[i][m] = mfma_mx_sel(i, m, w[d][i], sw[d], h[d][m], sh[d], acc[i][m]);
      }
      load(s + 4 * (D + d), d);
    }
  }
  const int col = lane & 15, blk = lane >> 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4 *>(&red[wave][(16 * m + col) * LDR + 16 * i + 4 * blk]) = acc[i][m];
  __syncthreads();
  for (int t = threadIdx.x; t < 16 * MT * 16; t += 256) {
    const int m = t >> 4, v = 4 * (t & 15);
    if (m >= a.M) break;
    f32x4 z = *reinterpret_cast<const f32x4 *>(&red[0][m * LDR + v]);
#pragma unroll
    for (int q = 1; q < 4; ++q) {
      const f32x4 o = *reinterpret_cast<const f32x4 *>(&red[q][m * LDR + v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] += o[e];
    }
    store4(a, m, 64 * (int)g + v, z);
  }
}

// ------------------------------------------------------------- many hidden rows
__device__ inline void raw_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// f(0), f(1), .. f(N - 1) with each number a constant.
template <class F, int... I>
__device__ __forceinline__ void each_impl(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
  each_impl(f, std::make_integer_sequence<int, N>{});
}

// At most N of this wave's memory reads pending, no LDS read.
template <int N>
__device__ inline void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (((N >> 4) & 3) << 14) | (0x7 << 4));
}

// The matrix instruction with its accumulator as both operand and result, in accumulation
// registers: left to itself the compiler gives this instruction another result register and
// moves accumulators about, some 200 moves for 64 instructions. It also knows no hazards of
// inline assembly, so two idle states stand before each (a vector write of an operand needs
// them) and settle() stands between the last one and the first read of a result.
#define SD_MX_INTO(SA0, SA1, SB0, SB1)                                                         \
  asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[" #SA0       \
      "," #SB0 ",0] op_sel_hi:[" #SA1 "," #SB1 ",0] cbsz:4 blgp:4"                              \
      : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb) : "memory")

__device__ __forceinline__ void mfma_mx_into(int sel_a, int sel_b, const u32x4 &a, int sa, const u32x4 &b, int sb,
                                             f32x4 &c) {
  switch (sel_a * 4 + sel_b) {
    case 0: SD_MX_INTO(0, 0, 0, 0); break;
    case 1: SD_MX_INTO(0, 0, 1, 0); break;
    case 2: SD_MX_INTO(0, 0, 0, 1); break;
    case 3: SD_MX_INTO(0, 0, 1, 1); break;
    case 4: SD_MX_INTO(1, 0, 0, 0); break;
    case 5: SD_MX_INTO(1, 0, 1, 0); break;
    case 6: SD_MX_INTO(1, 0, 0, 1); break;
    case 7: SD_MX_INTO(1, 0, 1, 1); break;
    case 8: SD_MX_INTO(0, 1, 0, 0); break;
    case 9: SD_MX_INTO(0, 1, 1, 0); break;
    case 10: SD_MX_INTO(0, 1, 0, 1); break;
    case 11: SD_MX_INTO(0, 1, 1, 1); break;
    case 12: SD_MX_INTO(1, 1, 0, 0); break;
    case 13: SD_MX_INTO(1, 1, 1, 0); break;
    case 14: SD_MX_INTO(1, 1, 0, 1); break;
    default: SD_MX_INTO(1, 1, 1, 1); break;
  }
}
#undef SD_MX_INTO

__device__ __forceinline__ void settle() { asm volatile("s_nop 12"); }

// n rows of W results of type T from a wave's part of LDS (rows ROW bytes apart) to rows m0 .. of
// the output at column v0: 16 bytes a lane along the rows where they are aligned and whole, else
// an element a lane.
template <class T, int W, int ROW>
__device__ __forceinline__ void store_rows(const MxGemmArgs &a, const LDSP uint8_t *part, int64_t m0, int n, int v0, int lane) {
  constexpr int E = 16 / sizeof(T), LPR = W / E;     // elements a lane, lanes a row
  static_assert(64 % LPR == 0, "whole rows a store");
  const int rows = (int)min((int64_t)n, a.M - m0);
  T *out = reinterpret_cast<T *>(a.out) + m0 * a.ld + v0;
  if (a.wide && v0 + W <= a.V) {
    for (int r = lane / LPR; r < rows; r += 64 / LPR) {
      const u32x4 x = *(const LDSP u32x4 *)(part + r * ROW + (lane % LPR) * 16);
      __builtin_nontemporal_store(x, reinterpret_cast<u32x4 *>(out + r * a.ld + (lane % LPR) * E));
    }
  } else {
    for (int r = 0; r < rows; ++r)
      for (int v = lane; v < W && v0 + v < a.V; v += 64)
        out[r * a.ld + v] = *(const LDSP T *)(part + r * ROW + v * (int)sizeof(T));
  }
}

// A workgroup of four waves computes 64 GV ids by 64 GM hidden rows, each wave 16 TV by 16 TM
// (WV by WM waves). A step's 128 columns of both operands come into one of NS LDS buffers by
// direct loads, NS - 1 steps ahead. While a wave's matrix instructions consume step k from
// registers it reads step k + 1's fragments from LDS, so with one wave a SIMD the matrix
// units still run back to back. One barrier a step: behind it every wave has read step k
// out of LDS, so its buffer takes step k + NS. 2048 rows by 129280 ids at depth 7168 in 256 x
// 256 tiles take 930 us (4.1 PFLOP/s). With the loads left out (copies of the kernel, for
// timing) it is 743 us, with the LDS reads left out too 642 us: 5.9 PFLOP/s, near the 6.0 -
// 6.8 of the bare instruction on random operands in registers (8.6 on zeros: the card's power
// sets its clock). So 290 us of feeding are not hidden behind the instructions; what holds
// them up is not known.
template <int WV, int WM, int TV, int TM, int NS>
__global__ __launch_bounds__(256, 1) void k_mx_tiled(MxGemmArgs a, int n_mt, int n_vt) {
  constexpr int GV = WV * TV / 4, GM = WM * TM / 4, G = GV + GM;
  constexpr int STAGE = G * (4096 + 256);
  constexpr int SPW = (G + 3) / 4;            // scale loads a wave
  constexpr int DPT = G + SPW;                // loads a wave and step
  static_assert(WV * WM == 4 && TV % 4 == 0 && TM % 4 == 0, "whole 64-row groups a wave");
  __shared__ __attribute__((aligned(16))) uint8_t S[NS * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wv = wave / WM, wm = wave % WM;
  // Tiles go to the XCDs (workgroup id mod 8) in contiguous runs with the hidden tile
  // running fastest: an XCD's workgroups share LM-head tiles and hidden tiles in its L2.
  const int nb = n_mt * n_vt, hb = blockIdx.x;
  const int per = nb / 8, rem = nb % 8, xcd = hb % 8, pos = hb / 8;
  const int logical = (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + pos;
  const int mt = logical % n_mt, vt = logical / n_mt;
  // Source of each of this wave's loads at step 0, the same address for all lanes; a step
  // further is 4096 (codes) or 256 (scales) bytes. Groups past the end repeat the last one;
  // their results are not stored.
  const int last_v = (a.V - 1) / 64, last_m = (a.M - 1) / 64;
  auto group = [&](int i, const uint8_t *w, const uint8_t *h, int64_t bytes) {
    return i < GV ? w + (int64_t)min(vt * GV + i, last_v) * a.steps * bytes
                  : h + (int64_t)min(mt * GM + i - GV, last_m) * a.steps * bytes;
  };
  const uint8_t *src[DPT];
#pragma unroll
  for (int i = 0; i < G; ++i) src[i] = group(i, a.wc, a.hc, 4096) + wave * 1024;
#pragma unroll
  for (int i = 0; i < SPW; ++i) src[G + i] = group(min(wave + 4 * i, G - 1), a.ws, a.hs, 256);
  const uint32_t lane16 = lane * 16, lane4 = lane * 4;
  // Load i of the DPT that bring step k in; kk: the step itself, or the last one past the end.
  auto issue = [&](int k, int kk, int i) __attribute__((always_inline)) {
    LDSP uint8_t *dst = (LDSP uint8_t *)S + (k % NS) * STAGE;
    if (i < G)
      __builtin_amdgcn_global_load_lds((const GLBP void *)(src[i] + (int64_t)kk * 4096 + lane16),
                                       (LDSP void *)(dst + i * 4096 + wave * 1024), 16, 0, 0);
    else
      __builtin_amdgcn_global_load_lds((const GLBP void *)(src[i] + (int64_t)kk * 256 + lane4),
                                       (LDSP void *)(dst + G * 4096 + min(wave + 4 * (i - G), G - 1) * 256), 4, 0, 0);
  };
  struct Frags {
    u32x4 w[TV], h[TM];
    int sw[TV / 4], sh[TM / 4];
  };
  // Read j of the FETCHES that take a step's fragments out of LDS.
  constexpr int FETCHES = TV + TM + TV / 4 + TM / 4;
  auto fetch = [&](int k, int j, Frags &f) __attribute__((always_inline)) {
    const LDSP uint8_t *b = (const LDSP uint8_t *)S + (k % NS) * STAGE;
    const LDSP uint8_t *sb = b + G * 4096 + lane4;
    if (j < TV / 4) f.sw[j] = *(const LDSP int *)(sb + (wv * TV / 4 + j) * 256);
    else if (j < TV / 4 + TM / 4) f.sh[j - TV / 4] = *(const LDSP int *)(sb + (GV + wm * TM / 4 + j - TV / 4) * 256);
    else if ((j -= TV / 4 + TM / 4) < TM) f.h[j] = *(const LDSP u32x4 *)(b + GV * 4096 + wm * TM * 1024 + lane16 + j * 1024);
    else f.w[j - TM] = *(const LDSP u32x4 *)(b + wv * TV * 1024 + lane16 + (j - TM) * 1024);
  };
  f32x4 acc[TV][TM];
#pragma unroll
  for (int i = 0; i < TV; ++i)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Step k: its fragments are in `now`; the next step's go to `next`. The reads and loads
  // stand between the matrix instructions, where they are written: all at once, they would
  // fill their queues and hold up the instructions behind them.
  constexpr int MM = TV * TM;
  static_assert(FETCHES <= MM && DPT <= MM, "at most one of each before a matrix instruction");
  auto step = [&](int k, const Frags &now, Frags &next) __attribute__((always_inline)) {
    wait_loads<(NS - 2) * DPT>();      // step k + 1 has arrived
    raw_barrier();
    const int kk = min(k + NS, a.steps - 1);
    each<MM>([&](auto x) __attribute__((always_inline)) {
      if constexpr (x * FETCHES % MM < FETCHES) fetch(k + 1, x * FETCHES / MM, next);
      if constexpr (x * DPT % MM < DPT) issue(k + NS, kk, x * DPT / MM);
      constexpr int i = x / TM, m = x % TM;
      mfma_mx_into(i % 4, m % 4, now.w[i], now.sw[i / 4], now.h[m], now.sh[m / 4], acc[i][m]);
    });
    settle();
  };
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int i = 0; i < DPT; ++i) issue(k, min(k, a.steps - 1), i);
  wait_loads<(NS - 1) * DPT>();
  raw_barrier();
  Frags f0, f1;
#pragma unroll
  for (int j = 0; j < FETCHES; ++j) fetch(0, j, f0);
  int k = 0;
  for (; k + 1 < a.steps; k += 2) {
    step(k, f0, f1);
    step(k + 1, f1, f0);
  }
  if (k < a.steps) {
    each<MM>([&](auto x) __attribute__((always_inline)) {
      constexpr int i = x / TM, m = x % TM;
      mfma_mx_into(i % 4, m % 4, f0.w[i], f0.sw[i / 4], f0.h[m], f0.sh[m / 4], acc[i][m]);
    });
    settle();
  }
  wait_loads<0>();                     // the trailing loads land before LDS is used again
  raw_barrier();
  // The results cross LDS so that a wave's stores run along the rows: out of the accumulators
  // a store would touch 16 rows with 32 or 64 bytes each. Each wave has a part of LDS to
  // itself, rows 16 bytes apart from a power of two so that neighbouring rows start on other
  // banks; 16-bit results cross at once, 32-bit ones in two halves of the rows.
  const int col = lane & 15, blk = lane >> 4;
  const int64_t m0 = (int64_t)mt * 64 * GM + wm * TM * 16;
  const int v0 = vt * 64 * GV + wv * TV * 16;
  constexpr int PART = NS * STAGE / 4 / 16 * 16;
  LDSP uint8_t *part = (LDSP uint8_t *)S + wave * PART;
  if (a.type == SD_F32) {
    constexpr int ROW = TV * 16 * 4 + 16;
    static_assert(ROW * TM * 8 <= PART, "half the rows in fp32");
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int m = 0; m < TM / 2; ++m)
#pragma unroll
        for (int i = 0; i < TV; ++i)
          *(LDSP f32x4 *)(part + (16 * m + col) * ROW + (16 * i + 4 * blk) * 4) = acc[i][half * TM / 2 + m];
      store_rows<float, TV * 16, ROW>(a, part, m0 + half * TM * 8, TM * 8, v0, lane);
    }
  } else {
    constexpr int ROW = TV * 16 * 2 + 16;
    static_assert(ROW * TM * 16 <= PART, "the rows in 16 bits");
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int i = 0; i < TV; ++i)
        *(LDSP u32x2 *)(part + (16 * m + col) * ROW + (16 * i + 4 * blk) * 2) = pack4(acc[i][m], a.type);
    store_rows<uint16_t, TV * 16, ROW>(a, part, m0, TM * 16, v0, lane);
  }
}

template <class F>
void by_type(int32_t type, F f) {
  if (type == SD_F32) f(std::integral_constant<int, SD_F32>{});
  else if (type == SD_BF16) f(std::integral_constant<int, SD_BF16>{});
  else f(std::integral_constant<int, SD_F16>{});
}

// launch(type, items a thread, grid) for items of eight columns. Four a thread once every CU
// has several workgroups of them. bf16, us for one / four a thread (quantise; back):
//   2^16 items 3.5 / 4.1; 3.5 / 4.2   2^21 items 9.5 / 8.5; 9.6 / 9.2   2^25 items 125 / 122; 138 / 115
template <class F>
hipError_t by_items(int32_t type, int64_t items, F launch) {
  by_type(type, [&](auto T) {
    if (items >= 1 << 21) launch(T, std::integral_constant<int, 4>{}, dim3((unsigned)((items + 1023) / 1024)));
    else launch(T, std::integral_constant<int, 1>{}, dim3((unsigned)((items + 255) / 256)));
  });
  return hipGetLastError();
}

template <int WV, int WM, int TV, int TM, int NS>
hipError_t launch_tiled(const MxGemmArgs &a, hipStream_t stream) {
  const int n_mt = (a.M + 16 * WM * TM - 1) / (16 * WM * TM), n_vt = (a.V + 16 * WV * TV - 1) / (16 * WV * TV);
  hipLaunchKernelGGL((k_mx_tiled<WV, WM, TV, TM, NS>), dim3((unsigned)((int64_t)n_mt * n_vt)), dim3(256), 0,
                     stream, a, n_mt, n_vt);
  return hipGetLastError();
}

// Rounds over 256 CUs of the workgroups of a tiling.
double rounds(int M, int V, int ids, int rows) {
  const int64_t n = (int64_t)((V + ids - 1) / ids) * ((M + rows - 1) / rows);
  return (double)((n + 255) / 256);
}

bool vec_rows(const void *x, int32_t type, int64_t stride, int elems) {
  const int64_t size = type == SD_F32 ? 4 : 2, bytes = size * elems;
  return reinterpret_cast<uintptr_t>(x) % bytes == 0 && stride * size % bytes == 0;
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, int32_t type, int64_t rows, int d, int64_t stride,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const bool vec = vec_rows(x, type, stride, type == SD_F32 ? 4 : 8);
  const MxArgs a{x, type, rows, stride, d, mx_padded(d), vec, codes, scales};
  return by_items(type, rows * (a.kp / 8), [&](auto T, auto U, dim3 grid) {
    hipLaunchKernelGGL((k_mx_quantize<T, U>), grid, dim3(256), 0, stream, a);
  });
}

hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int d,
                                void *x, int32_t type, int64_t stride, hipStream_t stream) {
  const bool vec = vec_rows(x, type, stride, type == SD_F32 ? 4 : 8);
  const MxArgs a{nullptr, type, rows, stride, d, mx_padded(d), vec, const_cast<uint8_t *>(codes),
                 const_cast<uint8_t *>(scales)};
  return by_items(type, rows * ((d + 7) / 8), [&](auto T, auto U, dim3 grid) {
    hipLaunchKernelGGL((k_mx_dequantize<T, U>), grid, dim3(256), 0, stream, a, x);
  });
}

size_t mx_tiled_bytes(int64_t rows, int d, size_t *scales) {
  const size_t tiles = (size_t)((rows + 63) / 64) * (mx_padded(d) / 128);
  if (scales) *scales = tiles * 4096;
  return tiles * (4096 + 256);
}

hipError_t launch_mx_head(const uint8_t *codes, const uint8_t *scales, int V, int d, uint8_t *head,
                          hipStream_t stream) {
  size_t so;
  const int64_t tiles = mx_tiled_bytes(V, d, &so) / (4096 + 256);
  hipLaunchKernelGGL(k_mx_tile, dim3((unsigned)tiles), dim3(256), 0, stream, codes, scales, V, mx_padded(d),
                     head, head + so);
  return hipGetLastError();
}

size_t mx_logits_workspace_bytes(int M, int d) {
  return align_up(sizeof(WsHeader) + mx_tiled_bytes(M, d, nullptr), 256);
}

hipError_t launch_mx_logits(const void *hidden, int32_t hidden_type, int M, int d, int64_t stride,
                            const uint8_t *head, int V, void *logits, int32_t type, int64_t ld,
                            void *workspace, hipStream_t stream) {
  size_t hs, ws;
  mx_tiled_bytes(M, d, &hs);
  mx_tiled_bytes(V, d, &ws);
  uint8_t *h = reinterpret_cast<uint8_t *>(workspace) + sizeof(WsHeader);
  const MxArgs q{hidden, hidden_type, M, stride, d, mx_padded(d),
                 vec_rows(hidden, hidden_type, stride, hidden_type == SD_F32 ? 4 : 8), h, h + hs};
  by_type(hidden_type, [&](auto T) {
    hipLaunchKernelGGL((k_mx_quantize_tiles<T>), dim3((unsigned)(hs / 4096)), dim3(256), 0, stream, q);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const MxGemmArgs a{h, h + hs, head, head + ws, M, V, mx_padded(d) / 128, logits, type, ld,
                     vec_rows(logits, type, ld, 4), vec_rows(logits, type, ld, type == SD_F32 ? 4 : 8)};
  if (M <= 32) {
    auto *k = M <= 16 ? &k_mx_skinny<1> : &k_mx_skinny<2>;
    hipLaunchKernelGGL(k, dim3((V + 63) / 64), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  // The tiling whose rounds over the 256 CUs cost least. Costs are times of a round at
  // depth 7168 relative to 256 x 256 (61 us), from calls of many rounds; the 64-row and the
  // 128 x 128 tilings run two workgroups a CU, at half a round each; 64 rows are for calls
  // of no more, as every 64 rows would read the LM head again. Measured (us, ids x rows
  // of a tile 256 x 256 / 256 x 128 / 128 x 128 / 256 x 64), V x depth, M:
  //   129280 x 7168:  64: - / 95 / 97 / 91      128: 129 / 97 / 107 / -    300: 233 / 215 / 216 / -
  //                  512: 245 / 285 / 295 / -
  //    32000 x 4096: 128: 36 / 26 / 23 / -      256: 36 / 29 / 33 / -      512: 43 / 49 / 53 / -
  //   151936 x 4096:  64: - / 78 / 68 / 68      128: 113 / 81 / 76 / -     512: 197 / 218 / 214 / -
  const double cost[4] = {rounds(M, V, 256, 256), 0.58 * rounds(M, V, 256, 128), 0.32 * rounds(M, V, 128, 128),
                          0.33 * rounds(M, V, 256, 64)};
  int best = 0;
  for (int i = 1; i < (M <= 64 ? 4 : 3); ++i) if (cost[i] < cost[best]) best = i;
  if (best == 0) return launch_tiled<2, 2, 8, 8, 4>(a, stream);
  if (best == 1) return launch_tiled<2, 2, 8, 4, 4>(a, stream);
  if (best == 2) return launch_tiled<2, 2, 4, 4, 4>(a, stream);
  return launch_tiled<4, 1, 4, 4, 3>(a, stream);
}

}  // namespace sdv
