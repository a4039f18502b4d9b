// Logits of hidden rows under LM heads of 8-bit (MXFP8) and 4-bit (integer, group scales)
// weights (gfx950).
//
// Both run on the 16-bit matrix instructions: an e4m3 value under its block's scale and a code
// 0 .. 15 are bf16 numbers (the latter fp16 numbers too), products of bf16 or fp16 numbers are
// exact in fp32, and these instructions add in fp32: 4096 terms of normal data come out 9e-8 off
// (relative). The 8-bit instructions have twice the rate and are not used: they cut the products of
// eight columns to 13 bits under the largest before they add them, 1.4e-5 on normal data but whole
// logits where large products cancel (224 and -224 in turn beside products of 0.012).
//
// Weights are re-laid once into tiles of 64 rows by 128 columns, each four fragments of 16 rows
// in the order the matrix instruction takes them: lane l holds row l % 16, q = l / 16, and of the
// four instructions (t) a fragment feeds eight columns each.
//   MXFP8  columns 64 (t / 2) + 16 q + 8 (t % 2) .. + 7: the bytes of t = 0, 1 are 16 columns of
//          one block, and so are those of t = 2, 3
//          codes  [ceil(V / 64)][kp / 128][4 fragments][2 halves][64 lanes][16 bytes]
//          scales [ceil(V / 64)][kp / 128][4 blocks][16 rows][4 fragments] bytes
//          a block that reads as NaN has NaN codes and scale 1
//   4 bits columns 32 t + 8 q .. + 7, so that an instruction's 32 columns lie in one group
//          codes  [ceil(V / 64)][kp / 128][4 fragments][64 lanes][4 words]; nibble 2 b of a word is
//                 column b of its eight, nibble 2 b + 1 column b + 4
//          scales [ceil(V / 64)][kp / 128][128 / G groups][16 rows][4 fragments] of 16 bits
//          zeros  the same in bytes (asymmetric form)
#include "sd_launch.h"
#include "sd_mx8.h"

namespace sdv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kMx8Tile = 8192, kMx8Scales = 256, kW4Tile = 4096;

// ---------------------------------------------------------------- LM heads, re-laid
// 129280 x 7168: 560 us (1.9 GB, 3.4 TB/s), once per model load.
__global__ __launch_bounds__(256) void k_mx8_head(const uint8_t *codes, const uint8_t *scales, int V, int kp,
                                                  uint8_t *out, uint8_t *out_scales) {
  const int steps = kp / 128, lane = threadIdx.x & 63, frag = threadIdx.x >> 6;
  const int64_t tile = blockIdx.x;
  const int64_t group = tile / steps;
  const int step = (int)(tile - group * steps), q = lane >> 4;
  const int64_t row = 64 * group + 16 * frag + (lane & 15);
  uint8_t s = 0;
  if (row < V) s = scales[row * (kp / 32) + 4 * step + q];
  out_scales[tile * kMx8Scales + lane * 4 + frag] = s == 255 ? 127 : s;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x4 w = {0u, 0u, 0u, 0u};
    if (row < V) {
      w = *reinterpret_cast<const u32x4 *>(codes + row * kp + 128 * step + 64 * h + 16 * q);
      if (scales[row * (kp / 32) + 4 * step + 2 * h + q / 2] == 255) w = u32x4{~0u, ~0u, ~0u, ~0u};
    }
    *reinterpret_cast<u32x4 *>(out + tile * kMx8Tile + frag * 2048 + h * 1024 + lane * 16) = w;
  }
}

// Eight nibbles in column order to the order above.
__device__ __forceinline__ uint32_t interleave(uint32_t w) {
  uint32_t r = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) r |= (w >> (4 * b) & 15) << (8 * b) | (w >> (4 * b + 16) & 15) << (8 * b + 4);
  return r;
}

// 129280 x 7168 with zeros in groups of 128: 390 us (1.0 GB, 2.5 TB/s), once per model load.
__global__ __launch_bounds__(256) void k_w4_head(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                                                 int V, int d, int group, int steps, uint8_t *out,
                                                 uint16_t *out_scales, uint8_t *out_zeros) {
  const int lane = threadIdx.x & 63, frag = threadIdx.x >> 6, q = lane >> 4, groups = 128 / group;
  const int64_t tile = blockIdx.x;
  const int64_t block = tile / steps;
  const int step = (int)(tile - block * steps);
  const int64_t row = 64 * block + 16 * frag + (lane & 15);
  u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int col = 128 * step + 32 * t + 8 * q;
    if (row < V && col < d) w[t] = interleave(*reinterpret_cast<const uint32_t *>(codes + row * (d / 2) + col / 2));
  }
  *reinterpret_cast<u32x4 *>(out + tile * kW4Tile + frag * 1024 + lane * 16) = w;
  const int g = 128 / group * step + q;
  if (q < groups) {
    const bool in = row < V && g < d / group;
    const int64_t at = (tile * groups + q) * 64 + (lane & 15) * 4 + frag;
    out_scales[at] = in ? scales[row * (d / group) + g] : 0;
    if (zeros) out_zeros[at] = in ? zeros[row * (d / group) + g] : 0;
  }
}

// ---------------------------------------------------------------- formats and hidden rows
// 16-bit types of the hidden rows in the matrix instructions, D += A B^T over 32 columns: lane l
// holds eight columns of row l % 16 of A and of B, of D the row 4 (l / 16) + e of A and row
// l % 16 of B. Hidden rows are A.
template <int H>
__device__ __forceinline__ f32x4 mfma16(const u32x4 &a, const u32x4 &b, const f32x4 &c) {
  if constexpr (H == SD_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two e4m3 bytes (SEL: which half of w) times a power of two, as 16-bit numbers.
template <int H, int SEL>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, float scale) {
  if constexpr (H == SD_F16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, SEL));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, SEL));
}

__device__ __forceinline__ u32x4 decode8(uint32_t w0, uint32_t w1, float scale) {
  return u32x4{e4m3_pair<SD_BF16, 0>(w0, scale), e4m3_pair<SD_BF16, 1>(w0, scale),
               e4m3_pair<SD_BF16, 0>(w1, scale), e4m3_pair<SD_BF16, 1>(w1, scale)};
}

// Codes 0 .. 15 of eight columns: as e4m3 bytes 0 .. 15 they are 0 .. 15 times 2^-9 (subnormals
// and the first normal binade), so the conversion under a scale of 2^9 gives the codes.
template <int H>
__device__ __forceinline__ u32x4 decode4(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = w >> 4 & 0x0f0f0f0fu;
  return u32x4{e4m3_pair<H, 0>(lo, 512.f), e4m3_pair<H, 1>(lo, 512.f), e4m3_pair<H, 0>(hi, 512.f),
               e4m3_pair<H, 1>(hi, 512.f)};
}

__device__ __forceinline__ float byte_scale(uint32_t word, int i) {
  return __uint_as_float((word >> (8 * i) & 255) << 23);
}

// A half of a word as a scale in fp16 (F16) or bf16.
template <bool F16>
__device__ __forceinline__ float wide_scale(uint32_t word, int half) {
  if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)(word >> (16 * half)));
  return __uint_as_float(half ? word & 0xffff0000u : word << 16);
}

struct NarrowArgs {
  const void *hidden;       // 16-bit rows, or MXFP8 codes [M][kp]
  const uint8_t *hscales;   // MXFP8: [M][kp / 32]
  int64_t hstride;          // elements from row to row
  const uint8_t *codes;     // LM head, tiled
  const uint8_t *scales;
  const uint8_t *zeros;
  bool scale_f16;           // scales of the 4-bit form in fp16, else bf16
  int M, V, steps;          // steps: 128-column steps
  void *out;
  int32_t type;
  int64_t ld;
  bool vec, wide;           // four-element and 16-byte stores allowed
  const float *sums;        // tiled kernel, 4-bit form: see k_w4_rows
};

__device__ inline void store4(const NarrowArgs &a, int m, int v, const f32x4 &z) {
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
#pragma unroll
      for (int i = 0; i < 4; ++i) if (v + i < a.V) p[i] = (uint16_t)(h[i / 2] >> (16 * (i & 1)));
    }
  }
}

// One step's weights of 64 G ids and their use. `Hid` is what a step of the hidden rows is.
//
// MXFP8 x MXFP8: each weight and hidden value is decoded under its scale into bf16.
template <int TV>
struct Mx8Step {
  u32x4 w[TV][2];
  uint32_t s[TV / 4][2];
  __device__ __forceinline__ void load(const NarrowArgs &a, int64_t group, int k, int lane) {
#pragma unroll
    for (int i = 0; i < TV; ++i) {
      const int64_t tile = min(group + i / 4, (int64_t)(a.V - 1) / 64) * a.steps + k;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[i][h] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4 *>(a.codes + tile * kMx8Tile + (i % 4) * 2048 + h * 1024) + lane);
      if (i % 4 == 0) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(a.scales + tile * kMx8Scales) + (lane & 15);
#pragma unroll
        for (int h = 0; h < 2; ++h) s[i / 4][h] = __builtin_nontemporal_load(p + 16 * (2 * h + (lane >> 5)));
      }
    }
  }
  template <int MT>
  __device__ __forceinline__ void use(const u32x4 (&h)[MT][4], f32x4 (&acc)[TV][MT]) const {
#pragma unroll
    for (int i = 0; i < TV; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const u32x4 x = decode8(w[i][t / 2][t % 2 * 2], w[i][t / 2][t % 2 * 2 + 1], byte_scale(s[i / 4][t / 2], i % 4));
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = mfma16<SD_BF16>(h[m][t], x, acc[i][m]);
      }
  }
};

// Eight codes under a scale byte in bf16; NaN under byte 255.
__device__ __forceinline__ u32x4 decode_row8(uint32_t w0, uint32_t w1, uint32_t byte) {
  const uint32_t nan = byte == 255 ? ~0u : 0u;
  return decode8(w0 | nan, w1 | nan, __uint_as_float(min(byte, 254u) << 23));
}

// Hidden rows in MXFP8 already.
struct Mx8 {
  template <int TV, int MT>
  struct Step : Mx8Step<TV> {
    u32x4 h[MT][2];
    uint32_t hs[MT];
  };
  template <int TV, int MT>
  static __device__ __forceinline__ void load(const NarrowArgs &a, int64_t group, int k, int lane,
                                              Step<TV, MT> &st) {
    st.Mx8Step<TV>::load(a, group, k, lane);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = min(16 * m + (lane & 15), a.M - 1);
      const uint8_t *p = reinterpret_cast<const uint8_t *>(a.hidden) + row * a.hstride + 128 * k + 16 * (lane >> 4);
      st.h[m][0] = *reinterpret_cast<const u32x4 *>(p);
      st.h[m][1] = *reinterpret_cast<const u32x4 *>(p + 64);
      st.hs[m] = *reinterpret_cast<const uint32_t *>(a.hscales + row * (a.hstride / 32) + 4 * k);
    }
  }
  template <int TV, int MT>
  static __device__ __forceinline__ void use(const Step<TV, MT> &st, int lane, f32x4 (&acc)[TV][MT]) {
    const int q = lane >> 4;
    u32x4 h[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        h[m][t] = decode_row8(st.h[m][t / 2][t % 2 * 2], st.h[m][t / 2][t % 2 * 2 + 1],
                              st.hs[m] >> (8 * (t / 2 * 2 + q / 2)) & 255);
    st.template use<MT>(h, acc);
  }
};

// Hidden rows of a 16-bit type T, quantised by every workgroup for itself: a block's 32 columns lie in
// this lane and the one 16 further or before. The codes are those of k_mx8_quantize.
template <int T>
struct Mx8Of {
  template <int TV, int MT>
  struct Step : Mx8Step<TV> {
    Raw8<T> x[MT][4];
  };
  template <int TV, int MT>
  static __device__ __forceinline__ void load(const NarrowArgs &a, int64_t group, int k, int lane,
                                              Step<TV, MT> &st) {
    st.Mx8Step<TV>::load(a, group, k, lane);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = min(16 * m + (lane & 15), a.M - 1);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        st.x[m][t] = load8<T>(a.hidden, row * a.hstride + 128 * k + 64 * (t / 2) + 16 * (lane >> 4) + 8 * (t % 2), 8, true);
    }
  }
  template <int TV, int MT>
  static __device__ __forceinline__ void use(const Step<TV, MT> &st, int, f32x4 (&acc)[TV][MT]) {
    u32x4 h[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t top = max(top8<T>(st.x[m][2 * half]), top8<T>(st.x[m][2 * half + 1]));
        top = max(top, (uint32_t)__builtin_amdgcn_ds_swizzle((int)top, 0x401f));     // lane ^ 16
        const int byte = mx8_scale(top);
#pragma unroll
        for (int t = 2 * half; t < 2 * half + 2; ++t) {
          f32x4 lo, hi;
          widen8<T>(st.x[m][t], lo, hi);
          const u32x2 w = mx8_codes(lo, hi, min(byte, 246));     // of byte 255: unused
          h[m][t] = decode_row8(w[0], w[1], byte);
        }
      }
    st.template use<MT>(h, acc);
  }
};

// 4-bit codes of NG groups a step, hidden rows in 16 bits as they are. Of each group the sum of
// code products c h and the sum of the h (a product with ones) are formed in fp32, and
// s (sum c h - z sum h) is added to the logit: no weight is rounded. Where z is 8 throughout, the
// code products start from -8 sum h.
template <int H, int NG, bool ASYM, bool SF16>
struct W4 {
  template <int TV, int MT>
  struct Step {
    u32x4 w[TV];
    u32x2 s[TV / 4][NG];
    uint32_t z[TV / 4][NG];
    u32x4 h[MT][4];
  };
  template <int TV, int MT>
  static __device__ __forceinline__ void load(const NarrowArgs &a, int64_t group, int k, int lane,
                                              Step<TV, MT> &st) {
#pragma unroll
    for (int i = 0; i < TV; ++i) {
      const int64_t tile = min(group + i / 4, (int64_t)(a.V - 1) / 64) * a.steps + k;
      st.w[i] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4 *>(a.codes + tile * kW4Tile + (i % 4) * 1024) + lane);
      if (i % 4 == 0) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int64_t at = (tile * NG + g) * 16 + (lane & 15);
          st.s[i / 4][g] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(a.scales) + at);
          if (ASYM) st.z[i / 4][g] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(a.zeros) + at);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = min(16 * m + (lane & 15), a.M - 1);
      const uint16_t *p = reinterpret_cast<const uint16_t *>(a.hidden) + row * a.hstride + 128 * k + 8 * (lane >> 4);
#pragma unroll
      for (int t = 0; t < 4; ++t) st.h[m][t] = *reinterpret_cast<const u32x4 *>(p + 32 * t);
    }
  }
  template <int TV, int MT>
  static __device__ __forceinline__ void use(const Step<TV, MT> &st, int lane, f32x4 (&acc)[TV][MT]) {
    constexpr int KS = 4 / NG;
    const uint32_t one = H == SD_F16 ? 0x3c003c00u : 0x3f803f80u;
    const u32x4 ones = {one, one, one, one};
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4 sum[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sum[m] = zero4;
#pragma unroll
        for (int t = 0; t < KS; ++t) sum[m] = mfma16<H>(st.h[m][g * KS + t], ones, sum[m]);
        if (!ASYM)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[m][e] *= -8.f;
      }
#pragma unroll
      for (int i = 0; i < TV; ++i) {
        f32x4 part[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) part[m] = ASYM ? zero4 : sum[m];
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          const u32x4 w = decode4<H>(st.w[i][g * KS + t]);
#pragma unroll
          for (int m = 0; m < MT; ++m) part[m] = mfma16<H>(st.h[m][g * KS + t], w, part[m]);
        }
        const float s = wide_scale<SF16>(st.s[i / 4][g][i % 4 / 2], i % 2);
        const float z = ASYM ? (float)(st.z[i / 4][g] >> (8 * (i % 4)) & 255) : 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][m][e] = fmaf(s, ASYM ? fmaf(-z, sum[m][e], part[m][e]) : part[m][e], acc[i][m][e]);
      }
    }
  }
};

// ---------------------------------------------------------------- few hidden rows
// Up to 16 MT rows: the LM head's bytes bound the call. One workgroup
// per 16 TV ids; its NW waves take the 128-column steps in turn, straight into registers: each
// weight is used by one wave only, so LDS would add a copy and share nothing. The hidden rows are
// read by every workgroup and come from L2. The waves' partial sums meet in LDS in wave order.
// 129280 x 7168, us: MXFP8 under 1 row 142 (6.7 TB/s), 16 rows 149; 4 bits with zeros in groups of 128
// under 1 row 80 (6.0 TB/s), 16 rows 82; in groups of 64 under 16 rows 90, of 32 107, without zeros 90:
// scales and sums come back at every 32 columns, and the vector units bound it. Held to 128 registers,
// so that two workgroups of eight waves fit a compute unit, the last two took 115 and 144 us when they
// took 108 and 96 (spills). fp16 scales cost the same, but for 32 rows under zeros in groups of 64: that
// form spills 5 registers and takes 26 us at 32000 x 4096, with bf16 scales 20.
template <class F, int TV, int MT, int NW, int D>
__global__ __launch_bounds__(64 * NW, 2) void k_narrow_skinny(NarrowArgs a) {
  constexpr int IDS = 16 * TV, LDR = IDS + 4;
  __shared__ float red[NW][16 * MT * LDR];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t group = (int64_t)blockIdx.x * (TV / 4);
  f32x4 acc[TV][MT];
#pragma unroll
  for (int i = 0; i < TV; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  typename F::template Step<TV, MT> st[D];
  const int n = (a.steps - wave + NW - 1) / NW;       // steps of this wave; past its end the last one, unused
  auto load = [&](int j, typename F::template Step<TV, MT> &to) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    F::template load<TV, MT>(a, group, min(wave + NW * j, a.steps - 1), lane, to);
    __builtin_amdgcn_sched_barrier(0);       // whole sets of loads, in the order of their use
  };
#pragma unroll
  for (int x = 0; x < D; ++x) load(x, st[x]);
  int j = 0;
  for (; j + D <= n; j += D) {
#pragma unroll
    for (int x = 0; x < D; ++x) {
      F::template use<TV, MT>(st[x], lane, acc);
      load(j + x + D, st[x]);
    }
  }
#pragma unroll
  for (int x = 0; x + 1 < D; ++x)
    if (j + x < n) F::template use<TV, MT>(st[x], lane, acc);
  const int col = lane & 15, q = lane >> 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < TV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][(16 * m + 4 * q + e) * LDR + 16 * i + col] = acc[i][m][e];
  __syncthreads();
  for (int t = threadIdx.x; t < 16 * MT * IDS / 4; t += 64 * NW) {
    const int m = t / (IDS / 4), v = 4 * (t % (IDS / 4));
    if (m >= a.M) break;
    f32x4 z = *reinterpret_cast<const f32x4 *>(&red[0][m * LDR + v]);
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const f32x4 o = *reinterpret_cast<const f32x4 *>(&red[w][m * LDR + v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] += o[e];
    }
    store4(a, m, IDS * (int)blockIdx.x + v, z);
  }
}

// ---------------------------------------------------------------- many hidden rows
// What a wave of the tiled kernel keeps of one step's weights (a tile of 64 ids), and what it
// does with them and the hidden rows' fragments (frag(m, t)). chunk(): which 16 bytes of the 256 that
// a step takes of a hidden row instruction t reads for the lanes of q.
struct Mx8Tile {
  static constexpr int kSums = 0;
  u32x4 w[4][2];
  uint32_t s[2];
  __device__ __forceinline__ void load(const NarrowArgs &a, int64_t tile, int lane) {
    const u32x4 *c = reinterpret_cast<const u32x4 *>(a.codes + tile * kMx8Tile) + lane;
    const uint32_t *p = reinterpret_cast<const uint32_t *>(a.scales + tile * kMx8Scales) + (lane & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[i][h] = c[128 * i + 64 * h];
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h] = p[16 * (2 * h + (lane >> 5))];
  }
  // Reads every register that load() fills: the compiler waits for them here.
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(w[i][0]), "+v"(w[i][1]));
    asm volatile("" : "+v"(s[0]), "+v"(s[1]));
  }
  static __device__ __forceinline__ int chunk(int t, int q) { return 2 * q + (t & 1) + 8 * (t >> 1); }
  template <int TM, class Frag, class Sum>
  __device__ __forceinline__ void use(Frag frag, Sum, f32x4 (&acc)[4][TM]) const {
    u32x4 h[2][TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) h[0][m] = frag(m, 0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t < 3)
#pragma unroll
        for (int m = 0; m < TM; ++m) h[(t + 1) & 1][m] = frag(m, t + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4 x = decode8(w[i][t / 2][t % 2 * 2], w[i][t / 2][t % 2 * 2 + 1], byte_scale(s[t / 2], i));
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[i][m] = mfma16<SD_BF16>(h[t & 1][m], x, acc[i][m]);
      }
    }
  }
};

// The products of a group start from -zero times the row's sum over the group (sum(g, m): the
// four rows of fragment m, times -8 already in the symmetric form).
template <int H, int NG, bool ASYM, bool SF16>
struct W4Tile {
  static constexpr int kSums = NG;
  u32x4 w[4];
  u32x2 s[NG];
  uint32_t z[NG];
  __device__ __forceinline__ void load(const NarrowArgs &a, int64_t tile, int lane) {
    const u32x4 *c = reinterpret_cast<const u32x4 *>(a.codes + tile * kW4Tile) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = c[64 * i];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int64_t at = (tile * NG + g) * 16 + (lane & 15);
      s[g] = reinterpret_cast<const u32x2 *>(a.scales)[at];
      if (ASYM) z[g] = reinterpret_cast<const uint32_t *>(a.zeros)[at];
    }
  }
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(w[i]));
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      asm volatile("" : "+v"(s[g]));
      if (ASYM) asm volatile("" : "+v"(z[g]));
    }
  }
  static __device__ __forceinline__ int chunk(int t, int q) { return 4 * t + q; }
  template <int TM, class Frag, class Sum>
  __device__ __forceinline__ void use(Frag frag, Sum sum, f32x4 (&acc)[4][TM]) const {
    constexpr int KS = 4 / NG;
    u32x4 h[2][TM];
    f32x4 part[4][TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) h[0][m] = frag(m, 0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t < 3)
#pragma unroll
        for (int m = 0; m < TM; ++m) h[(t + 1) & 1][m] = frag(m, t + 1);
      const int g = t / KS;
      if (t % KS == 0) {
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          const f32x4 c = sum(g, m);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if constexpr (ASYM) {
              const float zero = (float)(z[g] >> (8 * i) & 255);
#pragma unroll
              for (int e = 0; e < 4; ++e) part[i][m][e] = zero * c[e];
            } else {
              part[i][m] = c;
            }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4 x = decode4<H>(w[i][t]);
#pragma unroll
        for (int m = 0; m < TM; ++m) part[i][m] = mfma16<H>(h[t & 1][m], x, part[i][m]);
      }
      if (t % KS == KS - 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float sc = wide_scale<SF16>(s[g][i / 2], i % 2);
#pragma unroll
          for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][m][e] = fmaf(sc, part[i][m][e], acc[i][m][e]);
        }
      }
    }
  }
};

// 16 or 4 bytes a lane from base + lane_at + at to LDS, lane after lane from dst on. Through a
// buffer descriptor: behind a direct load with plain addresses the compiler lets no other load be
// awaited alone.
__device__ __forceinline__ void to_lds16(const void *base, int lane_at, int at, LDSP uint8_t *dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, -1, 0x00020000),
                                           (LDSP void *)dst, 16, lane_at, at, 0, 0);
}
__device__ __forceinline__ void to_lds4(const void *base, int lane_at, int at, LDSP uint8_t *dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, -1, 0x00020000),
                                           (LDSP void *)dst, 4, lane_at, at, 0, 0);
}

// A workgroup of four waves computes 256 ids by 16 TM hidden rows, each wave 64 ids by all of
// them. A step's 128 columns of the hidden rows (and the rows' sums of its groups) come into one
// of three LDS buffers by direct loads, two steps ahead; chunk c of row r lies at place
// c ^ (r % 16), so that the 16 rows of a fragment are read without bank conflicts. Each weight is
// used by one wave alone: it comes from memory into that wave's registers, two steps ahead,
// and is decoded there. Every wave issues the same loads every step, past the end the last
// step's again: a step's weights are issued behind its hidden rows, so when the former have
// arrived the latter have, and behind the barrier those of all waves. Two workgroups a compute
// unit: one decodes and scales while the other multiplies.
//
// 512 rows by 129280 ids at depth 7168: 4 bits with zeros in groups of 128 920 us (1.03 PFLOP/s;
// 860 us: what torch.matmul takes for bf16 weights of that shape, with nothing to decode), without zeros
// 835 - 850, in groups of 64 1050, of 32 1335 - 1350. In copies of the kernel for timing, without the
// scaling of a group's sums 720 us, without the decoding too 670; without the weights' loads 840. Vector
// and matrix work hardly overlap, in whatever order they are written: the scales cost their own
// time. fp16 scales are within 3% of these, which are of bf16, but for zeros in groups of 64: that form
// spills 35 registers and takes 1600 us. MXFP8, 2048 rows: 3030 us (1.25 PFLOP/s).
template <class F, int TM>
__global__ __launch_bounds__(256, 2) void k_narrow_tiled(NarrowArgs a, int n_mt, int n_vt) {
  constexpr int NS = 3, ROWS = 16 * TM, STAGE = ROWS * 256 + F::kSums * 256;
  constexpr int LOADS = ROWS / 16;                 // of four rows, by each wave
  static_assert(ROWS <= 64, "a wave's load of a group's sums is 64 rows");
  __shared__ __attribute__((aligned(16))) uint8_t S[NS * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  // Tiles go to the XCDs (workgroup id mod 8) in contiguous runs with the hidden tile running
  // fastest: an XCD's workgroups share LM-head tiles and hidden tiles in its L2.
  const int nb = n_mt * n_vt, hb = blockIdx.x;
  const int per = nb / 8, rem = nb % 8, xcd = hb % 8, pos = hb / 8;
  const int logical = (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + pos;
  const int mt = logical % n_mt, vt = logical / n_mt;
  const int64_t row0 = (int64_t)mt * ROWS;
  const int64_t tile0 = min((int64_t)vt * 4 + wave, (int64_t)(a.V - 1) / 64) * a.steps;
  const uint8_t *rows = reinterpret_cast<const uint8_t *>(a.hidden) + row0 * a.hstride * 2;
  int src[LOADS];
#pragma unroll
  for (int n = 0; n < LOADS; ++n) {
    const int at = 4 * (wave * LOADS + n) + q;       // row of the tile
    src[n] = (int)(min((int64_t)at, a.M - 1 - row0) * a.hstride * 2) + ((r ^ (at & 15)) * 16);
  }
  const float *sums = a.sums + (int64_t)mt * a.steps * F::kSums * ROWS;
  auto issue = [&](int k) __attribute__((always_inline)) {
    LDSP uint8_t *dst = (LDSP uint8_t *)S + (k % NS) * STAGE;
    const int kk = min(k, a.steps - 1);
#pragma unroll
    for (int n = 0; n < LOADS; ++n)
      to_lds16(rows, src[n], kk * 256, dst + (wave * LOADS + n) * 1024);
    if constexpr (F::kSums > 0)
      to_lds4(sums, lane % ROWS * 4, (kk * F::kSums + wave % F::kSums) * ROWS * 4,
              dst + ROWS * 256 + (wave % F::kSums) * 256);
    asm volatile("" ::: "memory");
  };
  f32x4 acc[4][TM];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  F st[2];
  auto step = [&](int k, F &now) __attribute__((always_inline)) {
    now.arrived();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    raw_barrier();                     // and every wave has read step k - 1 out of LDS
    issue(k + NS - 1);
    const LDSP uint8_t *b = (const LDSP uint8_t *)S + (k % NS) * STAGE;
    auto frag = [&](int m, int t) __attribute__((always_inline)) {
      return *(const LDSP u32x4 *)(b + (16 * m + r) * 256 + ((F::chunk(t, q) ^ r) * 16));
    };
    auto sum = [&](int g, int m) __attribute__((always_inline)) {
      return *(const LDSP f32x4 *)(b + ROWS * 256 + (g * 64 + 16 * m + 4 * q) * 4);
    };
    now.template use<TM>(frag, sum, acc);
    now.load(a, tile0 + min(k + 2, a.steps - 1), lane);
  };
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    issue(k);
    st[k].load(a, tile0 + min(k, a.steps - 1), lane);
    asm volatile("" ::: "memory");
  }
  int k = 0;
  for (; k + 1 < a.steps; k += 2) {
    step(k, st[0]);
    step(k + 1, st[1]);
  }
  if (k < a.steps) step(k, st[0]);
  wait_loads<0>();                     // the trailing loads land before LDS is used again
  raw_barrier();
  // The results cross LDS so that stores run along the rows: a lane holds one id of four rows.
  const int64_t m0 = row0;
  const int v0 = vt * 256 + wave * 64;
  constexpr int PART = NS * STAGE / 4 / 16 * 16;
  LDSP uint8_t *part = (LDSP uint8_t *)S + wave * PART;
  if (a.type == SD_F32) {
    constexpr int ROW = 64 * 4 + 16;
    static_assert(ROW * ROWS / 2 <= PART, "half the rows in fp32");
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int m = 0; m < TM / 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *(LDSP float *)(part + (16 * m + 4 * q + e) * ROW + (16 * i + r) * 4) = acc[i][half * TM / 2 + m][e];
      store_rows<float, 64, ROW>(a, part, m0 + half * ROWS / 2, ROWS / 2, v0, lane);
    }
  } else {
    constexpr int ROW = 64 * 2 + 16;
    static_assert(ROW * ROWS <= PART, "the rows in 16 bits");
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x2 h = pack4(acc[i][m], a.type);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *(LDSP uint16_t *)(part + (16 * m + 4 * q + e) * ROW + (16 * i + r) * 2) = (uint16_t)(h[e / 2] >> (16 * (e & 1)));
      }
    store_rows<uint16_t, 64, ROW>(a, part, m0, ROWS, v0, lane);
  }
}

// ---------------------------------------------------------------- hidden rows made ready
// Whole 128-column steps of 16-bit rows, zeros behind column d (out null: not stored), and each
// group's sum of a row times `factor` (sums null: not formed): [ceil(rows / tile)][kp / G][tile],
// rows past the last left. An item is eight columns.
template <int H, int G>
__global__ __launch_bounds__(256) void k_w4_rows(const uint16_t *x, int64_t rows, int64_t stride, int d, int kp,
                                                 bool vec, uint16_t *out, float *sums, int tile, float factor) {
  const int per = kp / 8;
  const int64_t base = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256, row0 = base / per;
  const Item it = item_at(row0, (int)(base - row0 * per), threadIdx.x, per);
  const int left = it.row < rows ? d - 8 * it.c : 0;
  Raw8<H> raw{};
  if (left > 0) raw = load8<H>(x, it.row * stride + 8 * it.c, left, vec);
  if (out && it.row < rows) *reinterpret_cast<u32x4 *>(out + it.row * kp + 8 * it.c) = raw.w;
  if (!sums) return;
  f32x4 lo, hi;
  widen8<H>(raw, lo, hi);
  float s = ((lo[0] + lo[1]) + (lo[2] + lo[3])) + ((hi[0] + hi[1]) + (hi[2] + hi[3]));
  s = __uint_as_float(over_group<G>(__float_as_uint(s), [](uint32_t p, uint32_t q) {
    return __float_as_uint(__uint_as_float(p) + __uint_as_float(q));
  }));
  if (it.row < rows && it.c % (G / 8) == 0)
    sums[(it.row / tile * (kp / G) + it.c / (G / 8)) * tile + it.row % tile] = factor * s;
}

// Hidden rows of any type as the bf16 numbers of their MXFP8 form, [M][kp].
template <int T>
__global__ __launch_bounds__(256) void k_mx8_rows(const void *x, int64_t rows, int64_t stride, int d, int kp, bool vec,
                                                  uint16_t *out) {
  const int per = kp / 8;
  const int64_t base = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256, row0 = base / per;
  const Item it = item_at(row0, (int)(base - row0 * per), threadIdx.x, per);
  const int left = it.row < rows ? d - 8 * it.c : 0;
  Raw8<T> raw{};
  if (left > 0) raw = load8<T>(x, it.row * stride + 8 * it.c, left, vec);
  f32x4 lo, hi;
  widen8<T>(raw, lo, hi);
  const int byte = mx8_scale(block_top(top8<T>(raw)));
  const u32x2 w = byte == 255 ? u32x2{0u, 0u} : mx8_codes(lo, hi, byte);
  mx8_values(w, byte, lo, hi);
  if (it.row < rows) store8<SD_BF16>(out, it.row * kp + 8 * it.c, 8, true, lo, hi);
}

// The same from codes and scales.
__global__ __launch_bounds__(256) void k_mx8_decode(const uint8_t *codes, const uint8_t *scales, int64_t rows, int kp,
                                                    uint16_t *out) {
  const int64_t at = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x) * 8;
  if (at >= rows * kp) return;
  f32x4 lo, hi;
  mx8_values(*reinterpret_cast<const u32x2 *>(codes + at), scales[at / 32], lo, hi);
  store8<SD_BF16>(out, at, 8, true, lo, hi);
}

// A launch of n items of 256 threads a workgroup has under 2^32 threads along x.
dim3 item_groups(int64_t items) {
  const int64_t n = (items + 255) / 256, x = n < 1 << 20 ? n : 1 << 20;
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

// Rows that the streaming kernel takes: 16, and 32 of an LM head that gives the tiled kernels less
// than a workgroup of 256 ids for each compute unit. us, streaming / tiled of 32 rows, M = 32, at two
// depths each (with zeros; what a call's host side takes, some 8 us, is in the smallest):
//                      129280 x 7168, 2048          32000 x 7168, 2048         8000 x 7168, 2048
//   4 bits, G = 128:   130 / 115, 45 / 35           28 / 47, 11.6 / 18.4       19 / 45, 8.3 / 16.6
//   4 bits, G = 32:    156 / 146, 57 / 45           39 / 76, 15.0 / 25.6       21 / 75, 9.2 / 25.4
//   MXFP8, bf16:       179 / 164, 63 / 53           45 / 56, 17.6 / 16.2       21 / 40, 8.8 / 15.1
//   MXFP8, fp32:       195 / 168, 70 / 55           45 / 57, 17.9 / 16.4       21 / 40, 8.8 / 15.2
constexpr int kFewRows = 16;
bool few_rows(int M, int V) { return M <= kFewRows || (M <= 2 * kFewRows && V <= 256 * 256); }

// What the workgroups of 256 ids by `rows` rows cost that one of the 256 compute units gets: two at a
// time at `both` each, one alone at `one`.
double paired(const NarrowArgs &a, int rows, double one, double both) {
  const int64_t n = ((int64_t)a.V + 255) / 256 * (((int64_t)a.M + rows - 1) / rows), each = (n + 255) / 256;
  return (double)(each / 2) * 2 * both + (double)(each % 2) * one;
}

template <class F, int TV, int MT, int NW, int D>
hipError_t launch_skinny_of(const NarrowArgs &a, hipStream_t stream) {
  const unsigned n = (unsigned)((a.V + 16 * TV - 1) / (16 * TV));
  hipLaunchKernelGGL((k_narrow_skinny<F, TV, MT, NW, D>), dim3(n), dim3(64 * NW), 0, stream, a);
  return hipGetLastError();
}

template <class F, int TV, int NW, int D>
hipError_t launch_skinny(const NarrowArgs &a, hipStream_t stream) {
  return a.M <= 16 ? launch_skinny_of<F, TV, 1, NW, D>(a, stream) : launch_skinny_of<F, TV, 2, NW, D>(a, stream);
}

template <class F, int TM>
hipError_t launch_tiled(const NarrowArgs &a, hipStream_t stream) {
  const int n_mt = (a.M + 16 * TM - 1) / (16 * TM), n_vt = (a.V + 255) / 256;
  hipLaunchKernelGGL((k_narrow_tiled<F, TM>), dim3((unsigned)((int64_t)n_mt * n_vt)), dim3(256), 0, stream, a, n_mt, n_vt);
  return hipGetLastError();
}

// Rows of a tile of k_narrow_tiled by what the workgroups that a compute unit gets cost, in pairs of
// 64-row ones. us, 32 / 64 rows a tile, V x depth, M:
//   4 bits, G = 128
//   129280 x 7168:  64: 160 / 138    128: 292 / 254    512: 1068 / 908
//    32000 x 4096:  64: 31 / 43      128: 48 / 45      256: 81 / 72     512: 153 / 133
//     8000 x 2048:  64: 21 / 29      256: 22 / 30      512: 32 / 32
//   MXFP8, bf16 logits
//   129280 x 7168:  64: 224 / 173    128: 323 / 258    512: 985 / 788   2048: 3685 / 3027
//    32000 x 4096:  64: 31 / 37      128: 47 / 40      256: 79 / 64     512: 143 / 118
//     8000 x 2048:  64: 16.5 / 19.8  256: 19.5 / 21.1  512: 27 / 24     1024: 46 / 38
int tile_rows(const NarrowArgs &a) { return paired(a, 32, 0.92, 0.70) < paired(a, 64, 1.27, 1.0) ? 32 : 64; }

template <int H, int NG, bool ASYM, bool SF16>
hipError_t launch_w4_form(const NarrowArgs &a, hipStream_t stream) {
  if (!few_rows(a.M, a.V)) {
    using F = W4Tile<H, NG, ASYM, SF16>;
    return tile_rows(a) == 32 ? launch_tiled<F, 2>(a, stream) : launch_tiled<F, 4>(a, stream);
  }
  // 128 ids a workgroup share the hidden rows' loads; an LM head that gives few workgroups then is dealt
  // in 64s. G = 128, us, ids x waves x steps ahead 128 x 8 x 1 / 128 x 4 x 2 / 64 x 4 x 2, V x depth, M:
  //   129280 x 7168:  1: 81 / 81 / 80         16: 82 / 87 / 101
  //    32768 x 7168:  1: 21.3 / 21.8 / 20.9   16: 22.1 / 22.6 / 27.1  32: 28.6 / 29.0 / 40.9
  //    32768 x 2048:  1: 8.1 / 8.7 / 8.3      16: 8.8 / 9.1 / 10.5    32: 11.7 / 12.2 / 16.1
  //     8000 x 7168:  1: 16.4 / 16.2 / 10.1   16: 17.3 / 17.7 / 12.6  32: 23.6 / 24.2 / 19.2
  //     8000 x 2048:  1: 7.1 / 6.9 / 4.9      16: 7.5 / 7.9 / 5.9     32: 10.3 / 10.8 / 8.6
  using F = W4<H, NG, ASYM, SF16>;
  return a.V <= 128 * 128 ? launch_skinny<F, 4, 4, 2>(a, stream) : launch_skinny<F, 8, 8, 1>(a, stream);
}

template <int H, int NG>
hipError_t launch_w4_of(const NarrowArgs &a, hipStream_t stream) {
  if (a.zeros) return a.scale_f16 ? launch_w4_form<H, NG, true, true>(a, stream) : launch_w4_form<H, NG, true, false>(a, stream);
  return a.scale_f16 ? launch_w4_form<H, NG, false, true>(a, stream) : launch_w4_form<H, NG, false, false>(a, stream);
}

// The rows of a call made ready, its group sums among them where the tiled kernel runs, and the call.
template <int H, int G>
hipError_t launch_w4_group(NarrowArgs a, int d, uint16_t *copy, float *sums, hipStream_t stream) {
  const int kp = a.steps * 128;
  const bool vec = vec_rows(a.hidden, H, a.hstride, 8);
  // 64 rows of a tile are addressed by 32 bits
  if (vec && kp == d && a.hstride < 1 << 24) copy = nullptr;
  if (few_rows(a.M, a.V)) sums = nullptr;
  if (copy || sums) {
    hipLaunchKernelGGL((k_w4_rows<H, G>), item_groups((int64_t)a.M * (kp / 8)), dim3(256), 0, stream,
                       reinterpret_cast<const uint16_t *>(a.hidden), (int64_t)a.M, a.hstride, d, kp, vec, copy, sums,
                       tile_rows(a), a.zeros ? -1.f : -8.f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (copy) {
    a.hidden = copy;
    a.hstride = kp;
  }
  a.sums = sums;
  return launch_w4_of<H, 128 / G>(a, stream);
}

int64_t tiles_of(int64_t rows, int d) { return (rows + 63) / 64 * (mx_padded(d) / 128); }

}  // namespace

size_t mx8_head_bytes(int64_t V, int d) { return (size_t)tiles_of(V, d) * (kMx8Tile + kMx8Scales); }

hipError_t launch_mx8_head(const uint8_t *codes, const uint8_t *scales, int V, int d, uint8_t *head,
                           hipStream_t stream) {
  const int64_t n = tiles_of(V, d);
  hipLaunchKernelGGL(k_mx8_head, dim3((unsigned)n), dim3(256), 0, stream, codes, scales, V, mx_padded(d), head,
                     head + n * kMx8Tile);
  return hipGetLastError();
}

size_t w4_head_bytes(int64_t V, int d, int group, bool zeros) {
  return (size_t)tiles_of(V, d) * (kW4Tile + 128 / group * 64 * (zeros ? 3 : 2));
}

hipError_t launch_w4_head(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int V, int d,
                          int group, uint8_t *head, hipStream_t stream) {
  const int64_t n = tiles_of(V, d);
  uint8_t *s = head + n * kW4Tile;
  hipLaunchKernelGGL(k_w4_head, dim3((unsigned)n), dim3(256), 0, stream, codes, scales, zeros, V, d, group,
                     mx_padded(d) / 128, head, reinterpret_cast<uint16_t *>(s), s + n * (128 / group) * 128);
  return hipGetLastError();
}

// Codes and scales, or many rows in bf16.
size_t mx8_logits_workspace_bytes(int M, int d) {
  const size_t kp = mx_padded(d);
  return align_up(sizeof(WsHeader) + (M <= kFewRows ? M * kp + M * (kp / 32) : 2 * M * kp), 256);
}

hipError_t launch_mx8_logits(const void *hidden, int32_t hidden_type, const uint8_t *hidden_scales, int M, int d,
                             int64_t stride, const uint8_t *head, int V, void *logits, int32_t type, int64_t ld,
                             void *workspace, hipStream_t stream) {
  const int kp = mx_padded(d);
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace) + sizeof(WsHeader);
  NarrowArgs a{hidden, hidden_scales, kp, head, head + tiles_of(V, d) * kMx8Tile, nullptr, false, M, V, kp / 128,
               logits, type, ld, vec_rows(logits, type, ld, 4), vec_rows(logits, type, ld, type == SD_F32 ? 4 : 8),
               nullptr};
  const bool coded = hidden_type == SD_MXFP8;
  hipError_t e = hipSuccess;
  if (few_rows(M, V)) {
    // Whole 16-bit rows of one tile are quantised by each workgroup, not by a launch before: measured
    // (us, each workgroup / a launch before, 1 and 16 rows) 1000 x 1024: 4.2 / 5.3, 4.5 / 6.1;
    // 8000 x 2048: 6.6 / 8.0, 7.7 / 9.1; 32768 x 2048: 13.8 / 14.4, 15.4 / 16.2; but 129280 x 7168:
    // 142.5 / 142.2, 152.8 / 149.5, and 32768 x 2048 of fp32 rows 14.7 / 14.3, 19.3 / 16.0. Ids decide, not
    // the depth: 8000 x 7168 14.7 / 16.1, 17.7 / 19.2; 129280 x 2048 46.0 / 45.6, 53.6 / 51.2.
    if (M <= 16 && V <= 65536 && d == kp && hidden_type != SD_F32 && vec_rows(hidden, hidden_type, stride, 8) && !coded) {
      a.hstride = stride;
      return hidden_type == SD_BF16 ? launch_skinny_of<Mx8Of<SD_BF16>, 4, 1, 4, 2>(a, stream)
                                    : launch_skinny_of<Mx8Of<SD_F16>, 4, 1, 4, 2>(a, stream);
    }
    if (!coded) {
      uint8_t *scales = ws + (size_t)M * kp;
      e = launch_mx8_quantize(hidden, hidden_type, M, d, stride, ws, scales, stream);
      a.hidden = ws;
      a.hscales = scales;
    }
    if (e != hipSuccess) return e;
    return launch_skinny<Mx8, 4, 4, 2>(a, stream);
  }
  uint16_t *rows = reinterpret_cast<uint16_t *>(ws);
  const dim3 grid = item_groups((int64_t)M * (kp / 8));
  if (coded)
    hipLaunchKernelGGL(k_mx8_decode, grid, dim3(256), 0, stream, reinterpret_cast<const uint8_t *>(hidden), hidden_scales,
                       (int64_t)M, kp, rows);
  else
    by_type(hidden_type, [&](auto T) {
      hipLaunchKernelGGL((k_mx8_rows<T>), grid, dim3(256), 0, stream, hidden, (int64_t)M, stride, d, kp,
                         vec_rows(hidden, hidden_type, stride, hidden_type == SD_F32 ? 4 : 8), rows);
    });
  e = hipGetLastError();
  a.hidden = rows;
  return e != hipSuccess ? e : tile_rows(a) == 32 ? launch_tiled<Mx8Tile, 2>(a, stream)
                         : launch_tiled<Mx8Tile, 4>(a, stream);
}

// Where the group sums of many rows lie behind a copy of the rows.
size_t w4_sums_at(int M, int d) { return align_up(sizeof(WsHeader) + (size_t)M * mx_padded(d) * 2, 256); }

size_t w4_logits_workspace_bytes(int M, int d, int group) {
  const size_t at = w4_sums_at(M, d);
  return M <= kFewRows ? at : at + (size_t)((M + 63) / 64) * (mx_padded(d) / group) * 64 * 4;
}

hipError_t launch_w4_logits(const void *hidden, int32_t hidden_type, int M, int d, int64_t stride,
                            const uint8_t *head, int V, int group, int32_t scale_type, bool zeros, void *logits,
                            int32_t type, int64_t ld, void *workspace, hipStream_t stream) {
  const int64_t n = tiles_of(V, d);
  const uint8_t *s = head + n * kW4Tile;
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
  float *sums = reinterpret_cast<float *>(ws + w4_sums_at(M, d));
  uint16_t *copy = reinterpret_cast<uint16_t *>(ws + sizeof(WsHeader));
  const NarrowArgs a{hidden, nullptr, stride, head, s, zeros ? s + n * (128 / group) * 128 : nullptr,
                     scale_type == SD_F16, M, V, mx_padded(d) / 128, logits, type, ld, vec_rows(logits, type, ld, 4),
                     vec_rows(logits, type, ld, type == SD_F32 ? 4 : 8), nullptr};
  if (hidden_type == SD_BF16) {
    if (group == 128) return launch_w4_group<SD_BF16, 128>(a, d, copy, sums, stream);
    if (group == 64) return launch_w4_group<SD_BF16, 64>(a, d, copy, sums, stream);
    return launch_w4_group<SD_BF16, 32>(a, d, copy, sums, stream);
  }
  if (group == 128) return launch_w4_group<SD_F16, 128>(a, d, copy, sums, stream);
  if (group == 64) return launch_w4_group<SD_F16, 64>(a, d, copy, sums, stream);
  return launch_w4_group<SD_F16, 32>(a, d, copy, sums, stream);
}

}  // namespace sdv
