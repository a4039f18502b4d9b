// Logits of hidden rows under LM heads of 8-bit (MXFP8) and 4-bit (integer, group scales)
// weights (gfx950).
//
// Both run on the 16-bit matrix instructions: an e4m3 value under its block's scale and a code
// 0 .. 15 are bf16 numbers (the latter fp16 numbers too), products of bf16 or fp16 numbers are
// exact in fp32, and these instructions add in fp32. The 8-bit instructions do not: they align
// the products of a block and cut them, and sums of 4096 terms come out 1.4e-5 off (relative,
// normal data) where the 16-bit ones are 9e-8 off.
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

__device__ __forceinline__ float wide_scale(uint32_t bits, bool f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)bits) : __uint_as_float(bits << 16);
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
struct Mx8 {
  template <int TV, int MT>
  struct Step {
    u32x4 w[TV][2];
    uint32_t s[TV / 4][2];
    u32x4 h[MT][2];
    uint32_t hs[MT];
  };
  template <int TV, int MT>
  static __device__ __forceinline__ void load(const NarrowArgs &a, int64_t group, int row0, int k, int lane,
                                              Step<TV, MT> &st) {
    const int q = lane >> 4;
#pragma unroll
    for (int i = 0; i < TV; ++i) {
      const int64_t tile = min(group + i / 4, (int64_t)(a.V - 1) / 64) * a.steps + k;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        st.w[i][h] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4 *>(a.codes + tile * kMx8Tile + (i % 4) * 2048 + h * 1024) + lane);
      if (i % 4 == 0) {
        const uint32_t *s = reinterpret_cast<const uint32_t *>(a.scales + tile * kMx8Scales) + (lane & 15);
#pragma unroll
        for (int h = 0; h < 2; ++h) st.s[i / 4][h] = __builtin_nontemporal_load(s + 16 * (2 * h + q / 2));
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = min(row0 + 16 * m + (lane & 15), a.M - 1);
      const uint8_t *p = reinterpret_cast<const uint8_t *>(a.hidden) + row * a.hstride + 128 * k + 16 * q;
      st.h[m][0] = *reinterpret_cast<const u32x4 *>(p);
      st.h[m][1] = *reinterpret_cast<const u32x4 *>(p + 64);
      st.hs[m] = *reinterpret_cast<const uint32_t *>(a.hscales + row * (a.hstride / 32) + 4 * k);
    }
  }
  template <int TV, int MT>
  static __device__ __forceinline__ void use(const NarrowArgs &a, const Step<TV, MT> &st, int lane, f32x4 (&acc)[TV][MT]) {
    const int q = lane >> 4;
    u32x4 h[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t byte = st.hs[m] >> (8 * (t / 2 * 2 + q / 2)) & 255;
        const uint32_t nan = byte == 255 ? ~0u : 0u;
        h[m][t] = decode8(st.h[m][t / 2][t % 2 * 2] | nan, st.h[m][t / 2][t % 2 * 2 + 1] | nan,
                          __uint_as_float(min(byte, 254u) << 23));
      }
#pragma unroll
    for (int i = 0; i < TV; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const u32x4 w = decode8(st.w[i][t / 2][t % 2 * 2], st.w[i][t / 2][t % 2 * 2 + 1],
                                byte_scale(st.s[i / 4][t / 2], i % 4));
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = mfma16<SD_BF16>(h[m][t], w, acc[i][m]);
      }
  }
};

// 4-bit codes of NG groups a step, hidden rows in 16 bits as they are. Of each group the sum of
// code products c h and the sum of the h (a product with ones) are formed in fp32, and
// s (sum c h - z sum h) is added to the logit: no weight is rounded.
template <int H, int NG, bool ASYM>
struct W4 {
  template <int TV, int MT>
  struct Step {
    u32x4 w[TV];
    u32x2 s[TV / 4][NG];
    uint32_t z[TV / 4][NG];
    u32x4 h[MT][4];
  };
  template <int TV, int MT>
  static __device__ __forceinline__ void load(const NarrowArgs &a, int64_t group, int row0, int k, int lane,
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
      const int64_t row = min(row0 + 16 * m + (lane & 15), a.M - 1);
      const uint16_t *p = reinterpret_cast<const uint16_t *>(a.hidden) + row * a.hstride + 128 * k + 8 * (lane >> 4);
#pragma unroll
      for (int t = 0; t < 4; ++t) st.h[m][t] = *reinterpret_cast<const u32x4 *>(p + 32 * t);
    }
  }
  template <int TV, int MT>
  static __device__ __forceinline__ void use(const NarrowArgs &a, const Step<TV, MT> &st, int lane, f32x4 (&acc)[TV][MT]) {
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
      }
#pragma unroll
      for (int i = 0; i < TV; ++i) {
        f32x4 part[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) part[m] = zero4;
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          const u32x4 w = decode4<H>(st.w[i][g * KS + t]);
#pragma unroll
          for (int m = 0; m < MT; ++m) part[m] = mfma16<H>(st.h[m][g * KS + t], w, part[m]);
        }
        const float s = wide_scale(st.s[i / 4][g][i % 4 / 2] >> (16 * (i % 2)) & 0xffff, a.scale_f16);
        const float z = ASYM ? (float)(st.z[i / 4][g] >> (8 * (i % 4)) & 255) : 8.f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][m][e] = fmaf(s, fmaf(-z, sum[m][e], part[m][e]), acc[i][m][e]);
      }
    }
  }
};

// ---------------------------------------------------------------- few hidden rows
// Up to 16 MT rows (and more by blockIdx.y): the LM head's bytes bound the call. One workgroup
// per 16 TV ids; its NW waves take the 128-column steps in turn, straight into registers: each
// weight is used by one wave only, so LDS would add a copy and share nothing. The hidden rows are
// read by every workgroup and come from L2. The waves' partial sums meet in LDS in wave order.
template <class F, int TV, int MT, int NW, int D>
__global__ __launch_bounds__(64 * NW) void k_narrow_skinny(NarrowArgs a) {
  constexpr int IDS = 16 * TV, LDR = IDS + 4;
  __shared__ float red[NW][16 * MT * LDR];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t group = (int64_t)blockIdx.x * (TV / 4);
  const int row0 = 16 * MT * blockIdx.y;
  f32x4 acc[TV][MT];
#pragma unroll
  for (int i = 0; i < TV; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  typename F::template Step<TV, MT> st[D];
#pragma unroll
  for (int x = 0; x < D; ++x) F::template load<TV, MT>(a, group, row0, min(wave + NW * x, a.steps - 1), lane, st[x]);
  for (int k = wave; k < a.steps; k += NW * D) {
#pragma unroll
    for (int x = 0; x < D; ++x) {
      if (k + NW * x < a.steps) {
        F::template use<TV, MT>(a, st[x], lane, acc);
        // past the end: the last step again, unused
        F::template load<TV, MT>(a, group, row0, min(k + NW * (x + D), a.steps - 1), lane, st[x]);
      }
    }
  }
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
    if (row0 + m >= a.M) break;
    f32x4 z = *reinterpret_cast<const f32x4 *>(&red[0][m * LDR + v]);
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const f32x4 o = *reinterpret_cast<const f32x4 *>(&red[w][m * LDR + v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] += o[e];
    }
    store4(a, row0 + m, IDS * (int)blockIdx.x + v, z);
  }
}

// ---------------------------------------------------------------- hidden rows made ready
// 16-bit rows copied to whole 128-column steps, zeros behind column d.
__global__ __launch_bounds__(256) void k_pad_rows(const uint16_t *x, int64_t rows, int64_t stride, int d, int kp,
                                                  bool vec, uint16_t *out) {
  const int per = kp / 8;
  const int64_t base = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256, row0 = base / per;
  const Item it = item_at(row0, (int)(base - row0 * per), threadIdx.x, per);
  if (it.row >= rows) return;
  const int left = d - 8 * it.c;
  u32x4 w = {0u, 0u, 0u, 0u};
  if (left > 0) w = load8<SD_BF16>(x, it.row * stride + 8 * it.c, left, vec).w;
  *reinterpret_cast<u32x4 *>(out + it.row * kp + 8 * it.c) = w;
}

template <class F, int TV, int NW, int D>
hipError_t launch_skinny(const NarrowArgs &a, hipStream_t stream) {
  const unsigned n = (unsigned)((a.V + 16 * TV - 1) / (16 * TV));
  if (a.M <= 16)
    hipLaunchKernelGGL((k_narrow_skinny<F, TV, 1, NW, D>), dim3(n), dim3(64 * NW), 0, stream, a);
  else
    hipLaunchKernelGGL((k_narrow_skinny<F, TV, 2, NW, D>), dim3(n, (a.M + 31) / 32), dim3(64 * NW), 0, stream, a);
  return hipGetLastError();
}

template <int H, int NG>
hipError_t launch_w4_of(const NarrowArgs &a, hipStream_t stream) {
  return a.zeros ? launch_skinny<W4<H, NG, true>, 8, 4, 2>(a, stream)
                 : launch_skinny<W4<H, NG, false>, 8, 4, 2>(a, stream);
}

template <int H>
hipError_t launch_w4_group(const NarrowArgs &a, int group, hipStream_t stream) {
  if (group == 128) return launch_w4_of<H, 1>(a, stream);
  if (group == 64) return launch_w4_of<H, 2>(a, stream);
  return launch_w4_of<H, 4>(a, stream);
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

size_t mx8_logits_workspace_bytes(int M, int d) {
  const size_t kp = mx_padded(d);
  return align_up(sizeof(WsHeader) + M * kp + M * (kp / 32), 256);
}

hipError_t launch_mx8_logits(const void *hidden, int32_t hidden_type, const uint8_t *hidden_scales, int M, int d,
                             int64_t stride, const uint8_t *head, int V, void *logits, int32_t type, int64_t ld,
                             void *workspace, hipStream_t stream) {
  const int kp = mx_padded(d);
  const uint8_t *h = reinterpret_cast<const uint8_t *>(hidden), *hs = hidden_scales;
  if (hidden_type != SD_MXFP8) {
    uint8_t *q = reinterpret_cast<uint8_t *>(workspace) + sizeof(WsHeader), *qs = q + (size_t)M * kp;
    const hipError_t e = launch_mx8_quantize(hidden, hidden_type, M, d, stride, q, qs, stream);
    if (e != hipSuccess) return e;
    h = q;
    hs = qs;
  }
  const NarrowArgs a{h, hs, kp, head, head + tiles_of(V, d) * kMx8Tile, nullptr, false, M, V, kp / 128, logits, type, ld,
                     vec_rows(logits, type, ld, 4), vec_rows(logits, type, ld, type == SD_F32 ? 4 : 8)};
  return launch_skinny<Mx8, 4, 4, 2>(a, stream);
}

size_t w4_logits_workspace_bytes(int M, int d) {
  return align_up(sizeof(WsHeader) + (size_t)M * mx_padded(d) * 2, 256);
}

hipError_t launch_w4_logits(const void *hidden, int32_t hidden_type, int M, int d, int64_t stride,
                            const uint8_t *head, int V, int group, int32_t scale_type, bool zeros, void *logits,
                            int32_t type, int64_t ld, void *workspace, hipStream_t stream) {
  const int kp = mx_padded(d);
  const int64_t n = tiles_of(V, d);
  const bool vec = vec_rows(hidden, hidden_type, stride, 8);
  if (!vec || kp != d) {
    uint16_t *copy = reinterpret_cast<uint16_t *>(reinterpret_cast<uint8_t *>(workspace) + sizeof(WsHeader));
    const int64_t n = ((int64_t)M * (kp / 8) + 255) / 256, x = n < 1 << 20 ? n : 1 << 20;
    hipLaunchKernelGGL(k_pad_rows, dim3((unsigned)x, (unsigned)((n + x - 1) / x)), dim3(256), 0, stream,
                       reinterpret_cast<const uint16_t *>(hidden), (int64_t)M, stride, d, kp, vec, copy);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hidden = copy;
    stride = kp;
  }
  const uint8_t *s = head + n * kW4Tile;
  const NarrowArgs a{hidden, nullptr, stride, head, s, zeros ? s + n * (128 / group) * 128 : nullptr,
                     scale_type == SD_F16, M, V, kp / 128,
                     logits, type, ld, vec_rows(logits, type, ld, 4), vec_rows(logits, type, ld, type == SD_F32 ? 4 : 8)};
  return hidden_type == SD_BF16 ? launch_w4_group<SD_BF16>(a, group, stream) : launch_w4_group<SD_F16>(a, group, stream);
}

}  // namespace sdv
