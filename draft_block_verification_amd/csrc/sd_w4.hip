// 4-bit integer weights with a scale per group of columns: quantisation and the values back
// (gfx950).
//
// A group of G (32, 64 or 128) consecutive columns of a row shares a 16-bit scale s and, in
// the asymmetric form, a zero z in 0 .. 15 (z = 8 in the symmetric form); a value is
// (c - z) s for its code c in 0 .. 15.
//   asymmetric  s = (max(x, 0) - min(x, 0)) / 15 rounded to fp32 and to its type,
//               z = -min(x, 0) / s rounded and held to 0 .. 15
//   symmetric   s = max |x| / 7 in fp32, rounded to its type
//   c = x / s rounded, plus z, held to 0 .. 15
// Quotients are rounded to fp32, then to the nearest integer, ties to even. A scale under the
// smallest normal fp32 number is 0 and its codes are z = 0 (8); a group that holds a NaN or an
// infinity, or whose scale passes its type, has a NaN scale.
#include "sd_launch.h"
#include "sd_rows.h"

namespace sdv {
namespace {

struct W4Args {
  const void *x;
  int64_t rows, stride;    // elements from row to row
  int d;
  bool vec, symmetric;
  int32_t scale_type;
  uint8_t *codes;          // [rows][d / 2]
  uint16_t *scales;        // [rows][d / G]
  uint8_t *zeros;          // [rows][d / G], null in the symmetric form
};

// The largest of eight values and of their negatives, 0 at least, as bits of the row's type: such
// numbers order as integers do, NaN and infinity on top.
struct Ends { uint32_t most, least; };

typedef short i16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ i16x2 max2(i16x2 a, i16x2 b) { return __builtin_elementwise_max(a, b); }

// Over the group: {most, least} as fp32 bits.
template <int T, int G>
__device__ __forceinline__ Ends group_ends(const Raw8<T> &r) {
  if constexpr (T == SD_F32) {
    int most = 0, least = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = __float_as_int(r.a[i]), b = __float_as_int(r.b[i]);
      most = max(most, max(a, b));
      least = max(least, max(a ^ INT32_MIN, b ^ INT32_MIN));
    }
    const auto larger = [](uint32_t p, uint32_t q) { return max(p, q); };
    return {over_group<G>(most, larger), over_group<G>(least, larger)};
  } else {
    i16x2 most = {0, 0}, least = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      most = max2(most, __builtin_bit_cast(i16x2, (uint32_t)r.w[i]));
      least = max2(least, __builtin_bit_cast(i16x2, (uint32_t)(r.w[i] ^ 0x80008000u)));
    }
    // most in the low half, least in the high one
    const uint32_t m = __builtin_bit_cast(uint32_t, most), l = __builtin_bit_cast(uint32_t, least);
    const i16x2 both = max2(__builtin_bit_cast(i16x2, (m & 0xffffu) | l << 16), __builtin_bit_cast(i16x2, m >> 16 | (l & 0xffff0000u)));
    const uint32_t e = over_group<G>(__builtin_bit_cast(uint32_t, both), [](uint32_t p, uint32_t q) {
      return __builtin_bit_cast(uint32_t, max2(__builtin_bit_cast(i16x2, p), __builtin_bit_cast(i16x2, q)));
    });
    if constexpr (T == SD_BF16) return {e << 16, e & 0xffff0000u};
    const f16x2 h = pair<f16x2>(e);
    return {__float_as_uint((float)h[0]), __float_as_uint((float)h[1])};
  }
}

// x / s rounded to nearest, r being near 1 / s: the quotient's error is taken from x by one fused
// operation (exactly but near the ends of fp32's range) and corrected by another, which leaves it
// 2^-44 off before it is rounded: quotients halfway between integers, fp32 numbers, come out exact.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

__device__ __forceinline__ float scale_value(uint16_t bits, int32_t type) {
  return type == SD_BF16 ? __uint_as_float((uint32_t)bits << 16) : (float)__builtin_bit_cast(_Float16, bits);
}

// An item is eight columns, G / 8 neighbouring threads hold a group; a thread takes U items 256
// apart, its loads issued together. 151936 x 4096 fp16 in groups of 32: 310 us (1.6 GB, 5.1 TB/s);
// 32768 x 2048 bf16 with zeros in groups of 128: 44 us in a row of calls (170 MB, 3.9 TB/s; some 13
// vector operations a column, the rounding of its quotient above all), 51 alone under the profiler.
template <int T, int U, int G>
__global__ __launch_bounds__(256) void k_w4_quantize(W4Args a) {
  const int per = a.d / 8;        // a multiple of G / 8: a group's items are all in or all out
  const int64_t base = (int64_t)blockIdx.x * 256 * U, row0 = base / per;
  const int c0 = (int)(base - row0 * per);
  Item it[U];
  Raw8<T> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    it[u] = item_at(row0, c0, threadIdx.x + 256 * u, per);
    raw[u] = Raw8<T>{};
    if (it[u].row < a.rows) raw[u] = load8<T>(a.x, it[u].row * a.stride + 8 * it[u].c, 8, a.vec);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    f32x4 lo, hi;
    widen8<T>(raw[u], lo, hi);
    const Ends ends = group_ends<T, G>(raw[u]);
    const uint32_t top = max(ends.most, ends.least);
    const float least = __uint_as_float(ends.least);
    float s;
    if (a.symmetric) {
      s = quotient(__uint_as_float(top), 7.f, 1.f / 7);
    } else {
      // The sum over 15, corrected as quotient() is.
      const double w = (double)__uint_as_float(ends.most) + (double)least, q = w * (1.0 / 15);
      s = (float)fma(fma(-15.0, q, w), 1.0 / 15, q);
    }
    const u32x2 packed = pack4(f32x4{s, s, s, s}, a.scale_type);
    uint16_t bits = (uint16_t)packed[0];
    s = scale_value(bits, a.scale_type);
    const bool bad = top >= 0x7f800000u || s > 3.4028234e38f, none = s < 1.17549435e-38f;
    if (bad) bits = a.scale_type == SD_BF16 ? 0x7fc0 : 0x7e00;
    else if (none) bits = 0;
    const float r = __builtin_amdgcn_rcpf(s);
    int z = a.symmetric ? 8 : (int)fminf(rintf(quotient(least, s, r)), 15.f);
    if (!a.symmetric && (bad || none)) z = 0;
    // A sum with 1.5 * 2^23 is rounded to an integer, which its low bits hold.
    constexpr float kInt = 12582912.f;
    const int off = z - __float_as_int(kInt);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = __float_as_int(quotient(i < 4 ? lo[i & 3] : hi[i & 3], s, r) + kInt) + off;
      word |= (uint32_t)min(max(c, 0), 15) << (4 * i);
    }
    if (bad || none) word = (uint32_t)z * 0x11111111u;
    const int64_t row = it[u].row;
    const int c = it[u].c;
    if (row >= a.rows) continue;
    *reinterpret_cast<uint32_t *>(a.codes + row * (a.d / 2) + 4 * c) = word;
    if (c % (G / 8) == 0) {
      const int64_t g = row * (a.d / G) + c / (G / 8);
      a.scales[g] = bits;
      if (!a.symmetric) a.zeros[g] = (uint8_t)z;
    }
  }
}

// x[row][8 c ..]: (code - zero) scale, exact in fp32, rounded once. 151936 x 4096 into bf16: 280 us
// (5.7 TB/s).
template <int T, int U, int G>
__global__ __launch_bounds__(256) void k_w4_dequantize(W4Args a, void *x) {
  const int per = a.d / 8;
  const int64_t base = (int64_t)blockIdx.x * 256 * U, row0 = base / per;
  const int c0 = (int)(base - row0 * per);
  Item it[U];
  uint32_t word[U];
  uint16_t s[U];
  uint8_t z[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    it[u] = item_at(row0, c0, threadIdx.x + 256 * u, per);
    if (it[u].row < a.rows) {
      const int64_t g = it[u].row * (a.d / G) + it[u].c / (G / 8);
      word[u] = *reinterpret_cast<const uint32_t *>(a.codes + it[u].row * (a.d / 2) + 4 * it[u].c);
      s[u] = a.scales[g];
      z[u] = a.symmetric ? 8 : a.zeros[g];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (it[u].row >= a.rows) continue;
    const float scale = scale_value(s[u], a.scale_type);
    f32x4 lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = (float)((int)(word[u] >> (4 * i) & 15) - z[u]) * scale;
      hi[i] = (float)((int)(word[u] >> (16 + 4 * i) & 15) - z[u]) * scale;
    }
    store8<T>(x, it[u].row * a.stride + 8 * it[u].c, 8, a.vec, lo, hi);
  }
}

template <class F>
hipError_t by_group(int group, F f) {
  if (group == 32) return f(std::integral_constant<int, 32>{});
  if (group == 64) return f(std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 128>{});
}

}  // namespace

hipError_t launch_w4_quantize(const void *x, int32_t type, int64_t rows, int d, int64_t stride, int group,
                              uint8_t *codes, uint16_t *scales, int32_t scale_type, uint8_t *zeros,
                              hipStream_t stream) {
  const W4Args a{x, rows, stride, d, vec_rows(x, type, stride, type == SD_F32 ? 4 : 8), zeros == nullptr,
                 scale_type, codes, scales, zeros};
  return by_group(group, [&](auto G) {
    return by_items(type, rows * (d / 8), [&](auto T, auto U, dim3 grid) {
      hipLaunchKernelGGL((k_w4_quantize<T, U, G>), grid, dim3(256), 0, stream, a);
    });
  });
}

hipError_t launch_w4_dequantize(const uint8_t *codes, const uint16_t *scales, int32_t scale_type,
                                const uint8_t *zeros, int64_t rows, int d, int group, void *x, int32_t type,
                                int64_t stride, hipStream_t stream) {
  const W4Args a{nullptr, rows, stride, d, vec_rows(x, type, stride, type == SD_F32 ? 4 : 8), zeros == nullptr,
                 scale_type, const_cast<uint8_t *>(codes), const_cast<uint16_t *>(scales),
                 const_cast<uint8_t *>(zeros)};
  return by_group(group, [&](auto G) {
    return by_items(type, rows * (d / 8), [&](auto T, auto U, dim3 grid) {
      hipLaunchKernelGGL((k_w4_dequantize<T, U, G>), grid, dim3(256), 0, stream, a, x);
    });
  });
}

}  // namespace sdv
