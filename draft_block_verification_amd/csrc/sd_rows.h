// Rows of the library's element types on the device, and launches over them: what the
// kernels of narrow rows and of the products with them share.
#pragma once

#include <type_traits>
#include <utility>

#include "sd_internal.h"

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

// Row and column group of item n: base (row, c) of the workgroup's first item, `per` a row.
struct Item { int64_t row; int c; };
__device__ __forceinline__ Item item_at(int64_t row0, int c0, int n, int per) {
  const unsigned at = c0 + n, q = at / (unsigned)per;
  return {row0 + q, (int)(at - q * per)};
}

// Rounded to nearest even, by the hardware's conversions.
__device__ inline u32x2 pack4(const f32x4 &z, int32_t type) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  return type == SD_BF16 ? __builtin_bit_cast(u32x2, __builtin_convertvector(z, bf16x4))
                         : __builtin_bit_cast(u32x2, __builtin_convertvector(z, f16x4));
}

// Eight values to a row of type T, rounded to nearest even; those past `left` are not written.
template <int T>
__device__ __forceinline__ void store8(void *x, int64_t at, int left, bool vec, const f32x4 &lo, const f32x4 &hi) {
  if constexpr (T == SD_F32) {
    float *p = reinterpret_cast<float *>(x) + at;
    if (vec && left >= 8) {
      *reinterpret_cast<f32x4 *>(p) = lo;
      *reinterpret_cast<f32x4 *>(p + 4) = hi;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) if (i < left) p[i] = i < 4 ? lo[i] : hi[i - 4];
    }
  } else {
    uint16_t *p = reinterpret_cast<uint16_t *>(x) + at;
    const u32x2 a = pack4(lo, T), b = pack4(hi, T);
    const u32x4 h = {a[0], a[1], b[0], b[1]};
    if (vec && left >= 8) {
      *reinterpret_cast<u32x4 *>(p) = h;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) if (i < left) p[i] = (uint16_t)(h[i / 2] >> (16 * (i & 1)));
    }
  }
}

// The eight values of a Raw8 in fp32.
template <int T>
__device__ __forceinline__ void widen8(const Raw8<T> &r, f32x4 &lo, f32x4 &hi) {
  if constexpr (T == SD_F32) {
    lo = r.a;
    hi = r.b;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x, y;
      if (T == SD_BF16) {
        x = __uint_as_float(r.w[i] << 16);
        y = __uint_as_float(r.w[i] & 0xffff0000u);
      } else {
        const f16x2 h = pair<f16x2>(r.w[i]);
        x = (float)h[0];
        y = (float)h[1];
      }
      if (i < 2) { lo[2 * i] = x; lo[2 * i + 1] = y; }
      else { hi[2 * i - 4] = x; hi[2 * i - 3] = y; }
    }
  }
}

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

// f over the G / 8 neighbouring threads of a group: quads, halves of 16 lanes, 16 lanes.
template <int G, class F>
__device__ __forceinline__ uint32_t over_group(uint32_t v, F f) {
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));                    // lane ^ 1
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));                    // lane ^ 2
  if (G >= 64) v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));      // 7 - lane of 8
  if (G >= 128) v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));     // 15 - lane of 16
  return v;
}

// n rows of W results of type T from a wave's part of LDS (rows ROW bytes apart) to rows m0 .. of
// the output at column v0: 16 bytes a lane along the rows where they are aligned and whole, else
// an element a lane.
template <class T, int W, int ROW, class Args>
__device__ __forceinline__ void store_rows(const Args &a, const LDSP uint8_t *part, int64_t m0, int n, int v0, int lane) {
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

bool vec_rows(const void *x, int32_t type, int64_t stride, int elems) {
  const int64_t size = type == SD_F32 ? 4 : 2, bytes = size * elems;
  return reinterpret_cast<uintptr_t>(x) % bytes == 0 && stride * size % bytes == 0;
}

}  // namespace
}  // namespace sdv
