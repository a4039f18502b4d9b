// Microscaled 8-bit floating point (MXFP8, e4m3): quantisation and the values back (gfx950).
//
// Rows are stored padded to a multiple of 128 columns: codes [rows][kp] bytes, scales
// [rows][kp / 32] bytes; padding is code 0, whole blocks of it under scale byte 0.
#include "sd_launch.h"
#include "sd_mx8.h"

namespace sdv {
namespace {

struct Mx8Args {
  const void *x;
  int64_t rows, stride;    // elements from row to row
  int d, kp;
  bool vec;
  uint8_t *codes, *scales;
};

// An item is eight columns, four neighbouring threads hold a block. A thread takes U items 256
// apart, its loads issued together. Bound by memory: 129280 x 7168 bf16 in 513 us (2.81 GB, 5.5 TB/s),
// back in 450 us (6.2 TB/s).
template <int T, int U>
__global__ __launch_bounds__(256) void k_mx8_quantize(Mx8Args a) {
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
    const int byte = mx8_scale(block_top(top8<T>(r[u])));
    f32x4 lo, hi;
    widen8<T>(r[u], lo, hi);
    const u32x2 w = byte == 255 ? u32x2{0u, 0u} : mx8_codes(lo, hi, byte);
    if (it[u].row >= a.rows) continue;
    *reinterpret_cast<u32x2 *>(a.codes + it[u].row * a.kp + 8 * it[u].c) = w;
    if ((it[u].c & 3) == 0) a.scales[it[u].row * (a.kp / 32) + it[u].c / 4] = (uint8_t)byte;
  }
}

// x[row][8 c ..] from the codes; x is written to column d - 1.
template <int T, int U>
__global__ __launch_bounds__(256) void k_mx8_dequantize(Mx8Args a, void *x) {
  const int per = (a.d + 7) / 8;
  const int64_t base = (int64_t)blockIdx.x * 256 * U, row0 = base / per;
  const int c0 = (int)(base - row0 * per);
  Item it[U];
  u32x2 w[U];
  int s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    it[u] = item_at(row0, c0, threadIdx.x + 256 * u, per);
    if (it[u].row < a.rows) {
      w[u] = *reinterpret_cast<const u32x2 *>(a.codes + it[u].row * a.kp + 8 * it[u].c);
      s[u] = a.scales[it[u].row * (a.kp / 32) + it[u].c / 4];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (it[u].row >= a.rows) continue;
    f32x4 lo, hi;
    mx8_values(w[u], s[u], lo, hi);
    store8<T>(x, it[u].row * a.stride + 8 * it[u].c, a.d - 8 * it[u].c, a.vec, lo, hi);
  }
}

}  // namespace

hipError_t launch_mx8_quantize(const void *x, int32_t type, int64_t rows, int d, int64_t stride,
                               uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const Mx8Args a{x, rows, stride, d, mx_padded(d), vec_rows(x, type, stride, type == SD_F32 ? 4 : 8), codes, scales};
  return by_items(type, rows * (a.kp / 8), [&](auto T, auto U, dim3 grid) {
    hipLaunchKernelGGL((k_mx8_quantize<T, U>), grid, dim3(256), 0, stream, a);
  });
}

hipError_t launch_mx8_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int d,
                                 void *x, int32_t type, int64_t stride, hipStream_t stream) {
  const Mx8Args a{nullptr, rows, stride, d, mx_padded(d), vec_rows(x, type, stride, type == SD_F32 ? 4 : 8),
                  const_cast<uint8_t *>(codes), const_cast<uint8_t *>(scales)};
  return by_items(type, rows * ((d + 7) / 8), [&](auto T, auto U, dim3 grid) {
    hipLaunchKernelGGL((k_mx8_dequantize<T, U>), grid, dim3(256), 0, stream, a, x);
  });
}

}  // namespace sdv
