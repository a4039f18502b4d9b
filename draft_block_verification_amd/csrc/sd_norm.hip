// Root-mean-square norm of rows, with the residual's addition before it and an output in the
// caller's type or as MXFP8 rows (gfx950).
//
//   s = x + r, rounded to r's type (x itself without a residual)
//   y = s / sqrt(mean(s^2) + eps) * (offset + w)
//
// A row belongs to NT threads of one workgroup, eight neighbouring columns (a chunk) a thread and turn,
// and stays in their registers between the sum of its squares and its output, so it is read
// once; rows past 32768 columns are read a second time. Squares and their sum, the root and the
// product are formed in fp64: the memory bounds the kernel (two conversions and three fp64
// operations a column against at least four bytes), and every output is then the
// formula's value rounded to fp32 and to the output type, also where an 8-bit code has its border
// within fp32's rounding of it. The sum's order is fixed. Rows that are not 16-byte aligned are read and
// written element by element: 2176 x 7168 bf16 with residual and sum 22 us, with x not aligned 30, at 7167
// columns with nothing aligned 63; 16000 x 2048 47, 65, at 2047 141.
#include "sd_launch.h"
#include "sd_mx8.h"

namespace sdv {
namespace {

constexpr int kNone = -1;     // no residual

struct NormLaunch : NormArgs {
  int chunks;                 // groups of eight columns, padding of an MXFP8 row counted in
  int kp;
  bool x_vec, r_vec, w_vec, sum_vec, y_vec;
};

// A launch has under 2^32 threads along x: workgroups past 2^20 go along y.
__device__ __forceinline__ int64_t row_group() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

dim3 groups_of(int64_t n) {
  const int64_t x = n < 1 << 20 ? n : 1 << 20;
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

// v plus the value of the lane that is CTRL's source, by a lane exchange inside rows of 16.
template <int CTRL>
__device__ __forceinline__ double add_lane(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  const u32x2 o = {(uint32_t)__builtin_amdgcn_mov_dpp((int)w[0], CTRL, 0xf, 0xf, true),
                   (uint32_t)__builtin_amdgcn_mov_dpp((int)w[1], CTRL, 0xf, 0xf, true)};
  return v + __builtin_bit_cast(double, o);
}

__device__ __forceinline__ double of_lane(double v, int lane) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)w[0], lane),
                                          (uint32_t)__builtin_amdgcn_readlane((int)w[1], lane)});
}

// Sum over the row's NT threads, in all of them; `part` holds a wave's sum each.
template <int NT>
__device__ __forceinline__ double row_sum(double v, double *part) {
  v = add_lane<0xb1>(v);        // lane ^ 1
  v = add_lane<0x4e>(v);        // lane ^ 2
  v = add_lane<0x141>(v);       // 7 - lane of 8: the other four
  v = add_lane<0x140>(v);       // 15 - lane of 16: the other eight
  v = (of_lane(v, 0) + of_lane(v, 16)) + (of_lane(v, 32) + of_lane(v, 48));
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += part[i];
  }
  return v;
}

template <int T>
__device__ __forceinline__ void round8(f32x4 &lo, f32x4 &hi) {
  if constexpr (T != SD_F32) {
    const u32x2 a = pack4(lo, T), b = pack4(hi, T);
    const Raw8<T> r{{a[0], a[1], b[0], b[1]}};
    widen8<T>(r, lo, hi);
  }
}

// The weight's eight values plus the offset.
__device__ __forceinline__ void weight8(const NormLaunch &a, int col, int left, double *f) {
  f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
  if (a.w_type == SD_F32) widen8<SD_F32>(load8<SD_F32>(a.w, col, left, a.w_vec), lo, hi);
  else if (a.w_type == SD_BF16) widen8<SD_BF16>(load8<SD_BF16>(a.w, col, left, a.w_vec), lo, hi);
  else widen8<SD_F16>(load8<SD_F16>(a.w, col, left, a.w_vec), lo, hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = (double)lo[i] + (double)a.offset;
    f[4 + i] = (double)hi[i] + (double)a.offset;
  }
}

// Output of eight columns of a row from s and the row's factor.
__device__ __forceinline__ void put8(const NormLaunch &a, int64_t row, int c, double inv, f32x4 lo, f32x4 hi) {
  const int col = 8 * c, left = a.d - col;
  double f[8];
  if (a.w && left > 0) {
    weight8(a, col, left, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.0;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = (float)((double)lo[i] * inv * f[i]);
    hi[i] = (float)((double)hi[i] * inv * f[4 + i]);
  }
  if (a.codes) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= left) lo[i] = 0.f;          // padding, also in a row whose factor is not finite
      if (4 + i >= left) hi[i] = 0.f;
      top = max(top, max(__float_as_uint(lo[i]) & 0x7fffffffu, __float_as_uint(hi[i]) & 0x7fffffffu));
    }
    const int byte = mx8_scale(block_top(top));
    const u32x2 w = byte == 255 ? u32x2{0u, 0u} : mx8_codes(lo, hi, byte);
    *reinterpret_cast<u32x2 *>(a.codes + row * a.kp + col) = w;
    if ((c & 3) == 0) a.scales[row * (a.kp / 32) + c / 4] = (uint8_t)byte;
  } else if (left > 0) {
    const int64_t at = row * a.y_stride + col;
    if (a.y_type == SD_F32) store8<SD_F32>(a.y, at, left, a.y_vec, lo, hi);
    else if (a.y_type == SD_BF16) store8<SD_BF16>(a.y, at, left, a.y_vec, lo, hi);
    else store8<SD_F16>(a.y, at, left, a.y_vec, lo, hi);
  }
}

// s of eight columns; the sum is stored where it is wanted.
template <int XT, int RT>
__device__ __forceinline__ void sum8(const NormLaunch &a, int64_t row, int col, int left, const Raw8<XT> &x,
                                     const Raw8<RT == kNone ? XT : RT> &r, f32x4 &lo, f32x4 &hi) {
  widen8<XT>(x, lo, hi);
  if constexpr (RT != kNone) {
    f32x4 rl, rh;
    widen8<RT>(r, rl, rh);
#pragma unroll
    for (int i = 0; i < 4; ++i) { lo[i] += rl[i]; hi[i] += rh[i]; }
    round8<RT>(lo, hi);
    if (a.sum && left > 0) store8<RT>(a.sum, row * a.sum_stride + col, left, a.sum_vec, lo, hi);
  }
}

__device__ __forceinline__ double squares(const f32x4 &lo, const f32x4 &hi, double t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t = fma((double)lo[i], (double)lo[i], t);
    t = fma((double)hi[i], (double)hi[i], t);
  }
  return t;
}

// Rows of up to 8 NT U columns. Blocks of four threads that share an MXFP8 block are whole:
// chunks are a multiple of 16 then.
template <int XT, int RT, int NT, int U>
__global__ __launch_bounds__(NT < 128 ? 256 : NT) void k_norm(NormLaunch a) {
  constexpr int PER = NT < 128 ? 256 / NT : 1;       // rows a workgroup
  constexpr int RR = RT == kNone ? XT : RT;
  __shared__ double part[NT / 64];
  const int t = threadIdx.x % NT;
  const int64_t row = row_group() * PER + threadIdx.x / NT;
  if (row >= a.rows) return;                         // whole waves, and all that share a row
  Raw8<XT> x[U];
  Raw8<RR> r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int col = 8 * (t + u * NT), left = a.d - col;
    x[u] = Raw8<XT>{};
    r[u] = Raw8<RR>{};
    if (left > 0) {
      x[u] = load8<XT>(a.x, row * a.x_stride + col, left, a.x_vec);
      if constexpr (RT != kNone) r[u] = load8<RR>(a.r, row * a.r_stride + col, left, a.r_vec);
    }
  }
  f32x4 lo[U], hi[U];
  double sum = 0.0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int col = 8 * (t + u * NT);
    sum8<XT, RT>(a, row, col, a.d - col, x[u], r[u], lo[u], hi[u]);
    sum = squares(lo[u], hi[u], sum);
  }
  sum = row_sum<NT>(sum, part);
  const double inv = 1.0 / sqrt(sum / a.d + (double)a.eps);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (t + u * NT < a.chunks) put8(a, row, t + u * NT, inv, lo[u], hi[u]);
}

// Longer rows: the second pass takes s from the sum where that is kept (it may have been written
// over x or the residual), each thread its own columns again.
template <int XT, int RT>
__global__ __launch_bounds__(1024) void k_norm_long(NormLaunch a) {
  constexpr int RR = RT == kNone ? XT : RT;
  __shared__ double part[16];
  const int64_t row = row_group();
  if (row >= a.rows) return;
  f32x4 lo, hi;
  auto s = [&](int c, bool again) {
    const int col = 8 * c, left = a.d - col;
    if (again && RT != kNone && a.sum) {
      Raw8<RR> r{};
      if (left > 0) r = load8<RR>(a.sum, row * a.sum_stride + col, left, a.sum_vec);
      widen8<RR>(r, lo, hi);
      return;
    }
    Raw8<XT> x{};
    Raw8<RR> r{};
    if (left > 0) {
      x = load8<XT>(a.x, row * a.x_stride + col, left, a.x_vec);
      if constexpr (RT != kNone) r = load8<RR>(a.r, row * a.r_stride + col, left, a.r_vec);
    }
    sum8<XT, RT>(a, row, col, left, x, r, lo, hi);
  };
  double sum = 0.0;
  for (int c = threadIdx.x; c < a.chunks; c += 1024) {
    s(c, false);
    sum = squares(lo, hi, sum);
  }
  sum = row_sum<1024>(sum, part);
  const double inv = 1.0 / sqrt(sum / a.d + (double)a.eps);
  for (int c = threadIdx.x; c < a.chunks; c += 1024) {
    s(c, true);
    put8(a, row, c, inv, lo, hi);
  }
}

template <int XT, int RT, int NT, int U>
void launch_rows(const NormLaunch &a, hipStream_t stream) {
  constexpr int PER = NT < 128 ? 256 / NT : 1;
  hipLaunchKernelGGL((k_norm<XT, RT, NT, U>), groups_of((a.rows + PER - 1) / PER),
                     dim3(NT < 128 ? 256 : NT), 0, stream, a);
}

template <int XT, int RT>
hipError_t launch_norm_of(const NormLaunch &a, hipStream_t stream) {
  // Few rows wait for themselves, one chunk a thread is quickest; many fill the chip, and two a thread
  // keep more loads on their way. us for a row of bf16 with residual and sum, threads x chunks:
  //      1 x 4096: 512 x 1 2.9, 256 x 2 3.5, 1024 x 1 3.1       128 x 7168: 1024 x 1 4.3, 512 x 2 4.6, 256 x 4 5.7
  //   2176 x 7168: 512 x 2 26, 256 x 4 30, 1024 x 1 32          2176 x 4096: 256 x 2 14.8, 512 x 1 14.8
  //  16000 x 2048: 128 x 2 44, 256 x 1 46 (5.9 TB/s), 512 x 1 62   16000 x 1024: 64 x 2 22.6, 128 x 1 22.3, 256 x 1 25
  const bool few = a.rows < 2048;
  if (a.chunks <= 64) launch_rows<XT, RT, 64, 1>(a, stream);
  else if (a.chunks <= 128) few ? launch_rows<XT, RT, 128, 1>(a, stream) : launch_rows<XT, RT, 64, 2>(a, stream);
  else if (a.chunks <= 256) few ? launch_rows<XT, RT, 256, 1>(a, stream) : launch_rows<XT, RT, 128, 2>(a, stream);
  else if (a.chunks <= 512) few ? launch_rows<XT, RT, 512, 1>(a, stream) : launch_rows<XT, RT, 256, 2>(a, stream);
  else if (a.chunks <= 1024) few ? launch_rows<XT, RT, 1024, 1>(a, stream) : launch_rows<XT, RT, 512, 2>(a, stream);
  else if (a.chunks <= 2048) launch_rows<XT, RT, 1024, 2>(a, stream);
  else if (a.chunks <= 4096) launch_rows<XT, RT, 1024, 4>(a, stream);
  else hipLaunchKernelGGL((k_norm_long<XT, RT>), groups_of(a.rows), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

bool vec8(const void *p, int32_t type, int64_t stride) {
  return vec_rows(p, type, stride, type == SD_F32 ? 4 : 8);
}

}  // namespace

hipError_t launch_norm(const NormArgs &n, hipStream_t stream) {
  NormLaunch a;
  static_cast<NormArgs &>(a) = n;
  a.kp = mx_padded(n.d);
  a.chunks = n.codes ? a.kp / 8 : (n.d + 7) / 8;
  a.x_vec = vec8(n.x, n.x_type, n.x_stride);
  a.r_vec = vec8(n.r, n.r_type, n.r_stride);
  a.w_vec = vec8(n.w, n.w_type, 8);
  a.sum_vec = vec8(n.sum, n.r_type, n.sum_stride);
  a.y_vec = vec8(n.y, n.y_type, n.y_stride);
  hipError_t e = hipSuccess;
  by_type(n.x_type, [&](auto T) {
    if (!n.r) e = launch_norm_of<T, kNone>(a, stream);
    else if (n.r_type == SD_F32) e = launch_norm_of<T, SD_F32>(a, stream);
    else if constexpr (T != SD_F32) e = launch_norm_of<T, T>(a, stream);
  });
  return e;
}

}  // namespace sdv
