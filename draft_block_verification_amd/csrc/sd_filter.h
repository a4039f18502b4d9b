// Filtered softmax of a logit row: temperature, top-k, top-p, min-p (gfx950).
//
// With m the row's largest logit, a logit l weighs w = 2^((l - m) log2(e) / T) in [0, 1].
// Rank the ids by larger logit, then lower id. Each filter keeps a leading run of that
// order, so their combination keeps the first n ids, n = min(n_k, n_p, n_m):
//   n_k = k;  n_p = shortest run whose weight reaches p times the weight of the first n_k;
//   n_m = ids with w >= min_p.
// The kept set is then stated by its last member alone: the pair (key, id) of a RowCut.
//
// Weights are formed in fp64 (relative error 4e-14) and summed as 64-bit integers in
// units of 2^-b: integer sums do not depend on order, so a call repeated gives the same
// bytes, and running sums of the same weights are exact in those units. b is 46, less for
// rows of more than 2^17 ids (45 up to 2^18, .. 42 at 2^21) so that V 2^b stays under 2^63.
// One weight's rounding is at most 2^-(b+1) of the row's largest, V 2^-(b+1) of it over a
// whole row, and a weight under 2^-(b+1) counts as 0. Where a row is passed in shares, the
// share that holds a draw is found by weights scaled from their bin, the id in it by single
// exponentials: a border may lie a few units elsewhere than under another split.
//
// The functions that hold workgroup barriers are forced inline: as calls they spill and read
// LDS through flat addresses.
#pragma once

#include <math.h>

#include "sd_internal.h"

namespace sdv {

constexpr int kFilterThreads = 512;    // three workgroups a compute unit in 80 registers a
                                     // lane; 1024 threads or fewer workgroups were no faster
constexpr int kFilterWaves = kFilterThreads / kWave;
constexpr int kGrid = 4096;          // bins of the first pass's histogram, half on each side
                                     // of its reference logit
constexpr int kBins = 2048;          // bins of the narrowing path's histogram
constexpr int kCandMax = 1536;       // ids that are ranked in LDS (three workgroups a compute unit)
constexpr int kCandPad = 2048;       // the same, up to a power of two
constexpr int kPerThread = kCandPad / kFilterThreads;
constexpr int kMaxShares = 256;      // parts a row's vectors are summed in
constexpr int kFixBits = 46;         // most fraction bits of the summed weights
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // key of -inf (sort_key)

typedef unsigned long long u64;

struct RowSettings {
  double sl;      // log2(e) / T
  double unit;    // 2^b, the summed weights' units in 1
  double p;       // top-p share, 1 when off
  double min_p;   // 0 when off, at most 1
  float T;
  int k;          // top-k, 0x7fffffff when off
  bool greedy;    // temperature 0
};

// 2^b for rows of V ids: b = min(46, 63 - ceil(log2 V)).
__device__ inline double fix_unit(int V) {
  const int lg = V > 1 ? 32 - __clz(V - 1) : 0;
  const int b = 63 - lg < kFixBits ? 63 - lg : kFixBits;
  return (double)(1ull << b);
}

// Settings of request i for rows of V ids. A temperature that is NaN, infinite or negative
// counts as 0, a NaN top_p or min_p as off; each raises SD_FLAG_SAMPLING.
__device__ inline RowSettings load_settings(const SampleSettings &s, int i, int V, WsHeader *ws) {
  RowSettings r;
  r.unit = fix_unit(V);
  float T = s.temperature ? s.temperature[i] : 1.f;
  const int k = s.top_k ? s.top_k[i] : 0;
  float p = s.top_p ? s.top_p[i] : 1.f;
  float mp = s.min_p ? s.min_p[i] : 0.f;
  bool bad = false;
  if (!(T >= 0.f && T < INFINITY)) { T = 0.f; bad = true; }
  if (p != p) { p = 1.f; bad = true; }
  if (mp != mp) { mp = 0.f; bad = true; }
  if (bad) raise_flag(ws, SD_FLAG_SAMPLING);
  r.T = T;
  r.greedy = T == 0.f;
  r.sl = r.greedy ? 0.0 : 1.4426950408889634 / (double)T;
  r.k = k > 0 ? k : 0x7fffffff;
  r.p = p >= 1.f ? 1.0 : (double)p;
  r.min_p = mp <= 0.f ? 0.0 : (mp > 1.f ? 1.0 : (double)mp);
  return r;
}

// What keeps an id of a row: a logit above `val`, or equal to it and id <= `id`.
struct RowCut {
  float m;        // largest logit of the row, -inf when the row has none
  float val;
  int32_t id;
  int32_t n;      // ids kept (at least: some calls only tell none from some)
  u64 S;          // their weight, in RowSettings::unit
  int32_t pad[2];
};
static_assert(sizeof(RowCut) == 32, "row cuts are 32 bytes");

// ------------------------------------------------------------------ elements
// NaN counts as -inf (never kept): the maximum of a NaN and a number is the number.
__device__ inline float canonical(float x) { return __builtin_fmaxf(x, -INFINITY); }

// Order-preserving bits: a > b <=> sort_key(a) > sort_key(b) for canonical values (-0 has the
// key of +0).
__device__ inline uint32_t sort_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ inline float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

struct ElemF32 {
  static constexpr uint32_t kNegInf = 0xff800000u;   // a word of -inf
  using S = float;
  static constexpr int VE = 4;
  __device__ static float get(S x) { return x; }
  __device__ static void unpack(u32x4 q, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(q[i]);
  }
};

struct ElemBF16 {
  static constexpr uint32_t kNegInf = 0xff80ff80u;   // a word of -inf
  using S = uint16_t;
  static constexpr int VE = 8;
  __device__ static float get(S x) { return bf16_to_f32(x); }
  __device__ static void unpack(u32x4 q, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
};

struct ElemF16 {
  static constexpr uint32_t kNegInf = 0xfc00fc00u;   // a word of -inf
  using S = _Float16;
  static constexpr int VE = 8;
  __device__ static float get(S x) { return (float)x; }
  __device__ static void unpack(u32x4 q, float (&v)[8]) {
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    const h8 h = __builtin_bit_cast(h8, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  }
};

// A row as 16-byte vectors: vector j holds ids off + j VE .. + VE - 1, off <= 0 chosen so
// that every vector that lies in the row whole is 16-byte aligned; the first and the last
// may lie in it in part and are read id by id.
template <class E>
struct RowView {
  const typename E::S *p;
  int V, off, nv;
  __device__ RowView(const typename E::S *row, int V_) : p(row), V(V_) {
    const int head = (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(typename E::S));
    off = head ? head - E::VE : 0;
    nv = (V - off + E::VE - 1) / E::VE;
  }
  __device__ int id(int j, int i) const { return off + j * E::VE + i; }
  __device__ bool whole(int j) const {
    const int b = off + j * E::VE;
    return b >= 0 && b + E::VE <= V;
  }
  __device__ float at(int x) const { return canonical(E::get(p[x])); }
  // Canonical values of vector j, which lies in the row whole.
  __device__ void load_whole(int j, float (&v)[E::VE]) const {
    unpack(*reinterpret_cast<const u32x4 *>(p + off + j * E::VE), v);
  }
  __device__ static void unpack(const u32x4 &q, float (&v)[E::VE]) {
    E::unpack(q, v);
#pragma unroll
    for (int i = 0; i < E::VE; ++i) v[i] = canonical(v[i]);
  }
  // Canonical values of any vector, -inf outside the row.
  __device__ void load(int j, float (&v)[E::VE]) const {
    if (whole(j)) {
      load_whole(j, v);
    } else {
#pragma unroll
      for (int i = 0; i < E::VE; ++i) {
        const int x = id(j, i);
        v[i] = x >= 0 && x < V ? at(x) : -INFINITY;
      }
    }
  }
};

// f(v, id0) for vectors j0 .. j1 - 1, taken by the calling wave: VE values as they lie in
// memory (NaN among them) and the first one's id. Lanes without a vector get -inf, so f needs
// no mask. The whole vectors go first, a round's loads issued before the round ahead of it is
// used; then the row's first and last vector if it holds them and they lie in it in part, an
// element a lane. N: ids a lane and round.
template <int N = 8, class E, class F>
__device__ __forceinline__ void wave_vecs(const RowView<E> &r, int j0, int j1, F f) {
  const int lane = threadIdx.x & 63;
  j0 = __builtin_amdgcn_readfirstlane(j0);
  j1 = __builtin_amdgcn_readfirstlane(j1);
  constexpr int U = N > E::VE ? N / E::VE : 1;
  const bool head = j0 == 0 && j0 < j1 && !r.whole(0);
  const bool tail = j1 == r.nv && j0 < j1 && !r.whole(r.nv - 1) && !(head && r.nv == 1);
  const int a = j0 + head, n = j1 - tail - a;      // whole vectors
  if (n > 0) {
    // The wave's place in the row is one number for all its lanes: addresses are a scalar base
    // and a lane's constant offset.
    const char *base = reinterpret_cast<const char *>(r.p + r.off) + 16 * (size_t)a;
    auto fetch = [&](int t, u32x4 (&q)[U]) {
      const char *p = base + (size_t)t * (1024 * U);
      if ((t + 1) * 64 * U <= n) {
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = *reinterpret_cast<const u32x4 *>(p + (u * 1024 + lane * 16));
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
          q[u] = *reinterpret_cast<const u32x4 *>(base + 16 * (size_t)min(t * 64 * U + 64 * u + lane, n - 1));
      }
    };
    u32x4 next[U];
    fetch(0, next);
    for (int t = 0; t * 64 * U < n; ++t) {
      u32x4 now[U];
#pragma unroll
      for (int u = 0; u < U; ++u) now[u] = next[u];
      if ((t + 1) * 64 * U < n) fetch(t + 1, next);
      if ((t + 1) * 64 * U > n) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (t * 64 * U + 64 * u + lane >= n) now[u] = u32x4{E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf};
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[E::VE];
        E::unpack(now[u], v);
        f(v, r.id(a + t * 64 * U + 64 * u + lane, 0));
      }
    }
  }
  if (head || tail) {
    const bool second = lane >= E::VE;
    const int x = r.id(second ? r.nv - 1 : 0, second ? lane - E::VE : lane);
    const bool in = lane < 2 * E::VE && (second ? tail : head) && x >= 0 && x < r.V;
    float v[E::VE];
#pragma unroll
    for (int i = 0; i < E::VE; ++i) v[i] = -INFINITY;
    if (in) v[0] = E::get(r.p[x]);
    f(v, x);
  }
}

// f(value, id) for their ids, canonical values above -inf only.
template <int N = 8, class E, class F>
__device__ __forceinline__ void wave_ids(const RowView<E> &r, int j0, int j1, F f) {
  wave_vecs<N>(r, j0, j1, [&](const float (&v)[E::VE], int id) {
#pragma unroll
    for (int i = 0; i < E::VE; ++i)
      if (v[i] > -INFINITY) f(v[i], id + i);
  });
}

// ------------------------------------------------------------------ weights
// 2^x in fp64: 2^n (1 + f q(f)) for the nearest whole n and f = x - n. q is the polynomial of
// degree 8 through (2^f - 1) / f at the nine Chebyshev points of [-1/2, 1/2]; the relative
// error of the result is at most 4e-14, and f = 0 gives exactly 2^n. Every fused step is
// written out and the compiler may form no other: a weight formed in two places must be the
// same number, or a running sum could miss a border by a unit.
__device__ inline double exp2_f64(double x) {
#pragma clang fp contract(off)
  const double n = __builtin_rint(x), f = x - n;
  double s = 1.0203121063391729e-07;
  s = __builtin_fma(s, f, 1.3255224878668817e-06);
  s = __builtin_fma(s, f, 1.525268684626772e-05);
  s = __builtin_fma(s, f, 0.00015403455852453838);
  s = __builtin_fma(s, f, 0.0013333558179043112);
  s = __builtin_fma(s, f, 0.009618129159402558);
  s = __builtin_fma(s, f, 0.055504108664760424);
  s = __builtin_fma(s, f, 0.2402265069581299);
  s = __builtin_fma(s, f, 0.6931471805599453);
  s = __builtin_fma(s, f, 1.0);
  return __builtin_ldexp(s, (int)n);
}

// Weight of a finite logit l under a finite row maximum m.
__device__ inline double weight_finite(float l, float m, double sl) {
#pragma clang fp contract(off)
  return exp2_f64(((double)l - (double)m) * sl);
}

// Weight of any logit above -inf: ids at a maximum of +inf share the whole weight.
__device__ inline double weight(float l, float m, double sl) {
  return l == m ? 1.0 : m == INFINITY ? 0.0 : weight_finite(l, m, sl);
}

// w * unit rounded to nearest, for results under 2^52: the fp64 sum's low 52 bits hold it.
__device__ inline u64 to_fix(double w, double unit) {
  const double s = __builtin_fma(w, unit, 4503599627370496.0);
  return (u64)__double_as_longlong(s) & 0xfffffffffffffull;
}

__device__ inline bool kept(const RowCut &c, float l, int id) {
  return l > c.val || (l == c.val && id <= c.id);
}

// ------------------------------------------------------------------ workgroup sums
// x of the lane that a data-parallel-primitive control names, 0 where it names none.
template <int CTRL, int ROWS>
__device__ inline u64 dpp_u64(u64 x) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(x >> 32), CTRL, ROWS, 0xf, false);
  return ((u64)hi << 32) | lo;
}

// Sum over lanes 0 .. own: by shifts inside each row of 16 lanes, then the rows' totals
// broadcast onwards (all lanes of the wave take part).
__device__ inline u64 wave_incl_scan_u64(u64 x) {
  x += dpp_u64<0x111, 0xf>(x);    // from 1, 2, 4 and 8 lanes below in the row
  x += dpp_u64<0x112, 0xf>(x);
  x += dpp_u64<0x114, 0xf>(x);
  x += dpp_u64<0x118, 0xf>(x);
  x += dpp_u64<0x142, 0xa>(x);    // lane 15 of rows 0 and 2 into rows 1 and 3
  x += dpp_u64<0x143, 0xc>(x);    // lane 31 into rows 2 and 3
  return x;
}

__device__ inline u64 wave_sum_u64(u64 x) {
  x = wave_incl_scan_u64(x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, 63);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), 63);
  return ((u64)hi << 32) | lo;
}

// Shared memory of one workgroup's row.
struct FilterSmem {
  union {
    u64 grid[kGrid + 64];  // first pass: weight (or count) by bin, then spare words
    double scale[kGrid + 64];   // second pass: a bin's lower end's weight, spare words 0
    struct {               // narrowing path
      u64 mass[kBins];
      uint32_t cnt[kBins];
    };
    struct {               // choosing from the list
      u64 bucket[kFilterThreads];
      u64 sub[kCandMax], sub_w[kCandMax];
    };
  };
  u64 cand[kCandPad];
  u64 red[kFilterWaves];
  u64 share[kMaxShares];   // weight of the kept ids by share of the row
  uint32_t n_cand, n_sub;
  int hit;
  uint32_t key;
  int32_t id;
  u64 acc, acc2, word;
};

// Sum over the workgroup; every thread gets it.
__device__ __forceinline__ u64 block_sum_u64(u64 x, FilterSmem &s) {
  x = wave_sum_u64(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.red[threadIdx.x >> 6] = x;
  __syncthreads();
  u64 t = 0;
#pragma unroll
  for (int w = 0; w < kFilterWaves; ++w) t += s.red[w];
  return t;
}

// Exclusive scan over the workgroup's threads.
__device__ __forceinline__ u64 block_excl_scan_u64(u64 x, FilterSmem &s) {
  const u64 incl = wave_incl_scan_u64(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.red[threadIdx.x >> 6] = incl;
  __syncthreads();
  u64 before = 0;
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) before += s.red[w];
  return before + incl - x;
}

// s.cand[0 .. n), n a power of two, sorted in descending order. Up to 128 of them are sorted
// by the first wave alone: its LDS accesses take effect in order, so its steps need no barrier.
__device__ __forceinline__ void sort_desc(FilterSmem &s, int n) {
  __syncthreads();
  if (n <= 128) {
    if (threadIdx.x < 64) {
      for (int size = 2; size <= n; size <<= 1) {
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
          const int t = threadIdx.x;
          const int i = 2 * t - (t & (stride - 1)), j = i + stride;
          if (t < n / 2) {
            const u64 a = s.cand[i], b = s.cand[j];
            if ((a < b) == ((i & size) == 0)) { s.cand[i] = b; s.cand[j] = a; }
          }
          asm volatile("" ::: "memory");
        }
      }
    }
    __syncthreads();
    return;
  }
  for (int size = 2; size <= n; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n / 2; t += kFilterThreads) {
        const int i = 2 * t - (t & (stride - 1)), j = i + stride;
        const u64 a = s.cand[i], b = s.cand[j];
        if ((a < b) == ((i & size) == 0)) { s.cand[i] = b; s.cand[j] = a; }
      }
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------ the narrowing path
// Bins of the mass histogram: equal steps of (m - l), which falls as the rank rises, over
// max(33 T, 16). A logit past that range weighs under 2^-47 (33 T are 47.6 octaves), so its
// summed weight is 0 and no filter but the count of top-k can end among those ids: the last
// bin stands for them, without weight. Equal steps spread a row's logits over many bins, so
// that lanes seldom meet on one LDS counter and a bin holds few ids to rank; the last bin's
// ids are counted in registers.
struct BinScale {
  float m, scale;
  __device__ BinScale(float m_, float T) : m(m_), scale((float)(kBins - 1) / fmaxf(33.f * T, 16.f)) {}
  // Bin of a logit, kBins - 1 past the range.
  __device__ int of(float l) const {
    const float d = l == m ? 0.f : (m - l) * scale;
    return d < (float)(kBins - 1) ? (int)d : kBins - 1;
  }
};

// First rank position, over the bins in order, at which a running total reaches `need`:
// the bin, and the totals before it. Bin totals come from f(bin) (count or mass).
// Returns kBins when the sum over all bins stays under need.
template <class F>
__device__ __forceinline__ int find_bin(FilterSmem &s, u64 need, F f, u64 *before) {
  constexpr int P = kBins / kFilterThreads;
  const int b = P * threadIdx.x;
  u64 x[P], own = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) { x[i] = f(b + i); own += x[i]; }
  u64 run = block_excl_scan_u64(own, s);
  if (threadIdx.x == 0) { s.hit = kBins; s.acc = 0; }
  __syncthreads();
  // Exactly one bin has before < need <= before + own (need >= 1).
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (run < need && run + x[i] >= need) { s.hit = b + i; s.acc = run; }
    run += x[i];
  }
  __syncthreads();
  const int hit = s.hit;
  *before = s.acc;
  __syncthreads();
  return hit;
}

// Smallest whole t >= 1 with t >= x.
__device__ inline u64 at_least(double x) {
  const double c = ceil(x);
  return c < 1.0 ? 1ull : (u64)c;
}

// Last member of a leading run: its key and id, and the run's count and weight.
struct CutAt {
  uint32_t key;
  int32_t id;
  u64 n, mass;
};

// The run that ends at the need-th id (by_mass false) or at the first id whose running
// weight reaches need (by_mass true), known to end in bin cb; the bins before it hold
// n_before ids of weight mass_before. Overwrites the histogram when it has to narrow.

template <class E>
__device__ __forceinline__ CutAt cut_in_bin(const RowView<E> &r, FilterSmem &s, const BinScale &bins,
                            const RowSettings &set, int cb, bool by_mass, u64 need, u64 n_before, u64 mass_before) {
  const int tid = threadIdx.x, wave = tid >> 6;
  const int per = (r.nv + kFilterWaves - 1) / kFilterWaves;
  const int j0 = wave * per, j1 = min(r.nv, j0 + per);
  // Narrow by key digits (11, 11, 10 bits) while the bin holds more ids than are ranked in
  // LDS. fixed: bits of the key known so far; prefix: their value.
  uint32_t prefix = 0, n_in = s.cnt[cb];
  int known = 0;
  __syncthreads();
  while (n_in > kCandMax && known < 32) {
    const int width = known == 22 ? 10 : 11, shift = 32 - known - width;
    for (int b = tid; b < kBins; b += kFilterThreads) { s.mass[b] = 0; s.cnt[b] = 0; }
    __syncthreads();
    wave_ids<4>(r, j0, j1, [&](float l, int) {
      if (l == -INFINITY || bins.of(l) != cb) return;
      const uint32_t k = sort_key(l);
      if (known && (k >> (32 - known)) != prefix) return;
      // Digit 0 is the largest.
      const uint32_t g = ((1u << width) - 1) - ((k >> shift) & ((1u << width) - 1));
      atomicAdd(&s.cnt[g], 1u);
      atomicAdd(&s.mass[g], to_fix(weight(l, bins.m, set.sl), set.unit));
    });
    __syncthreads();
    u64 before;
    const int g = by_mass
        ? find_bin(s, need - mass_before, [&](int b) { return s.mass[b]; }, &before)
        : find_bin(s, need - n_before, [&](int b) { return (u64)s.cnt[b]; }, &before);
    // Totals of both kinds before digit g.
    u64 nb = 0, mb = 0;
    for (int b = tid; b < g; b += kFilterThreads) { nb += s.cnt[b]; mb += s.mass[b]; }
    nb = block_sum_u64(nb, s);
    mb = block_sum_u64(mb, s);
    n_before += nb;
    mass_before += mb;
    n_in = s.cnt[g];
    prefix = (prefix << width) | (((1u << width) - 1) - g);
    known += width;
    __syncthreads();
  }
  if (known == 32 && n_in > kCandMax) {
    // One key, many ids of equal weight: how many of them, then the id of the last.
    const u64 w = to_fix(weight(key_value(prefix), bins.m, set.sl), set.unit);
    const u64 take = by_mass ? (need - mass_before + w - 1) / w : need - n_before;
    u64 left = take;      // ids still to pass, in id order
    int a = 0, b = r.nv;
    while (b - a > 64) {
      const int step = (b - a + kFilterWaves - 1) / kFilterWaves;
      const int w0 = a + wave * step, w1 = min(b, w0 + step);
      u64 c = 0;
      wave_ids<4>(r, w0, w1, [&](float l, int) { c += l > -INFINITY && sort_key(l) == prefix; });
      c = wave_sum_u64(c);
      __syncthreads();
      if ((tid & 63) == 0) s.red[wave] = c;
      __syncthreads();
      int v = 0;
      while (v < kFilterWaves - 1 && s.red[v] < left) left -= s.red[v++];
      a = a + v * step;
      b = min(b, a + step);
      __syncthreads();
    }
    if (wave == 0) {
      const int lane = tid, j = a + lane;
      float v[E::VE];
      u64 c = 0;
      if (j < b) {
        r.load(j, v);
#pragma unroll
        for (int i = 0; i < E::VE; ++i) c += v[i] > -INFINITY && sort_key(v[i]) == prefix;
      }
      const u64 ex = wave_incl_scan_u64(c) - c;
      if (j < b && ex < left && ex + c >= left) {
        u64 seen = ex;
#pragma unroll
        for (int i = 0; i < E::VE; ++i) {
          const bool is = v[i] > -INFINITY && sort_key(v[i]) == prefix;
          seen += is;
          if (is && seen == left) s.id = r.id(j, i);
        }
      }
    }
    __syncthreads();
    CutAt c{prefix, s.id, n_before + take, mass_before + take * w};
    __syncthreads();
    return c;
  }
  // Rank the ids in LDS.
  if (tid == 0) s.n_cand = 0;
  __syncthreads();
  wave_ids<4>(r, j0, j1, [&](float l, int id) {
    if (l == -INFINITY || bins.of(l) != cb) return;
    const uint32_t k = sort_key(l);
    if (known && (known == 32 ? k : k >> (32 - known)) != prefix) return;
    const uint32_t at = atomicAdd(&s.n_cand, 1u);
    if (at < kCandMax) s.cand[at] = ((u64)k << 32) | (uint32_t)~id;
  });
  __syncthreads();
  const int n = (int)s.n_cand;
  int pow2 = 2;
  while (pow2 < n) pow2 <<= 1;
  for (int i = n + tid; i < pow2; i += kFilterThreads) s.cand[i] = 0;
  sort_desc(s, pow2);
  // Thread t holds ranks kPerThread t .. .
  u64 w[kPerThread], own = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int at = kPerThread * tid + i;
    w[i] = at < n ? to_fix(weight(key_value((uint32_t)(s.cand[at] >> 32)), bins.m, set.sl), set.unit) : 0;
    own += w[i];
  }
  u64 run = mass_before + block_excl_scan_u64(own, s);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int at = kPerThread * tid + i;
    const u64 incl = run + w[i];
    const bool is = at < n && (by_mass ? (run < need && incl >= need) : n_before + at + 1 == need);
    if (is) {
      s.key = (uint32_t)(s.cand[at] >> 32);
      s.id = (int)~(uint32_t)s.cand[at];
      s.acc = n_before + at + 1;
      s.acc2 = incl;
    }
    run = incl;
  }
  __syncthreads();
  CutAt c{s.key, s.id, s.acc, s.acc2};
  __syncthreads();
  return c;
}

// The narrowing path: the cut of a row whose largest logit c.m is known, for every row that the
// single-pass path leaves: more ids at the cut than are ranked in LDS, a top-k past them, a
// top-k that ends under the grid, logits too large for the grid's arithmetic, +inf among them,
// and of the rows dealt to several workgroups those whose largest logit lies past the grid
// that their sample gave (under it: a mask that left the sample nothing). One row of 151936
// fp32 ids: 10 ids allowed 125 us, those 10 with the others at fp32's lowest value 200, an
// unsampled peak 15 over the rest at T = 0.3 under top-p 198, top-k 2000 265, T = 3 under
// top-p 0.85 393, against 28 for top-k 50 and 40 for top-p 0.9 on the single-pass path.
// totals (as for row_plan): probabilities are taken from the cut, and an id past the range has
// one as long as it is kept. A draw sums such weights to 0, so it does without the last member
// of a top-k run that ends there: c.n is right, and ids behind that run are not told apart.
template <class E>
__device__ __forceinline__ void cut_narrowing(const RowView<E> &r, const RowSettings &set, bool totals, RowCut &c,
                                              FilterSmem &s) {
  const int tid = threadIdx.x, wave = tid >> 6;
  c.val = -INFINITY;
  c.id = -1;
  const int per = (r.nv + kFilterWaves - 1) / kFilterWaves;
  const int j0 = wave * per, j1 = min(r.nv, j0 + per);
  const BinScale bins(c.m, set.T);
  __syncthreads();
  for (int b = tid; b < kBins; b += kFilterThreads) { s.mass[b] = 0; s.cnt[b] = 0; }
  __syncthreads();
  uint32_t n_m = 0, low = 0xffffffffu, past = 0;
  wave_ids<4>(r, j0, j1, [&](float l, int) {
    if (l == -INFINITY) return;
    const double w = weight(l, c.m, set.sl);
    if (w >= set.min_p) { ++n_m; low = min(low, sort_key(l)); }
    const int b = bins.of(l);
    if (b == kBins - 1) { ++past; return; }
    atomicAdd(&s.cnt[b], 1u);
    atomicAdd(&s.mass[b], to_fix(w, set.unit));
  });
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) low = min(low, (uint32_t)__shfl_xor((int)low, off));
  // Both counts in one sum (each under 2^31).
  const u64 both = block_sum_u64(((u64)past << 32) | n_m, s);
  __syncthreads();
  if ((tid & 63) == 0) s.red[wave] = low;
  __syncthreads();
  for (int w = 0; w < kFilterWaves; ++w) low = min(low, (uint32_t)s.red[w]);
  __syncthreads();
  n_m = (uint32_t)both;
  past = (uint32_t)(both >> 32);
  u64 n = n_m;                           // w >= min_p (all of them when min_p is off)
  if (set.min_p > 0.0) { c.val = key_value(low); c.id = 0x7fffffff; }
  {
    u64 total = 0, in_bins = 0;
    for (int b = tid; b < kBins; b += kFilterThreads) { total += s.mass[b]; in_bins += s.cnt[b]; }
    total = block_sum_u64(total, s);
    in_bins = block_sum_u64(in_bins, s);
    CutAt at{kKeyNegInf, -1, in_bins + past, total};
    const u64 rankable = totals ? at.n : in_bins;
    if ((u64)set.k >= rankable && (u64)set.k < at.n) at.n = set.k;
    // First the end of the top-k run, then that of the top-p run inside it.
#pragma unroll 1
    for (int by_mass = 0; by_mass < 2; ++by_mass) {
      if (by_mass ? !(set.p < 1.0) : !((u64)set.k < rankable)) continue;
      const u64 need = by_mass ? at_least(set.p * (double)at.mass) : (u64)set.k;
      // The histogram again: narrowing the top-k run may have overwritten it.
      __syncthreads();
      for (int b = tid; b < kBins; b += kFilterThreads) { s.mass[b] = 0; s.cnt[b] = 0; }
      __syncthreads();
      wave_ids<4>(r, j0, j1, [&](float l, int) {
        if (l == -INFINITY) return;
        const int b = bins.of(l);
        if (b == kBins - 1) return;
        atomicAdd(&s.cnt[b], 1u);
        atomicAdd(&s.mass[b], to_fix(weight(l, c.m, set.sl), set.unit));
      });
      if (tid == 0) s.cnt[kBins - 1] = past;
      __syncthreads();
      u64 before, n_before = 0, mass_before = 0;
      const int bin = find_bin(s, need, [&](int b) { return by_mass ? s.mass[b] : (u64)s.cnt[b]; }, &before);
      for (int b = tid; b < bin; b += kFilterThreads) { n_before += s.cnt[b]; mass_before += s.mass[b]; }
      n_before = block_sum_u64(n_before, s);
      mass_before = block_sum_u64(mass_before, s);
      const CutAt q = cut_in_bin(r, s, bins, set, bin, by_mass, need, n_before, mass_before);
      if (q.n < at.n) at = q;
    }
    // The shorter of the two runs.
    if (at.n < n) {
      n = at.n;
      c.val = key_value(at.key);
      c.id = at.id;
    }
  }
  c.n = (int)n;
}

// ------------------------------------------------------------------ the cut
// How a row's cut is found.
enum CutKind {
  kCutOne,     // the likeliest id alone: no weights
  kCutCount,   // top-k: ids are counted by bin
  kCutMass,    // top-p without top-k (or totals alone are wanted): weights are summed by bin
  kCutSum      // no ranking: weights are summed where they are drawn from
};

// totals: only the kept set and its weight are wanted, not a draw.
__device__ inline CutKind cut_kind(const RowSettings &set, int V, bool totals) {
  if (set.greedy || set.k == 1 || set.p <= 0.0) return kCutOne;
  if (set.k < V) return kCutCount;
  return set.p < 1.0 || totals ? kCutMass : kCutSum;
}

// Bins of the first pass: steps of the logit's distance from a reference logit, kGrid / 2 on
// each side; 33 T (or 16 when ids are counted, so that small temperatures still spread them)
// fill one side. With the row's largest logit at or above the reference and inside the grid,
// a logit under its lower end weighs less than 2^-47 of it.
struct Grid {
  double k, c;        // position of logit l in bins from the lower end: l k + c
  bool fine;          // positions are good to 3e-11 bins, weights to 5e-13
  __device__ Grid(float ref, float T, bool count) {
    k = (double)(kGrid / 2) / (count ? fmax(33.0 * (double)T, 16.0) : 33.0 * (double)T);
    c = (double)(kGrid / 2) - (double)ref * k;
    fine = fabs(c) < 262144.0;
  }
  __device__ double pos(float l) const { return __builtin_fma((double)l, k, c); }
};

// x towards 0, saturating (a C++ conversion leaves positions outside int undefined).
__device__ inline uint32_t whole_part(double x) {
  int i;
  asm("v_cvt_i32_f64 %0, %1" : "=v"(i) : "v"(x));
  return (uint32_t)i;
}

// A bin sums its weights relative to its own lower end, e^(a y) for the position y in [0, 1)
// inside it with a = 33 / (kGrid / 2): bins need no common scale and the pass over the row no
// maximum to start from. The polynomial goes through e^(a y) at five Chebyshev points of
// [0, 1]; its relative error is 2e-14.
constexpr double kBinOctaves = 33.0 * 1.4426950408889634 / (kGrid / 2);

__device__ inline double bin_weight(double y) {
  static_assert(kGrid == 4096, "the coefficients are those of a = 33 / 2048");
  double s = 2.8315539305093126e-09;
  s = __builtin_fma(s, y, 6.972496547552619e-07);
  s = __builtin_fma(s, y, 0.00012981892343785);
  s = __builtin_fma(s, y, 0.016113281249110118);
  return __builtin_fma(s, y, 1.0000000000000178);
}

// Unit of the bins' sums: up to V weights under 1.02 stay under 2^64.
__device__ inline double bin_unit(const RowSettings &set) { return set.unit * 0.25; }

// Smallest value (not -inf) for which `ok`, which holds from some value on; +inf has to be
// one. Each wave searches by itself, 64 probes a step: first those around a guess, which is
// nearly always within a few steps of fp32 of the border.
template <class F>
__device__ __forceinline__ float smallest(double guess, F ok) {
  const int lane = threadIdx.x & 63;
  uint32_t lo = kKeyNegInf + 1, hi = 0xff800000u;   // keys of the lowest finite value and +inf
  const uint32_t mid = min(max(sort_key(canonical((float)guess)), lo + 64), hi - 64);
  const u64 near = __ballot(ok(key_value(mid - 32 + lane)));
  if (near && !(near & 1)) return key_value(mid - 32 + (__ffsll((long long)near) - 1));
  while (hi > lo) {
    const uint32_t step = (hi - lo + 63) / 64;
    const uint32_t probe = (uint32_t)lane * step < hi - lo ? lo + (uint32_t)lane * step : hi;
    const u64 m = __ballot(ok(key_value(probe)));
    if (m == 0) { lo = lo + 63 * step < hi ? lo + 63 * step + 1 : hi; continue; }
    const int first = __ffsll((long long)m) - 1;
    const uint32_t at = (uint32_t)first * step < hi - lo ? lo + (uint32_t)first * step : hi;
    if (first == 0) { hi = lo; break; }
    lo = at - step + 1;
    hi = at;
  }
  return key_value(hi);
}

// Smallest value at or above the lower end of bin b.
__device__ __forceinline__ float bin_floor(const Grid &g, int b) {
  return smallest(((double)b - g.c) / g.k, [&](float l) { return g.pos(l) >= (double)b; });
}

// Lane's part of the first pass over vectors j0 .. j1 - 1: the largest logit (best), and by
// kind the lowest id that attains it (at), the ids above -inf (any), the grid's bins in LDS.
struct PassOut {
  float best = -INFINITY;
  int at = 0x7fffffff;
  uint32_t any = 0;
};

template <class E>
__device__ __forceinline__ void bin_pass(const RowView<E> &r, const Grid &g, CutKind kind, double unit, int j0, int j1,
                                         PassOut &o, FilterSmem &s) {
  // An id outside the grid adds to one of 64 words behind it, a lane's own, unread: without a
  // branch around the add. A NaN's position converts to 0: bin 0 is not read either.
  const uint32_t spare = kGrid + (threadIdx.x & 63);
  if (kind == kCutMass) {
    wave_vecs(r, j0, j1, [&](const float (&v)[E::VE], int) {
#pragma unroll
      for (int i = 0; i < E::VE; ++i) {
        o.best = fmaxf(o.best, v[i]);
        const double x = g.pos(v[i]);
        const uint32_t b = whole_part(x);
        atomicAdd(&s.grid[b < kGrid ? b : spare], to_fix(bin_weight(__builtin_amdgcn_fract(x)), unit));
      }
    });
  } else if (kind == kCutCount) {
    wave_vecs(r, j0, j1, [&](const float (&v)[E::VE], int) {
#pragma unroll
      for (int i = 0; i < E::VE; ++i) {
        o.best = fmaxf(o.best, v[i]);
        o.any += __popcll(__ballot(v[i] > -INFINITY));
        const uint32_t b = whole_part(g.pos(v[i]));
        atomicAdd(reinterpret_cast<uint32_t *>(&s.grid[b < kGrid ? b : spare]), 1u);
      }
    });
    o.any = (threadIdx.x & 63) == 0 ? o.any : 0;       // counted once a wave
  } else {
    wave_ids(r, j0, j1, [&](float l, int id) {
      if (l > o.best || (l == o.best && id < o.at)) { o.best = l; o.at = id; }
    });
  }
}

// Larger logit first, then lower id; 0 for none.
__device__ inline u64 rank_word(float l, int id) { return l > -INFINITY ? ((u64)sort_key(l) << 32) | (uint32_t)~id : 0; }
__device__ inline float word_value(u64 w) { return w ? key_value((uint32_t)(w >> 32)) : -INFINITY; }
__device__ inline int word_id(u64 w) { return w ? (int)~(uint32_t)w : -1; }

__device__ __forceinline__ u64 block_max_u64(u64 k, FilterSmem &s) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const u64 o = __shfl_xor(k, off);
    k = o > k ? o : k;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.red[threadIdx.x >> 6] = k;
  __syncthreads();
  for (int w = 0; w < kFilterWaves; ++w) k = s.red[w] > k ? s.red[w] : k;
  return k;
}

// What the second pass does with an id: from t_hi up it is kept without ranking, from t_lo up
// it is listed (with `list` every id from t_lo up is).
struct CutPlan {
  float t_lo, t_hi;
  float t_m;       // smallest logit that min-p keeps, -inf when it is off
  bool list;
  bool narrow;     // left to the narrowing path
  bool listed;     // the first pass has listed the ids already
  u64 need;        // weight at which the top-p run of a kCutMass row ends, 0 without one
  u64 above;       // kCutMass: weight of the ids from t_hi up, by the bins
  u64 in_bin;      // kCutMass: weight of the ids in the bin of the cut
};

// Smallest logit that min-p keeps under maximum m.
__device__ __forceinline__ float min_p_floor(const RowSettings &set, float m) {
  return smallest((double)m + log2((double)set.min_p) / set.sl,
                  [&](float l) { return l >= m || weight_finite(l, m, set.sl) >= set.min_p; });
}

// The plan of a row with largest logit m (above -inf) and `any` ids above -inf (kCutCount),
// from the grid in LDS. Every thread gets it. Thread t holds the kPlan bins from kGrid - 1 -
// kPlan t down, so one scan over the threads runs in rank order.
constexpr int kPlan = kGrid / kFilterThreads;

__device__ __forceinline__ CutPlan make_plan(const RowSettings &set, CutKind kind, const Grid &g, float m, u64 any,
                                             FilterSmem &s) {
  const int tid = threadIdx.x, b0 = kGrid - 1 - kPlan * tid;
  const float lowest = key_value(kKeyNegInf + 1);
  CutPlan p{lowest, lowest, -INFINITY, false, m == INFINITY || !g.fine || !(g.pos(m) < (double)kGrid), false, 0, 0, 0};
  const bool min_p = set.min_p > 0.0;
  if (p.narrow) return p;
  const float t_m = min_p ? min_p_floor(set, m) : lowest;
  if (min_p) p.t_m = t_m;
  if (kind == kCutSum) {
    p.t_lo = p.t_hi = t_m;
    return p;
  }
  // Bin totals: counts, or weights under the row's maximum in its unit.
  const double xm = g.pos(m), scale = set.unit / bin_unit(set);
  u64 raw[kPlan], total[kPlan], own = 0;
#pragma unroll
  for (int i = 0; i < kPlan; ++i) {
    raw[i] = b0 - i > 0 ? s.grid[b0 - i] : 0;
    if (kind == kCutCount) total[i] = (uint32_t)raw[i];
    else total[i] = raw[i] ? (u64)((double)raw[i] * scale * exp2_f64(((double)(b0 - i) - xm) * kBinOctaves)) : 0;
    own += total[i];
  }
  const u64 before = block_excl_scan_u64(own, s);
  if (tid == kFilterThreads - 1) s.acc = before + own;
  if (tid == 0) s.hit = -1;
  __syncthreads();
  const u64 all = s.acc;
  // The bin with the cut, counted from below, and the total up to and including it.
  u64 need = 0;
  if (kind == kCutCount) need = (u64)set.k;
  else if (set.p < 1.0) need = p.need = at_least(set.p * (double)all);
  if (need > before && need <= before + own) {
    u64 run = before;
#pragma unroll
    for (int i = 0; i < kPlan; ++i) {
      if (run < need && run + total[i] >= need) { s.hit = b0 - i; s.acc2 = run + total[i]; }
      run += total[i];
    }
  }
  __syncthreads();
  int cb = s.hit;
  if (kind == kCutCount) {
    p.list = true;
    const u64 upto = cb < 0 ? all : s.acc2;
    p.narrow = upto > kCandMax || (cb < 0 && all != any);   // fewer than k in the grid
    if (cb >= 0) p.t_lo = bin_floor(g, cb);
    return p;
  }
  // That of top-p, or of min-p's bound if it is higher. A bound under bin 1 (bin 0 is not read)
  // parts ids without weight: the bins name no cut, min_p_floor's value alone states the run.
  p.t_lo = p.t_hi = t_m;
  if (min_p) {
    const int mb = (int)whole_part(g.pos(t_m));
    if (mb > max(cb, 0)) { cb = mb; p.need = 0; }
  }
  // No bin holds more ids than its weights say: each is at least 1 (to 2e-14).
  const double per_id = 1.001 / bin_unit(set);
  u64 above = 0, ids = 0;
  if (tid == 0) s.acc2 = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlan; ++i) {
    if (b0 - i > cb) above += total[i];
    if (b0 - i == cb) s.acc2 = total[i];
    if (b0 - i >= cb) ids += (u64)((double)raw[i] * per_id);
  }
  p.above = block_sum_u64(above, s);
  p.in_bin = s.acc2;
  if (cb >= 0) {
    ids = block_sum_u64(ids, s);
    const u64 in_bin = (u64)((double)s.grid[cb] * per_id);
    p.narrow = in_bin > kCandMax;
    p.list = ids <= kCandMax;
    p.t_lo = fmaxf(bin_floor(g, cb), t_m);
    p.t_hi = bin_floor(g, cb + 1);
  }
  return p;
}

// Weights of the bins' lower ends under maximum m, times the unit, in s.scale for collect_pass.
__device__ __forceinline__ void scale_table(const Grid &g, float m, double unit, FilterSmem &s) {
  const double xm = g.pos(m);
  for (int b = threadIdx.x; b < kGrid + 64; b += kFilterThreads)
    s.scale[b] = b < kGrid && (double)b <= xm ? unit * exp2_f64(((double)b - xm) * kBinOctaves) : 0.0;
}

// Lists the ids id + i whose values v[i] `take` names. One counter update a wave and vector;
// the lanes' places follow from the ballots.
template <int VE, class F>
__device__ __forceinline__ void list_ids(const float (&v)[VE], int id, F take, FilterSmem &s) {
  u64 m[VE];
  uint32_t count = 0;
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    m[i] = __ballot(take(v[i]));
    count += __popcll(m[i]);
  }
  if (count == 0) return;
  uint32_t at = 0;
  if ((threadIdx.x & 63) == 0) at = atomicAdd(&s.n_cand, count);
  at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    const uint32_t mine = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(m[i] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m[i], 0));
    if (take(v[i]) && mine < kCandMax) s.cand[mine] = rank_word(v[i], id + i);
    at += __popcll(m[i]);
  }
}

// Second pass over vectors j0 .. j1 - 1: lists ids in s.cand (s.n_cand counts them) and, with
// `sums` (s.scale set), adds up the rest of the kept ones: a weight is its bin's scale times
// its weight inside the bin, half the work of an exponential.
template <int N = 8, class E>
__device__ __forceinline__ void collect_pass(const RowView<E> &r, const CutPlan &p, const Grid &g, bool sums, int j0, int j1,
                                             u64 *sum, uint32_t *n, FilterSmem &s) {
  const float lo = p.t_lo, hi = p.list ? INFINITY : p.t_hi;
  auto list = [&](const float (&v)[E::VE], int id) {
    list_ids<E::VE>(v, id, [&](float l) { return l >= lo && l < hi; }, s);
  };
  if (sums && !p.list) {
    uint32_t kept_n = 0;
    u64 kept_w = 0;
    wave_vecs(r, j0, j1, [&](const float (&v)[E::VE], int id) {
#pragma unroll
      for (int i = 0; i < E::VE; ++i) {
        const bool k = v[i] >= hi;
        kept_n += __popcll(__ballot(k));
        // An id that is not kept takes part as the lowest finite value, under the grid.
        const double x = g.pos(k ? v[i] : -3.402823466e38f);
        const uint32_t b = min(whole_part(x), (uint32_t)kGrid);
        const double w = __builtin_fma(bin_weight(__builtin_amdgcn_fract(x)), s.scale[b], 4503599627370496.0);
        kept_w += (u64)__double_as_longlong(w) & 0xfffffffffffffull;
      }
      list(v, id);
    });
    *sum += kept_w;
    *n += (threadIdx.x & 63) == 0 ? kept_n : 0;        // counted once a wave
  } else if (lo < hi) {
    wave_vecs<N>(r, j0, j1, [&](const float (&v)[E::VE], int id) { list(v, id); });
  }
}

// ------------------------------------------------------------------ choosing from the list
// The item of s.cand[0 .. n) at which the running total of weights wt(word), taken in
// descending order of the distinct numbers ord(word), first reaches need (at least 1, at most
// the total): its ord, and the total up to and including it. bucket(word) in [0,
// kFilterThreads) may not fall as ord falls. Two levels: the bucket that holds it, then every
// item of that bucket against every other.
template <class Ord, class Bucket, class Wt>
__device__ __forceinline__ u64 pick(FilterSmem &s, int n, u64 need, Ord ord, Bucket bucket, Wt wt, u64 *upto) {
  const int tid = threadIdx.x;
  __syncthreads();
  s.bucket[tid] = 0;
  if (tid == 0) s.n_sub = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kFilterThreads) {
    const u64 x = s.cand[i], w = wt(x);
    if (w) atomicAdd(&s.bucket[bucket(x)], w);
  }
  __syncthreads();
  const u64 own = s.bucket[tid], before = block_excl_scan_u64(own, s);
  if (before < need && before + own >= need) { s.hit = tid; s.acc = before; }
  __syncthreads();
  const int hit = s.hit;
  for (int i = tid; i < n; i += kFilterThreads) {
    const u64 x = s.cand[i];
    if (bucket(x) != hit) continue;
    const u64 w = wt(x);
    if (!w) continue;
    const uint32_t at = atomicAdd(&s.n_sub, 1u);
    s.sub[at] = ord(x);
    s.sub_w[at] = w;
  }
  __syncthreads();
  const int m = (int)s.n_sub;
  for (int i = tid; i < m; i += kFilterThreads) {
    const u64 x = s.sub[i], w = s.sub_w[i];
    u64 run = s.acc;
#pragma unroll 8
    for (int j = 0; j < m; ++j) run += s.sub[j] > x ? s.sub_w[j] : 0;
    if (run < need && run + w >= need) { s.word = x; s.acc2 = run + w; }
  }
  __syncthreads();
  *upto = s.acc2;
  return s.word;
}

__device__ inline u64 swap_halves(u64 x) { return (x << 32) | (x >> 32); }

// Cuts the list s.cand[0 .. nc) by rank: c.val, c.id, c.n, c.S, given the ids kept without
// ranking (n_above of them, weight c.S). Returns the last listed word that is kept, 0 when
// all are.
__device__ __forceinline__ u64 cut_list(const RowSettings &set, CutKind kind, const CutPlan &p, int nc, uint32_t n_above,
                                        RowCut &c, FilterSmem &s) {
  const int tid = threadIdx.x;
  const u64 mass_above = c.S;
  c.val = p.t_hi; c.id = 0x7fffffff;
  c.n = (int)n_above;
  if (nc == 0) return 0;
  float lo = p.t_lo;
  if (lo == key_value(kKeyNegInf + 1)) {                 // every finite id is listed
    u64 low = 0;
    for (int i = tid; i < nc; i += kFilterThreads) low = ~s.cand[i] > low ? ~s.cand[i] : low;
    lo = word_value(~block_max_u64(low, s));
  }
  const float hi = p.list ? c.m : p.t_hi, per = (float)(kFilterThreads - 1) / (hi - lo);
  auto ord = [](u64 x) { return x; };
  auto bucket = [&](u64 x) { return (int)fminf(fmaxf((hi - word_value(x)) * per, 0.f), (float)(kFilterThreads - 1)); };
  auto mass = [&](u64 x) { return to_fix(weight_finite(word_value(x), c.m, set.sl), set.unit); };
  // Weight and number of the listed words from x up.
  auto totals = [&](u64 x, u64 *n) __attribute__((always_inline)) {
    u64 w = 0, m = 0;
    for (int i = tid; i < nc; i += kFilterThreads) {
      if (s.cand[i] < x) continue;
      w += mass(s.cand[i]);
      ++m;
    }
    *n = block_sum_u64(m, s);
    return block_sum_u64(w, s);
  };
  u64 last = 0, upto, n;
  if (kind == kCutCount && nc > set.k) last = pick(s, nc, (u64)set.k, ord, bucket, [](u64) { return 1ull; }, &upto);
  u64 total = totals(last, &n), need = 0;
  if (kind == kCutCount && set.p < 1.0) need = at_least(set.p * (double)total);
  if (kind == kCutMass && p.need > 0) {
    if (p.need <= mass_above) return ~0ull;              // nothing of the list
    need = p.need - mass_above < total ? p.need - mass_above : total;
  }
  const u64 first = last;
  if (need > 0) last = pick(s, nc, need, ord, bucket, [&](u64 x) { return x >= first ? mass(x) : 0ull; }, &upto);
  // Min-p's own run if it ends earlier, not before top-p's share is taken: that is one of the
  // whole top-k run. Nothing under the list is kept, whatever min-p says.
  if (kind == kCutCount && p.t_m > -INFINITY) {
    const u64 floor = ((u64)sort_key(fmaxf(p.t_m, p.t_lo)) << 32) | (uint32_t)~0x7fffffff;
    last = floor > last ? floor : last;
  }
  if (last != first) total = totals(last, &n);
  c.n = (int)n_above + (int)n;
  c.S = mass_above + total;
  if (last) { c.val = word_value(last); c.id = word_id(last); }
  else { c.val = p.t_lo; c.id = 0x7fffffff; }
  return last;
}

// Where the kept ids' weights are after the cut.
enum RowMode {
  kModeTop,      // at most one id, c.id
  kModeList,     // the words of s.cand[0 .. s.n_cand) from `last` up
  kModeShares,   // s.share, by share of the vectors
  kModeNone,     // not summed yet (c.S unset)
  kModeNarrow    // not cut: the narrowing path's
};

// Adds the kept listed ids' weights to the shares (of `step` vectors) they lie in.
template <class E>
__device__ __forceinline__ void add_listed(const RowView<E> &r, const RowSettings &set, const RowCut &c, int nc, u64 last,
                                           int step, FilterSmem &s) {
  for (int i = threadIdx.x; i < nc; i += kFilterThreads) {
    const u64 x = s.cand[i];
    if (x >= last)
      atomicAdd(&s.share[(word_id(x) - r.off) / E::VE / step], to_fix(weight_finite(word_value(x), c.m, set.sl), set.unit));
  }
}

__device__ inline RowMode cut_top(const RowSettings &set, u64 top, RowCut &c) {
  c.m = word_value(top);
  c.id = word_id(top);
  c.val = top ? c.m : INFINITY;
  c.n = top ? 1 : 0;
  c.S = top ? to_fix(1.0, set.unit) : 0;
  return kModeTop;
}

// First bin from above at which the running count of s.grid reaches need, 0 when none does.
__device__ __forceinline__ int bin_of_count(u64 need, FilterSmem &s) {
  const int tid = threadIdx.x, b0 = kGrid - 1 - kPlan * tid;
  u64 own = 0;
#pragma unroll
  for (int i = 0; i < kPlan; ++i) own += b0 - i > 0 ? (uint32_t)s.grid[b0 - i] : 0;
  if (tid == 0) s.hit = 0;
  u64 run = block_excl_scan_u64(own, s);
  if (run < need && run + own >= need) {
#pragma unroll
    for (int i = 0; i < kPlan; ++i) {
      const u64 n = b0 - i > 0 ? (uint32_t)s.grid[b0 - i] : 0;
      if (run < need && run + n >= need) s.hit = b0 - i;
      run += n;
    }
  }
  __syncthreads();
  return s.hit;
}

// From a sample of the row, 128 runs of eight vectors spread evenly: the largest logit, which
// the grid is laid around, and for a top-k of few ids a logit that somewhat more than k ids of
// the row reach (`guess`; NaN without one). With F the sampled fraction, the sample's rank
// k F + 4 sqrt(k F) + 6 is taken: less than k ids reach it, or more than can be listed, about
// as seldom as a normal variable lies 4 deviations out. Both are noticed; they cost a second
// look at the row, and a row of several workgroups the narrowing path.
template <class E>
__device__ __forceinline__ float row_sample(const RowView<E> &r, const RowSettings &set, CutKind kind, float *guess,
                                            FilterSmem &s) {
  constexpr int U = 1024 / kFilterThreads;
  float v[U][E::VE], ref = -INFINITY;
  const int taken = min(r.nv, 1024);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = threadIdx.x + u * kFilterThreads;
    const int j = r.nv <= 1024 ? i : (int)((int64_t)(i >> 3) * (r.nv - 8) / 127) + (i & 7);
#pragma unroll
    for (int e = 0; e < E::VE; ++e) v[u][e] = -INFINITY;
    if (i < taken) r.load(j, v[u]);
#pragma unroll
    for (int e = 0; e < E::VE; ++e) ref = fmaxf(ref, v[u][e]);
  }
  ref = word_value(block_max_u64(rank_word(ref, 0), s));
  *guess = NAN;
  if (kind != kCutCount) return ref;
  const double share = (double)taken / (double)r.nv, kf = (double)set.k * share;
  const double rank = taken == r.nv ? (double)set.k : kf + 4.0 * sqrt(kf) + 6.0;
  if (rank / share * (1.0 + (taken == r.nv ? 0.0 : 4.0 / sqrt(rank))) > (double)kCandMax) return ref;
  const Grid g(ref, set.T, true);
  if (ref == -INFINITY || ref == INFINITY || !g.fine) return ref;
  for (int b = threadIdx.x; b < kGrid; b += kFilterThreads) s.grid[b] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < E::VE; ++e) {
      const uint32_t b = whole_part(g.pos(v[u][e]));
      if (b > 0 && b < kGrid) atomicAdd(reinterpret_cast<uint32_t *>(&s.grid[b]), 1u);
    }
  __syncthreads();
  const int bin = bin_of_count(at_least(rank), s);
  *guess = bin > 0 ? bin_floor(g, bin) : key_value(kKeyNegInf + 1);
  return ref;
}

// Lists the ids of vectors j0 .. j1 - 1 from `lo` up in s.cand (s.n_cand counts them).
template <int N = 8, class E>
__device__ __forceinline__ void list_pass(const RowView<E> &r, float lo, int j0, int j1, FilterSmem &s) {
  wave_vecs<N>(r, j0, j1, [&](const float (&v)[E::VE], int id) {
    list_ids<E::VE>(v, id, [&](float l) { return l >= lo; }, s);
  });
}

// Whether n ids from `guess` up hold the first k and fit the list.
__device__ inline bool guess_holds(const RowSettings &set, float guess, u64 n) {
  return n <= kCandMax && (n >= (u64)set.k || guess == key_value(kKeyNegInf + 1));
}

// Plan of a row whose ids from `guess` up are listed.
__device__ __forceinline__ CutPlan listed_plan(const RowSettings &set, float guess, float m) {
  const bool narrow = m == INFINITY;
  return {guess, guess, set.min_p > 0.0 && !narrow ? min_p_floor(set, m) : -INFINITY, true, narrow, true, 0, 0, 0};
}

// The cut of one row by one workgroup and the weight of what it keeps; every thread gets both.
//   1. One pass bins the row (bin_pass), around a reference taken from a sample; a row whose
//      largest logit lies past the grid is passed again around that. For a top-k of few ids
//      the sample also gives a logit that slightly more than k ids reach: one pass lists
//      those (list_pass), and if it got them all the row is not passed again.
//   2. The bin that holds the cut, and the smallest logits of it and of the bin above, follow
//      from the bins' totals (make_plan). Both steps: row_plan.
//   3. A second pass lists the ids in that bin and, where a draw follows, sums the weights of
//      those above it by wave; when all kept ids are few they are listed and nothing is
//      summed by pass (collect_pass).
//   4. The list is cut (cut_list). Both steps: row_rest.
// totals: only the kept set and its weight are wanted; the bins give the weight above the cut.
// A row that this leaves to the narrowing path is cut by row_cut_narrowing.
struct RowPlan {
  CutKind kind;
  float ref;       // the grid's reference
  CutPlan plan;
};

// kModeTop: c is the cut; kModeNarrow; else c.m is set and row_rest comes next.
template <class E>
__device__ __forceinline__ RowMode row_plan(const RowView<E> &r, const RowSettings &set, bool totals, RowPlan &o, RowCut &c,
                                            FilterSmem &s) {
  const int tid = threadIdx.x, wave = tid >> 6;
  const int per = (r.nv + kFilterWaves - 1) / kFilterWaves;
  const int j0 = min(r.nv, wave * per), j1 = min(r.nv, j0 + per);
  const CutKind kind = o.kind = cut_kind(set, r.V, totals);
  const bool binned = kind == kCutCount || kind == kCutMass;
  float guess = NAN, ref = binned ? row_sample(r, set, kind, &guess, s) : 0.f;
  if (kind == kCutCount && guess == guess) {
    if (tid == 0) s.n_cand = 0;
    __syncthreads();
    list_pass(r, guess, j0, j1, s);
    __syncthreads();
    const uint32_t n = s.n_cand;
    if (guess_holds(set, guess, n)) {
      u64 top = 0;
      for (uint32_t i = tid; i < n; i += kFilterThreads) top = s.cand[i] > top ? s.cand[i] : top;
      top = block_max_u64(top, s);
      if (!top) return cut_top(set, top, c);
      c.m = word_value(top);
      o.ref = ref;
      o.plan = listed_plan(set, guess, c.m);
      return o.plan.narrow ? kModeNarrow : kModeNone;
    }
    __syncthreads();
  }
  u64 any = 0, top;
  for (int attempt = 0;; ++attempt) {
    const Grid g(ref, set.T, kind == kCutCount);
    if (binned) {
      for (int b = tid; b < kGrid; b += kFilterThreads) s.grid[b] = 0;
      __syncthreads();
    }
    PassOut o;
    bin_pass(r, g, kind, bin_unit(set), j0, j1, o, s);
    top = block_max_u64(rank_word(o.best, o.at), s);
    if (kind == kCutCount) any = block_sum_u64(o.any, s);
    c.m = word_value(top);
    if (!binned || attempt == 1 || !top || (g.fine && g.pos(c.m) < (double)kGrid)) break;
    ref = c.m;
    __syncthreads();
  }
  if (!top || kind == kCutOne) return cut_top(set, top, c);
  __syncthreads();
  o.ref = kind == kCutSum ? c.m : ref;
  o.plan = make_plan(set, kind, Grid(o.ref, set.T, kind == kCutCount), c.m, any, s);
  return o.plan.narrow ? kModeNarrow : kModeNone;
}

template <int N = 8, class E>
__device__ __forceinline__ RowMode row_rest(const RowView<E> &r, const RowSettings &set, bool totals, const RowPlan &o,
                                            RowCut &c, u64 *last, FilterSmem &s) {
  const int tid = threadIdx.x, wave = tid >> 6;
  const int per = (r.nv + kFilterWaves - 1) / kFilterWaves;
  const int j0 = min(r.nv, wave * per), j1 = min(r.nv, j0 + per);
  const CutPlan &p = o.plan;
  const Grid g(o.ref, set.T, o.kind == kCutCount);
  c.S = 0;
  const bool sums = !totals && !p.list;
  __syncthreads();
  if (sums) scale_table(g, c.m, set.unit, s);
  u64 sum = 0;
  uint32_t n_sum = 0;
  if (!p.listed) {
    if (tid == 0) s.n_cand = 0;
    __syncthreads();
    collect_pass<N>(r, p, g, sums, j0, j1, &sum, &n_sum, s);
  }
  if (totals && !p.list) {
    c.S = p.above;
    n_sum = 1;                     // some
  }
  __syncthreads();
  if (sums) {
    sum = wave_sum_u64(sum);
    if ((tid & 63) == 0) s.share[wave] = sum;
    n_sum = (uint32_t)block_sum_u64(n_sum, s);
    for (int w = 0; w < kFilterWaves; ++w) c.S += s.share[w];
  }
  const int nc = min((int)s.n_cand, kCandMax);
  *last = cut_list(set, o.kind, p, nc, n_sum, c, s);
  if (sums) add_listed(r, set, c, nc, *last, per, s);
  __syncthreads();
  return p.list ? kModeList : sums ? kModeShares : kModeNone;
}

template <class E>
__device__ __forceinline__ RowMode row_cut(const RowView<E> &r, const RowSettings &set, RowCut &c, u64 *last, FilterSmem &s) {
  RowPlan o;
  const RowMode mode = row_plan(r, set, false, o, c, s);
  return mode == kModeNone ? row_rest(r, set, false, o, c, last, s) : mode;
}

// The cut of a row that row_cut leaves (c.S unset).
template <class E>
__device__ __forceinline__ void row_cut_narrowing(const RowView<E> &r, const RowSettings &set, bool totals, RowCut &c,
                                                  FilterSmem &s) {
  const int per = (r.nv + kFilterWaves - 1) / kFilterWaves, j0 = min(r.nv, (int)(threadIdx.x >> 6) * per);
  float m = -INFINITY;
  wave_ids<4>(r, j0, min(r.nv, j0 + per), [&](float l, int) { m = fmaxf(m, l); });
  c.m = word_value(block_max_u64(rank_word(m, 0), s));
  c.S = 0;
  cut_narrowing(r, set, totals, c, s);
}

// ------------------------------------------------------------------ the draw
// Weights of vector j's kept ids in id order, 0 for the others.
template <class E>
__device__ inline void kept_weights(const RowView<E> &r, const RowCut &c, const RowSettings &set,
                                    int j, u64 (&w)[E::VE]) {
  float v[E::VE];
  r.load(j, v);
#pragma unroll
  for (int i = 0; i < E::VE; ++i)
    w[i] = v[i] > -INFINITY && kept(c, v[i], r.id(j, i)) ? to_fix(weight(v[i], c.m, set.sl), set.unit) : 0;
}

// Weights f(j, w) of vectors a .. b - 1 summed by shares of *step vectors, a multiple of 64:
// s.share[0 .. *n) afterwards, and their total.
template <int VE, class F>
__device__ __forceinline__ u64 sum_shares(F f, int a, int b, int *n, int *step, FilterSmem &s) {
  const int per = 64 * ((b - a + 64 * kMaxShares - 1) / (64 * kMaxShares)), count = (b - a + per - 1) / per;
  u64 own = 0;
  __syncthreads();
  for (int w = threadIdx.x >> 6; w < count; w += kFilterWaves) {
    u64 m = 0;
    const int j0 = a + w * per, j1 = min(b, j0 + per);
    for (int j = j0 + (int)(threadIdx.x & 63); j < j1; j += 64) {
      u64 x[VE];
      f(j, x);
#pragma unroll
      for (int i = 0; i < VE; ++i) m += x[i];
    }
    own += m;
    m = wave_sum_u64(m);
    if ((threadIdx.x & 63) == 0) s.share[w] = m;
  }
  *n = count;
  *step = per;
  return block_sum_u64(own, s);
}

// The running total that a draw for uniform u of total S > 0 has to reach: the least whole
// number over u S. u outside [0, 1) is taken as the nearest end of the range, NaN as 0.
__device__ inline u64 draw_need(float u, u64 S) {
  const u64 t = (u64)((u >= 1.f ? 0.99999994 : (u > 0.f ? (double)u : 0.0)) * (double)S) + 1;
  return t < S ? t : S;
}

// Position (vector VE + element) of the first weight at which the running sum reaches need,
// given the sums of n contiguous shares of `step` of all nv vectors in s.share: the share that
// holds the crossing is split again until a vector a thread covers it. The shares may come
// from another form of the weights, units apart: a need past the sum of the parts is taken as
// that sum. -1 when nothing there has weight.
template <int VE, class F>
__device__ __forceinline__ int draw_in_shares(F f, int nv, int n, int step, u64 need, FilterSmem &s) {
  const int tid = threadIdx.x;
  int a = 0, b = nv;
  // The running sums over the threads' x: whether this thread's holds the crossing.
  auto crosses = [&](u64 x, u64 *before) __attribute__((always_inline)) {
    *before = block_excl_scan_u64(x, s);
    u64 total = 0;
#pragma unroll
    for (int w = 0; w < kFilterWaves; ++w) total += s.red[w];
    need = need < total ? need : total;
    return *before < need && *before + x >= need;
  };
  u64 before;
  for (;;) {
    if (tid == 0) s.hit = -1;
    if (crosses(tid < n ? s.share[tid] : 0, &before)) { s.hit = tid; s.acc = before; }
    __syncthreads();
    if (s.hit < 0) return -1;
    need -= s.acc;
    a += s.hit * step;
    b = min(b, a + step);
    if (b - a <= kFilterThreads) break;
    sum_shares<VE>(f, a, b, &n, &step, s);
  }
  u64 w[VE], own = 0;
#pragma unroll
  for (int i = 0; i < VE; ++i) w[i] = 0;
  if (a + tid < b) f(a + tid, w);
#pragma unroll
  for (int i = 0; i < VE; ++i) own += w[i];
  if (tid == 0) s.id = -1;
  if (crosses(own, &before)) {
    u64 run = before;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if (run < need && run + w[i] >= need) s.id = (a + tid) * VE + i;
      run += w[i];
    }
  }
  __syncthreads();
  const int at = s.id;
  __syncthreads();
  return at;
}

// Sets c.S when the cut left it out.
template <class E>
__device__ __forceinline__ void row_total(const RowView<E> &r, RowCut &c, const RowSettings &set, FilterSmem &s) {
  if (c.n == 0 || c.S > 0) return;
  int n, step;
  c.S = sum_shares<E::VE>([&](int j, u64 (&w)[E::VE]) { kept_weights(r, c, set, j, w); }, 0, r.nv, &n, &step, s);
}

// The row's draw for uniform u: the smallest kept id whose running weight, in id order, passes
// u times the total (set in c.S when the cut left it out), with its logit; -1 for an empty row.
// n shares of `step` vectors are in s.share in kModeShares, nc words in s.cand in kModeList.
template <class E>
__device__ __forceinline__ int row_draw(const RowView<E> &r, RowCut &c, const RowSettings &set, RowMode mode, int n, int step,
                                        int nc, u64 last, float u, float *l, FilterSmem &s) {
  *l = c.m;
  if (mode == kModeTop) return c.n ? c.id : -1;
  if (mode == kModeList) {
    u64 upto;
    const float per = (float)kFilterThreads / (float)r.V;
    const u64 x = pick(s, nc, draw_need(u, c.S), swap_halves,
                       [&](u64 w) { return min((int)((float)word_id(w) * per), kFilterThreads - 1); },
                       [&](u64 w) { return w >= last ? to_fix(weight_finite(word_value(w), c.m, set.sl), set.unit) : 0ull; }, &upto);
    *l = word_value(swap_halves(x));
    return word_id(swap_halves(x));
  }
  auto f = [&](int j, u64 (&w)[E::VE]) { kept_weights(r, c, set, j, w); };
  if (mode == kModeNone) c.S = sum_shares<E::VE>(f, 0, r.nv, &n, &step, s);
  if (c.n == 0 || c.S == 0) return -1;
  const int at = draw_in_shares<E::VE>(f, r.nv, n, step, draw_need(u, c.S), s);
  if (at < 0) return -1;
  *l = r.at(r.off + at);
  return r.off + at;
}

}  // namespace sdv
