// Filtered softmax of a logit row: temperature, top-k, top-p, min-p (gfx950).
//
// With m the row's largest logit, a logit l weighs w = 2^((l - m) log2(e) / T) in [0, 1].
// Rank the ids by larger logit, then lower id. Each filter keeps a leading run of that
// order, so their combination keeps the first n ids, n = min(n_k, n_p, n_m):
//   n_k = k;  n_p = shortest run whose weight reaches p times the weight of the first n_k;
//   n_m = ids with w >= min_p.
// The kept set is then stated by its last member alone: the pair (key, id) of a RowCut.
//
// Weights are formed in fp64 (relative error about 1e-14) and summed as 64-bit integers in
// units of 2^-b: integer sums do not depend on order, so results are the same whatever
// the split over lanes, waves and workgroups, and every running sum is exact in those
// units. b is 46, less for rows of more than 2^17 ids so that V 2^b stays under 2^63. One
// weight's rounding is at most 2^-(b+1) of the row's largest, a few 1e-12 of the total
// over a whole row, and a weight under 2^-47 counts as 0.
//
// The functions that hold workgroup barriers are forced inline: as calls they spill and read
// LDS through flat addresses.
#pragma once

#include <math.h>

#include "sd_internal.h"

namespace sdv {

constexpr int kFilterThreads = 1024;
constexpr int kFilterWaves = kFilterThreads / kWave;
constexpr int kBins = 2048;          // linear bins of the mass histogram
constexpr int kCandMax = 4096;       // ids of a cut bin that are ranked in LDS
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

// What keeps an id of a row: sort key above `key`, or equal to it and id <= `id`.
struct RowCut {
  float m;        // largest logit of the row, -inf when the row has none
  uint32_t key;
  int32_t id;
  int32_t n;      // ids kept
  u64 S;          // their weight, in RowSettings::unit
  int32_t top;    // lowest id that attains m, -1 when the row has none
  int32_t pad;
};
static_assert(sizeof(RowCut) == 32, "row cuts are 32 bytes");

// ------------------------------------------------------------------ elements
// NaN counts as -inf (never kept) and -0 as +0, so that equal values have equal keys.
__device__ inline float canonical(float x) { return x != x ? -INFINITY : x + 0.f; }

// Order-preserving bits: a > b <=> sort_key(a) > sort_key(b) for canonical values.
__device__ inline uint32_t sort_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ inline float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

struct ElemF32 {
  using S = float;
  static constexpr int VE = 4;
  __device__ static float get(S x) { return x; }
  __device__ static void unpack(u32x4 q, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(q[i]);
  }
};

struct ElemBF16 {
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
  // Canonical values of vector j, -inf outside the row.
  __device__ void load(int j, float (&v)[E::VE]) const {
    const int b = off + j * E::VE;
    if (b >= 0 && b + E::VE <= V) {
      E::unpack(*reinterpret_cast<const u32x4 *>(p + b), v);
    } else {
#pragma unroll
      for (int i = 0; i < E::VE; ++i) v[i] = b + i >= 0 && b + i < V ? E::get(p[b + i]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < E::VE; ++i) v[i] = canonical(v[i]);
  }
};

// f(value, id) for the ids of vectors j0 .. j1 - 1, taken by the calling wave in order;
// four vectors a lane are in flight at once.
template <class E, class F>
__device__ inline void wave_ids(const RowView<E> &r, int j0, int j1, F f) {
  const int lane = threadIdx.x & 63;
  constexpr int U = E::VE == 4 ? 2 : 1;
  int j = j0 + lane;
  for (; j + 64 * (U - 1) < j1; j += 64 * U) {
    float v[U][E::VE];
#pragma unroll
    for (int u = 0; u < U; ++u) r.load(j + 64 * u, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < E::VE; ++i) f(v[u][i], r.id(j + 64 * u, i));
  }
  for (; j < j1; j += 64) {
    float v[E::VE];
    r.load(j, v);
#pragma unroll
    for (int i = 0; i < E::VE; ++i) f(v[i], r.id(j, i));
  }
}

// ------------------------------------------------------------------ weights
// 2^x for x <= 0 in fp64: 2^n times the Taylor series of e^(f ln 2), |f| <= 1/2. The first
// term left out, (ln(2) / 2)^12 / 12!, is 6e-15.
__device__ inline double exp2_neg(double x) {
  if (x < -1000.0) return 0.0;
  const double n = __builtin_rint(x);
  const double y = (x - n) * 0.6931471805599453;
  double s = 1.0 / 39916800.0;
  s = __builtin_fma(s, y, 1.0 / 3628800.0);
  s = __builtin_fma(s, y, 1.0 / 362880.0);
  s = __builtin_fma(s, y, 1.0 / 40320.0);
  s = __builtin_fma(s, y, 1.0 / 5040.0);
  s = __builtin_fma(s, y, 1.0 / 720.0);
  s = __builtin_fma(s, y, 1.0 / 120.0);
  s = __builtin_fma(s, y, 1.0 / 24.0);
  s = __builtin_fma(s, y, 1.0 / 6.0);
  s = __builtin_fma(s, y, 0.5);
  s = __builtin_fma(s, y, 1.0);
  s = __builtin_fma(s, y, 1.0);
  return __builtin_ldexp(s, (int)n);
}

// Weight of logit l under row maximum m. The maximum itself weighs 1 also when infinite.
__device__ inline double weight(float l, float m, double sl) {
#pragma clang fp contract(off)
  return l == m ? 1.0 : exp2_neg(((double)l - (double)m) * sl);
}

// w * unit rounded to nearest, for results under 2^52: the fp64 sum's low 52 bits hold it.
__device__ inline u64 to_fix(double w, double unit) {
  const double s = __builtin_fma(w, unit, 4503599627370496.0);
  return (u64)__double_as_longlong(s) & 0xfffffffffffffull;
}

__device__ inline bool kept(const RowCut &c, float l, int id) {
  const uint32_t k = sort_key(l);
  return k > c.key || (k == c.key && id <= c.id);
}

// ------------------------------------------------------------------ workgroup sums
__device__ inline u64 wave_sum_u64(u64 x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

__device__ inline u64 wave_incl_scan_u64(u64 x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const u64 o = __shfl_up(x, off);
    if (lane >= off) x += o;
  }
  return x;
}

// Shared memory of one workgroup's row.
struct FilterSmem {
  u64 mass[kBins];
  uint32_t cnt[kBins];
  u64 cand[kCandMax];
  u64 red[kFilterWaves];
  u64 red2[kFilterWaves];
  uint32_t n_cand;
  int hit;
  uint32_t key;
  int32_t id;
  u64 acc, acc2;
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

// s.cand[0 .. n), n a power of two, sorted in descending order.
__device__ __forceinline__ void sort_desc(FilterSmem &s, int n) {
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

// ------------------------------------------------------------------ the cut
// Largest logit of the row, the lowest id that attains it (-1 in a row without any), and the
// count of ids above -inf.
template <class E>
__device__ __forceinline__ void row_max(const RowView<E> &r, FilterSmem &s, float *m, int *top, int *n) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (r.nv + kFilterWaves - 1) / kFilterWaves;
  float best = -INFINITY;
  int at = 0x7fffffff;
  uint32_t any = 0;
  wave_ids(r, wave * per, min(r.nv, wave * per + per), [&](float l, int id) {
    if (l > best) { best = l; at = id; }
    any += l > -INFINITY;
  });
  *n = (int)block_sum_u64(any, s);
  // Larger key first, then lower id.
  u64 k = best > -INFINITY ? ((u64)sort_key(best) << 32) | (uint32_t)~at : 0;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const u64 o = __shfl_xor(k, off);
    k = o > k ? o : k;
  }
  __syncthreads();
  if (lane == 0) s.red[wave] = k;
  __syncthreads();
  for (int w = 0; w < kFilterWaves; ++w) k = s.red[w] > k ? s.red[w] : k;
  __syncthreads();
  *m = k ? key_value((uint32_t)(k >> 32)) : -INFINITY;
  *top = k ? (int)~(uint32_t)k : -1;
}

// Bins of the mass histogram: equal steps of (m - l), which falls as the rank rises, over
// max(33 T, 16). A logit past that range weighs under 2^-47 (33 T are 47.6 octaves), so its
// summed weight is 0 and no filter but the count of top-k can reach it: those ids are
// counted, not binned. Equal steps spread a row's logits over many bins, so that lanes
// seldom meet on one LDS counter and a bin holds few ids to rank.
struct BinScale {
  float m, scale;
  __device__ BinScale(float m_, float T) : m(m_), scale((float)(kBins - 1) / fmaxf(33.f * T, 16.f)) {}
  // Bin of a logit, kBins - 1 and up: past the range.
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
  const int b = 2 * threadIdx.x;
  const u64 x0 = f(b), x1 = f(b + 1);
  const u64 ex = block_excl_scan_u64(x0 + x1, s);
  if (threadIdx.x == 0) { s.hit = kBins; s.acc = 0; }
  __syncthreads();
  // Exactly one bin has before < need <= before + own (need >= 1).
  if (ex < need && ex + x0 >= need) { s.hit = b; s.acc = ex; }
  else if (ex + x0 < need && ex + x0 + x1 >= need) { s.hit = b + 1; s.acc = ex + x0; }
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
    wave_ids(r, j0, j1, [&](float l, int) {
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
      wave_ids(r, w0, w1, [&](float l, int) { c += l > -INFINITY && sort_key(l) == prefix; });
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
  wave_ids(r, j0, j1, [&](float l, int id) {
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
  // Thread t holds ranks 4 t .. 4 t + 3.
  u64 w[4], own = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = 4 * tid + i;
    w[i] = at < n ? to_fix(weight(key_value((uint32_t)(s.cand[at] >> 32)), bins.m, set.sl), set.unit) : 0;
    own += w[i];
  }
  u64 run = mass_before + block_excl_scan_u64(own, s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = 4 * tid + i;
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

// The cut of one row; every thread of the workgroup gets it. The pass over the row that
// forms the histogram is left out when neither top-k nor top-p is set. S is set only by
// row_mass.
template <class E>
__device__ __forceinline__ RowCut row_cut(const RowView<E> &r, const RowSettings &set, FilterSmem &s) {
  const int tid = threadIdx.x, wave = tid >> 6;
  RowCut c;
  c.S = 0;
  c.pad = 0;
  row_max(r, s, &c.m, &c.top, &c.n);
  if (c.top < 0) {                       // nothing to keep: every id is masked
    c.key = 0xffffffffu; c.id = -1; c.n = 0;
    return c;
  }
  if (set.greedy || set.k == 1 || set.p <= 0.0) {
    c.key = sort_key(c.m); c.id = c.top; c.n = 1;
    return c;
  }
  c.key = kKeyNegInf; c.id = -1;
  if (set.k >= r.V && set.p >= 1.0 && set.min_p <= 0.0) return c;
  const int per = (r.nv + kFilterWaves - 1) / kFilterWaves;
  const int j0 = wave * per, j1 = min(r.nv, j0 + per);
  const BinScale bins(c.m, set.T);
  const bool ranks = set.k < r.V || set.p < 1.0;
  for (int b = tid; b < kBins; b += kFilterThreads) { s.mass[b] = 0; s.cnt[b] = 0; }
  __syncthreads();
  uint32_t n_m = 0, low = 0xffffffffu, past = 0;
  wave_ids(r, j0, j1, [&](float l, int) {
    if (l == -INFINITY) return;
    const double w = weight(l, c.m, set.sl);
    if (w >= set.min_p) { ++n_m; low = min(low, sort_key(l)); }
    if (!ranks) return;
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
  if (set.min_p > 0.0) { c.key = low; c.id = 0x7fffffff; }
  if (ranks) {
    u64 mass_k, n_k = (u64)set.k, cnt_before, mass_before;
    u64 total = 0, in_bins = 0;
    for (int b = tid; b < kBins; b += kFilterThreads) { total += s.mass[b]; in_bins += s.cnt[b]; }
    total = block_sum_u64(total, s);
    in_bins = block_sum_u64(in_bins, s);
    CutAt at{kKeyNegInf, -1, in_bins + past, total};
    if (n_k < in_bins) {
      const int kb = find_bin(s, n_k, [&](int b) { return (u64)s.cnt[b]; }, &cnt_before);
      mass_before = 0;
      for (int b = tid; b < kb; b += kFilterThreads) mass_before += s.mass[b];
      mass_before = block_sum_u64(mass_before, s);
      at = cut_in_bin(r, s, bins, set, kb, false, n_k, cnt_before, mass_before);
    } else if (n_k < in_bins + past) {
      // The run ends among ids without weight: they count, and cannot be drawn.
      at.n = n_k;
    }
    mass_k = at.mass;
    if (set.p < 1.0) {
      // The histogram again: narrowing the top-k cut may have overwritten it.
      const u64 need = at_least(set.p * (double)mass_k);
      for (int b = tid; b < kBins; b += kFilterThreads) { s.mass[b] = 0; s.cnt[b] = 0; }
      __syncthreads();
      wave_ids(r, j0, j1, [&](float l, int) {
        if (l == -INFINITY) return;
        const int b = bins.of(l);
        if (b == kBins - 1) return;
        atomicAdd(&s.cnt[b], 1u);
        atomicAdd(&s.mass[b], to_fix(weight(l, c.m, set.sl), set.unit));
      });
      __syncthreads();
      const int pb = find_bin(s, need, [&](int b) { return s.mass[b]; }, &mass_before);
      cnt_before = 0;
      for (int b = tid; b < pb; b += kFilterThreads) cnt_before += s.cnt[b];
      cnt_before = block_sum_u64(cnt_before, s);
      const CutAt q = cut_in_bin(r, s, bins, set, pb, true, need, cnt_before, mass_before);
      if (q.n < at.n) at = q;
    }
    // The shorter of the two runs.
    if (at.n < n) {
      n = at.n;
      c.key = at.key;
      c.id = at.id;
    }
  }
  c.n = (int)n;
  return c;
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

// Sum of f's weights over vectors a .. b - 1, dealt to the waves in contiguous shares of
// `step` vectors; s.red holds each wave's part afterwards. f(j, w) gives vector j's weights.
template <int VE, class F>
__device__ __forceinline__ u64 range_mass(F f, int a, int b, int step, FilterSmem &s) {
  const int w0 = a + (int)(threadIdx.x >> 6) * step, w1 = min(b, w0 + step);
  u64 m = 0;
#pragma unroll 2
  for (int j = w0 + (int)(threadIdx.x & 63); j < w1; j += 64) {
    u64 w[VE];
    f(j, w);
#pragma unroll
    for (int i = 0; i < VE; ++i) m += w[i];
  }
  return block_sum_u64(m, s);
}

// Position (vector VE + element) of the first weight whose running sum passes u times the
// total *S, -1 when the total is 0: shares of the vectors are summed by wave, and the
// share that holds the crossing is split again until one wave load covers it. u outside
// [0, 1) is taken as the nearest end of the range, NaN as 0.
template <int VE, class F>
__device__ __forceinline__ int split_draw(F f, int nv, float u, u64 *S, FilterSmem &s) {
  int a = 0, b = nv, step = (b + kFilterWaves - 1) / kFilterWaves;
  *S = range_mass<VE>(f, a, b, step, s);
  if (*S == 0) return -1;
  const double t = (u >= 1.f ? 0.99999994 : (u > 0.f ? (double)u : 0.0)) * (double)*S;
  u64 before = 0;
  for (;;) {
    int w = 0;
    while (w < kFilterWaves - 1 && !((double)(before + s.red[w]) > t)) before += s.red[w++];
    a += w * step;
    b = min(b, a + step);
    if (b - a <= 64) break;
    step = (b - a + kFilterWaves - 1) / kFilterWaves;
    range_mass<VE>(f, a, b, step, s);
  }
  if (threadIdx.x < 64) {
    const int j = a + threadIdx.x;
    u64 w[VE], own = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) w[i] = 0;
    if (j < b) f(j, w);
#pragma unroll
    for (int i = 0; i < VE; ++i) own += w[i];
    u64 run = before + wave_incl_scan_u64(own) - own;
    // The total passes t (u < 1), so exactly one lane crosses it.
    if (!((double)run > t) && (double)(run + own) > t) {
      bool done = false;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        run += w[i];
        if (!done && (double)run > t) { s.id = j * VE + i; done = true; }
      }
    }
  }
  __syncthreads();
  const int at = s.id;
  __syncthreads();
  return at;
}

// Sets c.S and returns the row's draw for uniform u: the smallest kept id whose running
// weight, in id order, passes u times the total; -1 for an empty row.
template <class E>
__device__ __forceinline__ int row_draw(const RowView<E> &r, RowCut &c, const RowSettings &set, float u,
                        FilterSmem &s) {
  if (c.n <= 1) {
    c.S = c.n ? to_fix(1.0, set.unit) : 0;
    return c.n ? c.top : -1;
  }
  const int at = split_draw<E::VE>([&](int j, u64 (&w)[E::VE]) { kept_weights(r, c, set, j, w); },
                                   r.nv, u, &c.S, s);
  return r.off + at;
}

// Sets c.S alone.
template <class E>
__device__ __forceinline__ void row_total(const RowView<E> &r, RowCut &c, const RowSettings &set, FilterSmem &s) {
  if (c.n <= 1) {
    c.S = c.n ? to_fix(1.0, set.unit) : 0;
    return;
  }
  c.S = range_mass<E::VE>([&](int j, u64 (&w)[E::VE]) { kept_weights(r, c, set, j, w); }, 0, r.nv,
                          (r.nv + kFilterWaves - 1) / kFilterWaves, s);
}

}  // namespace sdv
