// Sampling under temperature, top-k, top-p and min-p, and rejection acceptance of a
// drafted block whose target and drafter are both filtered that way (gfx950).
//
// DSpark summary, "Problem definition": rejection sampling keeps the output distribution
// that of the target; a server samples its target through these filters, so the target
// distribution of the rule is the filtered one, and the drafter's is whatever its tokens
// were drawn from -- its own filtered one.
#include <math.h>

#include "sd_filter.h"
#include "sd_launch.h"

namespace sdv {
namespace {

// Where rows come from and what becomes of them. with(i, f) calls f(view, settings) for row i
// of the grid, or not at all for a row that is not used; finish() has the row's cut.
struct SampleArgs {
  const void *logits;
  int64_t stride;        // elements from row to row
  int R, V, rows_per;
  const float *u;
  SampleSettings set;
  int32_t *tokens;
  int64_t token_stride;
  int32_t *kept;         // or null
  float *logprob;        // or null
  WsHeader *ws;
};

template <class E>
struct SampleRows {
  SampleArgs a;
  static constexpr bool kTotals = false;
  template <class F>
  __device__ __forceinline__ void with(int row, F f) const {
    f(RowView<E>(reinterpret_cast<const typename E::S *>(a.logits) + row * a.stride, a.V),
      load_settings(a.set, row / a.rows_per, a.V, threadIdx.x == 0 ? a.ws : nullptr));
  }
  __device__ __forceinline__ void finish(int row, const RowView<E> &r, const RowSettings &set, RowCut &c, RowMode mode,
                                         int n, int step, int nc, u64 last, FilterSmem &s) const {
    float l;
    const int id = row_draw(r, c, set, mode, n, step, nc, last, a.u[row], &l, s);
    if (threadIdx.x == 0) {
      if (id < 0) raise_flag(a.ws, SD_FLAG_EMPTY_ROW);
      a.tokens[row * a.token_stride] = id;
      if (a.kept) a.kept[row] = c.n;
      if (a.logprob) {
        float lp = id < 0 ? -INFINITY : 0.f;
        if (id >= 0 && c.n > 1) lp = (float)log(weight(l, c.m, set.sl) * set.unit / (double)c.S);
        a.logprob[row] = lp;
      }
    }
  }
};

// A row after the first of its two passes: its weight S lies in [s_lo, s_hi] (in
// RowSettings::unit), ids from plan.t_hi up are kept and ids under plan.t_lo are not.
struct RowBound {
  CutPlan plan;
  float m, ref;
  double s_lo, s_hi;
  uint32_t open;        // 0: the cut itself is known
  uint32_t pad;
};
static_assert(sizeof(RowBound) == 72, "row bounds are 72 bytes");

struct FilteredArgs {
  const float *logits;           // [cap][V]
  const uint16_t *draft_logits;  // bf16 [B][gamma][V]
  const int32_t *draft_tokens;
  const int32_t *verify_len;
  RowMap rm;
  const float *u_accept, *u_resample;
  SampleSettings set;            // per request
  int V;
  int32_t *accept_len, *next_token;
  int64_t *counters;
  RowCut *cut_p;                 // [B][gamma + 1]
  RowCut *cut_q;                 // [B][gamma]
  RowBound *bound;               // [B (2 gamma + 1)], or null: every cut is exact
  uint32_t *todo;                // rows to be cut: their number, then from word 64 on the rows
  u64 *share;                    // [B][kMaxShares][2] sums of the draw's weights
  WsHeader *ws;
};

// First row of request r, or -1 when rows r .. r + L would leave the row capacity.
__device__ inline int first_row(const RowMap &rm, int r, int L, WsHeader *ws) {
  const int cap = rm.B * (rm.gamma + 1);
  const int base = rm.row_offsets ? rm.row_offsets[r] : r * (rm.gamma + 1);
  if (base < 0 || base >= cap - L) {
    raise_flag(ws, SD_FLAG_ROW_OFFSETS);
    return -1;
  }
  return base;
}

// The B (gamma + 1) target rows, then the B gamma drafter rows.
struct AcceptRows {
  FilteredArgs a;
  static constexpr bool kTotals = true;
  template <class F>
  __device__ __forceinline__ void with(int row, F f) const {
    const int g = a.rm.gamma, targets = a.rm.B * (g + 1);
    const bool draft = row >= targets;
    const int i = draft ? row - targets : row, per = draft ? g : g + 1;
    const int r = i / per, j = i - r * per;
    const int L = clamp_len(a.verify_len, r, g, nullptr);
    const int base = first_row(a.rm, r, L, nullptr);
    if (base < 0 || j > L || (draft && j == L)) return;
    const RowSettings set = load_settings(a.set, r, a.V, nullptr);
    if (draft) f(RowView<ElemBF16>(a.draft_logits + (size_t)i * a.V, a.V), set);
    else f(RowView<ElemF32>(a.logits + (size_t)(base + j) * a.V, a.V), set);
  }
  template <class E>
  __device__ __forceinline__ void finish(int row, const RowView<E> &r, const RowSettings &set, RowCut &c, RowMode, int,
                                         int, int, u64, FilterSmem &s) const {
    row_total(r, c, set, s);
    const int targets = a.rm.B * (a.rm.gamma + 1);
    if (threadIdx.x == 0) (row < targets ? a.cut_p[row] : a.cut_q[row - targets]) = c;
  }
};

// ------------------------------------------------------------------ one workgroup a row
// 1088 rows of 151936 fp32 ids under top-p (662 MB): 360 - 380 us. The first pass takes 151 of
// them (134 without its bins: the rate at which rows arrive), the second, which also forms the
// weights of what is kept and lists the bin of the cut, the rest (100 for the rows alone, as
// more rows are in work than the memory-side cache holds).
// todo[row] says whether the row is left to k_rows_narrow: its code would cost the others
// registers, and with them one workgroup in three on each compute unit.
template <class Rows>
__global__ __launch_bounds__(kFilterThreads, 6) void k_rows(Rows rows, uint32_t *todo) {
  __shared__ FilterSmem s;
  const int row = blockIdx.x;
  if (threadIdx.x == 0) todo[row] = 0;
  rows.with(row, [&](const auto &r, const RowSettings &set) {
    RowCut c;
    u64 last = 0;
    const RowMode mode = row_cut(r, set, c, &last, s);
    if (mode == kModeNarrow) {
      if (threadIdx.x == 0) todo[row] = 1;
      return;
    }
    const int nc = min((int)s.n_cand, kCandMax);
    rows.finish(row, r, set, c, mode, kFilterWaves, (r.nv + kFilterWaves - 1) / kFilterWaves, nc, last, s);
  });
}

template <class Rows>
__global__ __launch_bounds__(kFilterThreads) void k_rows_narrow(Rows rows, const uint32_t *todo) {
  __shared__ FilterSmem s;
  const int row = blockIdx.x;
  if (!todo[row]) return;
  rows.with(row, [&](const auto &r, const RowSettings &set) {
    RowCut c;
    row_cut_narrowing(r, set, Rows::kTotals, c, s);
    rows.finish(row, r, set, c, kModeNone, 0, 0, 0, 0, s);
  });
}

// ------------------------------------------------------------------ several workgroups a row
// For few rows: the steps of row_plan and row_rest as launches, a row's vectors dealt to C
// workgroups in contiguous shares. Bins and lists meet in the workspace through integer
// atomics, whose order does not change a sum; the list is ranked before it is used. No
// workgroup waits for another: the last of a row to arrive goes on with it. One row of 151936
// ids under top-k 50 and top-p: 24.6 us, 6 to sample it, 7 to list, 10 to cut and draw; a
// launch for the cut alone, in place of the last workgroup, made it 25.9.
struct TeamRow {
  u64 top, any;
  uint32_t n_list, n_above;
  float ref, guess;
  uint32_t done;     // workgroups whose bins are in
  uint32_t cut;      // workgroups whose lists and sums are in
  CutPlan plan;
};
static_assert(sizeof(TeamRow) <= 128, "team rows are 128 bytes");

struct Team {
  int C;
  TeamRow *row;       // [R], 128 bytes apart
  u64 *grid;          // [R][kGrid]
  u64 *list;          // [R][kCandMax]
  u64 *share;         // [R][kMaxShares]
  __device__ TeamRow &at(int i) const { return *reinterpret_cast<TeamRow *>(reinterpret_cast<char *>(row) + 128 * (size_t)i); }
};

// Reference of the row's grid, and its counters and bins cleared.
template <class Rows>
__global__ __launch_bounds__(kFilterThreads) void k_team_start(Rows rows, Team t) {
  __shared__ FilterSmem s;
  const int row = blockIdx.y;
  rows.with(row, [&](const auto &r, const RowSettings &set) {
    const CutKind kind = cut_kind(set, r.V, Rows::kTotals);
    const bool binned = kind == kCutCount || kind == kCutMass;
    float guess = NAN;
    const float ref = binned ? row_sample(r, set, kind, &guess, s) : 0.f;
    if (binned && guess != guess)
      for (int b = threadIdx.x; b < kGrid; b += kFilterThreads) t.grid[(size_t)row * kGrid + b] = 0;
    if (threadIdx.x == 0) {
      TeamRow &o = t.at(row);
      o.top = o.any = 0;
      o.n_list = o.n_above = o.done = o.cut = 0;
      o.ref = ref;
      o.guess = guess;
    }
  });
}

// Vectors of the calling wave in workgroup x of the C that a row's vectors are dealt to: share
// 8 x + wave of 8 C.
struct Part {
  int step, j0, j1, share;
  __device__ Part(int nv, int C, int x) {
    step = part_step(nv, C);
    share = x * kFilterWaves + (int)(threadIdx.x >> 6);
    j0 = min(nv, share * step);
    j1 = min(nv, j0 + step);
  }
  __device__ static int part_step(int nv, int C) { return (nv + C * kFilterWaves - 1) / (C * kFilterWaves); }
};

// Adds s.cand[0 .. nc) to the row's list.
__device__ __forceinline__ void append_list(const Team &t, int row, TeamRow &o, uint32_t nc, FilterSmem &s) {
  if (threadIdx.x == 0) s.key = nc ? atomicAdd(&o.n_list, nc) : 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < nc; i += kFilterThreads)
    if (s.key + i < (uint32_t)kCandMax)
      __hip_atomic_store(&t.list[(size_t)row * kCandMax + s.key + i], s.cand[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Counts this workgroup in once its atomics are over; whether it is the row's last. What it
// then takes from the others, it reads by atomics too.
__device__ __forceinline__ bool last_in(uint32_t *count, int C, FilterSmem &s) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) s.n_sub = atomicAdd(count, 1u);
  __syncthreads();
  return s.n_sub == (uint32_t)C - 1;
}

template <class T>
__device__ __forceinline__ T from_all(const T *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Bins by workgroup, then in the workspace. The row's last workgroup to arrive makes the plan.
template <class Rows>
__global__ __launch_bounds__(kFilterThreads, 6) void k_team_bins(Rows rows, Team t) {
  __shared__ FilterSmem s;
  const int row = blockIdx.y, tid = threadIdx.x;
  rows.with(row, [&](const auto &r, const RowSettings &set) {
    const CutKind kind = cut_kind(set, r.V, Rows::kTotals);
    TeamRow &o = t.at(row);
    const Part part(r.nv, t.C, blockIdx.x);
    const float guess = o.guess;
    const bool listed = kind == kCutCount && guess == guess, binned = !listed && (kind == kCutCount || kind == kCutMass);
    u64 *grid = t.grid + (size_t)row * kGrid;
    u64 top = 0, any = 0;
    if (listed) {
      if (tid == 0) s.n_cand = 0;
      __syncthreads();
      list_pass(r, guess, part.j0, part.j1, s);
      __syncthreads();
      any = s.n_cand;
      const uint32_t nc = min((uint32_t)any, (uint32_t)kCandMax);
      for (uint32_t i = tid; i < nc; i += kFilterThreads) top = s.cand[i] > top ? s.cand[i] : top;
      top = block_max_u64(top, s);
      append_list(t, row, o, nc, s);
    } else {
      const Grid g(o.ref, set.T, kind == kCutCount);
      if (binned) {
        for (int b = tid; b < kGrid; b += kFilterThreads) s.grid[b] = 0;
        __syncthreads();
      }
      PassOut out;
      bin_pass(r, g, kind, bin_unit(set), part.j0, part.j1, out, s);
      top = block_max_u64(rank_word(out.best, out.at), s);
      any = kind == kCutCount ? block_sum_u64(out.any, s) : 0;
      __syncthreads();
      if (binned) {
        // Where this workgroup's own counts reach k from above, the row's do: the bins below
        // cannot hold the end of the run.
        const int low = kind == kCutCount ? bin_of_count((u64)set.k, s) : 0;
        for (int b = low + tid; b < kGrid; b += kFilterThreads)
          if (s.grid[b]) atomicAdd(&grid[b], s.grid[b]);
      }
    }
    if (tid == 0) {
      atomicMax(&o.top, top);
      if (any) atomicAdd(&o.any, any);
    }
    if (!last_in(&o.done, t.C, s)) return;
    top = from_all(&o.top);
    any = from_all(&o.any);
    if (!top || kind == kCutOne) return;
    if (listed) {
      CutPlan p = listed_plan(set, guess, word_value(top));
      p.narrow = p.narrow || !guess_holds(set, guess, any);
      if (tid == 0) o.plan = p;
      return;
    }
    if (binned) {
      for (int b = tid; b < kGrid; b += kFilterThreads)
        s.grid[b] = from_all(&grid[b]);
      __syncthreads();
    }
    const float m = word_value(top);
    const CutPlan p = make_plan(set, kind, Grid(kind == kCutSum ? m : o.ref, set.T, kind == kCutCount), m, any, s);
    if (tid == 0) o.plan = p;
  });
}

// Lists and sums by workgroup, where the plan asks for them; the row's last workgroup to arrive
// (or its first, when there is nothing to wait for) cuts the list and finishes the row.
template <class Rows>
__global__ __launch_bounds__(kFilterThreads, 6) void k_team_cut(Rows rows, Team t) {
  __shared__ FilterSmem s;
  const int row = blockIdx.y, tid = threadIdx.x;
  rows.with(row, [&](const auto &r, const RowSettings &set) {
    const CutKind kind = cut_kind(set, r.V, Rows::kTotals);
    TeamRow &o = t.at(row);
    const u64 top = o.top;
    RowCut c;
    c.S = 0;
    c.m = word_value(top);
    const bool one = !top || kind == kCutOne;
    const CutPlan p = o.plan;
    const int step = Part::part_step(r.nv, t.C), shares = t.C * kFilterWaves;
    const bool sums = !Rows::kTotals && !p.list;
    RowMode mode = kModeNone;
    u64 last = 0;
    int nc = 0;
    if (one || p.narrow || p.listed) {
      if (blockIdx.x != 0) return;
    } else {
      const Grid g(kind == kCutSum ? c.m : o.ref, set.T, kind == kCutCount);
      if (sums) scale_table(g, c.m, set.unit, s);
      if (tid == 0) s.n_cand = 0;
      __syncthreads();
      const Part part(r.nv, t.C, blockIdx.x);
      u64 sum = 0;
      uint32_t n = 0;
      collect_pass(r, p, g, sums, part.j0, part.j1, &sum, &n, s);
      if (sums) {
        sum = wave_sum_u64(sum);
        if ((tid & 63) == 0)
          __hip_atomic_store(&t.share[(size_t)row * kMaxShares + part.share], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (n) atomicAdd(&o.n_above, n);       // one lane a wave
      }
      __syncthreads();
      append_list(t, row, o, min(s.n_cand, (uint32_t)kCandMax), s);
      if (!last_in(&o.cut, t.C, s)) return;
    }
    if (one) {
      mode = cut_top(set, top, c);
    } else if (p.narrow) {
      row_cut_narrowing(r, set, Rows::kTotals, c, s);
    } else {
      nc = min(from_all(&o.n_list), (uint32_t)kCandMax);
      for (int i = tid; i < nc; i += kFilterThreads) s.cand[i] = from_all(&t.list[(size_t)row * kCandMax + i]);
      const u64 share = sums && tid < shares ? from_all(&t.share[(size_t)row * kMaxShares + tid]) : 0;
      if (tid < shares) s.share[tid] = share;
      if (sums) c.S = block_sum_u64(share, s);
      else if (!p.list) c.S = p.above;
      __syncthreads();
      last = cut_list(set, kind, p, nc, sums || p.list ? from_all(&o.n_above) : 1, c, s);
      if (sums) add_listed(r, set, c, nc, last, step, s);
      __syncthreads();
      mode = p.list ? kModeList : sums ? kModeShares : kModeNone;
    }
    rows.finish(row, r, set, c, mode, shares, step, nc, last, s);
  });
}

// Workgroups a row's vectors are dealt to: 1024 in all, each with at least 10240 ids (its bins
// cost it the same whatever their number); 1: the row is one workgroup's. Measured (us):
//   128 bf16 rows of 129280 ids, workgroups in all: 512 85, 768 78, 1024 76, 2048 81
//   33 rows of 151936 ids (a block of 16), ids a workgroup: 4096 58, 10240 47, 24576 47
//   one row of 151936 ids: 4096 28.2, 10240 28.6, 24576 31.5
//   1088 rows of 151936 ids: one workgroup 362, two 370 - 377
int team_size(int rows, int V) {
  int c = rows < 1024 ? 1024 / rows : 0;
  if (c > V / 10240) c = V / 10240;
  return c < kMaxShares / kFilterWaves ? c : kMaxShares / kFilterWaves;
}

// Workspace of the rows: a word each for one workgroup a row, else the team's state.
struct TeamLayout {
  size_t row, grid, list, share, end;
  TeamLayout(size_t start, int rows, int V) : row(start), grid(start), list(start), share(start) {
    end = align_up(start + 4 * (size_t)rows, 256);
    if (team_size(rows, V) < 2) return;
    grid = align_up(row + 128 * (size_t)rows, 256);
    list = grid + (size_t)rows * kGrid * sizeof(u64);
    share = list + (size_t)rows * kCandMax * sizeof(u64);
    end = align_up(share + (size_t)rows * kMaxShares * sizeof(u64), 256);
  }
};

template <class Rows>
hipError_t launch_team(const Rows &rows, int n, int V, char *ws, const TeamLayout &l, hipStream_t stream) {
  const int C = team_size(n, V);
  const Team t{C, reinterpret_cast<TeamRow *>(ws + l.row), reinterpret_cast<u64 *>(ws + l.grid),
               reinterpret_cast<u64 *>(ws + l.list), reinterpret_cast<u64 *>(ws + l.share)};
  hipLaunchKernelGGL(k_team_start<Rows>, dim3(1, n), dim3(kFilterThreads), 0, stream, rows, t);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_team_bins<Rows>, dim3(C, n), dim3(kFilterThreads), 0, stream, rows, t);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(k_team_cut<Rows>, dim3(C, n), dim3(kFilterThreads), 0, stream, rows, t);
  return hipGetLastError();
}

template <class Rows>
hipError_t launch_rows(const Rows &rows, int n, int V, char *ws, const TeamLayout &l, hipStream_t stream) {
  if (team_size(n, V) >= 2) return launch_team(rows, n, V, ws, l, stream);
  uint32_t *todo = reinterpret_cast<uint32_t *>(ws + l.row);
  hipLaunchKernelGGL(k_rows<Rows>, dim3(n), dim3(kFilterThreads), 0, stream, rows, todo);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_rows_narrow<Rows>, dim3(n), dim3(kFilterThreads), 0, stream, rows, todo);
  return hipGetLastError();
}

// ------------------------------------------------------------ filtered acceptance
// After the rows' cuts:
//   k_filtered_shares  (request, share): p'_j(x_j) / q'_j(x_j) at each kept position and the
//                      first rejection a_r (every workgroup decides for itself, the first
//                      one writes), then the sum of the draw's weights over one share of the
//                      row: max(0, p' - q') after a rejection, p' for the bonus row;
//   k_filtered_pick    (request): the share that holds the draw, and the id in it.

// Probability of an id with canonical logit l under a row's cut; per = unit / S.
__device__ inline double prob(const RowCut &c, double per, const RowSettings &set, float l, int x) {
  return l > -INFINITY && c.n > 0 && kept(c, l, x) ? weight(l, c.m, set.sl) * per : 0.0;
}

__device__ inline double per_weight(const RowCut &c, const RowSettings &set) {
  return c.n > 0 ? set.unit / (double)c.S : 0.0;
}

// The probability as far as it is known. An open row's bounds are taken 1e-9 wider than the
// sums they come from, which are good to 1e-12.
struct Between { double lo, hi; };
__device__ inline Between prob_between(const RowCut &c, const RowBound *b, const RowSettings &set, float l, int x) {
  if (!b || !b->open) {
    const double p = prob(c, per_weight(c, set), set, l, x);
    return {p, p};
  }
  if (b->plan.narrow) return {0.0, INFINITY};
  if (l < b->plan.t_lo) return {0.0, 0.0};
  const double w = weight(l, b->m, set.sl) * set.unit;
  return {l >= b->plan.t_hi ? w / b->s_hi : 0.0, w / b->s_lo};
}

// Acceptance probability of a token of probabilities p and q: one that the target does not
// keep is rejected, whatever the drafter's. It rises with p and falls with q.
__device__ inline double accept_prob(double p, double q) { return p >= q ? (p > 0.0 ? 1.0 : 0.0) : p / q; }

enum Verdict { kAccept, kReject, kUnsure };

// Position `lane` of request r, whose token is drawn against u.
__device__ __forceinline__ Verdict judge(const FilteredArgs &a, int r, int base, const RowSettings &set) {
  const int lane = threadIdx.x & 63, g = a.rm.gamma;
  const size_t rj = (size_t)r * g + lane;
  const int x = a.draft_tokens[rj];
  if (x < 0 || x >= a.V) return kReject;
  const RowBound *bp = a.bound ? a.bound + rj + r : nullptr;
  const RowBound *bq = a.bound ? a.bound + (size_t)a.rm.B * (g + 1) + rj : nullptr;
  const Between p = prob_between(a.cut_p[rj + r], bp, set, canonical(a.logits[(size_t)(base + lane) * a.V + x]), x);
  const Between q = prob_between(a.cut_q[rj], bq, set, canonical(bf16_to_f32(a.draft_logits[rj * a.V + x])), x);
  const double u = (double)a.u_accept[rj];
  return u < accept_prob(p.lo, q.hi) ? kAccept : !(u < accept_prob(p.hi, q.lo)) ? kReject : kUnsure;
}

// a_r of request r by one wave, lane j deciding position j. Positions up to a_r are sure
// (k_filtered_need); those behind it may say anything.
__device__ __forceinline__ int first_rejection(const FilteredArgs &a, int r, int L, int base, const RowSettings &set) {
  const u64 m = __ballot((int)(threadIdx.x & 63) < L && judge(a, r, base, set) == kReject);
  return m ? __ffsll((long long)m) - 1 : L;
}

// Many rows: two passes over all of them cost twice the bytes, and the second one is needed of
// few. The first pass leaves bounds (k_filtered_bounds) that decide nearly every position: the
// weight of a top-p run is its needed weight and less than one id more, so only a token in the
// bin of the cut or a uniform within some 1e-5 of the border stays open. 128 ragged requests
// of up to 16 drafts, 129280 ids, top-p (some 1800 rows in use, 687 MB): 241 us for the bounds,
// 8 to decide, 42 for the rows that are cut, 66 + 8 for the draws; cutting every row took
// 395 - 440 in place of the first three. Rows of open positions up to the first sure
// rejection, and of that one (or the bonus row), whose distribution is drawn from, are listed
// (k_filtered_need) and cut (k_filtered_cut).
__global__ __launch_bounds__(kFilterThreads, 6) void k_filtered_bounds(AcceptRows rows) {
  __shared__ FilterSmem s;
  const int row = blockIdx.x, tid = threadIdx.x;
  const FilteredArgs &a = rows.a;
  if (row == 0 && tid == 0) a.todo[0] = 0;
  rows.with(row, [&](const auto &r, const RowSettings &set) {
    RowCut c;
    RowPlan o;
    const RowMode mode = row_plan(r, set, true, o, c, s);
    // A count's second pass is needed for its weight; without a cut nothing is left to pass.
    const bool open = mode == kModeNarrow || (mode == kModeNone && o.kind == kCutMass && o.plan.t_lo < o.plan.t_hi);
    if (tid == 0) {
      RowBound b;
      b.open = open;
      if (open) {
        b.plan = o.plan;
        b.m = c.m;
        b.ref = o.ref;
        // A top-p run weighs what it needs, unless min-p ends it earlier, and less than its
        // last id more; any kept set holds the largest logit and what lies above the bin.
        const CutPlan &p = o.plan;
        const double above = fmax((double)p.above, set.unit), need = (double)p.need;
        const double one = weight(p.t_hi, fmaxf(c.m, p.t_hi), set.sl) * set.unit;
        b.s_lo = (p.need && set.min_p == 0.0 ? need : above) * (1.0 - 1e-9);
        b.s_hi = (p.need ? need + one : above + (double)p.in_bin) * (1.0 + 1e-9);
      }
      a.bound[row] = b;
    }
    if (open) return;
    u64 last = 0;
    const RowMode m = mode == kModeNone ? row_rest(r, set, true, o, c, &last, s) : mode;
    rows.finish(row, r, set, c, m, 0, 0, 0, last, s);
  });
}

// Position `lane` of request `blockIdx.x`.
__global__ __launch_bounds__(kWave) void k_filtered_need(FilteredArgs a) {
  const int r = blockIdx.x, g = a.rm.gamma, lane = threadIdx.x;
  const int L = clamp_len(a.verify_len, r, g, nullptr);
  const int base = first_row(a.rm, r, L, nullptr);
  if (base < 0) return;
  const RowSettings set = load_settings(a.set, r, a.V, nullptr);
  const Verdict v = lane < L ? judge(a, r, base, set) : kAccept;
  const u64 rejects = __ballot(v == kReject);
  const int stop = rejects ? __ffsll((long long)rejects) - 1 : L;
  const bool need = lane < L && (lane == stop || (lane < stop && v == kUnsure));
  const uint32_t target = (uint32_t)(r * (g + 1) + lane), draft = (uint32_t)(a.rm.B * (g + 1) + r * g + lane);
  const bool t = need && a.bound[target].open, d = need && a.bound[draft].open;
  const u64 tm = __ballot(t), dm = __ballot(d);
  const uint32_t nt = __popcll(tm), nd = __popcll(dm), bonus = (uint32_t)(r * (g + 1) + L);
  const bool with_bonus = stop == L && a.bound[bonus].open;
  uint32_t at = 0;
  if (lane == 0 && nt + nd + with_bonus) {
    at = atomicAdd(&a.todo[0], nt + nd + with_bonus);
    if (with_bonus) a.todo[64 + at + nt + nd] = bonus;
  }
  at = __builtin_amdgcn_readfirstlane(at);
  const u64 below = (1ull << lane) - 1;
  if (t) a.todo[64 + at + __popcll(tm & below)] = target;
  if (d) a.todo[64 + at + nt + __popcll(dm & below)] = draft;
}

__global__ __launch_bounds__(kFilterThreads, 4) void k_filtered_cut(AcceptRows rows) {
  __shared__ FilterSmem s;
  const uint32_t n = rows.a.todo[0];
  for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int row = (int)rows.a.todo[64 + i];
    rows.with(row, [&](const auto &r, const RowSettings &set) {
      RowBound &b = rows.a.bound[row];
      RowCut c;
      u64 last = 0;
      if (b.plan.narrow) {
        row_cut_narrowing(r, set, true, c, s);
      } else {
        c.m = b.m;
        const RowPlan o{kCutMass, b.ref, b.plan};
        row_rest<32>(r, set, true, o, c, &last, s);
      }
      rows.finish(row, r, set, c, kModeNone, 0, 0, 0, last, s);
      __syncthreads();
      if (threadIdx.x == 0) b.open = 0;
    });
  }
}

// Residual weights are summed in units of 2^-51: they add up to at most 1 (and a little), so a
// sum over 2^21 ids is off by 2^-31 of a unit row at the very worst, 2^-42 for random roundings.
constexpr double kResidualUnit = 2251799813685248.0;

// Weights of vector j of target row v in id order: max(0, p' - q'), and p' alone (wp), which is
// drawn from when the former have no mass. All in kResidualUnit. has_q false: p' as both.
struct Residual {
  RowView<ElemF32> v;
  const uint16_t *q;
  RowCut cp, cq;
  RowSettings set;
  double pp, pq;
  __device__ Residual(const FilteredArgs &a, const RowView<ElemF32> &v_, int r, int acc, bool has_q, const RowCut &cp_,
                      const RowSettings &set_)
      : v(v_), q(has_q ? a.draft_logits + ((size_t)r * a.rm.gamma + acc) * a.V : nullptr), cp(cp_), set(set_) {
    pp = per_weight(cp, set);
    pq = 0.0;
    if (q) {
      cq = a.cut_q[(size_t)r * a.rm.gamma + acc];
      pq = per_weight(cq, set);
    }
  }
  __device__ void raw_q(int j, uint2 &h) const {
    const int x0 = v.id(j, 0);
    if (v.whole(j) && (reinterpret_cast<uintptr_t>(q + x0) & 7) == 0) {
      h = *reinterpret_cast<const uint2 *>(q + x0);
    } else {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = x0 + i >= 0 && x0 + i < v.V ? q[x0 + i] : 0;
      h = uint2{b[0] | b[1] << 16, b[2] | b[3] << 16};
    }
  }
  __device__ void weights(int j, const float (&l)[4], const uint2 &h, u64 (&w)[4], u64 (&wp)[4]) const {
    const float lq[4] = {__uint_as_float(h.x << 16), __uint_as_float(h.x & 0xffff0000u), __uint_as_float(h.y << 16),
                         __uint_as_float(h.y & 0xffff0000u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = wp[i] = 0;
      const double p = prob(cp, pp, set, l[i], v.id(j, i));
      if (p > 0.0) {
        w[i] = wp[i] = to_fix(p, kResidualUnit);
        if (q) w[i] = to_fix(fmax(p - prob(cq, pq, set, canonical(lq[i]), v.id(j, i)), 0.0), kResidualUnit);
      }
    }
  }
  __device__ void operator()(int j, bool only_p, u64 (&w)[4]) const {
    float l[4];
    uint2 h = {0u, 0u};
    v.load(j, l);
    if (q) raw_q(j, h);
    u64 wp[4];
    weights(j, l, h, w, wp);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = only_p ? wp[i] : w[i];
  }
};

__global__ __launch_bounds__(kFilterThreads, 6) void k_filtered_shares(FilteredArgs a) {
  const int r = blockIdx.x, part = blockIdx.y, g = a.rm.gamma, tid = threadIdx.x;
  WsHeader *ws = part == 0 && tid == 0 ? a.ws : nullptr;
  const int L = clamp_len(a.verify_len, r, g, ws);
  const int base = first_row(a.rm, r, L, ws);
  const RowSettings set = load_settings(a.set, r, a.V, ws);
  if (base < 0) {
    if (part == 0 && tid == 0) { a.accept_len[r] = 0; a.next_token[r] = -1; }
    return;
  }
  const int acc = first_rejection(a, r, L, base, set);   // the same in every wave
  if (part == 0 && tid == 0) {
    a.accept_len[r] = acc;
    if (a.counters) {
      atomicAdd(reinterpret_cast<u64 *>(a.counters), (u64)L);
      atomicAdd(reinterpret_cast<u64 *>(a.counters + 1), (u64)acc);
    }
  }
  const RowView<ElemF32> v(a.logits + (size_t)(base + acc) * a.V, a.V);
  const RowCut cp = a.cut_p[(size_t)r * (g + 1) + acc];
  const Part mine(v.nv, gridDim.y, part);
  const Residual f(a, v, r, acc, acc < L, cp, set);
  // Two vectors of both rows a lane are in flight.
  u64 sum = 0, sum_p = 0;
  for (int j = mine.j0 + (tid & 63); j < mine.j1; j += 2 * kWave) {
    float l[2][4];
    uint2 h[2] = {{0u, 0u}, {0u, 0u}};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int jj = min(j + u * kWave, mine.j1 - 1);
      v.load(jj, l[u]);
      if (f.q) f.raw_q(jj, h[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (j + u * kWave < mine.j1) {
        u64 w[4], wp[4];
        f.weights(j + u * kWave, l[u], h[u], w, wp);
        sum += (w[0] + w[1]) + (w[2] + w[3]);
        sum_p += (wp[0] + wp[1]) + (wp[2] + wp[3]);
      }
    }
  }
  sum = wave_sum_u64(sum);
  sum_p = wave_sum_u64(sum_p);
  if ((tid & 63) == 0) {
    a.share[((size_t)r * kMaxShares + mine.share) * 2] = sum;
    a.share[((size_t)r * kMaxShares + mine.share) * 2 + 1] = sum_p;
  }
}

__global__ __launch_bounds__(kFilterThreads) void k_filtered_pick(FilteredArgs a, int shares) {
  __shared__ FilterSmem s;
  const int r = blockIdx.x, g = a.rm.gamma, tid = threadIdx.x;
  const int L = clamp_len(a.verify_len, r, g, nullptr);
  const int base = first_row(a.rm, r, L, nullptr);
  if (base < 0) return;
  const int acc = a.accept_len[r];
  const RowSettings set = load_settings(a.set, r, a.V, nullptr);
  const RowView<ElemF32> v(a.logits + (size_t)(base + acc) * a.V, a.V);
  RowCut cp = a.cut_p[(size_t)r * (g + 1) + acc];
  const float u = a.u_resample[(size_t)r * (g + 1) + acc];
  u64 w = 0, wp = 0;
  if (tid < shares) {
    w = a.share[((size_t)r * kMaxShares + tid) * 2];
    wp = a.share[((size_t)r * kMaxShares + tid) * 2 + 1];
  }
  u64 S = block_sum_u64(w, s);
  const bool only_p = S == 0;        // no residual mass: the target's own distribution
  if (only_p) {
    S = block_sum_u64(wp, s);
    w = wp;
  }
  if (tid < shares) s.share[tid] = w;
  __syncthreads();
  int id = -1;
  if (S > 0) {
    if (only_p && tid == 0) raise_flag(a.ws, SD_FLAG_NO_RESIDUAL);
    const Residual f(a, v, r, acc, acc < L, cp, set);
    const int at = draw_in_shares<4>([&](int j, u64 (&x)[4]) { f(j, only_p, x); }, v.nv, shares,
                                     Part::part_step(v.nv, shares / kFilterWaves), draw_need(u, S), s);
    if (at >= 0) id = v.off + at;
  }
  if (tid == 0) {
    if (id < 0) raise_flag(a.ws, SD_FLAG_EMPTY_ROW);
    a.next_token[r] = id;
  }
}

// Workgroups that sum the draw's row of a request, at least 2048 ids each, 1024 in all: one
// request of 151936 ids 9 us, 128 requests of 129280 66 us.
int draw_shares(int B, int V) {
  int c = B < 1024 ? 1024 / B : 1;
  if (c > V / 2048) c = V / 2048;
  return c < 1 ? 1 : (c > kMaxShares / kFilterWaves ? kMaxShares / kFilterWaves : c);
}

struct FilteredLayout {
  size_t cut_p, cut_q, share;
  TeamLayout team;
  size_t bound, todo, end;
  FilteredLayout(int B, int gamma, int V)
      : cut_p(sizeof(WsHeader)),
        cut_q(align_up(cut_p + (size_t)B * (gamma + 1) * sizeof(RowCut), 256)),
        share(align_up(cut_q + (size_t)B * gamma * sizeof(RowCut), 256)),
        team(align_up(share + (size_t)B * kMaxShares * 2 * sizeof(u64), 256), B * (2 * gamma + 1), V),
        bound(team.row), todo(team.row), end(team.end) {
    const size_t rows = (size_t)B * (2 * gamma + 1);
    if (team_size((int)rows, V) >= 2) return;
    todo = align_up(bound + rows * sizeof(RowBound), 256);
    end = align_up(todo + (64 + rows) * sizeof(uint32_t), 256);
  }
};

}  // namespace

size_t sample_workspace_layout(int R, int V) { return TeamLayout(sizeof(WsHeader), R, V).end; }

hipError_t launch_sample(const void *logits, int32_t type, int64_t stride, int R, int V,
                         const float *u, const SampleSettings &set, int rows_per,
                         int32_t *tokens, int64_t token_stride, int32_t *kept, float *logprob,
                         void *workspace, hipStream_t stream) {
  const SampleArgs a{logits, stride, R, V, rows_per, u, set, tokens, token_stride, kept, logprob,
                     reinterpret_cast<WsHeader *>(workspace)};
  char *ws = reinterpret_cast<char *>(workspace);
  const TeamLayout l(sizeof(WsHeader), R, V);
  if (type == SD_F32) return launch_rows(SampleRows<ElemF32>{a}, R, V, ws, l, stream);
  if (type == SD_BF16) return launch_rows(SampleRows<ElemBF16>{a}, R, V, ws, l, stream);
  return launch_rows(SampleRows<ElemF16>{a}, R, V, ws, l, stream);
}

size_t accept_filtered_workspace_layout(int B, int gamma, int V) { return FilteredLayout(B, gamma, V).end; }

hipError_t launch_accept_filtered(const float *logits, const uint16_t *draft_logits,
                                  const int32_t *draft_tokens, const int32_t *verify_len,
                                  const RowMap &rm, const float *u_accept,
                                  const float *u_resample, const SampleSettings &set, int V,
                                  int32_t *accept_len, int32_t *next_token, int64_t *counters,
                                  void *workspace, hipStream_t stream) {
  const FilteredLayout l(rm.B, rm.gamma, V);
  char *w = reinterpret_cast<char *>(workspace);
  const int rows = rm.B * (2 * rm.gamma + 1);
  const bool team = team_size(rows, V) >= 2;
  const FilteredArgs a{logits, draft_logits, draft_tokens, verify_len, rm, u_accept, u_resample, set, V,
                       accept_len, next_token, counters, reinterpret_cast<RowCut *>(w + l.cut_p),
                       reinterpret_cast<RowCut *>(w + l.cut_q), team ? nullptr : reinterpret_cast<RowBound *>(w + l.bound),
                       reinterpret_cast<uint32_t *>(w + l.todo), reinterpret_cast<u64 *>(w + l.share),
                       reinterpret_cast<WsHeader *>(workspace)};
  hipError_t e;
  if (team) {
    e = launch_team(AcceptRows{a}, rows, V, w, l.team, stream);
  } else {
    hipLaunchKernelGGL(k_filtered_bounds, dim3(rows), dim3(kFilterThreads), 0, stream, AcceptRows{a});
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(k_filtered_need, dim3(rm.B), dim3(kWave), 0, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(k_filtered_cut, dim3(rows < 512 ? rows : 512), dim3(kFilterThreads), 0, stream, AcceptRows{a});
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  const int shares = draw_shares(rm.B, V);
  hipLaunchKernelGGL(k_filtered_shares, dim3(rm.B, shares), dim3(kFilterThreads), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(k_filtered_pick, dim3(rm.B), dim3(kFilterThreads), 0, stream, a, shares * kFilterWaves);
  return hipGetLastError();
}

}  // namespace sdv
