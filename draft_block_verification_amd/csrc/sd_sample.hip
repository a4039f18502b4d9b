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

// One workgroup per row.
template <class E>
__global__ __launch_bounds__(kFilterThreads, 4) void k_sample(SampleArgs a) {
  __shared__ FilterSmem s;
  const int row = blockIdx.x;
  const RowView<E> r(reinterpret_cast<const typename E::S *>(a.logits) + row * a.stride, a.V);
  const RowSettings set = load_settings(a.set, row / a.rows_per, a.V, threadIdx.x == 0 ? a.ws : nullptr);
  RowCut c;
  const RowMode mode = row_cut(r, set, false, c, s);
  const int id = row_draw(r, c, set, mode, kFilterWaves, (r.nv + kFilterWaves - 1) / kFilterWaves, a.u[row], s);
  if (threadIdx.x == 0) {
    if (id < 0) raise_flag(a.ws, SD_FLAG_EMPTY_ROW);
    a.tokens[row * a.token_stride] = id;
    if (a.kept) a.kept[row] = c.n;
    if (a.logprob) {
      float lp = id < 0 ? -INFINITY : 0.f;
      if (c.n > 1) {
        const double w = weight(r.at(id), c.m, set.sl);
        lp = (float)log(w * set.unit / (double)c.S);
      }
      a.logprob[row] = lp;
    }
  }
}

// ------------------------------------------------------------ filtered acceptance
// Three kernels:
//   k_filter_rows      (row): the cut and total of every verified target row and every kept
//                      drafter row;
//   k_filtered_decide  (request): p'_j(x_j) / q'_j(x_j) at each kept position, the first
//                      rejection a_r, the counters;
//   k_filtered_draw    (request): the token from norm(max(0, p' - q')) at a_r, or from p'
//                      at the bonus row.
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
  WsHeader *ws;
};

// First row of request r, or -1 when rows r .. r + L would leave the row capacity.
__device__ inline int first_row(const RowMap &rm, int r, int L, WsHeader *ws) {
  const int cap = rm.B * (rm.gamma + 1);
  const int base = rm.row_offsets ? rm.row_offsets[r] : r * (rm.gamma + 1);
  if (base < 0 || base + L >= cap) {
    raise_flag(ws, SD_FLAG_ROW_OFFSETS);
    return -1;
  }
  return base;
}

__global__ __launch_bounds__(kFilterThreads, 4) void k_filter_rows(FilteredArgs a) {
  __shared__ FilterSmem s;
  const int g = a.rm.gamma, targets = a.rm.B * (g + 1);
  const bool draft = (int)blockIdx.x >= targets;
  const int i = draft ? blockIdx.x - targets : blockIdx.x;
  const int r = i / (draft ? g : g + 1), j = i - r * (draft ? g : g + 1);
  const int L = clamp_len(a.verify_len, r, g, nullptr);
  const int base = first_row(a.rm, r, L, nullptr);
  if (base < 0 || j > L || (draft && j == L)) return;
  const RowSettings set = load_settings(a.set, r, a.V, nullptr);
  if (draft) {
    const RowView<ElemBF16> v(a.draft_logits + (size_t)i * a.V, a.V);
    RowCut c;
    row_cut(v, set, true, c, s);
    row_total(v, c, set, s);
    if (threadIdx.x == 0) a.cut_q[i] = c;
  } else {
    const RowView<ElemF32> v(a.logits + (size_t)(base + j) * a.V, a.V);
    RowCut c;
    row_cut(v, set, true, c, s);
    row_total(v, c, set, s);
    if (threadIdx.x == 0) a.cut_p[i] = c;
  }
}

// Probability of id x, whose logit is l, under a row's cut.
__device__ inline double prob(const RowCut &c, const RowSettings &set, float l, int x) {
  l = canonical(l);
  return l > -INFINITY && c.n > 0 && kept(c, l, x) ? weight(l, c.m, set.sl) * set.unit / (double)c.S : 0.0;
}

// One wave per request, lane j decides position j.
__global__ __launch_bounds__(256) void k_filtered_decide(FilteredArgs a) {
  const int lane = threadIdx.x & 63, g = a.rm.gamma;
  const int r = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= a.rm.B) return;
  WsHeader *ws = lane == 0 ? a.ws : nullptr;
  const int L = clamp_len(a.verify_len, r, g, ws);
  const int base = first_row(a.rm, r, L, ws);
  const RowSettings set = load_settings(a.set, r, a.V, ws);
  if (base < 0) {
    if (lane == 0) { a.accept_len[r] = 0; a.next_token[r] = -1; }
    return;
  }
  bool miss = false;
  if (lane < L) {
    const int x = a.draft_tokens[(size_t)r * g + lane];
    miss = true;
    if (x >= 0 && x < a.V) {
      const double p = prob(a.cut_p[(size_t)r * (g + 1) + lane], set, a.logits[(size_t)(base + lane) * a.V + x], x);
      const size_t rj = (size_t)r * g + lane;
      const double q = prob(a.cut_q[rj], set, bf16_to_f32(a.draft_logits[rj * a.V + x]), x);
      // 0 / 0 compares false: a token that neither side keeps is rejected.
      miss = !((double)a.u_accept[rj] < (p >= q ? (p > 0.0 ? 1.0 : 0.0) : p / q));
    }
  }
  const u64 m = __ballot(miss);
  if (lane == 0) {
    const int acc = m ? __ffsll((long long)m) - 1 : L;
    a.accept_len[r] = acc;
    if (a.counters) {
      atomicAdd(reinterpret_cast<u64 *>(a.counters), (u64)L);
      atomicAdd(reinterpret_cast<u64 *>(a.counters + 1), (u64)acc);
    }
  }
}

// Residual weights are summed in units of 2^-51: they add up to at most 1, so a sum over
// 2^21 ids is off by 2^-31 of a unit row at the very worst, 2^-42 for random roundings.
constexpr double kResidualUnit = 2251799813685248.0;

__global__ __launch_bounds__(kFilterThreads) void k_filtered_draw(FilteredArgs a) {
  __shared__ FilterSmem s;
  const int r = blockIdx.x, g = a.rm.gamma;
  const int L = clamp_len(a.verify_len, r, g, nullptr);
  const int base = first_row(a.rm, r, L, nullptr);
  if (base < 0) return;
  const int acc = a.accept_len[r];
  const RowSettings set = load_settings(a.set, r, a.V, nullptr);
  const RowView<ElemF32> v(a.logits + (size_t)(base + acc) * a.V, a.V);
  RowCut cp = a.cut_p[(size_t)r * (g + 1) + acc];
  const float u = a.u_resample[(size_t)r * (g + 1) + acc];
  int id = -1;
  if (acc < L && cp.n > 0) {
    const uint16_t *q = a.draft_logits + ((size_t)r * g + acc) * a.V;
    const RowCut cq = a.cut_q[(size_t)r * g + acc];
    auto f = [&](int j, u64 (&w)[4]) {
      float l[4];
      v.load(j, l);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x = v.id(j, i);
        const double p = prob(cp, set, l[i], x);
        w[i] = p > 0.0 ? to_fix(fmax(p - prob(cq, set, bf16_to_f32(q[x]), x), 0.0), kResidualUnit) : 0;
      }
    };
    const int step = (v.nv + kFilterWaves - 1) / kFilterWaves;
    const u64 S = sum_shares<4>(f, 0, v.nv, step, s);
    if (S > 0) id = v.off + draw_in_shares<4>(f, v.nv, kFilterWaves, step, draw_target(u, S), s);
    else if (threadIdx.x == 0) raise_flag(a.ws, SD_FLAG_NO_RESIDUAL);
  }
  if (id < 0) id = row_draw(v, cp, set, kModeNone, 0, 0, u, s);
  if (threadIdx.x == 0) {
    if (id < 0) raise_flag(a.ws, SD_FLAG_EMPTY_ROW);
    a.next_token[r] = id;
  }
}

}  // namespace

// One workgroup per row keeps all of a row's state in LDS: the workspace is its header.
size_t sample_workspace_layout(int, int) { return sizeof(WsHeader); }

hipError_t launch_sample(const void *logits, int32_t type, int64_t stride, int R, int V,
                         const float *u, const SampleSettings &set, int rows_per,
                         int32_t *tokens, int64_t token_stride, int32_t *kept, float *logprob,
                         void *workspace, hipStream_t stream) {
  SampleArgs a{logits, stride, R, V, rows_per, u, set, tokens, token_stride, kept, logprob,
               reinterpret_cast<WsHeader *>(workspace)};
  auto *k = type == SD_F32 ? &k_sample<ElemF32> : type == SD_BF16 ? &k_sample<ElemBF16> : &k_sample<ElemF16>;
  hipLaunchKernelGGL(k, dim3(R), dim3(kFilterThreads), 0, stream, a);
  return hipGetLastError();
}

size_t accept_filtered_workspace_layout(int B, int gamma, size_t *cut_p, size_t *cut_q) {
  const size_t p = sizeof(WsHeader);
  const size_t q = align_up(p + (size_t)B * (gamma + 1) * sizeof(RowCut), 256);
  if (cut_p) *cut_p = p;
  if (cut_q) *cut_q = q;
  return align_up(q + (size_t)B * gamma * sizeof(RowCut), 256);
}

hipError_t launch_accept_filtered(const float *logits, const uint16_t *draft_logits,
                                  const int32_t *draft_tokens, const int32_t *verify_len,
                                  const RowMap &rm, const float *u_accept,
                                  const float *u_resample, const SampleSettings &set, int V,
                                  int32_t *accept_len, int32_t *next_token, int64_t *counters,
                                  void *workspace, hipStream_t stream) {
  size_t po, qo;
  accept_filtered_workspace_layout(rm.B, rm.gamma, &po, &qo);
  char *w = reinterpret_cast<char *>(workspace);
  FilteredArgs a{logits, draft_logits, draft_tokens, verify_len, rm, u_accept, u_resample, set, V,
                 accept_len, next_token, counters, reinterpret_cast<RowCut *>(w + po),
                 reinterpret_cast<RowCut *>(w + qo), reinterpret_cast<WsHeader *>(workspace)};
  hipLaunchKernelGGL(k_filter_rows, dim3(rm.B * (2 * rm.gamma + 1)), dim3(kFilterThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_filtered_decide, dim3((rm.B + 3) / 4), dim3(256), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(k_filtered_draw, dim3(rm.B), dim3(kFilterThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace sdv
