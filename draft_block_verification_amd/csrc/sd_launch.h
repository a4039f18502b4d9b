// Host-side launchers and workspace layouts of the HIP library (defined in sd_gemm.hip,
// sd_accept.hip, sd_sched.hip, sd_sample.hip, sd_mxfp4.hip, sd_norm.hip, sd_mxfp8.hip, sd_w4.hip and
// sd_narrow.hip; called by sd_api.hip). Each launcher enqueues its kernels on `stream` and returns the
// hipError_t of the launch.
#pragma once

#include "sd_internal.h"

namespace sdv {

// Bytes of verify workspace (header, then the row partials) for these sizes.
size_t verify_workspace_layout(int B, int gamma, int V, size_t *part_off, int *part_stride,
                               size_t *zx_off);

// LM-head verify.
hipError_t launch_verify(const VerifyArgs &a, hipStream_t stream);
// Greedy verify in two launches: the contraction, then one kernel that merges each
// request's row statistics and decides acceptance (temperature 0, stats written too).
hipError_t launch_verify_greedy(const VerifyArgs &a, int32_t *accept_len, int32_t *next_token,
                                int64_t *counters, hipStream_t stream);
// The contraction kernel alone; *n_part receives the partial columns written per row and
// *zx_done whether it also wrote the drafted-token logits to a.zx. With
// a.greedy_accept_len set, *greedy_done (when given) says whether the launch also wrote
// the greedy statistics and decisions (small streaming grids); otherwise the caller
// still has to.
// With a.dpart and a.draft_logits set, a streaming contraction may also write the drafter
// chunk partials of every kept draft row (workgroups appended to its grid); *draft_done
// (when given) says whether it did.
hipError_t launch_contraction(const VerifyArgs &a, hipStream_t stream, int *n_part,
                              bool *zx_done, bool *greedy_done = nullptr,
                              bool *draft_done = nullptr);
// Row statistics from the contraction's n_part partial columns (k_row_merge), with the
// drafted-token logits of a.zx when the contraction formed them (zx_done).
hipError_t launch_row_merge(const VerifyArgs &a, int n_part, bool zx_done, hipStream_t stream);
// Rejection verify's row merge and decision (k_merge_decide, gamma <= kDecideMaxGamma):
// statistics of every verified
// row, drafter log-normalisers, a_r and the counters, from the contraction's n_part
// partial columns, the drafter chunk partials and a.zx.
hipError_t launch_merge_decide(const VerifyArgs &a, const DecideArgs &o, int n_part,
                               hipStream_t stream);

// Workgroups of 256 threads of kernel fn that the current device holds at once.
int resident_workgroups(const void *fn);

// Stage-major blocked copy of a bf16 LM head (the layout VerifyArgs::w_blocked reads).
hipError_t launch_block_lm_head(const uint16_t *W, int V, int d, uint16_t *out,
                                hipStream_t stream);

hipError_t launch_truncate(const float *conf, int B, int gamma, float threshold,
                           int32_t *verify_len, int32_t *row_offsets, hipStream_t stream);

hipError_t launch_schedule(const float *conf, const float *conf_stale, int R, int gamma,
                           const float *sps, int mode, int32_t *verify_len, int32_t *row_offsets,
                           hipStream_t stream);

hipError_t launch_accept_greedy(const sd_row_stats *stats, const int32_t *draft_tokens,
                                const int32_t *verify_len, const RowMap &rm,
                                int32_t *accept_len, int32_t *next_token, int64_t *counters,
                                hipStream_t stream);

// Byte offsets inside the rejection-accept workspace.
struct AcceptLayout {
  int chunks;       // vocabulary chunks per row
  size_t lse_q;     // double [B][gamma] drafter log-normalisers (right after the header)
  size_t rec;       // DrawRec [B] draw records
  size_t qx;        // float [B][gamma] drafter logits of the drafted tokens
  size_t dpart;     // drafter chunk partials [B][gamma][chunks]
  size_t csum;      // double [B][chunks][2] draw-weight chunk sums
};
size_t accept_workspace_layout(int B, int gamma, int V, AcceptLayout *lay);

// Rejection verify in one call: the contraction (v.logits and v.stats set), the drafter
// normaliser, k_merge_decide and the draws; v.draft_logits and v.draft_tokens are required.
hipError_t launch_verify_rejection(VerifyArgs v, const float *u_accept, const float *u_resample,
                                   int32_t *accept_len, int32_t *next_token, int64_t *counters,
                                   double *accept_rate, void *accept_workspace,
                                   hipStream_t stream);

// Rejection acceptance.
hipError_t launch_accept_rejection(const float *logits, const sd_row_stats *stats,
                                   const uint16_t *draft_logits, const int32_t *draft_tokens,
                                   const int32_t *verify_len, const RowMap &rm,
                                   const float *u_accept, const float *u_resample, int V,
                                   float temperature, int32_t *accept_len, int32_t *next_token,
                                   int64_t *counters, double *accept_rate, void *workspace,
                                   hipStream_t stream);

// MXFP4 rows: columns padded to one matrix instruction's depth.
constexpr int mx_padded(int d) { return (d + 127) / 128 * 128; }

// Codes and scales by row.
hipError_t launch_mx_quantize(const void *x, int32_t type, int64_t rows, int d, int64_t stride,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int d,
                                void *x, int32_t type, int64_t stride, hipStream_t stream);
// Bytes of the tiled form of [rows][d]; *scales: where its scales start.
size_t mx_tiled_bytes(int64_t rows, int d, size_t *scales);
hipError_t launch_mx_head(const uint8_t *codes, const uint8_t *scales, int V, int d, uint8_t *head,
                          hipStream_t stream);

// Logits under a tiled MXFP4 LM head; the workspace holds the quantised hidden rows.
size_t mx_logits_workspace_bytes(int M, int d);
hipError_t launch_mx_logits(const void *hidden, int32_t hidden_type, int M, int d, int64_t stride,
                            const uint8_t *head, int V, void *logits, int32_t type, int64_t ld,
                            void *workspace, hipStream_t stream);

// RMS norm of rows; r (the residual) and sum may be null, w too; the output goes to y or, where
// codes is not null, to MXFP8 rows.
struct NormArgs {
  const void *x;
  int32_t x_type;
  int64_t x_stride;
  const void *r;
  int32_t r_type;           // of r and sum: x_type or SD_F32
  int64_t r_stride;
  const void *w;
  int32_t w_type;
  float offset, eps;
  int64_t rows;
  int d;
  void *sum;
  int64_t sum_stride;
  void *y;
  int32_t y_type;
  int64_t y_stride;
  uint8_t *codes, *scales;
};
hipError_t launch_norm(const NormArgs &a, hipStream_t stream);

// MXFP8 rows, an LM head of them re-laid into tiles, and logits under it.
hipError_t launch_mx8_quantize(const void *x, int32_t type, int64_t rows, int d, int64_t stride,
                               uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t launch_mx8_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int d,
                                 void *x, int32_t type, int64_t stride, hipStream_t stream);
size_t mx8_head_bytes(int64_t V, int d);
hipError_t launch_mx8_head(const uint8_t *codes, const uint8_t *scales, int V, int d, uint8_t *head,
                           hipStream_t stream);
size_t mx8_logits_workspace_bytes(int M, int d);
hipError_t launch_mx8_logits(const void *hidden, int32_t hidden_type, const uint8_t *hidden_scales, int M, int d,
                             int64_t stride, const uint8_t *head, int V, void *logits, int32_t type, int64_t ld,
                             void *workspace, hipStream_t stream);

// 4-bit integer weights with group scales (zeros null: symmetric), likewise.
hipError_t launch_w4_quantize(const void *x, int32_t type, int64_t rows, int d, int64_t stride, int group,
                              uint8_t *codes, uint16_t *scales, int32_t scale_type, uint8_t *zeros,
                              hipStream_t stream);
hipError_t launch_w4_dequantize(const uint8_t *codes, const uint16_t *scales, int32_t scale_type,
                                const uint8_t *zeros, int64_t rows, int d, int group, void *x, int32_t type,
                                int64_t stride, hipStream_t stream);
size_t w4_head_bytes(int64_t V, int d, int group, bool zeros);
hipError_t launch_w4_head(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int V, int d,
                          int group, uint8_t *head, hipStream_t stream);
size_t w4_logits_workspace_bytes(int M, int d, int group);
hipError_t launch_w4_logits(const void *hidden, int32_t hidden_type, int M, int d, int64_t stride,
                            const uint8_t *head, int V, int group, int32_t scale_type, bool zeros, void *logits,
                            int32_t type, int64_t ld, void *workspace, hipStream_t stream);

// Filtered sampling and acceptance.
hipError_t launch_sample(const void *logits, int32_t type, int64_t stride, int R, int V,
                         const float *u, const SampleSettings &set, int rows_per,
                         int32_t *tokens, int64_t token_stride, int32_t *kept, float *logprob,
                         void *workspace, hipStream_t stream);
size_t sample_workspace_layout(int R, int V);
size_t accept_filtered_workspace_layout(int B, int gamma, int V);
hipError_t launch_accept_filtered(const float *logits, const uint16_t *draft_logits,
                                  const int32_t *draft_tokens, const int32_t *verify_len,
                                  const RowMap &rm, const float *u_accept,
                                  const float *u_resample, const SampleSettings &set, int V,
                                  int32_t *accept_len, int32_t *next_token, int64_t *counters,
                                  void *workspace, hipStream_t stream);
}  // namespace sdv
