/*
 * sd_verify.h -- C ABI of the draft-block verification library (libsdverify.so).
 *
 * One verify round of speculative decoding on an AMD MI355X (gfx950):
 *   1. sd_truncate_by_confidence  keep each request's confident draft prefix
 *      sd_schedule_prefix         or choose the prefixes that maximise throughput
 *   2. sd_verify_logits           LM-head logits at every kept position plus the
 *                                 bonus position, with per-row statistics
 *   3. sd_accept_greedy           greedy prefix acceptance + correction/bonus token
 *      sd_accept_rejection        rejection-sampling acceptance + residual/bonus draw
 *      sd_accept_filtered         the same under top-k, top-p and min-p
 * before it
 *      sd_rms_norm                the last residual addition and norm, which make the hidden rows
 * and, on the drafter's side:
 *      sd_mxfp4_logits            logits under a 4-bit copy of the LM head
 *      sd_mxfp8_logits            the same under an 8-bit copy
 *      sd_w4_logits               the same under 4-bit integer weights with group scales
 *      sd_sample                  draws under temperature, top-k, top-p and min-p
 *
 * Conventions shared by every call
 *   - All tensors are row-major, contiguous, caller-owned DEVICE memory unless
 *     stated otherwise. The library never allocates; scratch memory comes from a
 *     caller-provided workspace sized by the *_workspace_bytes functions.
 *   - bf16 tensors are passed as uint16_t bit patterns.
 *   - `stream` is a hipStream_t (NULL = the default stream). Calls only enqueue
 *     work; outputs are valid once the stream has been synchronised.
 *   - Host-checkable errors (null pointers, bad sizes, misalignment, small
 *     workspace) are returned synchronously before any GPU work is enqueued.
 *     SD_EDEVICE reports a failed kernel launch. Nothing is printed.
 *   - Device-side anomalies (a verify length outside [0, gamma], row offsets
 *     that disagree with the lengths, a residual with no positive mass) are
 *     clamped or handled by a documented fallback and raise bits in a sticky
 *     flag word inside the workspace, read with sd_device_flags.
 *   - Identical inputs give identical output bytes (fixed-order reductions, no
 *     floating-point atomics).
 *   - Rows: request r verifies L_r kept drafts (0 <= L_r <= gamma) plus one bonus
 *     row, M = sum_r (L_r + 1) rows in total, packed with no padding. Row m of
 *     request r, block position j (0 <= j <= L_r) is m = row_offsets[r] + j and
 *     reads hidden[r][j][:]. Per-row outputs have capacity B * (gamma + 1) rows;
 *     only the first M are written.
 *
 * The operations follow these passages:
 *   DSpark summary (GeekNews), "Problem definition": the target checks a drafted
 *     block in one forward pass and rejection sampling accepts the longest
 *     prefix consistent with the target distribution, losslessly.
 *   DSpark summary, "Architecture" (decode-round example, confidence head,
 *     prefix scheduler): per-position survival confidences; the scheduler keeps
 *     the confident prefix and cuts the rest; on the first rejection the target
 *     emits a correction token.
 *   DSpark summary, "Production deployment": the LM head maps the d-dimensional
 *     hidden state to V logits; variable-length requests are flattened into
 *     independent elements instead of padded.
 *   LFM2.5-DSpark blog, "How DSpark works" and "Quality parity": verification
 *     shares one weight load across the block; in greedy decoding a draft is
 *     kept only if it matches the target and is otherwise replaced by the
 *     target's token, so the output equals the target's own greedy output.
 */
#ifndef SD_VERIFY_H
#define SD_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifndef SD_API
#define SD_API __attribute__((visibility("default")))
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point (as int32_t). */
enum {
    SD_OK = 0,
    SD_EINVAL = 1,      /* null required pointer, bad temperature or threshold   */
    SD_ESHAPE = 2,      /* B < 1, gamma outside [1, 64], d % 8 != 0, V < 1, a row stride
                           shorter than its row, size overflow                            */
    SD_EALIGN = 3,      /* a bf16 / fp32 tensor not 16-byte aligned, stats not 8-byte aligned */
    SD_EWORKSPACE = 4,  /* workspace pointer null or smaller than required       */
    SD_EDEVICE = 5,     /* a HIP launch or copy failed                           */
    SD_ESCRATCH = 6     /* the problem needs more scratch than the allocation-free
                           entry point holds (SD_NOALLOC_SCRATCH_BYTES)            */
};

/* Sticky device flags (bit mask) accumulated in a workspace. */
enum {
    SD_FLAG_VERIFY_LEN = 1,   /* a verify_len entry was outside [0, gamma] and was clamped */
    SD_FLAG_ROW_OFFSETS = 2,  /* row_offsets disagreed with verify_len or overflowed the row capacity */
    SD_FLAG_NO_RESIDUAL = 4,  /* a residual max(0, p - q) had no positive mass; drew from p instead */
    SD_FLAG_WAIT = 8,         /* a workgroup's bounded wait for results that other workgroups
                                 of the same launch publish ran out (sd_verify_rejection's
                                 one-launch draw, sd_verify_greedy's in-launch decision);
                                 the tokens of that call are not valid */
    SD_FLAG_SAMPLING = 16,    /* a sampling setting was not a number (temperature: or negative
                                 or infinite) and was replaced as sd_sampling documents      */
    SD_FLAG_EMPTY_ROW = 32    /* a sampled row had no logit above -inf: its token is -1      */
};

/* Per verified row statistics (32 bytes, 8-byte aligned). */
typedef struct sd_row_stats {
    int32_t argmax;   /* lowest vocabulary id attaining max_v z[v]                        */
    float top1;       /* z[argmax] (fp32 logit)                                          */
    float top2;       /* largest z[v] over v != argmax (equals top1 on an exact tie)      */
    int32_t pos;      /* block position j of this row (0..L_r; L_r is the bonus row)      */
    double lse;       /* log sum_v exp(z[v] / T) when T > 0, else 0                      */
    double z_draft;   /* logit of the drafted token x[r][j] for j < L_r, as an fp64 dot of
                         the bf16 inputs; 0 on the bonus row                              */
} sd_row_stats;

/* ABI version of this header (incremented on any signature or layout change). */
SD_API int32_t sd_abi_version(void);

/* Static text for a status code. */
SD_API const char *sd_status_string(int32_t status);

/* Workspace bytes sd_verify_logits needs for these sizes (0 on invalid sizes). */
SD_API size_t sd_verify_workspace_bytes(int32_t B, int32_t gamma, int32_t d, int32_t V);

/* Workspace bytes sd_accept_rejection needs for these sizes (0 on invalid sizes). */
SD_API size_t sd_accept_workspace_bytes(int32_t B, int32_t gamma, int32_t V);

/* Prepare a freshly allocated workspace: clears its 256-byte header (flag word and
 * counters) and, in a workspace of at least 256 + 1049600 bytes (every verify workspace),
 * sets the 1049600-byte publication area that follows the header to all ones bytes (the
 * state sd_verify_greedy's in-launch decision expects; every later verify call leaves it so).
 * Must be called once per workspace before its first use; enqueued on `stream`.
 * Calls in turn may share a workspace of the largest size among them, calls at the same time
 * may not. A workspace serves the verify calls or the others (acceptance, sampling, MXFP4
 * logits): those keep scratch in that area, so it becomes a verify workspace only by being
 * prepared again. */
SD_API int32_t sd_workspace_init(void *workspace, size_t workspace_bytes, void *stream);

/* Synchronise `stream`, copy the sticky flag word of `workspace` to *flags (host) and,
 * if clear != 0, reset it to zero. */
SD_API int32_t sd_device_flags(void *workspace, void *stream, uint32_t *flags, int32_t clear);

/*
 * Confidence truncation (DSpark summary, "Architecture": the scheduler keeps
 * the confident prefix E F G and cuts the low-confidence H).
 *   conf        fp32 [B][gamma]  per-position prefix-survival confidences
 *   threshold   keep leading positions with conf >= threshold (finite, any value)
 *   verify_len  int32 [B]        out: L_r = number of leading positions kept
 *   row_offsets int32 [B + 1]    out: exclusive prefix sum of (L_r + 1); row_offsets[B] = M
 */
SD_API int32_t sd_truncate_by_confidence(const float *conf, int32_t B, int32_t gamma, float threshold,
                                  int32_t *verify_len, int32_t *row_offsets, void *stream);

/* Modes of sd_schedule_prefix. */
enum {
    SD_SCHED_EARLY_STOP = 0,  /* synchronous: admit by survival, stop when throughput drops */
    SD_SCHED_TOP_K = 1        /* asynchronous: K from (stale) confidences over every K, then top-K */
};

/* Largest R * gamma sd_schedule_prefix accepts (all candidates are sorted in one workgroup). */
#define SD_SCHED_MAX_CANDIDATES 16384

/*
 * Hardware-aware prefix scheduler (DSpark summary, "Architecture" ->
 * "Confidence-Scheduled Verification": survival-ordered admission that maximises
 * throughput tau * SPS(B) over a cost table profiled once, with early stopping;
 * "Engineering": the asynchronous form that sizes the batch from two-step-old
 * confidences by a search over every K and admits the current top-K). A drop-in
 * replacement for sd_truncate_by_confidence.
 *   conf        fp32 [R][gamma]  conditional confidences c[r][k] of the current step
 *   conf_stale  fp32 [R][gamma]  confidences of an earlier step (SD_SCHED_TOP_K only,
 *               may be NULL: then conf); must be NULL with SD_SCHED_EARLY_STOP
 *   sps         fp32 [n_sps]     steps per second at a batch of B target rows, for
 *               B = 0 .. n_sps - 1; n_sps >= R * (gamma + 1) + 1; finite and positive
 *   mode        SD_SCHED_EARLY_STOP or SD_SCHED_TOP_K
 *   verify_len  int32 [R]        out: admitted drafts of request r (a prefix of its block)
 *   row_offsets int32 [R + 1]    out: exclusive prefix sum of (verify_len + 1)
 * Survival a[r][j] = product of clamp(c[r][k], 0, 1) over k <= j (NaN counts as 0),
 * taken left to right in fp32. Candidates are ordered by larger survival, then lower
 * request, then lower position. With K admitted, the batch is B = R + K rows and
 * Theta_K = (R * 2^40 + sum over the first K candidates of floor(a * 2^40)) * SPS(B),
 * the integer converted to fp64 (round to nearest even) and one fp64 multiply.
 * SD_SCHED_EARLY_STOP: K = first K with Theta_{K+1} < Theta_K, else R * gamma.
 * SD_SCHED_TOP_K: K = smallest K attaining the largest Theta_K over K = 0 .. R * gamma
 * (computed from conf_stale when given); the admitted set is the first K candidates
 * in the order of conf.
 * Errors: SD_EINVAL for a null output or conf/sps, a bad mode or a stale array with
 * SD_SCHED_EARLY_STOP; SD_ESHAPE for R < 1, gamma outside [1, 64],
 * R * gamma > SD_SCHED_MAX_CANDIDATES or a short sps table; SD_EALIGN for arrays not
 * 4-byte aligned. One workgroup, no workspace.
 */
SD_API int32_t sd_schedule_prefix(const float *conf, const float *conf_stale, int32_t R,
                                  int32_t gamma, const float *sps, int32_t n_sps, int32_t mode,
                                  int32_t *verify_len, int32_t *row_offsets, void *stream);

/*
 * Target logits at every verified row and their statistics (LFM2.5-DSpark
 * blog, "How DSpark works"; DSpark summary, "Production deployment").
 *   hidden       bf16 [B][gamma + 1][d]  target hidden states before the LM head
 *   lm_head      bf16 [V][d]             LM-head weight, d-contiguous rows
 *   draft_tokens int32 [B][gamma] or NULL drafted tokens (for z_draft); NULL -> z_draft = 0
 *   verify_len   int32 [B] or NULL       kept drafts per request; NULL -> gamma for all
 *   row_offsets  int32 [B + 1] or NULL   packed row starts; NULL -> r * (gamma + 1).
 *                                        verify_len and row_offsets are both NULL or both set.
 *   temperature  >= 0; 0 computes argmax/top1/top2 only (lse = 0)
 *   logits       fp32 [B * (gamma + 1)][V] or NULL: out, z[m][v] for m < M
 *   stats        sd_row_stats [B * (gamma + 1)]: out, rows m < M
 *   workspace    device scratch of sd_verify_workspace_bytes(B, gamma, d, V) bytes
 * z[m][v] = sum_k hidden_row(m)[k] * lm_head[v][k], bf16 products accumulated in fp32.
 */
SD_API int32_t sd_verify_logits(const uint16_t *hidden, const uint16_t *lm_head,
                         const int32_t *draft_tokens, const int32_t *verify_len,
                         const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                         int32_t V, float temperature, float *logits, sd_row_stats *stats,
                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * The LM-head contraction stage of sd_verify_logits on its own (same passages):
 * writes the fp32 logits (when logits != NULL) and leaves per-row partial
 * statistics in `workspace`; it does not produce sd_row_stats. It runs exactly the
 * contraction kernel sd_verify_logits runs first, so it serves to time that kernel
 * alone, and callers that only need the logits can use it. Arguments as for
 * sd_verify_logits.
 */
SD_API int32_t sd_verify_contraction(const uint16_t *hidden, const uint16_t *lm_head,
                                     const int32_t *verify_len, const int32_t *row_offsets,
                                     int32_t B, int32_t gamma, int32_t d, int32_t V,
                                     float temperature, float *logits, void *workspace,
                                     size_t workspace_bytes, void *stream);

/*
 * Greedy verify of a drafted block in one call (LFM2.5-DSpark blog, "How DSpark
 * works" and "Quality parity"): the LM-head contraction at temperature 0 followed
 * by one kernel that merges each request's row statistics and decides acceptance.
 * When the streaming contraction runs (B * (gamma + 1) <= 64, d % 128 == 0) for at most
 * 16 requests of at most 12 rows (gamma <= 11) on a grid that leaves a compute unit for
 * each request (up to about V = 16000 on MI355X), workgroups appended to its launch merge
 * and decide instead (no second launch): the contraction's workgroups publish their row
 * partials in the workspace's publication area, which the call leaves as it found it.
 * Outputs are the same bytes as sd_verify_logits (temperature 0, logits NULL)
 * followed by sd_accept_greedy, with one or two launches fewer.
 *   hidden, lm_head, draft_tokens, verify_len, row_offsets, B, gamma, d, V
 *                as for sd_verify_logits (draft_tokens required)
 *   stats        sd_row_stats [B * (gamma + 1)]  out, as for sd_verify_logits
 *   accept_len, next_token, counters  as for sd_accept_greedy
 *   workspace    the verify workspace (sd_verify_workspace_bytes)
 * Errors: as for sd_verify_logits and sd_accept_greedy.
 */
SD_API int32_t sd_verify_greedy(const uint16_t *hidden, const uint16_t *lm_head,
                                const int32_t *draft_tokens, const int32_t *verify_len,
                                const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                                int32_t V, sd_row_stats *stats, int32_t *accept_len,
                                int32_t *next_token, int64_t *counters, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * sd_verify_greedy for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, and harnesses that forbid hipMalloc. The verify
 * workspace (header, per-tile row partials, drafted-token logits) lives in a file-scope
 * device array of the library, SD_NOALLOC_SCRATCH_BYTES bytes on every GPU the library
 * runs on, held until the process ends; its address is looked up once per device on
 * the first call made with that device current. The call itself allocates nothing
 * (no hipMalloc, hipFree or allocating library routine).
 *   hidden, lm_head, draft_tokens, verify_len, row_offsets, B, gamma, d, V, stats,
 *   accept_len, next_token, counters   as for sd_verify_greedy (bf16 [V][d] LM head)
 *   flags   device uint32 [1] out, 4-byte aligned, or NULL: this call's sticky device
 *           flag word (SD_FLAG_*); the scratch's flag word is cleared at the start of
 *           every call, so flags cover this call only (the first call on a device also
 *           prepares the scratch as sd_workspace_init prepares a workspace)
 *   stream  hipStream_t of the device that is current at the call
 * Limit: sd_verify_workspace_bytes(B, gamma, d, V) <= SD_NOALLOC_SCRATCH_BYTES, else
 * SD_ESCRATCH before any GPU work (16 MiB holds, for example, 64 rows at V = 151936 or
 * 400 rows at V = 32768). Every call on one GPU shares that GPU's scratch: calls that
 * overlap on one GPU (other streams, other host threads) race and must be serialised
 * by the caller. Outputs are the bytes sd_verify_greedy writes for the same inputs.
 * Errors: as for sd_verify_greedy (SD_EWORKSPACE does not occur), SD_ESCRATCH, and
 * SD_EDEVICE when the scratch address cannot be looked up.
 */
#define SD_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
SD_API int32_t sd_verify_greedy_noalloc(const uint16_t *hidden, const uint16_t *lm_head,
                                        const int32_t *draft_tokens, const int32_t *verify_len,
                                        const int32_t *row_offsets, int32_t B, int32_t gamma,
                                        int32_t d, int32_t V, sd_row_stats *stats,
                                        int32_t *accept_len, int32_t *next_token,
                                        int64_t *counters, uint32_t *flags, void *stream);

/*
 * W12 LM head (SpecPilot page, "Reasons": a lossless 12-bit weight format whose three
 * 4-bit planes the GEMM rebuilds in registers). This library's layout:
 *   - a bf16 weight's low byte (exponent bit 0, 7 mantissa bits) is kept verbatim;
 *   - its high byte (sign, exponent bits 7..1 = e2) becomes the 4-bit code
 *     sign << 3 | t: t = 0 for e2 = 0 (zeros, subnormals), t = e2 - b2 + 1 for e2 in
 *     the tensor's window [b2, b2 + 6], b2 = max(1, largest nonzero e2 - 6);
 *   - every other weight is coded as a signed zero and its exact bits go to a
 *     correction slot of its region of 64 LM-head rows by 128 columns: uint32
 *     k_local | row_local << 7 | bits << 16, sorted by (row_local, k_local), 0 = empty;
 *   - a group of 8 columns 8 g .. 8 g + 7 of one row is 12 bytes: the 8 low bytes, then
 *     byte 8 + i = code of column 8 g + 2 i | code of column 8 g + 2 i + 1 << 4; groups
 *     are stored region by region, [ceil(V / 64)][d / 128][64 rows][16 groups][12 bytes],
 *     rows past V zero (one region = one contiguous 12 KB block).
 * Decoding gives back every bf16 bit pattern exactly.
 */
typedef struct sd_w12 {
    const uint8_t *codes;    /* [ceil(V/64)][d/128][64][16][12], device, 16-byte aligned */
    const uint32_t *corr;    /* [ceil(V / 64)][d / 128][cap] correction slots, device     */
    int32_t cap;             /* slots per region: a multiple of 4 in [4, 64] for the GEMM */
    int32_t b2;              /* window start, 1..121                                     */
} sd_w12;

/*
 * Encode a bf16 LM head into W12 (host memory in and out; runs on the host).
 *   W      bf16 [V][d] (d a multiple of 128)
 *   codes  uint8 [ceil(V / 64)][d / 128][64][16][12] out (ignored by the sizing call)
 *   corr   uint32 [ceil(V / 64)][d / 128][*cap] out, or NULL for the sizing call
 *   cap    in: slots per region of corr; out: the slots needed (sizing call), or used
 *   b2     out: window start
 * A sizing call (corr NULL) sets *cap and *b2 only. SD_EWORKSPACE (with *cap set to
 * the need) when *cap is too small; SD_ESHAPE for V < 1 or d not a positive multiple
 * of 128.
 */
SD_API int32_t sd_w12_encode(const uint16_t *W, int32_t V, int32_t d, uint8_t *codes,
                             uint32_t *corr, int32_t *cap, int32_t *b2);

/*
 * sd_verify_logits, sd_verify_contraction and sd_verify_greedy with the LM head
 * given as W12 (lm_head:
 * host struct of device pointers). The contraction decodes the 12-bit groups in
 * registers and adds the corrected weights' products, so every result is that of
 * the bf16 LM head (logits up to fp32 summation order). Restricted to the streaming
 * regime: d % 128 == 0, B * (gamma + 1) <= 64 and cap <= 64, else SD_ESHAPE.
 * Other arguments, outputs and errors as for the bf16 calls.
 */
SD_API int32_t sd_verify_logits_w12(const uint16_t *hidden, const sd_w12 *lm_head,
                                    const int32_t *draft_tokens, const int32_t *verify_len,
                                    const int32_t *row_offsets, int32_t B, int32_t gamma,
                                    int32_t d, int32_t V, float temperature, float *logits,
                                    sd_row_stats *stats, void *workspace, size_t workspace_bytes,
                                    void *stream);
SD_API int32_t sd_verify_contraction_w12(const uint16_t *hidden, const sd_w12 *lm_head,
                                         const int32_t *verify_len, const int32_t *row_offsets,
                                         int32_t B, int32_t gamma, int32_t d, int32_t V,
                                         float temperature, float *logits, void *workspace,
                                         size_t workspace_bytes, void *stream);
SD_API int32_t sd_verify_greedy_w12(const uint16_t *hidden, const sd_w12 *lm_head,
                                    const int32_t *draft_tokens, const int32_t *verify_len,
                                    const int32_t *row_offsets, int32_t B, int32_t gamma,
                                    int32_t d, int32_t V, sd_row_stats *stats,
                                    int32_t *accept_len, int32_t *next_token, int64_t *counters,
                                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * Blocked bf16 LM head: the same weights re-laid once so that the streaming
 * contraction reads each of its stages (64 LM-head rows by 128 columns) as one
 * contiguous 16 KB block. Layout: [d/128][ceil(V/64)][64][128] bf16, stage-major: block
 * (st, s) holds LM-head rows 64 s .. 64 s + 63 at columns 128 st .. 128 st + 127, so the
 * blocks of one column range are adjacent. Within a block, row r's 16-byte chunk j
 * (columns 8j .. 8j + 7) sits at chunk position j ^ (r & 15); rows past V are zero. The values, and so every verify output, are those of the bf16
 * [V][d] LM head. The LM head is static, so the copy is made once, beside the original.
 *
 * sd_lm_head_block_bytes: bytes of the copy (0 unless V >= 1 and d is a positive
 * multiple of 128).
 * sd_lm_head_block: writes the copy on `stream`.
 *   lm_head  bf16 [V][d], 16-byte aligned; blocked: device buffer of
 *   sd_lm_head_block_bytes(V, d) bytes, 16-byte aligned, not overlapping lm_head.
 *   Errors: SD_EINVAL (null pointer), SD_ESHAPE (V < 1, d % 128 != 0), SD_EALIGN,
 *   SD_EWORKSPACE (blocked_bytes too small), SD_EDEVICE.
 * sd_verify_logits_blocked / sd_verify_contraction_blocked / sd_verify_greedy_blocked:
 * sd_verify_logits / sd_verify_contraction / sd_verify_greedy reading the blocked copy
 * (lm_head_blocked) instead of the [V][d] LM head; the streaming regime only, like W12:
 * d % 128 == 0 and B * (gamma + 1) <= 64, else SD_ESHAPE. All other arguments, outputs
 * and errors are those of the [V][d] calls.
 */
SD_API size_t sd_lm_head_block_bytes(int32_t V, int32_t d);
SD_API int32_t sd_lm_head_block(const uint16_t *lm_head, int32_t V, int32_t d, uint16_t *blocked,
                                size_t blocked_bytes, void *stream);
SD_API int32_t sd_verify_logits_blocked(const uint16_t *hidden, const uint16_t *lm_head_blocked,
                                        const int32_t *draft_tokens, const int32_t *verify_len,
                                        const int32_t *row_offsets, int32_t B, int32_t gamma,
                                        int32_t d, int32_t V, float temperature, float *logits,
                                        sd_row_stats *stats, void *workspace,
                                        size_t workspace_bytes, void *stream);
SD_API int32_t sd_verify_contraction_blocked(const uint16_t *hidden,
                                             const uint16_t *lm_head_blocked,
                                             const int32_t *verify_len,
                                             const int32_t *row_offsets, int32_t B, int32_t gamma,
                                             int32_t d, int32_t V, float temperature,
                                             float *logits, void *workspace,
                                             size_t workspace_bytes, void *stream);
SD_API int32_t sd_verify_greedy_blocked(const uint16_t *hidden, const uint16_t *lm_head_blocked,
                                        const int32_t *draft_tokens, const int32_t *verify_len,
                                        const int32_t *row_offsets, int32_t B, int32_t gamma,
                                        int32_t d, int32_t V, sd_row_stats *stats,
                                        int32_t *accept_len, int32_t *next_token,
                                        int64_t *counters, void *workspace,
                                        size_t workspace_bytes, void *stream);

/*
 * Greedy acceptance (LFM2.5-DSpark blog, "Quality parity"): a_r = first j < L_r
 * with stats[row_offsets[r] + j].argmax != draft_tokens[r][j], else L_r; the
 * emitted token is the target argmax of row a_r (a correction when a_r < L_r,
 * the bonus token otherwise).
 *   stats        from sd_verify_logits
 *   draft_tokens int32 [B][gamma]
 *   verify_len, row_offsets  as for sd_verify_logits (both NULL or both set)
 *   accept_len   int32 [B]  out: a_r
 *   next_token   int32 [B]  out
 *   counters     int64 [2] or NULL: counters[0] += sum_r L_r (drafts verified),
 *                counters[1] += sum_r a_r (drafts accepted)
 */
SD_API int32_t sd_accept_greedy(const sd_row_stats *stats, const int32_t *draft_tokens,
                         const int32_t *verify_len, const int32_t *row_offsets, int32_t B,
                         int32_t gamma, int32_t *accept_len, int32_t *next_token,
                         int64_t *counters, void *stream);

/*
 * Rejection-sampling acceptance (DSpark summary, "Problem definition":
 * lossless acceptance of the longest consistent prefix; "Architecture":
 * correction token on the first rejection). With p_j = softmax(z_j / T) and
 * q_j = softmax(draft_logits[r][j] / T):
 *   position j < L_r survives iff u_accept[r][j] < min(1, p_j(x_j) / q_j(x_j));
 *   a_r = first failing j, else L_r;
 *   if a_r < L_r the token is drawn from norm(max(0, p_a - q_a)), else from p_{L_r};
 *   draws are inverse-CDF in ascending vocabulary id: the smallest v whose running
 *   weight exceeds u_resample[r][a_r] times the total weight.
 *   logits       fp32 [B * (gamma + 1)][V] written by sd_verify_logits
 *   stats        from sd_verify_logits at the same temperature
 *   draft_logits bf16 [B][gamma][V]     drafter logits per block position
 *   draft_tokens int32 [B][gamma]
 *   u_accept     fp32 [B][gamma]        uniforms in [0, 1)
 *   u_resample   fp32 [B][gamma + 1]    uniforms in [0, 1), indexed by the row sampled
 *   temperature  > 0 (the same one given to sd_verify_logits)
 *   accept_len, next_token, counters   as for sd_accept_greedy
 *   workspace    device scratch of sd_accept_workspace_bytes(B, gamma, V) bytes
 */
SD_API int32_t sd_accept_rejection(const float *logits, const sd_row_stats *stats,
                            const uint16_t *draft_logits, const int32_t *draft_tokens,
                            const int32_t *verify_len, const int32_t *row_offsets,
                            const float *u_accept, const float *u_resample, int32_t B,
                            int32_t gamma, int32_t V, float temperature, int32_t *accept_len,
                            int32_t *next_token, int64_t *counters, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * sd_accept_rejection plus the analytic acceptance rate of every verified draft
 * position (DSpark summary, "Architecture": the confidence head learns, per drafted
 * position, the chance that rejection sampling keeps it, one minus the total-variation
 * distance between drafter and target distributions):
 *   accept_rate[r][j] = sum_v min(p_j(v), q_j(v)) = 1 - (1/2) sum_v |p_j(v) - q_j(v)|
 * for j < L_r, with p_j, q_j as above at the same temperature; -1 for j >= L_r and for
 * every position of a request whose rows leave the row capacity.
 *   accept_rate  fp64 [B][gamma], 8-byte aligned, or NULL (then identical to
 *                sd_accept_rejection)
 * All other arguments, outputs and errors are those of sd_accept_rejection; the
 * acceptance outputs are byte-identical to it. The extra work is one more pass over
 * the kept target and drafter rows (P * V * 6 bytes), with the same workspace.
 */
SD_API int32_t sd_accept_rejection_ex(const float *logits, const sd_row_stats *stats,
                            const uint16_t *draft_logits, const int32_t *draft_tokens,
                            const int32_t *verify_len, const int32_t *row_offsets,
                            const float *u_accept, const float *u_resample, int32_t B,
                            int32_t gamma, int32_t V, float temperature, int32_t *accept_len,
                            int32_t *next_token, int64_t *counters, double *accept_rate,
                            void *workspace, size_t workspace_bytes, void *stream);

/* LM-head layouts of sd_verify_rejection. */
enum {
    SD_LM_HEAD_ROWS = 0,     /* bf16 [V][d]                                              */
    SD_LM_HEAD_BLOCKED = 1,  /* the stage-major blocked copy written by sd_lm_head_block */
    SD_LM_HEAD_W12 = 2       /* lm_head points to an sd_w12 descriptor (host memory)     */
};

/*
 * Rejection verify of a drafted block in one call (DSpark summary, "Problem definition":
 * the target checks the block in one pass and rejection sampling keeps the longest
 * prefix consistent with its distribution; "Architecture": a correction token on the
 * first rejection, a bonus token when every draft survives): sd_verify_logits at
 * `temperature` followed by sd_accept_rejection_ex, in fewer launches. The row merge and
 * the acceptance test run in one kernel; in the streaming regime (d % 128 == 0,
 * B * (gamma + 1) <= 64) the contraction's launch also normalises the drafter rows when
 * the GPU has workgroup slots its grid leaves idle.
 *   hidden, draft_tokens, verify_len, row_offsets, B, gamma, d, V
 *                as for sd_verify_logits (draft_tokens required)
 *   lm_head      bf16 [V][d] (lm_head_layout SD_LM_HEAD_ROWS), its blocked copy
 *                (SD_LM_HEAD_BLOCKED), or a host sd_w12 descriptor of the W12 stream
 *                (SD_LM_HEAD_W12, checked as for sd_verify_logits_w12); the last two in
 *                the streaming regime only, else SD_ESHAPE
 *   draft_logits, u_accept, u_resample, temperature (> 0)
 *                as for sd_accept_rejection
 *   logits, stats  out, as for sd_verify_logits (both required)
 *   accept_len, next_token, counters, accept_rate (NULL: not computed)
 *                out, as for sd_accept_rejection_ex
 *   verify_workspace  sd_verify_workspace_bytes(B, gamma, d, V) bytes
 *   accept_workspace  sd_accept_workspace_bytes(B, gamma, V) bytes
 * The logits, argmax, top-1/top-2, drafted-token logits, accepted lengths, tokens,
 * counters and flags are those of the two separate calls; the per-row log-normalisers
 * (stats lse and the drafter's) are summed in another order and agree with them to
 * fp64 rounding.
 * Errors: those of sd_verify_logits and sd_accept_rejection_ex; SD_EINVAL for an unknown
 * lm_head_layout.
 */
SD_API int32_t sd_verify_rejection(const uint16_t *hidden, const void *lm_head,
                                   int32_t lm_head_layout, const uint16_t *draft_logits,
                                   const int32_t *draft_tokens, const int32_t *verify_len,
                                   const int32_t *row_offsets, const float *u_accept,
                                   const float *u_resample, int32_t B, int32_t gamma, int32_t d,
                                   int32_t V, float temperature, float *logits,
                                   sd_row_stats *stats, int32_t *accept_len,
                                   int32_t *next_token, int64_t *counters, double *accept_rate,
                                   void *verify_workspace, size_t verify_workspace_bytes,
                                   void *accept_workspace, size_t accept_workspace_bytes,
                                   void *stream);

/* Element types of the calls that take more than one. */
enum {
    SD_F32 = 0,
    SD_BF16 = 1,
    SD_F16 = 2,
    SD_MXFP8 = 3   /* hidden rows of sd_mxfp8_logits only */
};

/*
 * MXFP4 (OCP Microscaling Formats): a block of 32 consecutive columns of a row shares one
 * scale 2^e; a value is a 4-bit code, sign in bit 3, magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6
 * for codes 0..7. With kp = d rounded up to a multiple of 128 (sd_mxfp4_columns):
 *   codes   uint8 [rows][kp / 2]   column 2 i in the low half of byte i, 2 i + 1 in the high
 *   scales  uint8 [rows][kp / 32]  e + 127; 255: the block's values are NaN
 * Columns d .. kp - 1 hold code 0, whole blocks of them under scale byte 0. For d a multiple
 * of 128 this is the plain row-major form that checkpoints hold.
 * Quantisation: a = the block's largest magnitude, e = max(floor(log2 a) - 2, -127) (-127 for
 * a block of zeros), code = x / 2^e rounded to the nearest magnitude, ties to the even code,
 * over 6 to 6. A block that holds a NaN or an infinity gets scale byte 255.
 */
SD_API int32_t sd_mxfp4_columns(int32_t d);

/*
 * Quantise rows of x, and the values back.
 *   x       [rows][d] of type x_type (SD_F32, SD_BF16, SD_F16), row stride x_stride elements
 *           (>= d; any alignment of the element type, 16-byte aligned rows are fastest)
 *   rows    >= 1; d a positive multiple of 8, at most 2^20; rows * kp at most 2^37 - 2^13
 *   codes, scales  as above, 16-byte and 4-byte aligned
 * sd_mxfp4_dequantize writes x rounded once to x_type (exact in fp32 and, unless the scale
 * leaves its normal range, in bf16; scale bytes over 252, which quantisation never gives, can
 * pass the largest fp32 number and then give an infinity); nothing between row ends and
 * strides is written.
 * Errors: SD_EINVAL (null pointer, unknown type), SD_ESHAPE, SD_EALIGN, SD_EDEVICE.
 */
SD_API int32_t sd_mxfp4_quantize(const void *x, int32_t x_type, int32_t rows, int32_t d,
                                 int64_t x_stride, uint8_t *codes, uint8_t *scales, void *stream);
SD_API int32_t sd_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int32_t rows,
                                   int32_t d, void *x, int32_t x_type, int64_t x_stride,
                                   void *stream);

/*
 * The form of an MXFP4 LM head that sd_mxfp4_logits reads: the codes and scales above, re-laid
 * once into tiles of 64 rows by 128 columns (rows past V zero), in one device buffer.
 * sd_mxfp4_head_bytes: its size (0 unless V is in [1, 2^21], d is a positive multiple of 8 up to
 * 2^20, and there are fewer than 2^24 tiles).
 * sd_mxfp4_head: writes it on `stream`.
 *   codes, scales  as above, [V] rows
 *   head           sd_mxfp4_head_bytes(V, d) bytes, 256-byte aligned, apart from the inputs
 *   Errors: SD_EINVAL (null pointer), SD_ESHAPE, SD_EALIGN, SD_EWORKSPACE (head_bytes too
 *   small), SD_EDEVICE.
 */
SD_API size_t sd_mxfp4_head_bytes(int32_t V, int32_t d);
SD_API int32_t sd_mxfp4_head(const uint8_t *codes, const uint8_t *scales, int32_t V, int32_t d,
                             uint8_t *head, size_t head_bytes, void *stream);

/*
 * Logits of hidden rows under an MXFP4 LM head (LFM2.5-DSpark blog, "Training &
 * Architecture", and DSpark summary, "Training": drafter and target share the LM head). For
 * a drafter: verification keeps the target's distribution whatever the drafter's logits are,
 * so its copy of the LM head may be coarse.
 *   hidden   [M][d] of type hidden_type, row stride hidden_stride elements; quantised to
 *            MXFP4 in the call (into the workspace)
 *   head     the [V][d] LM head as sd_mxfp4_head wrote it
 *   logits   [M][V] of type logits_type, row stride logits_stride elements (>= V): out
 *   workspace  sd_mxfp4_logits_workspace_bytes(M, d) bytes
 * logits[m][v] = sum over blocks of 2^(eh + ew) sum of the code products, accumulated in
 * fp32, rounded once to logits_type. A row of hidden with a NaN or an infinity gives NaN.
 * Errors: SD_EINVAL (null pointer, unknown type), SD_ESHAPE (M < 1, d not a positive multiple
 * of 8 up to 2^20, V outside [1, 2^21], 2^24 or more tiles of hidden rows, of the LM head or, at
 * 128 x 128, of logits, short strides), SD_EALIGN, SD_EWORKSPACE, SD_EDEVICE.
 */
SD_API size_t sd_mxfp4_logits_workspace_bytes(int32_t M, int32_t d);
SD_API int32_t sd_mxfp4_logits(const void *hidden, int32_t hidden_type, int32_t M, int32_t d,
                               int64_t hidden_stride, const uint8_t *head, int32_t V,
                               void *logits, int32_t logits_type, int64_t logits_stride,
                               void *workspace, size_t workspace_bytes, void *stream);

/*
 * RMS norm of rows with the residual's addition (DSpark summary, "Production deployment": the
 * LM head maps the hidden state to logits; this is the step that makes that hidden state):
 *   s = x + residual, added in fp32 and rounded to the residual's type (s = x without one)
 *   y = s / sqrt(mean(s^2) + eps) * (weight_offset + weight)
 * with the mean, the root and the product in fp64 and y rounded to fp32, then to its type.
 *   x         [rows][d] of type x_type, row stride x_stride elements (>= d)
 *   residual  [rows][d] of type residual_type (x_type or SD_F32), or NULL
 *   weight    [d] of type weight_type, or NULL: no factor (weight_offset is not used then)
 *   eps       finite and >= 0 (a row of zeros under eps 0 gives NaN)
 *   sum       [rows][d] of residual_type or NULL: out, s; only with a residual
 *   sd_rms_norm:        y [rows][d] of type y_type: out
 *   sd_rms_norm_mxfp8:  codes, scales: out, y as MXFP8 rows (below; y's fp32 value is what is
 *                       quantised), d a multiple of 8
 * A row is read before any of it is written: sum or y may be x or the residual itself (same
 * address, type and stride), not the same one both; no other overlap is allowed. Any alignment of
 * the element types; 16-byte aligned rows are fastest. No workspace.
 * A NaN makes its row NaN. In a row with an infinity that column is NaN and the finite ones 0;
 * as MXFP8, where a block that holds a NaN reads as NaN, the other blocks 0.
 * Errors: SD_EINVAL (null pointer, unknown type, eps or weight_offset not finite, eps < 0, a sum
 * without a residual, y and sum the same), SD_ESHAPE (rows < 1, d outside [1, 2^20], d % 8 != 0 for MXFP8, short
 * strides), SD_EALIGN (an array not aligned to its elements; codes 16 bytes, scales 4), SD_EDEVICE.
 */
SD_API int32_t sd_rms_norm(const void *x, int32_t x_type, int64_t x_stride, const void *residual,
                           int32_t residual_type, int64_t residual_stride, const void *weight,
                           int32_t weight_type, float weight_offset, float eps, int32_t rows,
                           int32_t d, void *sum, int64_t sum_stride, void *y, int32_t y_type,
                           int64_t y_stride, void *stream);
SD_API int32_t sd_rms_norm_mxfp8(const void *x, int32_t x_type, int64_t x_stride,
                                 const void *residual, int32_t residual_type,
                                 int64_t residual_stride, const void *weight, int32_t weight_type,
                                 float weight_offset, float eps, int32_t rows, int32_t d, void *sum,
                                 int64_t sum_stride, uint8_t *codes, uint8_t *scales, void *stream);

/*
 * MXFP8 (OCP Microscaling Formats, e4m3): as MXFP4 with a byte a value, kp = sd_mxfp4_columns(d):
 *   codes   uint8 [rows][kp]       e4m3
 *   scales  uint8 [rows][kp / 32]  e + 127; 255: the block's values are NaN
 * Columns d .. kp - 1 hold code 0, whole blocks of them under scale byte 0.
 * Quantisation: a = the block's largest magnitude, e = max(floor(log2 a) - 8, -127), code =
 * x / 2^e rounded to the nearest e4m3 number, ties to the even code, over 448 to 448. A block that
 * holds a NaN or an infinity gets scale byte 255 and code 0.
 * Arguments and errors as for the MXFP4 calls. sd_mxfp8_dequantize rounds once to x_type (exact in
 * fp32 and bf16 unless the scale leaves their normal range; scale bytes over 246, which
 * quantisation never gives, can pass the largest fp32 number and then give an infinity).
 */
SD_API int32_t sd_mxfp8_quantize(const void *x, int32_t x_type, int32_t rows, int32_t d,
                                 int64_t x_stride, uint8_t *codes, uint8_t *scales, void *stream);
SD_API int32_t sd_mxfp8_dequantize(const uint8_t *codes, const uint8_t *scales, int32_t rows,
                                   int32_t d, void *x, int32_t x_type, int64_t x_stride,
                                   void *stream);

/*
 * The form of an MXFP8 LM head that sd_mxfp8_logits reads, made once: tiles of 64 rows by 128
 * columns in the order the matrix instructions take them. Arguments, limits and errors as for
 * sd_mxfp4_head_bytes and sd_mxfp4_head.
 */
SD_API size_t sd_mxfp8_head_bytes(int32_t V, int32_t d);
SD_API int32_t sd_mxfp8_head(const uint8_t *codes, const uint8_t *scales, int32_t V, int32_t d,
                             uint8_t *head, size_t head_bytes, void *stream);

/*
 * Logits of hidden rows under an MXFP8 LM head (a drafter's copy that is coarser than bf16 and
 * finer than MXFP4).
 *   hidden   hidden_type SD_F32, SD_BF16, SD_F16: [M][d], row stride hidden_stride elements,
 *            quantised to MXFP8 in the call; hidden_scales NULL
 *            hidden_type SD_MXFP8: codes [M][kp] as sd_rms_norm_mxfp8 or sd_mxfp8_quantize wrote
 *            them, 16-byte aligned, with hidden_scales [M][kp / 32], 4-byte aligned;
 *            hidden_stride kp
 *   head     the [V][d] LM head as sd_mxfp8_head wrote it
 *   logits   [M][V] of type logits_type, row stride logits_stride elements (>= V): out
 *   workspace  sd_mxfp8_logits_workspace_bytes(M, d) bytes; its header is left alone and need not
 *            have been prepared
 * logits[m][v] = the sum of the products of the values: every product exact, accumulated in fp32,
 * rounded once to logits_type, for any number of rows. Values are formed in bf16 (exact for scale
 * bytes 3 .. 246; smaller ones give values under bf16's smallest number, larger ones over its largest).
 * A row of hidden with a NaN or an infinity gives NaN.
 * Errors: as for sd_mxfp4_logits; SD_EINVAL also for hidden_scales that do not go with hidden_type.
 */
SD_API size_t sd_mxfp8_logits_workspace_bytes(int32_t M, int32_t d);
SD_API int32_t sd_mxfp8_logits(const void *hidden, int32_t hidden_type,
                               const uint8_t *hidden_scales, int32_t M, int32_t d,
                               int64_t hidden_stride, const uint8_t *head, int32_t V, void *logits,
                               int32_t logits_type, int64_t logits_stride, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * 4-bit integer weights with group scales: `group` (32, 64 or 128) consecutive columns of a row
 * share a scale and, in the asymmetric form, a zero; a value is (code - zero) * scale.
 *   codes   uint8 [rows][d / 2]      codes 0 .. 15, column 2 i in the low half of byte i
 *   scales  [rows][d / group]        of scale_type SD_BF16 or SD_F16
 *   zeros   uint8 [rows][d / group]  0 .. 15, or NULL: the symmetric form, every zero is 8
 * Quantisation:
 *   asymmetric  scale = (max(x, 0) - min(x, 0)) / 15, rounded to fp32 and to scale_type,
 *               zero = -min(x, 0) / scale, rounded and held to 15
 *   symmetric   scale = max |x| / 7 in fp32, rounded to scale_type
 *   code = x / scale rounded, plus zero, held to 0 .. 15
 * quotients in fp32, rounded to the nearest integer, ties to even. A scale under the smallest
 * normal fp32 number (2^-126) becomes 0, its zero 0 (8) and its codes that zero. A group that
 * holds a NaN or an infinity, or whose scale passes scale_type's largest number, has a NaN scale.
 *   x       [rows][d] of type x_type, row stride x_stride elements (any alignment of the element
 *           type, 16-byte aligned rows are fastest); rows >= 1, d a positive multiple of group, at
 *           most 2^20; rows * d at most 2^37 - 2^13
 *   codes, scales, zeros  16-, 4- and 4-byte aligned
 * sd_w4_dequantize writes the values, rounded once to x_type (products are exact in fp32).
 * Errors: SD_EINVAL (null pointer, unknown type), SD_ESHAPE (also a group not among the three),
 * SD_EALIGN, SD_EDEVICE.
 */
SD_API int32_t sd_w4_quantize(const void *x, int32_t x_type, int32_t rows, int32_t d,
                              int64_t x_stride, int32_t group, uint8_t *codes, void *scales,
                              int32_t scale_type, uint8_t *zeros, void *stream);
SD_API int32_t sd_w4_dequantize(const uint8_t *codes, const void *scales, int32_t scale_type,
                                const uint8_t *zeros, int32_t rows, int32_t d, int32_t group,
                                void *x, int32_t x_type, int64_t x_stride, void *stream);

/*
 * The form of such an LM head that sd_w4_logits reads, made once from any such codes, scales and
 * zeros: tiles of 64 rows by 128 columns in the order the matrix instructions take them.
 * sd_w4_head_bytes: its size (has_zeros: 1 with zeros, 0 without; 0 unless V is in [1, 2^21], d is
 * a positive multiple of group up to 2^20, group is 32, 64 or 128, and there are fewer than 2^24
 * tiles).
 * sd_w4_head: writes it on `stream`; head 256-byte aligned, apart from the inputs.
 *   Errors: SD_EINVAL (null pointer, unknown scale_type), SD_ESHAPE, SD_EALIGN, SD_EWORKSPACE
 *   (head_bytes too small), SD_EDEVICE.
 */
SD_API size_t sd_w4_head_bytes(int32_t V, int32_t d, int32_t group, int32_t has_zeros);
SD_API int32_t sd_w4_head(const uint8_t *codes, const void *scales, int32_t scale_type,
                          const uint8_t *zeros, int32_t V, int32_t d, int32_t group, uint8_t *head,
                          size_t head_bytes, void *stream);

/*
 * Logits of hidden rows under a 4-bit LM head with group scales; the hidden rows are not rounded.
 *   hidden   [M][d] of hidden_type SD_BF16 or SD_F16, row stride hidden_stride elements
 *   head, V, d, group, scale_type, has_zeros   as sd_w4_head wrote it
 *   logits   [M][V] of type logits_type, row stride logits_stride elements (>= V): out
 *   workspace  sd_w4_logits_workspace_bytes(M, d, group) bytes, as for sd_mxfp8_logits
 * logits[m][v] = sum over groups of scale * (sum code * hidden - zero * sum hidden), products
 * exact, sums in fp32, rounded once to logits_type. A row of hidden with a NaN or an infinity gives
 * NaN, and so may one whose sum of 15 |hidden| over a group passes the largest fp32 number.
 * Errors: SD_EINVAL (null pointer, unknown type), SD_ESHAPE (M < 1, V, d or group as above, 2^24
 * or more tiles of hidden rows, of the LM head or, at 128 x 128, of logits, short strides),
 * SD_EALIGN, SD_EWORKSPACE, SD_EDEVICE.
 */
SD_API size_t sd_w4_logits_workspace_bytes(int32_t M, int32_t d, int32_t group);
SD_API int32_t sd_w4_logits(const void *hidden, int32_t hidden_type, int32_t M, int32_t d,
                            int64_t hidden_stride, const uint8_t *head, int32_t V, int32_t group,
                            int32_t scale_type, int32_t has_zeros, void *logits,
                            int32_t logits_type, int64_t logits_stride, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * Sampling settings (host struct of device pointers, each may be NULL: that filter is off,
 * temperature 1). One value per request:
 *   temperature  fp32, finite and >= 0; 0 keeps the likeliest id alone
 *   top_k        int32; < 1 or >= V: off
 *   top_p        fp32; >= 1: off; <= 0 keeps the likeliest id alone
 *   min_p        fp32; <= 0: off; over 1 counts as 1
 * Out-of-range temperatures (NaN, infinite, negative) count as 0, a NaN top_p or min_p as
 * off; each raises SD_FLAG_SAMPLING.
 * The filtered distribution of a logit row z: rank the ids by larger logit, then lower id
 * (NaN counts as -inf; ids at -inf are never kept), with weights w = exp((z - max) / T);
 * top-k keeps the first k; top-p of these the shortest leading run that holds a share of at
 * least top_p of their weight; min-p of these the ids with w >= min_p. Probabilities are the
 * kept weights over their sum. With a logit of +inf the ids at +inf share the whole weight.
 */
typedef struct sd_sampling {
    const float *temperature;
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
} sd_sampling;

/*
 * Draw one token per logit row from its filtered distribution, by inverse CDF in ascending
 * vocabulary id: the smallest kept id whose running weight exceeds u times the total.
 *   logits    [R][V] of type logits_type, row stride logits_stride elements (>= V)
 *   u         fp32 [R], uniforms in [0, 1) (values outside count as the nearest in it)
 *   sampling  settings, row i reads entry i / rows_per_request of each
 *   tokens    int32 [R], element stride token_stride (>= 1): out; -1 for a row without any
 *             logit above -inf (SD_FLAG_EMPTY_ROW)
 *   kept      int32 [R] or NULL: out, size of the kept set
 *   logprob   fp32 [R] or NULL: out, log of the token's filtered probability (-inf with -1)
 *   workspace sd_sample_workspace_bytes(R, V) bytes
 * Weights are formed in fp64 and summed exactly in units of 2^-46 of the largest (V over 2^17:
 * 2^(ceil(log2 V) - 63), 2^-42 at 2^21): an id whose weight is below half a unit is never drawn,
 * and a border of top-p or of the draw is met to V / 2 units.
 * Errors: SD_EINVAL (null pointer, unknown type), SD_ESHAPE (R outside [1, 2^22], V outside
 * [1, 2^21], rows_per_request < 1, short strides), SD_EALIGN (an array not aligned to its elements),
 * SD_EWORKSPACE, SD_EDEVICE.
 */
SD_API size_t sd_sample_workspace_bytes(int32_t R, int32_t V);
SD_API int32_t sd_sample(const void *logits, int32_t logits_type, int64_t logits_stride, int32_t R,
                         int32_t V, const float *u, const sd_sampling *sampling,
                         int32_t rows_per_request, int32_t *tokens, int64_t token_stride,
                         int32_t *kept, float *logprob, void *workspace, size_t workspace_bytes,
                         void *stream);

/*
 * Rejection acceptance (sd_accept_rejection's rule) when the target is sampled through
 * temperature, top-k, top-p and min-p and the drafts were drawn from the drafter's logits
 * through the same settings (sd_sample): with p' and q' the filtered distributions of the
 * target row and the drafter row,
 *   position j < L_r survives iff u_accept[r][j] < min(1, p'_j(x_j) / q'_j(x_j)) (a token
 *   with p' = 0 never does);
 *   a_r = first failing j, else L_r;
 *   if a_r < L_r the token is drawn from norm(max(0, p'_a - q'_a)) (from p'_a, raising
 *   SD_FLAG_NO_RESIDUAL, when that has no mass), else from p'_{L_r}; draws as in sd_sample,
 *   probabilities in units of 2^-51: a residual under half of that at every id has no mass.
 * Lossless: the emitted tokens follow p', where the drafts were drawn from the very values of
 * draft_logits (drawn from finer logits that were rounded to bf16 afterwards, they follow
 * another q').
 *   logits    fp32 [B * (gamma + 1)][V] written by sd_verify_logits (any temperature)
 *   draft_logits bf16 [B][gamma][V], draft_tokens, verify_len, row_offsets, u_accept,
 *   u_resample, accept_len, next_token, counters   as for sd_accept_rejection
 *   sampling  settings of each request (temperature 0: both sides keep their likeliest id)
 *   workspace sd_accept_filtered_workspace_bytes(B, gamma, V) bytes
 * A target row without any logit above -inf emits -1 and raises SD_FLAG_EMPTY_ROW.
 * Errors: as for sd_accept_rejection; SD_ESHAPE also for B (2 gamma + 1) over 2^22.
 */
SD_API size_t sd_accept_filtered_workspace_bytes(int32_t B, int32_t gamma, int32_t V);
SD_API int32_t sd_accept_filtered(const float *logits, const uint16_t *draft_logits,
                                  const int32_t *draft_tokens, const int32_t *verify_len,
                                  const int32_t *row_offsets, const float *u_accept,
                                  const float *u_resample, const sd_sampling *sampling, int32_t B,
                                  int32_t gamma, int32_t V, int32_t *accept_len,
                                  int32_t *next_token, int64_t *counters, void *workspace,
                                  size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SD_VERIFY_H */
