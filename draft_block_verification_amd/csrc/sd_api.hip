// C ABI of libsdverify: argument validation, workspace layout and kernel dispatch.
// Every check that can be made on the host runs before any GPU work is enqueued.
#include <math.h>
#include <string.h>

#include <cmath>
#include <mutex>

#include "sd_launch.h"

using namespace sdv;

// Scratch of sd_verify_greedy_noalloc: the verify workspace for callers that cannot
// allocate. One copy per GPU, at its own address on each; host code uses only the
// address looked up per device (scratch_address), never this name.
static __device__ __align__(256) uint8_t scratch[SD_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int32_t kAbiVersion = 2;
constexpr int kMaxGamma = 64;        // one wavefront of draft positions per request
constexpr int kMaxVocab = 1 << 21;   // bound of the sampler's per-row tile table

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int32_t check_sizes(int32_t B, int32_t gamma, int32_t d, int32_t V) {
  if (B < 1 || gamma < 1 || gamma > kMaxGamma || d < 8 || (d % 8) != 0 || V < 1 ||
      V > kMaxVocab)
    return SD_ESHAPE;
  // Row capacity, logits and partial arrays must stay addressable.
  const int64_t cap = (int64_t)B * (gamma + 1);
  if (cap > (int64_t)1 << 30 || cap * (int64_t)V > ((int64_t)1 << 46) ||
      (int64_t)V * d > ((int64_t)1 << 46))
    return SD_ESHAPE;
  return SD_OK;
}

// Rows that one call of the filtered samplers takes: a workgroup of 512 threads each.
constexpr int64_t kMaxFilterRows = 1 << 22;

int32_t check_filtered(int32_t B, int32_t gamma, int32_t V) {
  const int32_t st = check_sizes(B, gamma, 8, V);
  if (st != SD_OK) return st;
  return (int64_t)B * (2 * gamma + 1) > kMaxFilterRows ? SD_ESHAPE : SD_OK;
}

bool known_type(int32_t t) { return t == SD_F32 || t == SD_BF16 || t == SD_F16; }

size_t type_size(int32_t t) { return t == SD_F32 ? 4 : 2; }

constexpr int kMaxMxColumns = 1 << 20;

// A launch has under 2^32 threads along x. Rows by row: four items of eight columns a thread,
// 256 threads a workgroup. Rows in tiles of 64 x 128: 256 threads a tile.
bool mx_rows_fit(int32_t rows, int32_t d) {
  return (int64_t)rows * (mx_padded(d) / 8) <= ((int64_t)1 << 34) - 1024;
}

bool mx_tiles_fit(int32_t rows, int32_t d) {
  return ((int64_t)rows + 63) / 64 * (mx_padded(d) / 128) < 1 << 24;
}

// Shared checks of the MXFP4 calls: [rows][d] of `type` beside its codes and scales.
int32_t check_mx(const void *x, int32_t type, int32_t rows, int32_t d, int64_t stride,
                 const uint8_t *codes, const uint8_t *scales) {
  if (!x || !codes || !scales || !known_type(type)) return SD_EINVAL;
  if (rows < 1 || d < 8 || d % 8 != 0 || d > kMaxMxColumns || stride < d ||
      stride > ((int64_t)1 << 40) || !mx_rows_fit(rows, d))
    return SD_ESHAPE;
  if (!aligned(x, type_size(type)) || !aligned(codes, 16) || !aligned(scales, 4)) return SD_EALIGN;
  return SD_OK;
}

bool stride_fits(int64_t stride, int64_t columns) { return stride >= columns && stride <= (int64_t)1 << 40; }

// Shared checks of the norms.
int32_t check_norm(const NormArgs &a) {
  if (!a.x || !known_type(a.x_type) || (a.w && !known_type(a.w_type)) || !(a.eps >= 0.f) ||
      !std::isfinite(a.eps) || !std::isfinite(a.offset) || (a.sum && !a.r))
    return SD_EINVAL;
  if (a.r && a.r_type != a.x_type && a.r_type != SD_F32) return SD_EINVAL;
  if (a.rows < 1 || a.d < 1 || a.d > kMaxMxColumns || !stride_fits(a.x_stride, a.d) ||
      (a.r && !stride_fits(a.r_stride, a.d)) || (a.sum && !stride_fits(a.sum_stride, a.d)))
    return SD_ESHAPE;
  if (!aligned(a.x, type_size(a.x_type)) || (a.r && !aligned(a.r, type_size(a.r_type))) ||
      (a.sum && !aligned(a.sum, type_size(a.r_type))) || (a.w && !aligned(a.w, type_size(a.w_type))))
    return SD_EALIGN;
  return SD_OK;
}

bool w4_group(int32_t d, int32_t group) {
  return (group == 32 || group == 64 || group == 128) && d >= group && d % group == 0 && d <= kMaxMxColumns;
}

bool w4_scale_type(int32_t t) { return t == SD_BF16 || t == SD_F16; }

// Shared checks of the 4-bit integer calls over rows.
int32_t check_w4(const void *x, int32_t type, int32_t rows, int32_t d, int64_t stride, int32_t group,
                 const uint8_t *codes, const void *scales, int32_t scale_type, const uint8_t *zeros) {
  if (!x || !codes || !scales || !known_type(type) || !w4_scale_type(scale_type)) return SD_EINVAL;
  if (rows < 1 || !w4_group(d, group) || !stride_fits(stride, d) || !mx_rows_fit(rows, d)) return SD_ESHAPE;
  if (!aligned(x, type_size(type)) || !aligned(codes, 16) || !aligned(scales, 4) || (zeros && !aligned(zeros, 4)))
    return SD_EALIGN;
  return SD_OK;
}

// The smallest output tile of the products' large calls is 128 x 128, by 256 threads; their small
// calls have a workgroup for 64 ids and 32 rows at least, or 64 rows and more at a time.
bool logits_fit(int32_t M, int32_t V) {
  return ((int64_t)M + 127) / 128 * (((int64_t)V + 127) / 128) < 1 << 24;
}

SampleSettings settings(const sd_sampling &s) {
  return SampleSettings{s.temperature, s.top_k, s.top_p, s.min_p};
}

bool aligned_settings(const sd_sampling &s) {
  return aligned(s.temperature, 4) && aligned(s.top_k, 4) && aligned(s.top_p, 4) && aligned(s.min_p, 4);
}

size_t verify_ws_bytes(int32_t B, int32_t gamma, int32_t V) {
  return verify_workspace_layout(B, gamma, V, nullptr, nullptr, nullptr);
}

size_t accept_ws_bytes(int32_t B, int32_t gamma, int32_t V) {
  return accept_workspace_layout(B, gamma, V, nullptr);
}

int32_t launch_status(hipError_t e) { return e == hipSuccess ? SD_OK : SD_EDEVICE; }

// Clears n 32-bit words with a kernel (no memset node, so it is safe under graph capture).
__global__ void k_clear_words(uint32_t *p, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0u;
}

hipError_t clear_words(void *p, int n, hipStream_t s) {
  hipLaunchKernelGGL(k_clear_words, dim3((n + 63) / 64), dim3(64), 0, s,
                     reinterpret_cast<uint32_t *>(p), n);
  return hipGetLastError();
}

__global__ void k_copy_word(const uint32_t *src, uint32_t *dst) { *dst = *src; }

// Sets the publication area after a verify workspace's header to kPubEmpty words.
__global__ void k_fill_pub(unsigned long long *p, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = kPubEmpty;
}

// A new workspace's header cleared and, when it is large enough to hold one, its
// publication area emptied.
hipError_t init_workspace(void *ws, size_t bytes, hipStream_t s) {
  hipError_t e = clear_words(ws, sizeof(WsHeader) / 4, s);
  if (e != hipSuccess || bytes < sizeof(WsHeader) + kPubBytes) return e;
  const int n = 2 * kPubWords;
  hipLaunchKernelGGL(k_fill_pub, dim3((n + 255) / 256), dim3(256), 0, s,
                     reinterpret_cast<unsigned long long *>(reinterpret_cast<char *>(ws) + sizeof(WsHeader)), n);
  return hipGetLastError();
}

// Device address of `scratch` on the current device, looked up on the first call made
// with that device current and kept for the process.
constexpr int kMaxScratchDevices = 256;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxScratchDevices] = {};

// The first lookup on a device also prepares the scratch as sd_workspace_init prepares
// a workspace (enqueued on s); the address is kept only once that is enqueued.
hipError_t scratch_address(void **out, hipStream_t s) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxScratchDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void *p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (!p) return hipErrorInvalidSymbol;
    e = init_workspace(p, SD_NOALLOC_SCRATCH_BYTES, s);
    if (e != hipSuccess) return e;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return hipSuccess;
}

}  // namespace

extern "C" {

int32_t sd_abi_version(void) { return kAbiVersion; }

const char *sd_status_string(int32_t status) {
  switch (status) {
    case SD_OK: return "ok";
    case SD_EINVAL: return "invalid argument (null pointer, temperature or threshold)";
    case SD_ESHAPE: return "invalid sizes (B, gamma, d or V)";
    case SD_EALIGN: return "misaligned tensor pointer";
    case SD_EWORKSPACE: return "workspace missing or too small";
    case SD_EDEVICE: return "HIP launch or copy failed";
    case SD_ESCRATCH: return "problem exceeds the allocation-free scratch (SD_NOALLOC_SCRATCH_BYTES)";
    default: return "unknown status";
  }
}

size_t sd_verify_workspace_bytes(int32_t B, int32_t gamma, int32_t d, int32_t V) {
  if (check_sizes(B, gamma, d, V) != SD_OK) return 0;
  return verify_ws_bytes(B, gamma, V);
}

size_t sd_accept_workspace_bytes(int32_t B, int32_t gamma, int32_t V) {
  if (check_sizes(B, gamma, 8, V) != SD_OK) return 0;
  return accept_ws_bytes(B, gamma, V);
}

int32_t sd_workspace_init(void *workspace, size_t workspace_bytes, void *stream) {
  if (!workspace || workspace_bytes < sizeof(WsHeader)) return SD_EWORKSPACE;
  if (!aligned(workspace, 256)) return SD_EALIGN;
  return launch_status(init_workspace(workspace, workspace_bytes, (hipStream_t)stream));
}

int32_t sd_device_flags(void *workspace, void *stream, uint32_t *flags, int32_t clear) {
  if (!workspace || !flags) return SD_EINVAL;
  hipStream_t s = (hipStream_t)stream;
  if (hipStreamSynchronize(s) != hipSuccess) return SD_EDEVICE;
  uint32_t v = 0;
  if (hipMemcpy(&v, workspace, sizeof(v), hipMemcpyDeviceToHost) != hipSuccess) return SD_EDEVICE;
  *flags = v;
  if (clear) {
    if (clear_words(workspace, 1, s) != hipSuccess) return SD_EDEVICE;
    if (hipStreamSynchronize(s) != hipSuccess) return SD_EDEVICE;
  }
  return SD_OK;
}

int32_t sd_truncate_by_confidence(const float *conf, int32_t B, int32_t gamma, float threshold,
                                  int32_t *verify_len, int32_t *row_offsets, void *stream) {
  if (!conf || !verify_len || !row_offsets) return SD_EINVAL;
  if (!isfinite(threshold)) return SD_EINVAL;
  if (check_sizes(B, gamma, 8, 1) != SD_OK) return SD_ESHAPE;
  if (!aligned(conf, 4) || !aligned(verify_len, 4) || !aligned(row_offsets, 4)) return SD_EALIGN;
  return launch_status(launch_truncate(conf, B, gamma, threshold, verify_len, row_offsets,
                                       (hipStream_t)stream));
}

int32_t sd_schedule_prefix(const float *conf, const float *conf_stale, int32_t R, int32_t gamma,
                           const float *sps, int32_t n_sps, int32_t mode, int32_t *verify_len,
                           int32_t *row_offsets, void *stream) {
  static_assert(kSchedMaxCandidates == SD_SCHED_MAX_CANDIDATES, "candidate bound");
  if (!conf || !sps || !verify_len || !row_offsets) return SD_EINVAL;
  if (mode != SD_SCHED_EARLY_STOP && mode != SD_SCHED_TOP_K) return SD_EINVAL;
  if (mode == SD_SCHED_EARLY_STOP && conf_stale) return SD_EINVAL;
  if (R < 1 || gamma < 1 || gamma > kMaxGamma) return SD_ESHAPE;
  if ((int64_t)R * gamma > kSchedMaxCandidates) return SD_ESHAPE;
  if ((int64_t)n_sps < (int64_t)R * (gamma + 1) + 1) return SD_ESHAPE;
  if (!aligned(conf, 4) || !aligned(sps, 4) || !aligned(verify_len, 4) ||
      !aligned(row_offsets, 4) || (conf_stale && !aligned(conf_stale, 4)))
    return SD_EALIGN;
  return launch_status(launch_schedule(conf, conf_stale, R, gamma, sps, mode, verify_len,
                                       row_offsets, (hipStream_t)stream));
}

}  // extern "C"

namespace {

// Shared validation and argument set-up of the verify calls.
int32_t verify_setup(const uint16_t *hidden, const uint16_t *lm_head, const sd_w12 *w12,
                     bool blocked, const int32_t *draft_tokens, const int32_t *verify_len,
                     const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d, int32_t V,
                     float temperature, float *logits, sd_row_stats *stats, bool need_stats,
                     void *workspace, size_t workspace_bytes, VerifyArgs *out) {
  if (!hidden || (!lm_head && !w12) || (need_stats && !stats)) return SD_EINVAL;
  if (w12) {
    if (!w12->codes || !w12->corr) return SD_EINVAL;
    if (w12->b2 < 1 || w12->b2 > 121) return SD_EINVAL;
    // The W12 stream is read by the skinny contraction only.
    if (d % 128 != 0 || (int64_t)B * (gamma + 1) > 64 || w12->cap < 4 || w12->cap % 4 != 0 ||
        w12->cap > kW12MaxCap)
      return SD_ESHAPE;
    if (!aligned(w12->codes, 16) || !aligned(w12->corr, 16)) return SD_EALIGN;
  }
  // The blocked bf16 LM head, like W12, is read by the skinny contraction only.
  if (blocked && (d % 128 != 0 || (int64_t)B * (gamma + 1) > 64)) return SD_ESHAPE;
  if ((verify_len == nullptr) != (row_offsets == nullptr)) return SD_EINVAL;
  if (!isfinite(temperature) || temperature < 0.f) return SD_EINVAL;
  const int32_t sz = check_sizes(B, gamma, d, V);
  if (sz != SD_OK) return sz;
  if (!aligned(hidden, 16) || (lm_head && !aligned(lm_head, 16)) || (stats && !aligned(stats, 8)) ||
      (logits && !aligned(logits, 16)) || (draft_tokens && !aligned(draft_tokens, 4)) ||
      (verify_len && (!aligned(verify_len, 4) || !aligned(row_offsets, 4))))
    return SD_EALIGN;
  if (!workspace || workspace_bytes < verify_ws_bytes(B, gamma, V)) return SD_EWORKSPACE;
  if (!aligned(workspace, 256)) return SD_EALIGN;
  size_t part_off = 0, zx_off = 0;
  int part_stride = 0;
  verify_workspace_layout(B, gamma, V, &part_off, &part_stride, &zx_off);
  char *wsb = reinterpret_cast<char *>(workspace);
  *out = VerifyArgs{};
  VerifyArgs &a = *out;
  a.hidden = hidden;
  a.W = w12 ? nullptr : lm_head;
  a.w_blocked = blocked;
  a.w12_codes = w12 ? w12->codes : nullptr;
  a.w12_corr = w12 ? w12->corr : nullptr;
  a.w12_cap = w12 ? w12->cap : 0;
  a.w12_lut0 = a.w12_lut1 = 0u;
  if (w12) {
    // High byte of code t (sign clear): 0 for t = 0, b2 + t - 1 otherwise.
    for (int t = 1; t < 8; ++t) {
      const uint32_t hb = (uint32_t)(w12->b2 + t - 1) << (8 * (t & 3));
      if (t < 4) a.w12_lut0 |= hb; else a.w12_lut1 |= hb;
    }
  }
  a.draft_tokens = draft_tokens;
  a.verify_len = verify_len;
  a.rm = RowMap{row_offsets, B, gamma};
  a.d = d;
  a.V = V;
  a.temperature = temperature;
  a.scale_log2 = temperature > 0.f ? (float)(1.4426950408889634 / (double)temperature) : 0.f;
  a.invT = temperature > 0.f ? 1.0 / (double)temperature : 0.0;
  a.logits = logits;
  a.partials = reinterpret_cast<TilePartial *>(wsb + part_off);
  a.part_stride = part_stride;
  a.zx = reinterpret_cast<double *>(wsb + zx_off);
  a.stats = stats;
  a.ws = reinterpret_cast<WsHeader *>(workspace);
  return SD_OK;
}

// The three verify calls for any LM-head form: bf16 [V][d] (lm_head), W12 (w12) or the
// blocked bf16 copy (lm_head with blocked).
int32_t verify_logits_impl(const uint16_t *hidden, const uint16_t *lm_head, const sd_w12 *w12,
                           bool blocked, const int32_t *draft_tokens, const int32_t *verify_len,
                           const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                           int32_t V, float temperature, float *logits, sd_row_stats *stats,
                           void *workspace, size_t workspace_bytes, void *stream) {
  VerifyArgs a;
  const int32_t st = verify_setup(hidden, lm_head, w12, blocked, draft_tokens, verify_len,
                                  row_offsets, B, gamma, d, V, temperature, logits, stats, true,
                                  workspace, workspace_bytes, &a);
  if (st != SD_OK) return st;
  return launch_status(launch_verify(a, (hipStream_t)stream));
}

int32_t verify_contraction_impl(const uint16_t *hidden, const uint16_t *lm_head,
                                const sd_w12 *w12, bool blocked, const int32_t *verify_len,
                                const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                                int32_t V, float temperature, float *logits, void *workspace,
                                size_t workspace_bytes, void *stream) {
  VerifyArgs a;
  const int32_t st = verify_setup(hidden, lm_head, w12, blocked, nullptr, verify_len, row_offsets,
                                  B, gamma, d, V, temperature, logits, nullptr, false, workspace,
                                  workspace_bytes, &a);
  if (st != SD_OK) return st;
  int n_part = 0;
  bool zx_done = false;
  return launch_status(launch_contraction(a, (hipStream_t)stream, &n_part, &zx_done));
}

int32_t verify_greedy_impl(const uint16_t *hidden, const uint16_t *lm_head, const sd_w12 *w12,
                           bool blocked, const int32_t *draft_tokens, const int32_t *verify_len,
                           const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                           int32_t V, sd_row_stats *stats, int32_t *accept_len,
                           int32_t *next_token, int64_t *counters, void *workspace,
                           size_t workspace_bytes, void *stream) {
  if (!draft_tokens || !accept_len || !next_token) return SD_EINVAL;
  if (!aligned(accept_len, 4) || !aligned(next_token, 4) || (counters && !aligned(counters, 8)))
    return SD_EALIGN;
  VerifyArgs a;
  const int32_t st = verify_setup(hidden, lm_head, w12, blocked, draft_tokens, verify_len,
                                  row_offsets, B, gamma, d, V, 0.f, nullptr, stats, true,
                                  workspace, workspace_bytes, &a);
  if (st != SD_OK) return st;
  return launch_status(launch_verify_greedy(a, accept_len, next_token, counters,
                                            (hipStream_t)stream));
}

// Bytes of the blocked copy of a [V][d] LM head: ceil(V/64) * (d/128) blocks of 16 KB.
size_t blocked_bytes(int32_t V, int32_t d) {
  return (size_t)((V + 63) / 64) * (size_t)(d / 128) * 16384u;
}

}  // namespace

extern "C" {

int32_t sd_verify_logits(const uint16_t *hidden, const uint16_t *lm_head,
                         const int32_t *draft_tokens, const int32_t *verify_len,
                         const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                         int32_t V, float temperature, float *logits, sd_row_stats *stats,
                         void *workspace, size_t workspace_bytes, void *stream) {
  return verify_logits_impl(hidden, lm_head, nullptr, false, draft_tokens, verify_len,
                            row_offsets, B, gamma, d, V, temperature, logits, stats, workspace,
                            workspace_bytes, stream);
}

int32_t sd_verify_contraction(const uint16_t *hidden, const uint16_t *lm_head,
                              const int32_t *verify_len, const int32_t *row_offsets, int32_t B,
                              int32_t gamma, int32_t d, int32_t V, float temperature,
                              float *logits, void *workspace, size_t workspace_bytes,
                              void *stream) {
  return verify_contraction_impl(hidden, lm_head, nullptr, false, verify_len, row_offsets, B,
                                 gamma, d, V, temperature, logits, workspace, workspace_bytes,
                                 stream);
}

int32_t sd_verify_greedy(const uint16_t *hidden, const uint16_t *lm_head,
                         const int32_t *draft_tokens, const int32_t *verify_len,
                         const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                         int32_t V, sd_row_stats *stats, int32_t *accept_len,
                         int32_t *next_token, int64_t *counters, void *workspace,
                         size_t workspace_bytes, void *stream) {
  return verify_greedy_impl(hidden, lm_head, nullptr, false, draft_tokens, verify_len,
                            row_offsets, B, gamma, d, V, stats, accept_len, next_token, counters,
                            workspace, workspace_bytes, stream);
}

int32_t sd_verify_greedy_noalloc(const uint16_t *hidden, const uint16_t *lm_head,
                                 const int32_t *draft_tokens, const int32_t *verify_len,
                                 const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                                 int32_t V, sd_row_stats *stats, int32_t *accept_len,
                                 int32_t *next_token, int64_t *counters, uint32_t *flags,
                                 void *stream) {
  // Every host check before the scratch lookup, so bad arguments never touch the runtime.
  if (!lm_head || !draft_tokens || !accept_len || !next_token) return SD_EINVAL;
  const int32_t sz = check_sizes(B, gamma, d, V);
  if (sz != SD_OK) return sz;
  if (verify_ws_bytes(B, gamma, V) > SD_NOALLOC_SCRATCH_BYTES) return SD_ESCRATCH;
  if (!aligned(accept_len, 4) || !aligned(next_token, 4) || (counters && !aligned(counters, 8)) ||
      (flags && !aligned(flags, 4)))
    return SD_EALIGN;
  VerifyArgs a;
  // The setup checks run against a stand-in workspace address (never dereferenced on the
  // host); the real scratch address replaces it below.
  void *const probe = reinterpret_cast<void *>((uintptr_t)1 << 12);
  int32_t st = verify_setup(hidden, lm_head, nullptr, false, draft_tokens, verify_len, row_offsets,
                            B, gamma, d, V, 0.f, nullptr, stats, true, probe,
                            SD_NOALLOC_SCRATCH_BYTES, &a);
  if (st != SD_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  void *ws = nullptr;
  if (scratch_address(&ws, s) != hipSuccess) return SD_EDEVICE;
  st = verify_setup(hidden, lm_head, nullptr, false, draft_tokens, verify_len, row_offsets, B,
                    gamma, d, V, 0.f, nullptr, stats, true, ws, SD_NOALLOC_SCRATCH_BYTES, &a);
  if (st != SD_OK) return st;
  // The flag word starts every call at zero. The rest of the header and the publication
  // area carry over from the previous call, as in a workspace; partials and drafted-token
  // logits are written in full by the contraction before they are read.
  if (clear_words(ws, 1, s) != hipSuccess) return SD_EDEVICE;
  hipError_t e = launch_verify_greedy(a, accept_len, next_token, counters, s);
  if (e == hipSuccess && flags) {
    hipLaunchKernelGGL(k_copy_word, dim3(1), dim3(1), 0, s, reinterpret_cast<const uint32_t *>(ws),
                       flags);
    e = hipGetLastError();
  }
  return launch_status(e);
}

int32_t sd_verify_logits_w12(const uint16_t *hidden, const sd_w12 *lm_head,
                             const int32_t *draft_tokens, const int32_t *verify_len,
                             const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                             int32_t V, float temperature, float *logits, sd_row_stats *stats,
                             void *workspace, size_t workspace_bytes, void *stream) {
  if (!lm_head) return SD_EINVAL;
  return verify_logits_impl(hidden, nullptr, lm_head, false, draft_tokens, verify_len,
                            row_offsets, B, gamma, d, V, temperature, logits, stats, workspace,
                            workspace_bytes, stream);
}

int32_t sd_verify_contraction_w12(const uint16_t *hidden, const sd_w12 *lm_head,
                                  const int32_t *verify_len, const int32_t *row_offsets, int32_t B,
                                  int32_t gamma, int32_t d, int32_t V, float temperature,
                                  float *logits, void *workspace, size_t workspace_bytes,
                                  void *stream) {
  if (!lm_head) return SD_EINVAL;
  return verify_contraction_impl(hidden, nullptr, lm_head, false, verify_len, row_offsets, B,
                                 gamma, d, V, temperature, logits, workspace, workspace_bytes,
                                 stream);
}

int32_t sd_verify_greedy_w12(const uint16_t *hidden, const sd_w12 *lm_head,
                             const int32_t *draft_tokens, const int32_t *verify_len,
                             const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                             int32_t V, sd_row_stats *stats, int32_t *accept_len,
                             int32_t *next_token, int64_t *counters, void *workspace,
                             size_t workspace_bytes, void *stream) {
  if (!lm_head) return SD_EINVAL;
  return verify_greedy_impl(hidden, nullptr, lm_head, false, draft_tokens, verify_len,
                            row_offsets, B, gamma, d, V, stats, accept_len, next_token, counters,
                            workspace, workspace_bytes, stream);
}

size_t sd_lm_head_block_bytes(int32_t V, int32_t d) {
  if (V < 1 || d < 128 || d % 128 != 0) return 0;
  return blocked_bytes(V, d);
}

int32_t sd_lm_head_block(const uint16_t *lm_head, int32_t V, int32_t d, uint16_t *blocked,
                         size_t blocked_bytes_given, void *stream) {
  if (!lm_head || !blocked) return SD_EINVAL;
  if (V < 1 || d < 128 || d % 128 != 0) return SD_ESHAPE;
  if (!aligned(lm_head, 16) || !aligned(blocked, 16)) return SD_EALIGN;
  if (blocked_bytes_given < blocked_bytes(V, d)) return SD_EWORKSPACE;
  return launch_status(launch_block_lm_head(lm_head, V, d, blocked, (hipStream_t)stream));
}

int32_t sd_verify_logits_blocked(const uint16_t *hidden, const uint16_t *lm_head_blocked,
                                 const int32_t *draft_tokens, const int32_t *verify_len,
                                 const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                                 int32_t V, float temperature, float *logits,
                                 sd_row_stats *stats, void *workspace, size_t workspace_bytes,
                                 void *stream) {
  return verify_logits_impl(hidden, lm_head_blocked, nullptr, true, draft_tokens, verify_len,
                            row_offsets, B, gamma, d, V, temperature, logits, stats, workspace,
                            workspace_bytes, stream);
}

int32_t sd_verify_contraction_blocked(const uint16_t *hidden, const uint16_t *lm_head_blocked,
                                      const int32_t *verify_len, const int32_t *row_offsets,
                                      int32_t B, int32_t gamma, int32_t d, int32_t V,
                                      float temperature, float *logits, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  return verify_contraction_impl(hidden, lm_head_blocked, nullptr, true, verify_len, row_offsets,
                                 B, gamma, d, V, temperature, logits, workspace, workspace_bytes,
                                 stream);
}

int32_t sd_verify_greedy_blocked(const uint16_t *hidden, const uint16_t *lm_head_blocked,
                                 const int32_t *draft_tokens, const int32_t *verify_len,
                                 const int32_t *row_offsets, int32_t B, int32_t gamma, int32_t d,
                                 int32_t V, sd_row_stats *stats, int32_t *accept_len,
                                 int32_t *next_token, int64_t *counters, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  return verify_greedy_impl(hidden, lm_head_blocked, nullptr, true, draft_tokens, verify_len,
                            row_offsets, B, gamma, d, V, stats, accept_len, next_token, counters,
                            workspace, workspace_bytes, stream);
}

int32_t sd_accept_greedy(const sd_row_stats *stats, const int32_t *draft_tokens,
                         const int32_t *verify_len, const int32_t *row_offsets, int32_t B,
                         int32_t gamma, int32_t *accept_len, int32_t *next_token,
                         int64_t *counters, void *stream) {
  if (!stats || !draft_tokens || !accept_len || !next_token) return SD_EINVAL;
  if ((verify_len == nullptr) != (row_offsets == nullptr)) return SD_EINVAL;
  if (check_sizes(B, gamma, 8, 1) != SD_OK) return SD_ESHAPE;
  if (!aligned(stats, 8) || !aligned(draft_tokens, 4) || !aligned(accept_len, 4) ||
      !aligned(next_token, 4) || (counters && !aligned(counters, 8)) ||
      (verify_len && (!aligned(verify_len, 4) || !aligned(row_offsets, 4))))
    return SD_EALIGN;
  RowMap rm{row_offsets, B, gamma};
  return launch_status(launch_accept_greedy(stats, draft_tokens, verify_len, rm, accept_len,
                                            next_token, counters, (hipStream_t)stream));
}

int32_t sd_accept_rejection(const float *logits, const sd_row_stats *stats,
                            const uint16_t *draft_logits, const int32_t *draft_tokens,
                            const int32_t *verify_len, const int32_t *row_offsets,
                            const float *u_accept, const float *u_resample, int32_t B,
                            int32_t gamma, int32_t V, float temperature, int32_t *accept_len,
                            int32_t *next_token, int64_t *counters, void *workspace,
                            size_t workspace_bytes, void *stream) {
  return sd_accept_rejection_ex(logits, stats, draft_logits, draft_tokens, verify_len,
                                row_offsets, u_accept, u_resample, B, gamma, V, temperature,
                                accept_len, next_token, counters, nullptr, workspace,
                                workspace_bytes, stream);
}

int32_t sd_accept_rejection_ex(const float *logits, const sd_row_stats *stats,
                               const uint16_t *draft_logits, const int32_t *draft_tokens,
                               const int32_t *verify_len, const int32_t *row_offsets,
                               const float *u_accept, const float *u_resample, int32_t B,
                               int32_t gamma, int32_t V, float temperature, int32_t *accept_len,
                               int32_t *next_token, int64_t *counters, double *accept_rate,
                               void *workspace, size_t workspace_bytes, void *stream) {
  if (!logits || !stats || !draft_logits || !draft_tokens || !u_accept || !u_resample ||
      !accept_len || !next_token)
    return SD_EINVAL;
  if ((verify_len == nullptr) != (row_offsets == nullptr)) return SD_EINVAL;
  if (!isfinite(temperature) || !(temperature > 0.f)) return SD_EINVAL;
  if (check_sizes(B, gamma, 8, V) != SD_OK) return SD_ESHAPE;
  if (!aligned(logits, 16) || !aligned(stats, 8) || !aligned(draft_logits, 16) ||
      !aligned(draft_tokens, 4) || !aligned(u_accept, 4) || !aligned(u_resample, 4) ||
      !aligned(accept_len, 4) || !aligned(next_token, 4) || (counters && !aligned(counters, 8)) ||
      (accept_rate && !aligned(accept_rate, 8)) ||
      (verify_len && (!aligned(verify_len, 4) || !aligned(row_offsets, 4))))
    return SD_EALIGN;
  if (!workspace || workspace_bytes < accept_ws_bytes(B, gamma, V)) return SD_EWORKSPACE;
  if (!aligned(workspace, 256)) return SD_EALIGN;
  RowMap rm{row_offsets, B, gamma};
  return launch_status(launch_accept_rejection(logits, stats, draft_logits, draft_tokens,
                                               verify_len, rm, u_accept, u_resample, V,
                                               temperature, accept_len, next_token, counters,
                                               accept_rate, workspace, (hipStream_t)stream));
}


int32_t sd_verify_rejection(const uint16_t *hidden, const void *lm_head,
                            int32_t lm_head_layout, const uint16_t *draft_logits,
                            const int32_t *draft_tokens, const int32_t *verify_len,
                            const int32_t *row_offsets, const float *u_accept,
                            const float *u_resample, int32_t B, int32_t gamma, int32_t d,
                            int32_t V, float temperature, float *logits, sd_row_stats *stats,
                            int32_t *accept_len, int32_t *next_token, int64_t *counters,
                            double *accept_rate, void *verify_workspace,
                            size_t verify_workspace_bytes, void *accept_workspace,
                            size_t accept_workspace_bytes, void *stream) {
  if (lm_head_layout != SD_LM_HEAD_ROWS && lm_head_layout != SD_LM_HEAD_BLOCKED &&
      lm_head_layout != SD_LM_HEAD_W12)
    return SD_EINVAL;
  if (!lm_head || !logits || !stats || !draft_logits || !draft_tokens || !u_accept ||
      !u_resample || !accept_len || !next_token)
    return SD_EINVAL;
  if (!isfinite(temperature) || !(temperature > 0.f)) return SD_EINVAL;
  const bool w12 = lm_head_layout == SD_LM_HEAD_W12;
  VerifyArgs a;
  const int32_t st = verify_setup(
      hidden, w12 ? nullptr : static_cast<const uint16_t *>(lm_head),
      w12 ? static_cast<const sd_w12 *>(lm_head) : nullptr, lm_head_layout == SD_LM_HEAD_BLOCKED,
      draft_tokens, verify_len, row_offsets, B, gamma, d, V, temperature, logits, stats, true,
      verify_workspace, verify_workspace_bytes, &a);
  if (st != SD_OK) return st;
  if (!aligned(draft_logits, 16) || !aligned(u_accept, 4) || !aligned(u_resample, 4) ||
      !aligned(accept_len, 4) || !aligned(next_token, 4) || (counters && !aligned(counters, 8)) ||
      (accept_rate && !aligned(accept_rate, 8)))
    return SD_EALIGN;
  if (!accept_workspace || accept_workspace_bytes < accept_ws_bytes(B, gamma, V))
    return SD_EWORKSPACE;
  if (!aligned(accept_workspace, 256)) return SD_EALIGN;
  a.draft_logits = draft_logits;
  return launch_status(launch_verify_rejection(a, u_accept, u_resample, accept_len, next_token,
                                               counters, accept_rate, accept_workspace,
                                               (hipStream_t)stream));
}

int32_t sd_mxfp4_columns(int32_t d) { return d < 8 || d % 8 != 0 || d > kMaxMxColumns ? 0 : mx_padded(d); }

int32_t sd_mxfp4_quantize(const void *x, int32_t x_type, int32_t rows, int32_t d, int64_t x_stride,
                          uint8_t *codes, uint8_t *scales, void *stream) {
  const int32_t st = check_mx(x, x_type, rows, d, x_stride, codes, scales);
  if (st != SD_OK) return st;
  return launch_status(launch_mx_quantize(x, x_type, rows, d, x_stride, codes, scales,
                                          (hipStream_t)stream));
}

int32_t sd_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int32_t rows, int32_t d,
                            void *x, int32_t x_type, int64_t x_stride, void *stream) {
  const int32_t st = check_mx(x, x_type, rows, d, x_stride, codes, scales);
  if (st != SD_OK) return st;
  return launch_status(launch_mx_dequantize(codes, scales, rows, d, x, x_type, x_stride,
                                            (hipStream_t)stream));
}

size_t sd_mxfp4_head_bytes(int32_t V, int32_t d) {
  if (V < 1 || V > kMaxVocab || d < 8 || d % 8 != 0 || d > kMaxMxColumns || !mx_tiles_fit(V, d)) return 0;
  return mx_tiled_bytes(V, d, nullptr);
}

int32_t sd_mxfp4_head(const uint8_t *codes, const uint8_t *scales, int32_t V, int32_t d, uint8_t *head,
                      size_t head_bytes, void *stream) {
  if (!codes || !scales || !head) return SD_EINVAL;
  const size_t need = sd_mxfp4_head_bytes(V, d);
  if (need == 0) return SD_ESHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(head, 256)) return SD_EALIGN;
  if (head_bytes < need) return SD_EWORKSPACE;
  return launch_status(launch_mx_head(codes, scales, V, d, head, (hipStream_t)stream));
}

size_t sd_mxfp4_logits_workspace_bytes(int32_t M, int32_t d) {
  if (M < 1 || d < 8 || d % 8 != 0 || d > kMaxMxColumns || !mx_tiles_fit(M, d)) return 0;
  return mx_logits_workspace_bytes(M, d);
}

int32_t sd_mxfp4_logits(const void *hidden, int32_t hidden_type, int32_t M, int32_t d,
                        int64_t hidden_stride, const uint8_t *head, int32_t V, void *logits,
                        int32_t logits_type, int64_t logits_stride, void *workspace,
                        size_t workspace_bytes, void *stream) {
  if (!hidden || !head || !logits || !known_type(hidden_type) || !known_type(logits_type)) return SD_EINVAL;
  const size_t need = sd_mxfp4_logits_workspace_bytes(M, d);
  if (need == 0 || sd_mxfp4_head_bytes(V, d) == 0 || hidden_stride < d || hidden_stride > ((int64_t)1 << 40) ||
      logits_stride < V || logits_stride > ((int64_t)1 << 40))
    return SD_ESHAPE;
  // The smallest output tile of a call of more than 64 rows is 128 x 128, by 256 threads.
  if (((int64_t)M + 127) / 128 * (((int64_t)V + 127) / 128) >= 1 << 24) return SD_ESHAPE;
  if (!aligned(hidden, type_size(hidden_type)) || !aligned(head, 256) || !aligned(logits, type_size(logits_type)))
    return SD_EALIGN;
  if (!workspace || workspace_bytes < need) return SD_EWORKSPACE;
  if (!aligned(workspace, 256)) return SD_EALIGN;
  return launch_status(launch_mx_logits(hidden, hidden_type, M, d, hidden_stride, head, V, logits,
                                        logits_type, logits_stride, workspace, (hipStream_t)stream));
}

int32_t sd_rms_norm(const void *x, int32_t x_type, int64_t x_stride, const void *residual,
                    int32_t residual_type, int64_t residual_stride, const void *weight,
                    int32_t weight_type, float weight_offset, float eps, int32_t rows, int32_t d, void *sum,
                    int64_t sum_stride, void *y, int32_t y_type, int64_t y_stride, void *stream) {
  const NormArgs a{x, x_type, x_stride, residual, residual_type, residual_stride, weight, weight_type,
                   weight_offset, eps, rows, d, sum, sum_stride, y, y_type, y_stride, nullptr, nullptr};
  if (!y || !known_type(y_type) || y == sum) return SD_EINVAL;
  const int32_t st = check_norm(a);
  if (st != SD_OK) return st;
  if (!stride_fits(y_stride, d)) return SD_ESHAPE;
  if (!aligned(y, type_size(y_type))) return SD_EALIGN;
  return launch_status(launch_norm(a, (hipStream_t)stream));
}

int32_t sd_rms_norm_mxfp8(const void *x, int32_t x_type, int64_t x_stride, const void *residual,
                          int32_t residual_type, int64_t residual_stride, const void *weight,
                          int32_t weight_type, float weight_offset, float eps, int32_t rows, int32_t d,
                          void *sum, int64_t sum_stride, uint8_t *codes, uint8_t *scales, void *stream) {
  const NormArgs a{x, x_type, x_stride, residual, residual_type, residual_stride, weight, weight_type,
                   weight_offset, eps, rows, d, sum, sum_stride, nullptr, SD_F32, 0, codes, scales};
  if (!codes || !scales) return SD_EINVAL;
  const int32_t st = check_norm(a);
  if (st != SD_OK) return st;
  if (d % 8 != 0) return SD_ESHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return SD_EALIGN;
  return launch_status(launch_norm(a, (hipStream_t)stream));
}

int32_t sd_mxfp8_quantize(const void *x, int32_t x_type, int32_t rows, int32_t d, int64_t x_stride,
                          uint8_t *codes, uint8_t *scales, void *stream) {
  const int32_t st = check_mx(x, x_type, rows, d, x_stride, codes, scales);
  if (st != SD_OK) return st;
  return launch_status(launch_mx8_quantize(x, x_type, rows, d, x_stride, codes, scales, (hipStream_t)stream));
}

int32_t sd_mxfp8_dequantize(const uint8_t *codes, const uint8_t *scales, int32_t rows, int32_t d,
                            void *x, int32_t x_type, int64_t x_stride, void *stream) {
  const int32_t st = check_mx(x, x_type, rows, d, x_stride, codes, scales);
  if (st != SD_OK) return st;
  return launch_status(launch_mx8_dequantize(codes, scales, rows, d, x, x_type, x_stride, (hipStream_t)stream));
}

size_t sd_mxfp8_head_bytes(int32_t V, int32_t d) {
  return sd_mxfp4_head_bytes(V, d) == 0 ? 0 : mx8_head_bytes(V, d);
}

int32_t sd_mxfp8_head(const uint8_t *codes, const uint8_t *scales, int32_t V, int32_t d, uint8_t *head,
                      size_t head_bytes, void *stream) {
  if (!codes || !scales || !head) return SD_EINVAL;
  const size_t need = sd_mxfp8_head_bytes(V, d);
  if (need == 0) return SD_ESHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(head, 256)) return SD_EALIGN;
  if (head_bytes < need) return SD_EWORKSPACE;
  return launch_status(launch_mx8_head(codes, scales, V, d, head, (hipStream_t)stream));
}

size_t sd_mxfp8_logits_workspace_bytes(int32_t M, int32_t d) {
  return sd_mxfp4_logits_workspace_bytes(M, d) == 0 ? 0 : mx8_logits_workspace_bytes(M, d);
}

int32_t sd_mxfp8_logits(const void *hidden, int32_t hidden_type, const uint8_t *hidden_scales, int32_t M,
                        int32_t d, int64_t hidden_stride, const uint8_t *head, int32_t V, void *logits,
                        int32_t logits_type, int64_t logits_stride, void *workspace, size_t workspace_bytes,
                        void *stream) {
  const bool coded = hidden_type == SD_MXFP8;
  if (!hidden || !head || !logits || (!coded && !known_type(hidden_type)) || !known_type(logits_type) ||
      coded != (hidden_scales != nullptr))
    return SD_EINVAL;
  const size_t need = sd_mxfp8_logits_workspace_bytes(M, d);
  if (need == 0 || sd_mxfp8_head_bytes(V, d) == 0 || !logits_fit(M, V) || !stride_fits(logits_stride, V) ||
      (coded ? hidden_stride != mx_padded(d) : !stride_fits(hidden_stride, d)))
    return SD_ESHAPE;
  if (!aligned(hidden, coded ? 16 : type_size(hidden_type)) || (coded && !aligned(hidden_scales, 4)) ||
      !aligned(head, 256) || !aligned(logits, type_size(logits_type)))
    return SD_EALIGN;
  if (!workspace || workspace_bytes < need) return SD_EWORKSPACE;
  if (!aligned(workspace, 256)) return SD_EALIGN;
  return launch_status(launch_mx8_logits(hidden, hidden_type, hidden_scales, M, d, hidden_stride, head, V, logits,
                                         logits_type, logits_stride, workspace, (hipStream_t)stream));
}

int32_t sd_w4_quantize(const void *x, int32_t x_type, int32_t rows, int32_t d, int64_t x_stride, int32_t group,
                       uint8_t *codes, void *scales, int32_t scale_type, uint8_t *zeros, void *stream) {
  const int32_t st = check_w4(x, x_type, rows, d, x_stride, group, codes, scales, scale_type, zeros);
  if (st != SD_OK) return st;
  return launch_status(launch_w4_quantize(x, x_type, rows, d, x_stride, group, codes,
                                          reinterpret_cast<uint16_t *>(scales), scale_type, zeros,
                                          (hipStream_t)stream));
}

int32_t sd_w4_dequantize(const uint8_t *codes, const void *scales, int32_t scale_type, const uint8_t *zeros,
                         int32_t rows, int32_t d, int32_t group, void *x, int32_t x_type, int64_t x_stride,
                         void *stream) {
  const int32_t st = check_w4(x, x_type, rows, d, x_stride, group, codes, scales, scale_type, zeros);
  if (st != SD_OK) return st;
  return launch_status(launch_w4_dequantize(codes, reinterpret_cast<const uint16_t *>(scales), scale_type, zeros,
                                            rows, d, group, x, x_type, x_stride, (hipStream_t)stream));
}

size_t sd_w4_head_bytes(int32_t V, int32_t d, int32_t group, int32_t has_zeros) {
  if (V < 1 || V > kMaxVocab || !w4_group(d, group) || has_zeros < 0 || has_zeros > 1 || !mx_tiles_fit(V, d)) return 0;
  return w4_head_bytes(V, d, group, has_zeros == 1);
}

int32_t sd_w4_head(const uint8_t *codes, const void *scales, int32_t scale_type, const uint8_t *zeros, int32_t V,
                   int32_t d, int32_t group, uint8_t *head, size_t head_bytes, void *stream) {
  if (!codes || !scales || !head || !w4_scale_type(scale_type)) return SD_EINVAL;
  const size_t need = sd_w4_head_bytes(V, d, group, zeros != nullptr);
  if (need == 0) return SD_ESHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 4) || (zeros && !aligned(zeros, 4)) || !aligned(head, 256))
    return SD_EALIGN;
  if (head_bytes < need) return SD_EWORKSPACE;
  return launch_status(launch_w4_head(codes, reinterpret_cast<const uint16_t *>(scales), zeros, V, d, group, head,
                                      (hipStream_t)stream));
}

size_t sd_w4_logits_workspace_bytes(int32_t M, int32_t d, int32_t group) {
  if (M < 1 || !w4_group(d, group) || !mx_tiles_fit(M, d)) return 0;
  return w4_logits_workspace_bytes(M, d, group);
}

int32_t sd_w4_logits(const void *hidden, int32_t hidden_type, int32_t M, int32_t d, int64_t hidden_stride,
                     const uint8_t *head, int32_t V, int32_t group, int32_t scale_type, int32_t has_zeros,
                     void *logits, int32_t logits_type, int64_t logits_stride, void *workspace,
                     size_t workspace_bytes, void *stream) {
  if (!hidden || !head || !logits || (hidden_type != SD_BF16 && hidden_type != SD_F16) ||
      !known_type(logits_type) || !w4_scale_type(scale_type) || has_zeros < 0 || has_zeros > 1)
    return SD_EINVAL;
  const size_t need = sd_w4_logits_workspace_bytes(M, d, group);
  if (need == 0 || sd_w4_head_bytes(V, d, group, has_zeros) == 0 || !logits_fit(M, V) ||
      !stride_fits(hidden_stride, d) || !stride_fits(logits_stride, V))
    return SD_ESHAPE;
  if (!aligned(hidden, 2) || !aligned(head, 256) || !aligned(logits, type_size(logits_type))) return SD_EALIGN;
  if (!workspace || workspace_bytes < need) return SD_EWORKSPACE;
  if (!aligned(workspace, 256)) return SD_EALIGN;
  return launch_status(launch_w4_logits(hidden, hidden_type, M, d, hidden_stride, head, V, group, scale_type,
                                        has_zeros == 1, logits, logits_type, logits_stride, workspace,
                                        (hipStream_t)stream));
}

size_t sd_sample_workspace_bytes(int32_t R, int32_t V) {
  if (R < 1 || R > kMaxFilterRows || V < 1 || V > kMaxVocab) return 0;
  return sample_workspace_layout(R, V);
}

int32_t sd_sample(const void *logits, int32_t logits_type, int64_t logits_stride, int32_t R, int32_t V,
                  const float *u, const sd_sampling *sampling, int32_t rows_per_request,
                  int32_t *tokens, int64_t token_stride, int32_t *kept, float *logprob,
                  void *workspace, size_t workspace_bytes, void *stream) {
  if (!logits || !u || !sampling || !tokens || !known_type(logits_type)) return SD_EINVAL;
  if (R < 1 || R > kMaxFilterRows || V < 1 || V > kMaxVocab || rows_per_request < 1 || logits_stride < V ||
      logits_stride > ((int64_t)1 << 40) || token_stride < 1 || token_stride > ((int64_t)1 << 30))
    return SD_ESHAPE;
  if (!aligned(logits, type_size(logits_type)) || !aligned(u, 4) || !aligned(tokens, 4) ||
      (kept && !aligned(kept, 4)) || (logprob && !aligned(logprob, 4)) || !aligned_settings(*sampling))
    return SD_EALIGN;
  if (!workspace || workspace_bytes < sample_workspace_layout(R, V)) return SD_EWORKSPACE;
  if (!aligned(workspace, 256)) return SD_EALIGN;
  return launch_status(launch_sample(logits, logits_type, logits_stride, R, V, u, settings(*sampling),
                                     rows_per_request, tokens, token_stride, kept, logprob,
                                     workspace, (hipStream_t)stream));
}

size_t sd_accept_filtered_workspace_bytes(int32_t B, int32_t gamma, int32_t V) {
  if (check_filtered(B, gamma, V) != SD_OK) return 0;
  return accept_filtered_workspace_layout(B, gamma, V);
}

int32_t sd_accept_filtered(const float *logits, const uint16_t *draft_logits,
                           const int32_t *draft_tokens, const int32_t *verify_len,
                           const int32_t *row_offsets, const float *u_accept,
                           const float *u_resample, const sd_sampling *sampling, int32_t B,
                           int32_t gamma, int32_t V, int32_t *accept_len, int32_t *next_token,
                           int64_t *counters, void *workspace, size_t workspace_bytes,
                           void *stream) {
  if (!logits || !draft_logits || !draft_tokens || !u_accept || !u_resample || !sampling ||
      !accept_len || !next_token)
    return SD_EINVAL;
  if ((verify_len == nullptr) != (row_offsets == nullptr)) return SD_EINVAL;
  if (check_filtered(B, gamma, V) != SD_OK) return SD_ESHAPE;
  if (!aligned(logits, 16) || !aligned(draft_logits, 16) || !aligned(draft_tokens, 4) ||
      !aligned(u_accept, 4) || !aligned(u_resample, 4) || !aligned(accept_len, 4) ||
      !aligned(next_token, 4) || (counters && !aligned(counters, 8)) || !aligned_settings(*sampling) ||
      (verify_len && (!aligned(verify_len, 4) || !aligned(row_offsets, 4))))
    return SD_EALIGN;
  if (!workspace || workspace_bytes < accept_filtered_workspace_layout(B, gamma, V))
    return SD_EWORKSPACE;
  if (!aligned(workspace, 256)) return SD_EALIGN;
  RowMap rm{row_offsets, B, gamma};
  return launch_status(launch_accept_filtered(logits, draft_logits, draft_tokens, verify_len, rm,
                                              u_accept, u_resample, settings(*sampling), V,
                                              accept_len, next_token, counters, workspace,
                                              (hipStream_t)stream));
}

}  // extern "C"
