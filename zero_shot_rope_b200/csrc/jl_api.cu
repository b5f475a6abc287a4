// Host side of the C ABI declared in include/jetlong.h: argument validation,
// status reporting and kernel dispatch.  Nothing here computes attention.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/jetlong.h"
#include "jl_common.cuh"
#include "jl_paged.cuh"

namespace jl {
cudaError_t launch_simt_prefill(bool bf16, int D, const void *q, const void *k, const void *v, void *out,
                                float *lse, const int32_t *cu, const int32_t *cu_k, int batch, int T_total,
                                int Tk, int Hq, int Hkv, long long w_pre, int w0, int window,
                                const InvFreq &inv, int plain, cudaStream_t st);
struct DecodePlan {
  int nsplit;
  int chunk;
  size_t smem_bytes;
};
DecodePlan decode_plan(int batch, int Hq, int Hkv, int D, int max_seqlen, int elem);
size_t decode_partial_rows(int batch, int Hq, int Hkv, int D, int max_seqlen);
size_t decode_plan_tab_bytes();
cudaError_t launch_decode(bool bf16, int D, int GS, const void *q, const void *kc, const void *vc,
                          const int32_t *seqlens, int B, int Lcap, int max_seqlen, int Hq, int Hkv,
                          long long w_pre, int w0, int window, const InvFreq &inv, int plain, float *part_o,
                          float *part_ml, int2 *plan_tab, int *err, void *out, float *lse, cudaStream_t st);
size_t tc_prefill_workspace(int batch, int T_total, int Hq, int Hkv, int D, uint32_t flags);
cudaError_t launch_tc_prefill(const void *q, const void *k, const void *v, void *out, float *lse,
                              const int32_t *cu, const int32_t *cu_k, int batch, int T_total, int Tk,
                              int max_seqlen, int Hq, int Hkv, int D, long long w_pre, int w0, int window,
                              const InvFreq &inv, int plain, uint32_t flags, void *ws, size_t ws_bytes,
                              cudaStream_t st, const char **why);
}  // namespace jl

namespace {

thread_local char g_err[320] = "";

jl_status fail(jl_status s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

jl_status ok() {
  g_err[0] = '\0';
  return JL_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

jl::InvFreq make_inv_freq(int D, double theta) {
  jl::InvFreq f;
  for (int k = 0; k < JL_MAX_HALF; ++k) f.v[k] = 0.0;
  for (int k = 0; k < D / 2; ++k) f.v[k] = std::pow(theta, -2.0 * (double)k / (double)D);
  return f;
}

// x modulo 1, times 2^64, to 2^-64 of a turn.
unsigned long long turn_bits(double x) {
  const double r = x - std::rint(x);  // exact
  return std::isfinite(r) ? (unsigned long long)std::llrint(std::ldexp(r, 63)) << 1 : 0ull;
}

// The same frequencies in turns per position, times 2^64 (modulo a turn).  1/(2 pi)
// as the sum of three doubles, so that a frequency above 1 keeps its fraction of
// a turn: the angle of any 31-bit number of positions is then known to 2^-30 turns.
jl::TurnFreq make_turn_freq(const jl::InvFreq &inv) {
  constexpr double c1 = 0x1.45f306dc9c883p-3, c2 = -0x1.6b01ec5417056p-57, c3 = -0x1.6447e493ad4cep-111;
  jl::TurnFreq f;
  for (int k = 0; k < JL_MAX_HALF; ++k) {
    const double w = inv.v[k], p1 = w * c1, p2 = w * c2;
    f.v[k] = turn_bits(p1) + turn_bits(std::fma(w, c1, -p1)) + turn_bits(p2) + turn_bits(std::fma(w, c2, -p2)) +
             turn_bits(w * c3);
  }
  return f;
}

// Both for the last (head_dim, theta) of the calling thread: a model has one,
// and 64 powers take as long as a launch.
struct Freqs {
  int D = 0;
  double theta = 0.0;
  jl::InvFreq inv;
  jl::TurnFreq turn;
};
const Freqs &freqs_of(int D, double theta) {
  static thread_local Freqs f;
  if (f.D != D || f.theta != theta) {
    f.inv = make_inv_freq(D, theta);
    f.turn = make_turn_freq(f.inv);
    f.D = D;
    f.theta = theta;
  }
  return f;
}

jl_status check_heads(int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hq <= 0 || Hkv <= 0) return fail(JL_ERR_INVALID_ARG, "head counts must be positive (Hq=%d, Hkv=%d)", Hq, Hkv);
  if (Hq % Hkv != 0) return fail(JL_ERR_INVALID_ARG, "n_q_heads (%d) is not a multiple of n_kv_heads (%d)", Hq, Hkv);
  if (D != 64 && D != 128) return fail(JL_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", D);
  return JL_OK;
}

// The kernels put one head (prefill: a query head or a pair of them; decode:
// a kv head) per y-block of their grid, whose extent is at most 65535.
constexpr int32_t kMaxGridY = 65535;

jl_status check_method(int64_t w_pre, int32_t w0, double theta) {
  if (w_pre < 1) return fail(JL_ERR_INVALID_ARG, "w_pretrained must be >= 1 (got %lld)", (long long)w_pre);
  if (w0 < 0) return fail(JL_ERR_INVALID_ARG, "w0 must be >= 0 (got %d)", w0);
  if (!(theta > 0.0) || !std::isfinite(theta)) return fail(JL_ERR_INVALID_ARG, "rope_theta must be finite and > 0");
  return JL_OK;
}

jl_status cuda_fail(cudaError_t e, const char *what) {
  return fail(JL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// What the paged-cache calls check alike.
jl_status check_pages(int32_t n_q_heads, int32_t page_size, int32_t n_pages, int32_t max_pages, int64_t table_stride,
                      int32_t batch, jl_dtype dtype) {
  if (n_q_heads > kMaxGridY)
    return fail(JL_ERR_UNSUPPORTED, "n_q_heads %d exceeds %d per call", n_q_heads, kMaxGridY);
  if (dtype != JL_BF16 && dtype != JL_FP32) return fail(JL_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (page_size < 1 || (page_size & (page_size - 1)) != 0)
    return fail(JL_ERR_INVALID_ARG, "page_size must be a power of two (got %d)", page_size);
  if (page_size < (1 << jl::PG_MIN_LOG2) || page_size > (1 << jl::PG_MAX_LOG2))
    return fail(JL_ERR_UNSUPPORTED, "page_size %d not supported (%d to %d)", page_size, 1 << jl::PG_MIN_LOG2,
                1 << jl::PG_MAX_LOG2);
  if (n_pages < 1 || max_pages < 1)
    return fail(JL_ERR_INVALID_ARG, "n_pages and max_pages must be >= 1 (got %d, %d)", n_pages, max_pages);
  if ((int64_t)max_pages * page_size > (int64_t)1 << 30)
    return fail(JL_ERR_UNSUPPORTED, "max_pages * page_size (%lld) exceeds 2^30", (long long)max_pages * page_size);
  if (table_stride < max_pages)
    return fail(JL_ERR_INVALID_ARG, "table_stride (%lld) < max_pages (%d)", (long long)table_stride, max_pages);
  if (batch < 0) return fail(JL_ERR_INVALID_ARG, "batch must be >= 0");
  if (batch > 65535) return fail(JL_ERR_UNSUPPORTED, "batch %d exceeds 65535 sequences per call", batch);
  return JL_OK;
}

jl_status check_pool(int32_t page_size, int64_t page_stride, int32_t Hkv, int32_t D, jl_dtype dtype) {
  if (page_stride < (int64_t)page_size * Hkv * D)
    return fail(JL_ERR_INVALID_ARG, "page_stride (%lld) < page_size * n_kv_heads * head_dim", (long long)page_stride);
  if (page_stride % (dtype == JL_BF16 ? 8 : 4) != 0)
    return fail(JL_ERR_INVALID_ARG, "page_stride (%lld elements) is not a multiple of 16 bytes", (long long)page_stride);
  return JL_OK;
}

// No length exceeds 2^30, so every larger w_pretrained means G = 1.
int64_t longest(int64_t w_pretrained) { return w_pretrained < ((int64_t)1 << 31) ? w_pretrained : (int64_t)1 << 31; }

int log2_of(int32_t x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

}  // namespace

namespace jl {
// Record a message for jl_last_error() from other translation units.
void set_last_error(const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
}
}  // namespace jl

extern "C" {

const char *jl_status_string(jl_status s) {
  switch (s) {
    case JL_OK: return "JL_OK";
    case JL_ERR_INVALID_ARG: return "JL_ERR_INVALID_ARG";
    case JL_ERR_UNSUPPORTED: return "JL_ERR_UNSUPPORTED";
    case JL_ERR_CUDA: return "JL_ERR_CUDA";
    case JL_ERR_WORKSPACE: return "JL_ERR_WORKSPACE";
  }
  return "JL_STATUS_UNKNOWN";
}

const char *jl_last_error(void) { return g_err; }

const char *jl_version(void) { return "jetlong-b200 0.1 sm_100a"; }

jl_status jl_group_size(int64_t L, int64_t w_pretrained, int64_t *G_out) {
  if (G_out == nullptr) return fail(JL_ERR_INVALID_ARG, "G_out is NULL");
  if (L < 0) return fail(JL_ERR_INVALID_ARG, "L must be >= 0 (got %lld)", (long long)L);
  if (w_pretrained < 1) return fail(JL_ERR_INVALID_ARG, "w_pretrained must be >= 1 (got %lld)", (long long)w_pretrained);
  // ceil without overflow for L near INT64_MAX
  const int64_t g = L / w_pretrained + (L % w_pretrained != 0 ? 1 : 0);
  *G_out = g < 1 ? 1 : g;
  return ok();
}

size_t jl_bifocal_prefill_workspace_size(int32_t batch, int32_t total_tokens, int32_t n_q_heads,
                                         int32_t n_kv_heads, int32_t head_dim, jl_dtype dtype,
                                         uint32_t flags) {
  if (batch < 0 || total_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0) return 0;
  if (n_q_heads % n_kv_heads != 0) return 0;
  const bool tc_shape = head_dim == 128 || head_dim == 64;
  if (dtype != JL_BF16 || (flags & JL_FLAG_SIMT) || !tc_shape) return 0;
  return jl::tc_prefill_workspace(batch, total_tokens, n_q_heads, n_kv_heads, head_dim, flags);
}

jl_status jl_bifocal_prefill_kv(const void *q, const void *k, const void *v, void *out, float *lse,
                                const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int32_t batch,
                                int32_t total_q, int32_t total_k, int32_t max_seqlen_q, int32_t n_q_heads,
                                int32_t n_kv_heads, int32_t head_dim, int64_t w_pretrained, int32_t w0,
                                int32_t window, double rope_theta, jl_dtype dtype, uint32_t flags,
                                void *workspace, size_t workspace_bytes, void *stream) {
  jl_status s;
  if ((s = check_heads(n_q_heads, n_kv_heads, head_dim)) != JL_OK) return s;
  if (n_q_heads > kMaxGridY)
    return fail(JL_ERR_UNSUPPORTED, "n_q_heads %d exceeds %d per call", n_q_heads, kMaxGridY);
  if ((s = check_method(w_pretrained, w0, rope_theta)) != JL_OK) return s;
  if (window < 0) return fail(JL_ERR_INVALID_ARG, "window must be >= 0 (0: no window), got %d", window);
  if (dtype != JL_BF16 && dtype != JL_FP32) return fail(JL_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (flags & ~(uint32_t)(JL_FLAG_PLAIN_CAUSAL | JL_FLAG_SIMT | JL_FLAG_PREROTATE_K))
    return fail(JL_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags);
  if (batch < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0)
    return fail(JL_ERR_INVALID_ARG, "batch, token counts and max_seqlen must be >= 0");
  if (batch == 0 || total_q == 0) return ok();  // nothing to attend
  if (batch > 65535)  // the kernels' grid takes one z-block per sequence
    return fail(JL_ERR_UNSUPPORTED, "batch %d exceeds 65535 sequences per call", batch);
  if (total_k < total_q)
    return fail(JL_ERR_INVALID_ARG, "total_k (%d) < total_q (%d): every sequence needs Lq <= Lk", total_k, total_q);
  if (cu_seqlens_q == nullptr || cu_seqlens_k == nullptr) return fail(JL_ERR_INVALID_ARG, "cu_seqlens is NULL");
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr)
    return fail(JL_ERR_INVALID_ARG, "q, k, v and out must be non-NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || (lse && !aligned16(lse)))
    return fail(JL_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if (max_seqlen_q == 0 || max_seqlen_q > total_q)
    return fail(JL_ERR_INVALID_ARG, "max_seqlen must be in [1, total query tokens] (got %d)", max_seqlen_q);

  const jl::InvFreq inv = make_inv_freq(head_dim, rope_theta);
  const int plain = (flags & JL_FLAG_PLAIN_CAUSAL) ? 1 : 0;
  cudaStream_t st = (cudaStream_t)stream;
  // tensor cores for bf16 at head_dim 64 and 128; the SIMT kernel otherwise
  const bool tc_shape = head_dim == 128 || head_dim == 64;
  const bool use_simt = dtype == JL_FP32 || (flags & JL_FLAG_SIMT) || !tc_shape;
  if (use_simt) {
    cudaError_t e = jl::launch_simt_prefill(dtype == JL_BF16, head_dim, q, k, v, out, lse, cu_seqlens_q,
                                            cu_seqlens_k, batch, total_q, total_k, n_q_heads, n_kv_heads,
                                            w_pretrained, w0, window, inv, plain, st);
    return e == cudaSuccess ? ok() : cuda_fail(e, "SIMT prefill launch");
  }
  const size_t need = jl::tc_prefill_workspace(batch, total_k, n_q_heads, n_kv_heads, head_dim, flags);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(JL_ERR_WORKSPACE, "prefill needs %zu workspace bytes (got %zu)", need, workspace_bytes);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(JL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const char *why = nullptr;
  cudaError_t e = jl::launch_tc_prefill(q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k,
                                        max_seqlen_q, n_q_heads, n_kv_heads, head_dim, w_pretrained, w0, window,
                                        inv, plain, flags, workspace, workspace_bytes, st, &why);
  return e == cudaSuccess ? ok() : cuda_fail(e, why ? why : "tensor-core prefill launch");
}

jl_status jl_bifocal_prefill(const void *q, const void *k, const void *v, void *out, float *lse,
                             const int32_t *cu_seqlens, int32_t batch, int32_t total_tokens,
                             int32_t max_seqlen, int32_t n_q_heads, int32_t n_kv_heads,
                             int32_t head_dim, int64_t w_pretrained, int32_t w0, double rope_theta,
                             jl_dtype dtype, uint32_t flags, void *workspace,
                             size_t workspace_bytes, void *stream) {
  // every token of every sequence is a query: the key prefix sums are the
  // query prefix sums
  return jl_bifocal_prefill_kv(q, k, v, out, lse, cu_seqlens, cu_seqlens, batch, total_tokens, total_tokens,
                               max_seqlen, n_q_heads, n_kv_heads, head_dim, w_pretrained, w0, 0, rope_theta,
                               dtype, flags, workspace, workspace_bytes, stream);
}

size_t jl_bifocal_decode_workspace_size(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads,
                                        int32_t head_dim, int32_t max_seqlen) {
  if (batch <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || max_seqlen < 0) return 0;
  if (n_q_heads % n_kv_heads != 0) return 0;
  // one layout serves every dtype and both decode kernels
  const size_t rows = jl::decode_partial_rows(batch, n_q_heads, n_kv_heads, head_dim, max_seqlen);
  return 256 + align256(rows * head_dim * sizeof(float)) + align256(rows * 2 * sizeof(float)) +
         align256(jl::decode_plan_tab_bytes());
}

jl_status jl_bifocal_decode_window(const void *q, const void *k_cache, const void *v_cache,
                                   const int32_t *seqlens, int32_t batch, int32_t cache_capacity,
                                   int32_t max_seqlen, int32_t n_q_heads, int32_t n_kv_heads,
                                   int32_t head_dim, int64_t w_pretrained, int32_t w0, int32_t window,
                                   double rope_theta, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, jl_dtype dtype, uint32_t flags, void *stream) {
  jl_status s;
  if (window < 0) return fail(JL_ERR_INVALID_ARG, "window must be >= 0 (0: no window), got %d", window);
  if ((s = check_heads(n_q_heads, n_kv_heads, head_dim)) != JL_OK) return s;
  if (n_kv_heads > kMaxGridY)
    return fail(JL_ERR_UNSUPPORTED, "n_kv_heads %d exceeds %d per call", n_kv_heads, kMaxGridY);
  const int gs = n_q_heads / n_kv_heads;
  if (gs != 1 && gs != 2 && gs != 4 && gs != 8)
    return fail(JL_ERR_UNSUPPORTED, "decode supports n_q_heads / n_kv_heads in {1,2,4,8} (got %d)", gs);
  if ((s = check_method(w_pretrained, w0, rope_theta)) != JL_OK) return s;
  if (dtype != JL_BF16 && dtype != JL_FP32) return fail(JL_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (flags & ~(uint32_t)JL_FLAG_PLAIN_CAUSAL) return fail(JL_ERR_INVALID_ARG, "unknown or prefill-only flag bits 0x%x", flags);
  if (batch < 0) return fail(JL_ERR_INVALID_ARG, "batch must be >= 0");
  if (batch == 0) return ok();
  if (batch > 65535)  // the kernels' grid takes one z-block per sequence
    return fail(JL_ERR_UNSUPPORTED, "batch %d exceeds 65535 sequences per call", batch);
  if (cache_capacity < 1 || max_seqlen < 1 || max_seqlen > cache_capacity)
    return fail(JL_ERR_INVALID_ARG, "need 1 <= max_seqlen <= cache_capacity (got %d, %d)", max_seqlen, cache_capacity);
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || out == nullptr || seqlens == nullptr)
    return fail(JL_ERR_INVALID_ARG, "q, k_cache, v_cache, seqlens and out must be non-NULL");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return fail(JL_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  const size_t need = jl_bifocal_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, max_seqlen);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(JL_ERR_WORKSPACE, "decode needs %zu workspace bytes (got %zu)", need, workspace_bytes);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(JL_ERR_WORKSPACE, "workspace must be 256-byte aligned");

  const size_t rows = jl::decode_partial_rows(batch, n_q_heads, n_kv_heads, head_dim, max_seqlen);
  int *err = (int *)workspace;
  float *part_o = (float *)((char *)workspace + 256);
  float *part_ml = (float *)((char *)workspace + 256 + align256(rows * head_dim * sizeof(float)));
  int2 *plan_tab = (int2 *)((char *)part_ml + align256(rows * 2 * sizeof(float)));
  const jl::InvFreq inv = make_inv_freq(head_dim, rope_theta);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaMemsetAsync(err, 0, sizeof(int), st);
  if (e == cudaSuccess)
    e = jl::launch_decode(dtype == JL_BF16, head_dim, gs, q, k_cache, v_cache, seqlens, batch, cache_capacity,
                          max_seqlen, n_q_heads, n_kv_heads, w_pretrained, w0, window, inv,
                          (flags & JL_FLAG_PLAIN_CAUSAL) ? 1 : 0, part_o, part_ml, plan_tab, err, out, lse, st);
  return e == cudaSuccess ? ok() : cuda_fail(e, "decode launch");
}

jl_status jl_bifocal_decode(const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *seqlens, int32_t batch, int32_t cache_capacity,
                            int32_t max_seqlen, int32_t n_q_heads, int32_t n_kv_heads,
                            int32_t head_dim, int64_t w_pretrained, int32_t w0, double rope_theta,
                            void *out, float *lse, void *workspace, size_t workspace_bytes,
                            jl_dtype dtype, uint32_t flags, void *stream) {
  return jl_bifocal_decode_window(q, k_cache, v_cache, seqlens, batch, cache_capacity, max_seqlen, n_q_heads,
                                  n_kv_heads, head_dim, w_pretrained, w0, 0, rope_theta, out, lse, workspace,
                                  workspace_bytes, dtype, flags, stream);
}

// ------------------------------------------------------------- paged cache
jl_status jl_paged_append(const void *k, const void *v, void *k_pages, void *v_pages, void *page_summary,
                          const int32_t *block_table, int64_t table_stride, int32_t max_pages,
                          const int32_t *cu_seqlens, const int32_t *seqlens, int32_t batch, int32_t total_tokens,
                          int32_t max_new, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                          int32_t page_size, int32_t n_pages, int64_t page_stride, const void *q, void *q_out,
                          double rope_theta, jl_dtype dtype, uint32_t flags, void *stream) {
  jl_status s;
  if ((s = check_heads(n_q_heads, n_kv_heads, head_dim)) != JL_OK) return s;
  if ((s = check_pages(n_q_heads, page_size, n_pages, max_pages, table_stride, batch, dtype)) != JL_OK) return s;
  if ((s = check_pool(page_size, page_stride, n_kv_heads, head_dim, dtype)) != JL_OK) return s;
  if (flags & ~(uint32_t)JL_FLAG_ROTATE) return fail(JL_ERR_INVALID_ARG, "unknown or unfitting flag bits 0x%x", flags);
  const bool rotate = (flags & JL_FLAG_ROTATE) != 0;
  if (rotate && (s = check_method(1, 0, rope_theta)) != JL_OK) return s;
  if ((q == nullptr) != (q_out == nullptr)) return fail(JL_ERR_INVALID_ARG, "q and q_out go together");
  if (q != nullptr && !rotate) return fail(JL_ERR_INVALID_ARG, "q needs JL_FLAG_ROTATE");
  if (total_tokens < 0 || max_new < 0) return fail(JL_ERR_INVALID_ARG, "total_tokens and max_new must be >= 0");
  if (batch == 0 || total_tokens == 0) return ok();
  if (max_new == 0 || max_new > total_tokens)
    return fail(JL_ERR_INVALID_ARG, "max_new must be in [1, total_tokens] (got %d)", max_new);
  if (k == nullptr || v == nullptr || k_pages == nullptr || v_pages == nullptr || block_table == nullptr ||
      cu_seqlens == nullptr || seqlens == nullptr)
    return fail(JL_ERR_INVALID_ARG, "k, v, k_pages, v_pages, block_table, cu_seqlens and seqlens must be non-NULL");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(page_summary) ||
      !aligned16(q) || !aligned16(q_out))
    return fail(JL_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  jl::PagedAppendArgs a;
  a.k = k;
  a.v = v;
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.summary = page_summary;
  a.q_out = q_out;
  a.table = block_table;
  a.table_stride = table_stride;
  a.cu = cu_seqlens;
  a.seqlens = seqlens;
  a.max_pages = max_pages;
  a.page_log2 = log2_of(page_size);
  a.n_pages = n_pages;
  a.T = total_tokens;
  a.max_new = max_new;
  a.Hkv = n_kv_heads;
  a.GS = n_q_heads / n_kv_heads;
  a.page_stride = page_stride;
  static const jl::TurnFreq none = {};  // (the thread's frequencies are kept for the calls that turn)
  const cudaError_t e = jl::launch_paged_append(dtype == JL_BF16, head_dim, rotate, a,
                                                rotate ? freqs_of(head_dim, rope_theta).turn : none, batch,
                                                (cudaStream_t)stream);
  return e == cudaSuccess ? ok() : cuda_fail(e, "paged append launch");
}

size_t jl_bifocal_select_pages_workspace_size(int32_t batch, int32_t n_kv_heads, int32_t max_pages, int32_t n_select) {
  if (batch <= 0 || n_kv_heads <= 0 || max_pages <= 0 || n_select <= 0 || max_pages <= n_select) return 0;
  const size_t n = (size_t)batch * n_kv_heads * max_pages;
  return 4 * align256(n * sizeof(float)) + align256(n * sizeof(double));
}

jl_status jl_bifocal_select_pages(const void *q, const void *page_summary, const int32_t *block_table,
                                  int64_t table_stride, int32_t max_pages, const int32_t *seqlens, int32_t batch,
                                  int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t page_size,
                                  int32_t n_pages, int32_t n_select, int32_t n_first, int32_t n_last,
                                  int64_t w_pretrained, int32_t w0, double rope_theta, int32_t *page_list,
                                  void *workspace, size_t workspace_bytes, jl_dtype dtype, uint32_t flags,
                                  void *stream) {
  jl_status s;
  if ((s = check_heads(n_q_heads, n_kv_heads, head_dim)) != JL_OK) return s;
  if ((s = check_method(w_pretrained, w0, rope_theta)) != JL_OK) return s;
  if ((s = check_pages(n_q_heads, page_size, n_pages, max_pages, table_stride, batch, dtype)) != JL_OK) return s;
  if (flags & ~(uint32_t)JL_FLAG_PLAIN_CAUSAL) return fail(JL_ERR_INVALID_ARG, "unknown or unfitting flag bits 0x%x", flags);
  if (n_select < 1) return fail(JL_ERR_INVALID_ARG, "n_select must be >= 1 (got %d)", n_select);
  if (n_first < 0 || n_last < 0 || (int64_t)n_first + n_last > n_select)
    return fail(JL_ERR_INVALID_ARG, "need n_first, n_last >= 0 and n_first + n_last <= n_select (got %d, %d, %d)", n_first,
                n_last, n_select);
  if (batch == 0) return ok();
  if (q == nullptr || page_summary == nullptr || block_table == nullptr || seqlens == nullptr || page_list == nullptr)
    return fail(JL_ERR_INVALID_ARG, "q, page_summary, block_table, seqlens and page_list must be non-NULL");
  if (!aligned16(q) || !aligned16(page_summary)) return fail(JL_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  const size_t need = jl_bifocal_select_pages_workspace_size(batch, n_kv_heads, max_pages, n_select);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(JL_ERR_WORKSPACE, "page selection needs %zu workspace bytes (got %zu)", need, workspace_bytes);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(JL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const size_t n = (size_t)batch * n_kv_heads * max_pages;
  jl::PagedSelectArgs a;
  a.q = q;
  a.summary = page_summary;
  a.table = block_table;
  a.table_stride = table_stride;
  a.seqlens = seqlens;
  a.B = batch;
  a.Hkv = n_kv_heads;
  a.GS = n_q_heads / n_kv_heads;
  a.max_pages = max_pages;
  a.page_log2 = log2_of(page_size);
  a.n_pages = n_pages;
  a.n_select = n_select;
  a.n_first = n_first;
  a.n_last = n_last;
  a.w_pre = longest(w_pretrained);
  a.w0 = w0;
  a.plain = (flags & JL_FLAG_PLAIN_CAUSAL) ? 1 : 0;
  a.list = page_list;
  a.score = (float *)workspace;
  a.size = (float *)((char *)workspace + align256(n * sizeof(float)));
  a.mark = (float *)((char *)workspace + 2 * align256(n * sizeof(float)));
  a.amb = (int32_t *)((char *)workspace + 3 * align256(n * sizeof(float)));
  a.fine = (double *)((char *)workspace + 4 * align256(n * sizeof(float)));
  const Freqs &f = freqs_of(head_dim, rope_theta);
  const cudaError_t e = jl::launch_paged_select(dtype == JL_BF16, head_dim, a, f.inv, f.turn, (cudaStream_t)stream);
  return e == cudaSuccess ? ok() : cuda_fail(e, "page selection launch");
}

size_t jl_bifocal_decode_paged_workspace_size(int32_t batch, int32_t head_dim) {
  if (batch <= 0 || head_dim <= 0) return 0;
  const size_t rows = (size_t)2 * jl::PD_MAX_CTAS * jl::PD_HEADS;
  return 256 + align256(jl::PD_MAX_CTAS * sizeof(int)) + align256(rows * head_dim * sizeof(float)) +
         align256(rows * 2 * sizeof(float)) + align256(((size_t)batch + 1) * sizeof(long long));
}

jl_status jl_bifocal_decode_paged(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                                  int64_t table_stride, int32_t max_pages, const int32_t *seqlens,
                                  const int32_t *page_list, int32_t n_list, int32_t batch, int32_t n_q_heads,
                                  int32_t n_kv_heads, int32_t head_dim, int32_t page_size, int32_t n_pages,
                                  int64_t page_stride, int64_t w_pretrained, int32_t w0, int32_t window,
                                  double rope_theta, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                  jl_dtype dtype, uint32_t flags, void *stream) {
  jl_status s;
  if (window < 0) return fail(JL_ERR_INVALID_ARG, "window must be >= 0 (0: no window), got %d", window);
  if ((s = check_heads(n_q_heads, n_kv_heads, head_dim)) != JL_OK) return s;
  if ((s = check_method(w_pretrained, w0, rope_theta)) != JL_OK) return s;
  if ((s = check_pages(n_q_heads, page_size, n_pages, max_pages, table_stride, batch, dtype)) != JL_OK) return s;
  if ((s = check_pool(page_size, page_stride, n_kv_heads, head_dim, dtype)) != JL_OK) return s;
  if (flags & ~(uint32_t)JL_FLAG_PLAIN_CAUSAL) return fail(JL_ERR_INVALID_ARG, "unknown or unfitting flag bits 0x%x", flags);
  if (n_list < 0 || n_list > (1 << 20)) return fail(JL_ERR_INVALID_ARG, "n_list must be in [0, 2^20] (got %d)", n_list);
  if (page_list == nullptr && n_list != 0) return fail(JL_ERR_INVALID_ARG, "n_list without a page_list");
  if (batch == 0) return ok();
  if (q == nullptr || k_pages == nullptr || v_pages == nullptr || block_table == nullptr || seqlens == nullptr ||
      out == nullptr)
    return fail(JL_ERR_INVALID_ARG, "q, k_pages, v_pages, block_table, seqlens and out must be non-NULL");
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
    return fail(JL_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  const size_t need = jl_bifocal_decode_paged_workspace_size(batch, head_dim);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(JL_ERR_WORKSPACE, "paged decode needs %zu workspace bytes (got %zu)", need, workspace_bytes);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(JL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const size_t rows = (size_t)2 * jl::PD_MAX_CTAS * jl::PD_HEADS;
  jl::PagedDecodeArgs a;
  a.q = q;
  a.k = k_pages;
  a.v = v_pages;
  a.table = block_table;
  a.table_stride = table_stride;
  a.seqlens = seqlens;
  a.list = page_list;
  a.n_list = n_list;
  a.max_pages = max_pages;
  a.page_log2 = log2_of(page_size);
  a.n_pages = n_pages;
  a.page_stride = page_stride;
  a.B = batch;
  a.Hq = n_q_heads;
  a.Hkv = n_kv_heads;
  a.GS = n_q_heads / n_kv_heads;
  a.HB = (a.GS + jl::PD_HEADS - 1) / jl::PD_HEADS;
  a.w_pre = longest(w_pretrained);
  a.w0 = w0;
  a.window = window;
  a.plain = (flags & JL_FLAG_PLAIN_CAUSAL) ? 1 : 0;
  a.err = (int *)workspace;
  a.cta_err = (int *)((char *)workspace + 256);
  a.part_o = (float *)((char *)a.cta_err + align256(jl::PD_MAX_CTAS * sizeof(int)));
  a.part_ml = (float *)((char *)a.part_o + align256(rows * head_dim * sizeof(float)));
  a.tab = (long long *)((char *)a.part_ml + align256(rows * 2 * sizeof(float)));
  a.out = out;
  a.lse = lse;
  const cudaError_t e =
      jl::launch_paged_decode(dtype == JL_BF16, head_dim, a, freqs_of(head_dim, rope_theta).turn, (cudaStream_t)stream);
  return e == cudaSuccess ? ok() : cuda_fail(e, "paged decode launch");
}

jl_status jl_paged_call(int32_t call, const int64_t *words, int32_t n_words) {
  static const int32_t kWords[3] = {25, 24, 27};
  if (call < 0 || call > 2 || words == nullptr || n_words != kWords[call])
    return fail(JL_ERR_INVALID_ARG, "jl_paged_call: no such call, or not its number of words (%d, %d)", call, n_words);
  bool fits = true;
  int at = 0;
  auto word = [&]() {
    int64_t w;
    memcpy(&w, reinterpret_cast<const char *>(words) + 8 * at++, 8);  // the words need not be aligned
    return w;
  };
  auto ptr = [&]() { return reinterpret_cast<void *>(word()); };
  auto i32 = [&]() {
    const int64_t w = word();
    fits = fits && w == (int32_t)w;
    return (int32_t)w;
  };
  auto u32 = [&]() {
    const int64_t w = word();
    fits = fits && w == (int64_t)(uint32_t)w;
    return (uint32_t)w;
  };
  auto f64 = [&]() {
    const int64_t w = word();
    double d;
    memcpy(&d, &w, 8);
    return d;
  };
  const char *kRange = "an argument does not fit 32 bits";
  if (call == JL_CALL_PAGED_APPEND) {
    const void *k = ptr(), *v = ptr();
    void *kp = ptr(), *vp = ptr(), *sum = ptr();
    const int32_t *table = (const int32_t *)ptr();
    const int64_t stride = word();
    const int32_t cols = i32();
    const int32_t *cu = (const int32_t *)ptr(), *lens = (const int32_t *)ptr();
    const int32_t batch = i32(), total = i32(), max_new = i32(), hq = i32(), hkv = i32(), d = i32(), page = i32(),
                  n = i32();
    const int64_t page_stride = word();
    const void *q = ptr();
    void *qo = ptr();
    const double theta = f64();
    const int32_t dtype = i32();
    const uint32_t flags = u32();
    void *stream = ptr();
    if (!fits) return fail(JL_ERR_INVALID_ARG, "%s", kRange);
    return jl_paged_append(k, v, kp, vp, sum, table, stride, cols, cu, lens, batch, total, max_new, hq, hkv, d, page, n,
                           page_stride, q, qo, theta, (jl_dtype)dtype, flags, stream);
  }
  const void *q = ptr(), *k = ptr(), *v = call == JL_CALL_BIFOCAL_DECODE_PAGED ? ptr() : nullptr;
  const int32_t *table = (const int32_t *)ptr();
  const int64_t stride = word();
  const int32_t cols = i32();
  const int32_t *lens = (const int32_t *)ptr();
  if (call == JL_CALL_BIFOCAL_SELECT_PAGES) {
    const int32_t batch = i32(), hq = i32(), hkv = i32(), d = i32(), page = i32(), n = i32(), n_select = i32(),
                  n_first = i32(), n_last = i32();
    const int64_t w_pre = word();
    const int32_t w0 = i32();
    const double theta = f64();
    int32_t *list = (int32_t *)ptr();
    void *ws = ptr();
    const size_t ws_bytes = (size_t)word();
    const int32_t dtype = i32();
    const uint32_t flags = u32();
    void *stream = ptr();
    if (!fits) return fail(JL_ERR_INVALID_ARG, "%s", kRange);
    return jl_bifocal_select_pages(q, k, table, stride, cols, lens, batch, hq, hkv, d, page, n, n_select, n_first,
                                   n_last, w_pre, w0, theta, list, ws, ws_bytes, (jl_dtype)dtype, flags, stream);
  }
  const int32_t *list = (const int32_t *)ptr();
  const int32_t n_list = i32(), batch = i32(), hq = i32(), hkv = i32(), d = i32(), page = i32(), n = i32();
  const int64_t page_stride = word(), w_pre = word();
  const int32_t w0 = i32(), window = i32();
  const double theta = f64();
  void *out = ptr();
  float *lse = (float *)ptr();
  void *ws = ptr();
  const size_t ws_bytes = (size_t)word();
  const int32_t dtype = i32();
  const uint32_t flags = u32();
  void *stream = ptr();
  if (!fits) return fail(JL_ERR_INVALID_ARG, "%s", kRange);
  return jl_bifocal_decode_paged(q, k, v, table, stride, cols, lens, list, n_list, batch, hq, hkv, d, page, n,
                                 page_stride, w_pre, w0, window, theta, out, lse, ws, ws_bytes, (jl_dtype)dtype, flags,
                                 stream);
}

}  // extern "C"

// ---------------------------------------------------------------- test hooks
namespace jl {
cudaError_t set_wait_limit_prefill(unsigned long long ns);
cudaError_t set_wait_limit_decode_tc(unsigned long long ns);
cudaError_t set_wait_limit_decode(unsigned long long ns);
cudaError_t set_wait_limit_paged(unsigned long long ns);
}  // namespace jl

extern "C" int jl_debug_set_wait_limit(unsigned long long ns) {
  if (ns == 0) ns = 2000000000ull;
  cudaError_t e = jl::set_wait_limit_prefill(ns);
  if (e == cudaSuccess) e = jl::set_wait_limit_decode_tc(ns);
  if (e == cudaSuccess) e = jl::set_wait_limit_decode(ns);
  if (e == cudaSuccess) e = jl::set_wait_limit_paged(ns);
  if (e != cudaSuccess) {
    fail(JL_ERR_CUDA, "setting the wait limit failed: %s", cudaGetErrorString(e));
    return -1;
  }
  return 0;
}

extern "C" void jl_debug_angle_cs(int32_t n, double inv_freq, float *c, float *s) {
  jl::angle_cs(n, inv_freq, *c, *s);
}

extern "C" void jl_debug_turn_cs(int32_t n, double inv_freq, float *c, float *s) {
  jl::InvFreq inv = {};
  inv.v[0] = inv_freq;
  jl::turn_cs(n, make_turn_freq(inv).v[0], *c, *s);
}
