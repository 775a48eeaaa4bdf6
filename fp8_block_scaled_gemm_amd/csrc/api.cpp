// C ABI of libdg.so: argument validation, device queries and dispatch to the
// gfx950 kernels.  Declarations and the contract of every entry point are in
// include/dg.h.  Nothing here allocates device memory or synchronises.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/dg.h"
#include "common.hpp"

namespace dg {

int launch_quant_token_group(const float* x, int64_t groups, int64_t m, int64_t k, uint8_t* q, float* sa,
                             int64_t ld_sa, hipStream_t stream);
int launch_quant_token_group_bf16(const uint16_t* x, int64_t groups, int64_t m, int64_t k, uint8_t* q, float* sa,
                                  int64_t ld_sa, hipStream_t stream);
int launch_quant_block(const float* w, int64_t groups, int64_t n, int64_t k, uint8_t* q, float* sb,
                       hipStream_t stream);
int launch_quant_channel_group(const float* x, int64_t mats, int64_t m, int64_t k, uint8_t* qt, float* st,
                               int64_t ld_st, hipStream_t stream);
int launch_quant_channel_group_bf16(const uint16_t* x, int64_t mats, int64_t m, int64_t k, uint8_t* qt, float* st,
                                    int64_t ld_st, hipStream_t stream);
int launch_transpose_blocks(const uint8_t* q, const float* s, int64_t groups, int64_t r, int64_t c, uint8_t* qt,
                            float* st, hipStream_t stream);
int launch_fill_zero_bf16(uint16_t* d, int64_t count, hipStream_t stream);
int launch_gemm(int layout, const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b,
                const float* sb, int64_t ld_sb, int64_t ld_ab, uint16_t* d, const int32_t* m_indices,
                const int32_t* masked_m,
                int64_t groups, int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes,
                hipStream_t stream, int num_cus);
size_t gemm_workspace_size(int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus);
int launch_gemm_fq(const void* x, bool x_bf16, const uint8_t* b, const float* sb, uint16_t* d, int64_t m, int64_t n,
                   int64_t k, void* ws, size_t ws_bytes, hipStream_t stream, int num_cus);
size_t gemm_fq_workspace_size(int64_t m, int64_t n, int64_t k, int num_cus);
void gemm_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, char* buf,
                      size_t len);
int read_diag(unsigned out[4], bool clear);
int launch_gemm_no_alloc(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                         uint16_t* d, int64_t m, int64_t n, int64_t k, hipStream_t stream, int num_cus);

int launch_route(const void* logits, int dtype, int64_t ld, const float* bias, int64_t tokens, int experts, int top_k,
                 int groups, int topk_groups, int group_top, bool softmax, bool renorm, float scale, int32_t* ids,
                 float* weights, hipStream_t stream);
int launch_route_grad(const float* dweights, const void* logits, int dtype, int64_t ld, const int32_t* ids,
                      int64_t tokens, int experts, int top_k, bool softmax, bool renorm, float scale, void* dlogits,
                      int64_t ld_out, hipStream_t stream);
size_t moe_layout_workspace_size(int64_t n, int64_t experts);
int launch_moe_layout(const int32_t* ids, int64_t n, int experts, int64_t rows_per_expert, int align,
                      int64_t rows_total, int32_t* rows, int32_t* sources, int32_t* m_indices, int32_t* counts,
                      void* ws, hipStream_t stream);
int launch_moe_dispatch(int form, const void* x, int dtype, const int32_t* rows, const int32_t* sources,
                        const int32_t* m_indices, int64_t tokens, int top_k, int64_t hidden, int64_t rows_total,
                        int64_t rows_per_expert, void* q, float* s, int64_t ld_s, float* s_tmp, hipStream_t stream);
size_t moe_dispatch_fp8_workspace_size(int64_t tokens, int64_t top_k, int64_t hidden);
int launch_moe_combine(const void* out, int dtype, const int32_t* rows, const float* weights, int64_t tokens, int top_k,
                       int64_t hidden, int64_t rows_total, void* y, hipStream_t stream);
int launch_moe_combine_grad(const void* dy, const void* out, int dtype, const int32_t* rows, const int32_t* sources,
                            const int32_t* m_indices, const float* weights, int64_t tokens, int top_k, int64_t hidden,
                            int64_t rows_total, void* dout, float* dweights, hipStream_t stream);
int launch_quant_int8(const void* x, int dtype, int64_t rows, int64_t k, int8_t* q, float* s, hipStream_t stream);
int launch_gemm_int8(int layout, const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d,
                     int out_dtype, const int32_t* m_indices, const int32_t* masked_m, int64_t groups, int64_t m,
                     int64_t n, int64_t k, void* ws, size_t ws_bytes, hipStream_t stream, int num_cus);
int launch_gemm_int8_act_quant(const void* x, int dtype, const int8_t* b, const float* sb, void* d, int out_dtype,
                               int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes, hipStream_t stream,
                               int num_cus);
void gemm_int8_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, char* buf,
                           size_t len);
size_t int8_workspace_size(int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus);
size_t int8_act_quant_workspace_size(int64_t m, int64_t n, int64_t k, int num_cus);

int launch_gemm_gated(int layout, const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                      int act, uint16_t* d, uint8_t* q, float* s, int64_t ld_s, uint16_t* pre, const int32_t* m_indices,
                      const int32_t* masked_m, int64_t groups, int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes,
                      hipStream_t stream, int num_cus);
size_t gemm_gated_workspace_size(int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus);
void gemm_gated_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, char* buf,
                            size_t len);
int launch_gated_act(int form, const void* pre, int dtype, int act, const int32_t* m_indices, const int32_t* masked_m,
                     int64_t rows_per_group, int64_t rows, int64_t n, void* h, float* scales, int64_t ld_s,
                     hipStream_t stream);
int launch_gated_act_grad(const void* dh, const void* pre, int dtype, int act, int64_t rows, int64_t n, void* dpre,
                          hipStream_t stream);
int launch_gated_act_grad_fp8(const void* dh, const void* pre, int dtype, int act, int64_t rows, int64_t n, uint8_t* q,
                              float* s, int64_t ld_s, uint8_t* qt, float* st, int64_t ld_st, uint8_t* ht, float* hst,
                              int64_t ld_hst, hipStream_t stream);
int launch_residual_norm(int out, const void* x, const void* residual, int dtype, int residual_dtype, const float* weight,
                         const void* gate, int64_t gate_rows, bool post_norm, const float* post_weight, float scale,
                         float eps, int64_t rows, int64_t hidden, void* sum, void* y, float* scales, int64_t ld_s,
                         hipStream_t stream);
size_t residual_norm_grad_workspace_size(int64_t rows, int64_t hidden);
int launch_residual_norm_grad(const void* dy, const void* dsum, const void* x, const void* sum, int dtype,
                              int residual_dtype, const float* weight, const void* gate, int64_t gate_rows, bool post_norm,
                              const float* post_weight, float scale, float eps, int64_t rows, int64_t hidden, void* dx,
                              void* dresidual, float* dweight, void* dgate, float* dpost, void* ws, hipStream_t stream);

static thread_local char g_msg[512] = "";

int set_error(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  if (debug_enabled()) std::fprintf(stderr, "[dg] %s\n", g_msg);
  return status;
}

bool debug_enabled() {
  const char* v = std::getenv("DG_DEBUG");
  return v != nullptr && v[0] != '\0' && !(v[0] == '0' && v[1] == '\0');
}

// ---- compute-unit cap (process-wide) ----------------------------------------
static std::atomic<int> g_cu_cap{0};      // 0 = not set: use every CU of the device
constexpr int kMaxDevices = 64;
static std::atomic<int> g_dev_cus[kMaxDevices];

// CUs of the current device (cached per device), or a negative status.
int device_cu_count() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return set_error(kHip, "hipGetDevice failed");
  if (dev < kMaxDevices) {
    const int cached = g_dev_cus[dev].load(std::memory_order_relaxed);
    if (cached > 0) return cached;
  }
  int cus = 0;
  const hipError_t e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess || cus <= 0) return set_error(kHip, "CU count query failed: %s", hipGetErrorString(e));
  if (dev < kMaxDevices) g_dev_cus[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

// The CU count the planner uses: the device's, capped by dg_set_num_cus.  With no device
// visible, a set cap stands in for it, so that the planning queries (configuration names,
// workspace sizes) also answer on a host without a GPU; launches still fail there.
static int effective_cus() {
  const int cap = g_cu_cap.load(std::memory_order_relaxed);
  const int cus = device_cu_count();
  if (cus < 0) return cap > 0 ? cap : cus;
  return (cap > 0 && cap < cus) ? cap : cus;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace dg

using namespace dg;

#define DG_REQUIRE(cond, ...)                           \
  do {                                                  \
    if (!(cond)) return set_error(kInvalidArg, __VA_ARGS__); \
  } while (0)

extern "C" {

const char* dg_status_string(int status) {
  switch (status) {
    case DG_OK: return "DG_OK";
    case DG_ERR_INVALID_ARG: return "DG_ERR_INVALID_ARG";
    case DG_ERR_UNSUPPORTED: return "DG_ERR_UNSUPPORTED";
    case DG_ERR_WORKSPACE: return "DG_ERR_WORKSPACE";
    case DG_ERR_HIP: return "DG_ERR_HIP";
    default: return "DG_ERR_UNKNOWN";
  }
}

const char* dg_last_error_message(void) { return g_msg; }

int dg_get_num_cus(void) { return effective_cus(); }

int dg_set_num_cus(int n) {
  DG_REQUIRE(n >= 1, "dg_set_num_cus: n must be >= 1 (got %d)", n);
  g_cu_cap.store(n, std::memory_order_relaxed);
  return DG_OK;
}

int dg_get_m_alignment_for_contiguous_layout(void) { return kGroup; }

int64_t dg_get_scale_ld(int64_t rows) { return rows <= 0 ? 0 : (rows + 3) / 4 * 4; }

size_t dg_gemm_workspace_size(int64_t m, int64_t n, int64_t k, int64_t num_groups) {
  if (m <= 0 || n <= 0 || k <= 0 || k % kKAlign || num_groups <= 0) return 0;
  const int cus = effective_cus();
  if (cus < 0) return 0;
  return gemm_workspace_size(m, n, k, num_groups, cus);
}

static int check_token_group(const void* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* q, float* sa,
                             int64_t ld_sa) {
  DG_REQUIRE(num_groups >= 0 && m >= 0 && k > 0 && k % kKAlign == 0,
             "quantize_per_token_group: need groups >= 0, m >= 0, k > 0, k %% 16 == 0 (m=%lld k=%lld)",
             (long long)m, (long long)k);
  DG_REQUIRE(ld_sa >= m && ld_sa % 4 == 0, "quantize_per_token_group: need ld_sa >= m and ld_sa %% 4 == 0 (ld_sa=%lld)",
             (long long)ld_sa);
  if (m == 0 || num_groups == 0) return DG_OK;
  DG_REQUIRE(x && q && sa, "quantize_per_token_group: null pointer");
  DG_REQUIRE(aligned16(x) && aligned16(q) && aligned16(sa), "quantize_per_token_group: pointers must be 16-byte aligned");
  return 1;   // proceed
}

int dg_quantize_per_token_group(const float* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* q,
                                float* sa, int64_t ld_sa, dg_stream_t stream) {
  const int c = check_token_group(x, num_groups, m, k, q, sa, ld_sa);
  if (c <= 0) return c;
  return launch_quant_token_group(x, num_groups, m, k, q, sa, ld_sa, static_cast<hipStream_t>(stream));
}

int dg_quantize_per_token_group_bf16(const uint16_t* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* q,
                                     float* sa, int64_t ld_sa, dg_stream_t stream) {
  const int c = check_token_group(x, num_groups, m, k, q, sa, ld_sa);
  if (c <= 0) return c;
  return launch_quant_token_group_bf16(x, num_groups, m, k, q, sa, ld_sa, static_cast<hipStream_t>(stream));
}

int dg_quantize_per_block(const float* w, int64_t num_groups, int64_t n, int64_t k, uint8_t* q,
                          float* sb, dg_stream_t stream) {
  DG_REQUIRE(num_groups >= 0 && n >= 0 && k > 0 && k % kKAlign == 0,
             "quantize_per_block: need groups >= 0, n >= 0, k > 0, k %% 16 == 0");
  if (num_groups == 0 || n == 0) return DG_OK;
  DG_REQUIRE(w && q && sb, "quantize_per_block: null pointer");
  DG_REQUIRE(aligned16(w) && aligned16(q) && aligned16(sb), "quantize_per_block: pointers must be 16-byte aligned");
  return launch_quant_block(w, num_groups, n, k, q, sb, static_cast<hipStream_t>(stream));
}

static int check_gemm_common(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b,
                             const float* sb, uint16_t* d, int64_t rows, int64_t n, int64_t k) {
  DG_REQUIRE(rows >= 0 && n >= 0 && k > 0 && k % kKAlign == 0, "gemm: need m >= 0, n >= 0, k > 0, k %% 16 == 0 (m=%lld n=%lld k=%lld)",
             (long long)rows, (long long)n, (long long)k);
  DG_REQUIRE(ld_sa >= rows && ld_sa % 4 == 0, "gemm: need ld_sa >= m and ld_sa %% 4 == 0 (ld_sa=%lld m=%lld)",
             (long long)ld_sa, (long long)rows);
  DG_REQUIRE(rows <= 0x7fffffffLL && n <= 0x7fffffffLL && k <= 0x7fffffffLL, "gemm: dimension too large");
  if (rows == 0 || n == 0) return DG_OK;
  DG_REQUIRE(a && sa && b && sb && d, "gemm: null pointer");
  DG_REQUIRE(aligned16(a) && aligned16(sa) && aligned16(b) && aligned16(sb) && aligned16(d),
             "gemm: pointers must be 16-byte aligned");
  return 1;   // proceed
}

int dg_gemm_fp8_nt(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b,
                   const float* sb, uint16_t* d, int64_t m, int64_t n, int64_t k, void* workspace,
                   size_t workspace_bytes, dg_stream_t stream) {
  const int c = check_gemm_common(a, sa, ld_sa, b, sb, d, m, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(workspace == nullptr || aligned16(workspace), "gemm: workspace must be 16-byte aligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm(0, a, sa, ld_sa, b, sb, 0, 0, d, nullptr, nullptr, 1, m, n, k, workspace,
                     workspace ? workspace_bytes : 0, static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_fp8_nt_no_alloc(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                            uint16_t* d, int64_t m, int64_t n, int64_t k, dg_stream_t stream) {
  const int c = check_gemm_common(a, sa, ld_sa, b, sb, d, m, n, k);
  if (c <= 0) return c;
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm_no_alloc(a, sa, ld_sa, b, sb, d, m, n, k, static_cast<hipStream_t>(stream), cus);
}

size_t dg_gemm_fp8_nt_act_quant_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || k <= 0 || k % kKAlign) return 0;
  const int cus = effective_cus();
  if (cus < 0) return 0;
  return gemm_fq_workspace_size(m, n, k, cus);
}

static int gemm_act_quant(const void* x, bool bf16, const uint8_t* b, const float* sb, uint16_t* d, int64_t m,
                          int64_t n, int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream) {
  DG_REQUIRE(m >= 0 && n >= 0 && k > 0 && k % kKAlign == 0,
             "gemm_act_quant: need m >= 0, n >= 0, k > 0, k %% 16 == 0 (m=%lld n=%lld k=%lld)", (long long)m,
             (long long)n, (long long)k);
  DG_REQUIRE(m <= 0x7fffffffLL && n <= 0x7fffffffLL && k <= 0x7fffffffLL, "gemm_act_quant: dimension too large");
  if (m == 0 || n == 0) return DG_OK;
  DG_REQUIRE(x && b && sb && d && workspace, "gemm_act_quant: null pointer");
  DG_REQUIRE(aligned16(x) && aligned16(b) && aligned16(sb) && aligned16(d) && aligned16(workspace),
             "gemm_act_quant: pointers must be 16-byte aligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm_fq(x, bf16, b, sb, d, m, n, k, workspace, workspace_bytes, static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_fp8_nt_act_quant(const float* x, const uint8_t* b, const float* sb, uint16_t* d, int64_t m, int64_t n,
                             int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream) {
  return gemm_act_quant(x, false, b, sb, d, m, n, k, workspace, workspace_bytes, stream);
}

int dg_gemm_fp8_nt_act_quant_bf16(const uint16_t* x, const uint8_t* b, const float* sb, uint16_t* d, int64_t m,
                                  int64_t n, int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream) {
  return gemm_act_quant(x, true, b, sb, d, m, n, k, workspace, workspace_bytes, stream);
}

int dg_gemm_fp8_grouped_contiguous(const uint8_t* a, const float* sa, int64_t ld_sa,
                                   const uint8_t* b, const float* sb, const int32_t* m_indices,
                                   int64_t num_groups, uint16_t* d, int64_t m_total, int64_t n,
                                   int64_t k, dg_stream_t stream) {
  DG_REQUIRE(num_groups >= 0, "contiguous gemm: num_groups must be >= 0");
  if (num_groups == 0) return DG_OK;
  DG_REQUIRE(m_total % kGroup == 0, "contiguous gemm: m_total must be a multiple of 128 (got %lld)", (long long)m_total);
  const int c = check_gemm_common(a, sa, ld_sa, b, sb, d, m_total, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(m_indices != nullptr, "contiguous gemm: m_indices is null");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm(1, a, sa, ld_sa, b, sb, 0, 0, d, m_indices, nullptr, num_groups, m_total, n, k,
                     nullptr, 0, static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_fp8_grouped_masked(const uint8_t* a, const float* sa, int64_t ld_sa,
                               const uint8_t* b, const float* sb, uint16_t* d,
                               const int32_t* masked_m, int64_t num_groups, int64_t m_max,
                               int64_t n, int64_t k, void* workspace, size_t workspace_bytes,
                               dg_stream_t stream) {
  DG_REQUIRE(num_groups >= 0, "masked gemm: num_groups must be >= 0");
  if (num_groups == 0) return DG_OK;
  DG_REQUIRE(num_groups <= 1024, "masked gemm: at most 1024 groups (got %lld)", (long long)num_groups);
  const int c = check_gemm_common(a, sa, ld_sa, b, sb, d, m_max, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(masked_m != nullptr, "masked gemm: masked_m is null");
  DG_REQUIRE(workspace == nullptr || aligned16(workspace), "gemm: workspace must be 16-byte aligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm(2, a, sa, ld_sa, b, sb, 0, 0, d, nullptr, masked_m, num_groups, m_max, n, k,
                     workspace, workspace ? workspace_bytes : 0, static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_fp8_nt_row_scaled(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b,
                              const float* sb, int64_t ld_sb, uint16_t* d, int64_t m, int64_t n, int64_t k,
                              void* workspace, size_t workspace_bytes, dg_stream_t stream) {
  const int c = check_gemm_common(a, sa, ld_sa, b, sb, d, m, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(ld_sb >= n && ld_sb % 4 == 0, "row-scaled gemm: need ld_sb >= n and ld_sb %% 4 == 0 (ld_sb=%lld n=%lld)",
             (long long)ld_sb, (long long)n);
  DG_REQUIRE(workspace == nullptr || aligned16(workspace), "gemm: workspace must be 16-byte aligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm(3, a, sa, ld_sa, b, sb, ld_sb, 0, d, nullptr, nullptr, 1, m, n, k, workspace,
                     workspace ? workspace_bytes : 0, static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_fp8_k_grouped_row_scaled(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b,
                                     const float* sb, int64_t ld_sb, uint16_t* d, const int64_t* group_tokens,
                                     int64_t num_groups, int64_t m, int64_t n, int64_t tokens_total, void* workspace,
                                     size_t workspace_bytes, dg_stream_t stream) {
  DG_REQUIRE(num_groups >= 0 && m >= 0 && n >= 0 && tokens_total >= 0,
             "k-grouped gemm: negative size (groups=%lld m=%lld n=%lld tokens=%lld)", (long long)num_groups,
             (long long)m, (long long)n, (long long)tokens_total);
  if (num_groups == 0 || m == 0 || n == 0) return DG_OK;
  DG_REQUIRE(group_tokens != nullptr, "k-grouped gemm: group_tokens is null");
  int64_t total = 0;
  for (int64_t g = 0; g < num_groups; ++g) {
    DG_REQUIRE(group_tokens[g] >= 0 && group_tokens[g] % kGroup == 0,
               "k-grouped gemm: group %lld has %lld tokens (need a multiple of 128)", (long long)g,
               (long long)group_tokens[g]);
    total += group_tokens[g];
  }
  DG_REQUIRE(total == tokens_total, "k-grouped gemm: group tokens sum to %lld, tokens_total is %lld", (long long)total,
             (long long)tokens_total);
  DG_REQUIRE(a && sa && b && sb && d, "k-grouped gemm: null pointer");
  DG_REQUIRE(aligned16(a) && aligned16(sa) && aligned16(b) && aligned16(sb) && aligned16(d),
             "k-grouped gemm: pointers must be 16-byte aligned");
  DG_REQUIRE(ld_sa >= m && ld_sa % 4 == 0 && ld_sb >= n && ld_sb % 4 == 0,
             "k-grouped gemm: need ld_sa >= m, ld_sb >= n, both multiples of 4");
  DG_REQUIRE((m * n) % 8 == 0, "k-grouped gemm: m * n must be a multiple of 8 (16-byte output blocks)");
  DG_REQUIRE(workspace == nullptr || aligned16(workspace), "gemm: workspace must be 16-byte aligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  int64_t start = 0;
  for (int64_t g = 0; g < num_groups; ++g) {
    const int64_t tk = group_tokens[g];
    uint16_t* dg_ = d + g * m * n;
    const int r = tk == 0 ? launch_fill_zero_bf16(dg_, m * n, s)
                          : launch_gemm(3, a + start, sa + (start / kGroup) * ld_sa, ld_sa, b + start,
                                        sb + (start / kGroup) * ld_sb, ld_sb, tokens_total, dg_, nullptr, nullptr, 1,
                                        m, n, tk, workspace, workspace ? workspace_bytes : 0, s, cus);
    if (r != kOk) return r;
    start += tk;
  }
  return DG_OK;
}

static int check_channel_group(const void* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* qt, float* st,
                               int64_t ld_st) {
  DG_REQUIRE(num_groups >= 0 && m >= 0 && m % kKAlign == 0 && k >= 0 && k % 4 == 0,
             "quantize_per_channel_group: need groups >= 0, m >= 0, m %% 16 == 0, k >= 0, k %% 4 == 0 "
             "(m=%lld k=%lld)", (long long)m, (long long)k);
  DG_REQUIRE(ld_st >= k && ld_st % 4 == 0, "quantize_per_channel_group: need ld_st >= k and ld_st %% 4 == 0 (ld_st=%lld)",
             (long long)ld_st);
  if (m == 0 || k == 0 || num_groups == 0) return DG_OK;
  DG_REQUIRE(x && qt && st, "quantize_per_channel_group: null pointer");
  DG_REQUIRE(aligned16(x) && aligned16(qt) && aligned16(st), "quantize_per_channel_group: pointers must be 16-byte aligned");
  return 1;   // proceed
}

int dg_quantize_per_channel_group(const float* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* qt, float* st,
                                  int64_t ld_st, dg_stream_t stream) {
  const int c = check_channel_group(x, num_groups, m, k, qt, st, ld_st);
  if (c <= 0) return c;
  return launch_quant_channel_group(x, num_groups, m, k, qt, st, ld_st, static_cast<hipStream_t>(stream));
}

int dg_quantize_per_channel_group_bf16(const uint16_t* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* qt,
                                       float* st, int64_t ld_st, dg_stream_t stream) {
  const int c = check_channel_group(x, num_groups, m, k, qt, st, ld_st);
  if (c <= 0) return c;
  return launch_quant_channel_group_bf16(x, num_groups, m, k, qt, st, ld_st, static_cast<hipStream_t>(stream));
}

int dg_transpose_blocks(const uint8_t* q, const float* s, int64_t num_groups, int64_t rows, int64_t cols, uint8_t* qt,
                        float* st, dg_stream_t stream) {
  DG_REQUIRE(num_groups >= 0 && rows >= 0 && cols >= 0 && rows % kKAlign == 0 && cols % kKAlign == 0,
             "transpose_blocks: need groups >= 0 and rows, cols >= 0 multiples of 16 (rows=%lld cols=%lld)",
             (long long)rows, (long long)cols);
  if (num_groups == 0 || rows == 0 || cols == 0) return DG_OK;
  DG_REQUIRE(q && s && qt && st, "transpose_blocks: null pointer");
  DG_REQUIRE(aligned16(q) && aligned16(qt), "transpose_blocks: code pointers must be 16-byte aligned");
  DG_REQUIRE(q != qt, "transpose_blocks: in-place transpose is not supported");
  return launch_transpose_blocks(q, s, num_groups, rows, cols, qt, st, static_cast<hipStream_t>(stream));
}

// ---- expert routing and the expert row layout ---------------------------------------------------
constexpr int64_t kMaxExperts = 1024, kMaxTopK = 64, kInt31 = 0x7fffffffLL;

static bool known_dtype(int dtype) { return dtype >= DG_DTYPE_F32 && dtype <= DG_DTYPE_F16; }
static size_t dtype_size(int dtype) { return dtype == DG_DTYPE_F32 ? 4 : 2; }
static bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

static int check_route(const char* what, int dtype, int64_t ld, int64_t tokens, int64_t experts, int64_t top_k, int score) {
  DG_REQUIRE(known_dtype(dtype), "%s: unknown dtype %d", what, dtype);
  DG_REQUIRE(tokens >= 0 && tokens <= kInt31 && experts >= 1 && experts <= kMaxExperts && top_k >= 1 &&
                 top_k <= kMaxTopK && top_k <= experts,
             "%s: need 0 <= tokens < 2^31, 1 <= experts <= 1024, 1 <= top_k <= min(64, experts) "
             "(tokens=%lld experts=%lld top_k=%lld)", what, (long long)tokens, (long long)experts, (long long)top_k);
  DG_REQUIRE(ld >= experts, "%s: need ld >= experts (ld=%lld)", what, (long long)ld);
  DG_REQUIRE(score == DG_MOE_SOFTMAX || score == DG_MOE_SIGMOID, "%s: unknown score %d", what, score);
  return DG_OK;
}

int dg_moe_route(const void* logits, int dtype, int64_t ld, const float* bias, int64_t tokens, int64_t experts,
                 int64_t top_k, int64_t num_groups, int64_t topk_groups, int group_top, int score, int renormalize,
                 float scale, int32_t* ids, float* weights, dg_stream_t stream) {
  const int c = check_route("moe_route", dtype, ld, tokens, experts, top_k, score);
  if (c != DG_OK) return c;
  DG_REQUIRE(num_groups >= 1 && num_groups <= 64 && experts % num_groups == 0 && topk_groups >= 1 &&
                 topk_groups <= num_groups && (group_top == 1 || group_top == 2),
             "moe_route: need 1 <= topk_groups <= num_groups <= 64, experts %% num_groups == 0, group_top 1 or 2 "
             "(num_groups=%lld topk_groups=%lld group_top=%d)", (long long)num_groups, (long long)topk_groups, group_top);
  if (tokens == 0) return DG_OK;
  DG_REQUIRE(logits && ids && weights, "moe_route: null pointer");
  DG_REQUIRE(aligned_to(logits, dtype_size(dtype)) && aligned_to(bias, 4) && aligned_to(ids, 4) && aligned_to(weights, 4),
             "moe_route: misaligned pointer");
  return launch_route(logits, dtype, ld, bias, tokens, (int)experts, (int)top_k, (int)num_groups, (int)topk_groups,
                      group_top, score == DG_MOE_SOFTMAX, renormalize != 0, scale, ids, weights,
                      static_cast<hipStream_t>(stream));
}

int dg_moe_route_grad(const float* dweights, const void* logits, int dtype, int64_t ld, const int32_t* ids,
                      int64_t tokens, int64_t experts, int64_t top_k, int score, int renormalize, float scale,
                      void* dlogits, int64_t ld_out, dg_stream_t stream) {
  const int c = check_route("moe_route_grad", dtype, ld, tokens, experts, top_k, score);
  if (c != DG_OK) return c;
  DG_REQUIRE(ld_out >= experts, "moe_route_grad: need ld_out >= experts (ld_out=%lld)", (long long)ld_out);
  if (tokens == 0) return DG_OK;
  DG_REQUIRE(dweights && logits && ids && dlogits, "moe_route_grad: null pointer");
  DG_REQUIRE(aligned_to(logits, dtype_size(dtype)) && aligned_to(dlogits, dtype_size(dtype)) && aligned_to(ids, 4) &&
                 aligned_to(dweights, 4), "moe_route_grad: misaligned pointer");
  return launch_route_grad(dweights, logits, dtype, ld, ids, tokens, (int)experts, (int)top_k, score == DG_MOE_SOFTMAX,
                           renormalize != 0, scale, dlogits, ld_out, static_cast<hipStream_t>(stream));
}

int64_t dg_moe_layout_rows(int64_t tokens, int64_t top_k, int64_t experts) {
  if (tokens <= 0 || top_k <= 0 || experts <= 0 || tokens > kInt31 || top_k > kMaxTopK) return 0;
  const int64_t n = tokens * top_k;
  // every expert in use may waste up to 127 rows
  return (n + (experts < n ? experts : n) * (kGroup - 1)) / kGroup * kGroup;
}

size_t dg_moe_layout_workspace_size(int64_t tokens, int64_t top_k, int64_t experts) {
  if (tokens <= 0 || top_k <= 0 || top_k > kMaxTopK || experts <= 0 || experts > kMaxExperts ||
      tokens * top_k > kInt31)
    return 0;
  return moe_layout_workspace_size(tokens * top_k, experts);
}

int dg_moe_layout(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts, int64_t rows_per_expert,
                  int64_t rows_total, int32_t* rows, int32_t* sources, int32_t* m_indices, int32_t* counts,
                  void* workspace, size_t workspace_bytes, dg_stream_t stream) {
  DG_REQUIRE(tokens >= 0 && tokens <= kInt31 && top_k >= 1 && top_k <= kMaxTopK && experts >= 1 && experts <= kMaxExperts &&
                 rows_per_expert >= 0 && rows_total >= 0,
             "moe_layout: need tokens >= 0, 1 <= top_k <= 64, 1 <= experts <= 1024, no negative size "
             "(tokens=%lld top_k=%lld experts=%lld)", (long long)tokens, (long long)top_k, (long long)experts);
  if (rows_per_expert > 0) {
    DG_REQUIRE(rows_per_expert <= kInt31 && rows_total == experts * rows_per_expert && m_indices == nullptr,
               "moe_layout: the masked layout has experts * rows_per_expert rows and no m_indices (rows_total=%lld)",
               (long long)rows_total);
  } else {
    DG_REQUIRE(rows_total % kGroup == 0 && rows_total >= dg_moe_layout_rows(tokens, top_k, experts),
               "moe_layout: the contiguous layout needs a multiple of 128 and at least %lld rows (rows_total=%lld)",
               (long long)dg_moe_layout_rows(tokens, top_k, experts), (long long)rows_total);
    DG_REQUIRE(m_indices != nullptr || rows_total == 0, "moe_layout: m_indices is null");
  }
  if (tokens * top_k > kInt31 || rows_total > kInt31) return set_error(kUnsupported, "moe_layout: 2^31 entries or rows");
  DG_REQUIRE(counts && (rows_total == 0 || sources) && (tokens == 0 || (ids && rows)), "moe_layout: null pointer");
  DG_REQUIRE(aligned_to(ids, 4) && aligned_to(rows, 4) && aligned_to(sources, 4) && aligned_to(m_indices, 4) &&
                 aligned_to(counts, 4) && aligned_to(workspace, 4), "moe_layout: misaligned pointer");
  const size_t need = dg_moe_layout_workspace_size(tokens, top_k, experts);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return set_error(kWorkspace, "moe_layout: workspace of %zu bytes, %zu needed", workspace_bytes, need);
  return launch_moe_layout(ids, tokens * top_k, (int)experts, rows_per_expert, kGroup, rows_total, rows, sources,
                           m_indices, counts, workspace, static_cast<hipStream_t>(stream));
}

static int check_rows(const char* what, int dtype, const int32_t* rows, const int32_t* sources, const int32_t* m_indices,
                      int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows_total) {
  DG_REQUIRE(known_dtype(dtype), "%s: unknown dtype %d", what, dtype);
  DG_REQUIRE(tokens >= 0 && top_k >= 1 && top_k <= kMaxTopK && hidden > 0 && hidden % kKAlign == 0 && rows_total >= 0,
             "%s: need tokens >= 0, 1 <= top_k <= 64, hidden > 0, hidden %% 16 == 0, rows_total >= 0 "
             "(tokens=%lld top_k=%lld hidden=%lld)", what, (long long)tokens, (long long)top_k, (long long)hidden);
  // tokens and rows each index a grid dimension with the padding's workgroups
  DG_REQUIRE(tokens <= kInt31 / 2 && tokens * top_k <= kInt31 && rows_total <= kInt31 && hidden <= kInt31 / 64,
             "%s: dimension too large", what);
  DG_REQUIRE(m_indices == nullptr || sources != nullptr, "%s: m_indices without sources", what);
  DG_REQUIRE(tokens == 0 || rows != nullptr, "%s: null pointer", what);
  DG_REQUIRE(aligned_to(rows, 4) && aligned_to(sources, 4) && aligned_to(m_indices, 4), "%s: misaligned pointer", what);
  return DG_OK;
}

static int moe_dispatch(const char* what, int form, const void* x, int dtype, const int32_t* rows, const int32_t* sources,
                        const int32_t* m_indices, int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows_total,
                        int64_t rows_per_expert, void* q, float* s, int64_t ld_s, float* s_tmp, dg_stream_t stream) {
  const int c = check_rows(what, dtype, rows, sources, m_indices, tokens, top_k, hidden, rows_total);
  if (c != DG_OK) return c;
  DG_REQUIRE(rows_per_expert >= 0 && (rows_per_expert == 0) == (m_indices != nullptr || rows_total == 0),
             "%s: m_indices for the contiguous layout, rows_per_expert for the masked one", what);
  DG_REQUIRE(rows_per_expert == 0 || rows_total % rows_per_expert == 0, "%s: rows_total is not whole experts", what);
  if (rows_total == 0) return DG_OK;
  DG_REQUIRE(q && (tokens == 0 || x) && (form == 0 || s), "%s: null pointer", what);
  DG_REQUIRE(aligned16(x) && aligned16(q) && aligned_to(s, 4), "%s: row data must be 16-byte aligned", what);
  return launch_moe_dispatch(form, x, dtype, rows, sources, m_indices, tokens, (int)top_k, hidden, rows_total,
                             rows_per_expert, q, s, ld_s, s_tmp, static_cast<hipStream_t>(stream));
}

int dg_moe_dispatch(const void* x, int dtype, const int32_t* rows, const int32_t* sources, const int32_t* m_indices,
                    int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows_total, int64_t rows_per_expert,
                    void* out, dg_stream_t stream) {
  return moe_dispatch("moe_dispatch", 0, x, dtype, rows, sources, m_indices, tokens, top_k, hidden, rows_total,
                      rows_per_expert, out, nullptr, 0, nullptr, stream);
}

size_t dg_moe_dispatch_fp8_workspace_size(int64_t tokens, int64_t top_k, int64_t hidden) {
  if (tokens <= 0 || tokens > kInt31 / 2 || top_k <= 0 || top_k > kMaxTopK || hidden <= 0 || hidden % kKAlign ||
      hidden > kInt31 / 64)
    return 0;
  return moe_dispatch_fp8_workspace_size(tokens, top_k, hidden);
}

int dg_moe_dispatch_fp8(const void* x, int dtype, const int32_t* rows, const int32_t* sources, const int32_t* m_indices,
                        int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows_total, int64_t rows_per_expert,
                        uint8_t* q, float* sa, int64_t ld_sa, void* workspace, size_t workspace_bytes,
                        dg_stream_t stream) {
  const int64_t need = rows_per_expert > 0 ? rows_per_expert : rows_total;
  DG_REQUIRE(ld_sa >= need && ld_sa % 4 == 0, "moe_dispatch_fp8: need ld_sa >= %lld and ld_sa %% 4 == 0 (ld_sa=%lld)",
             (long long)need, (long long)ld_sa);
  DG_REQUIRE(aligned_to(workspace, 4), "moe_dispatch_fp8: misaligned workspace");
  // without a workspace (or with too small a one) the scales go straight to their places
  const size_t tmp = dg_moe_dispatch_fp8_workspace_size(tokens, top_k, hidden);
  const bool moved = tmp > 0 && workspace != nullptr && workspace_bytes >= tmp && sources != nullptr;
  return moe_dispatch("moe_dispatch_fp8", 1, x, dtype, rows, sources, m_indices, tokens, top_k, hidden, rows_total,
                      rows_per_expert, q, sa, ld_sa, moved ? static_cast<float*>(workspace) : nullptr, stream);
}

int dg_moe_dispatch_int8(const void* x, int dtype, const int32_t* rows, const int32_t* sources,
                         const int32_t* m_indices, int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows_total,
                         int64_t rows_per_expert, int8_t* q, float* s, dg_stream_t stream) {
  return moe_dispatch("moe_dispatch_int8", 2, x, dtype, rows, sources, m_indices, tokens, top_k, hidden, rows_total,
                      rows_per_expert, q, s, 0, nullptr, stream);
}

int dg_moe_combine(const void* out, int dtype, const int32_t* rows, const float* weights, int64_t tokens, int64_t top_k,
                   int64_t hidden, int64_t rows_total, void* y, dg_stream_t stream) {
  const int c = check_rows("moe_combine", dtype, rows, nullptr, nullptr, tokens, top_k, hidden, rows_total);
  if (c != DG_OK) return c;
  if (tokens == 0) return DG_OK;
  DG_REQUIRE(y && (rows_total == 0 || out), "moe_combine: null pointer");
  DG_REQUIRE(aligned16(out) && aligned16(y) && aligned_to(weights, 4), "moe_combine: row data must be 16-byte aligned");
  return launch_moe_combine(out, dtype, rows, weights, tokens, (int)top_k, hidden, rows_total, y,
                            static_cast<hipStream_t>(stream));
}

int dg_moe_combine_grad(const void* dy, const void* out, int dtype, const int32_t* rows, const int32_t* sources,
                        const int32_t* m_indices, const float* weights, int64_t tokens, int64_t top_k, int64_t hidden,
                        int64_t rows_total, void* dout, float* dweights, dg_stream_t stream) {
  const int c = check_rows("moe_combine_grad", dtype, rows, sources, m_indices, tokens, top_k, hidden, rows_total);
  if (c != DG_OK) return c;
  DG_REQUIRE((tokens == 0 || (dy && weights && dweights)) && (rows_total == 0 || (out && dout)),
             "moe_combine_grad: null pointer");
  DG_REQUIRE(aligned16(dy) && aligned16(out) && aligned16(dout) && aligned_to(weights, 4) && aligned_to(dweights, 4),
             "moe_combine_grad: row data must be 16-byte aligned");
  return launch_moe_combine_grad(dy, out, dtype, rows, sources, m_indices, weights, tokens, (int)top_k, hidden, rows_total,
                                 dout, dweights, static_cast<hipStream_t>(stream));
}

// ---- 8-bit integer GEMMs ------------------------------------------------------------------------
constexpr int64_t kInt8MaxK = 131056;   // 16 * 8191: 2^14 per product, below 2^31 in all

int dg_quantize_int8_per_token(const void* x, int dtype, int64_t rows, int64_t k, int8_t* q, float* s,
                               dg_stream_t stream) {
  DG_REQUIRE(known_dtype(dtype), "quantize_int8_per_token: unknown dtype %d", dtype);
  DG_REQUIRE(rows >= 0 && k > 0 && k % kKAlign == 0,
             "quantize_int8_per_token: need rows >= 0, k > 0, k %% 16 == 0 (rows=%lld k=%lld)", (long long)rows, (long long)k);
  if (rows == 0) return DG_OK;
  DG_REQUIRE(x && q && s, "quantize_int8_per_token: null pointer");
  DG_REQUIRE(aligned16(x) && aligned16(q) && aligned_to(s, 4), "quantize_int8_per_token: row data must be 16-byte aligned");
  return launch_quant_int8(x, dtype, rows, k, q, s, static_cast<hipStream_t>(stream));
}

static int check_int8(const char* what, const void* a, const float* sa, const int8_t* b, const float* sb, const void* d,
                      int out_dtype, int64_t m, int64_t n, int64_t k) {
  DG_REQUIRE(known_dtype(out_dtype), "%s: unknown output dtype %d", what, out_dtype);
  DG_REQUIRE(m >= 0 && n >= 0 && k > 0 && k % kKAlign == 0, "%s: need m >= 0, n >= 0, k > 0, k %% 16 == 0 (m=%lld n=%lld k=%lld)",
             what, (long long)m, (long long)n, (long long)k);
  DG_REQUIRE(m <= kInt31 - 1024 && n <= kInt31 - 1024, "%s: dimension too large", what);
  if (k > kInt8MaxK)
    return set_error(kUnsupported, "%s: k = %lld, int32 sums hold at most %lld", what, (long long)k, (long long)kInt8MaxK);
  if (m == 0 || n == 0) return DG_OK;
  DG_REQUIRE(a && sa && b && sb && d, "%s: null pointer", what);
  DG_REQUIRE(aligned16(a) && aligned16(b) && aligned16(d) && aligned_to(sa, 4) && aligned_to(sb, 4),
             "%s: a, b and d must be 16-byte aligned", what);
  return 1;   // proceed
}

size_t dg_gemm_int8_workspace_size(int64_t m, int64_t n, int64_t k, int64_t num_groups) {
  if (m <= 0 || n <= 0 || k <= 0 || k % kKAlign || k > kInt8MaxK || num_groups <= 0 || num_groups > 1024) return 0;
  const int cus = effective_cus();
  return cus < 0 ? 0 : int8_workspace_size(m, n, k, num_groups, cus);
}

size_t dg_gemm_int8_nt_act_quant_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || k <= 0 || k % kKAlign || k > kInt8MaxK) return 0;
  const int cus = effective_cus();
  return cus < 0 ? 0 : int8_act_quant_workspace_size(m, n, k, cus);
}

int dg_gemm_int8_nt(const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d, int out_dtype,
                    int64_t m, int64_t n, int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream) {
  const int c = check_int8("int8 gemm", a, sa, b, sb, d, out_dtype, m, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(aligned16(workspace), "int8 gemm: workspace must be 16-byte aligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm_int8(0, a, sa, b, sb, d, out_dtype, nullptr, nullptr, 1, m, n, k, workspace,
                          workspace ? workspace_bytes : 0, static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_int8_nt_act_quant(const void* x, int dtype, const int8_t* b, const float* sb, void* d, int out_dtype,
                              int64_t m, int64_t n, int64_t k, void* workspace, size_t workspace_bytes,
                              dg_stream_t stream) {
  DG_REQUIRE(known_dtype(dtype), "int8 gemm with activation quantization: unknown dtype %d", dtype);
  const int c = check_int8("int8 gemm with activation quantization", x, sb, b, sb, d, out_dtype, m, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(aligned16(workspace), "int8 gemm with activation quantization: workspace must be 16-byte aligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  const size_t need = int8_act_quant_workspace_size(m, n, k, cus);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return set_error(kWorkspace, "int8 gemm with activation quantization: workspace of %zu bytes, %zu needed",
                     workspace ? workspace_bytes : (size_t)0, need);
  return launch_gemm_int8_act_quant(x, dtype, b, sb, d, out_dtype, m, n, k, workspace, workspace_bytes,
                                    static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_int8_grouped_contiguous(const int8_t* a, const float* sa, const int8_t* b, const float* sb,
                                    const int32_t* m_indices, int64_t num_groups, void* d, int out_dtype,
                                    int64_t m_total, int64_t n, int64_t k, dg_stream_t stream) {
  DG_REQUIRE(num_groups >= 0 && num_groups <= kInt31, "contiguous int8 gemm: num_groups must be >= 0");
  if (num_groups == 0) return DG_OK;
  DG_REQUIRE(m_total % kGroup == 0, "contiguous int8 gemm: m_total must be a multiple of 128 (got %lld)", (long long)m_total);
  const int c = check_int8("contiguous int8 gemm", a, sa, b, sb, d, out_dtype, m_total, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(m_indices != nullptr && aligned_to(m_indices, 4), "contiguous int8 gemm: m_indices is null or misaligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm_int8(1, a, sa, b, sb, d, out_dtype, m_indices, nullptr, num_groups, m_total, n, k, nullptr, 0,
                          static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_int8_grouped_masked(const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d,
                                int out_dtype, const int32_t* masked_m, int64_t num_groups, int64_t m_max, int64_t n,
                                int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream) {
  DG_REQUIRE(num_groups >= 0, "masked int8 gemm: num_groups must be >= 0");
  if (num_groups == 0) return DG_OK;
  DG_REQUIRE(num_groups <= 1024, "masked int8 gemm: at most 1024 groups (got %lld)", (long long)num_groups);
  const int c = check_int8("masked int8 gemm", a, sa, b, sb, d, out_dtype, m_max, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(masked_m != nullptr && aligned_to(masked_m, 4), "masked int8 gemm: masked_m is null or misaligned");
  DG_REQUIRE(aligned16(workspace), "masked int8 gemm: workspace must be 16-byte aligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm_int8(2, a, sa, b, sb, d, out_dtype, nullptr, masked_m, num_groups, m_max, n, k, workspace,
                          workspace ? workspace_bytes : 0, static_cast<hipStream_t>(stream), cus);
}

// ---- gated GEMMs ----------------------------------------------------------------------------------
static int gemm_gated(int layout, const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                      int act, uint16_t* d, uint8_t* q, float* s, int64_t ld_s, uint16_t* pre, const int32_t* m_indices,
                      const int32_t* masked_m, int64_t groups, int64_t m, int64_t n, int64_t k, void* workspace,
                      size_t workspace_bytes, dg_stream_t stream) {
  DG_REQUIRE(groups >= 0 && (layout != 2 || groups <= 1024), "gated gemm: need 0 <= num_groups, at most 1024 masked ones (got %lld)",
             (long long)groups);
  DG_REQUIRE(act == DG_ACT_SILU || act == DG_ACT_GELU, "gated gemm: unknown activation %d", act);
  if (groups == 0) return DG_OK;
  DG_REQUIRE(layout != 1 || m % kGroup == 0, "contiguous gated gemm: m_total must be a multiple of 128 (got %lld)", (long long)m);
  DG_REQUIRE((d == nullptr) != (q == nullptr) || m == 0 || n == 0, "gated gemm: one of d and q is given");
  const int c = check_gemm_common(a, sa, ld_sa, b, sb, d != nullptr ? d : reinterpret_cast<uint16_t*>(q), m, n, k);
  if (c <= 0) return c;
  DG_REQUIRE(q == nullptr || (s != nullptr && aligned_to(s, 4) && n % kKAlign == 0 && ld_s >= m && ld_s % 4 == 0),
             "gated gemm: quantized output needs scales, n %% 16 == 0, ld_s >= m, ld_s %% 4 == 0 (n=%lld ld_s=%lld)",
             (long long)n, (long long)ld_s);
  DG_REQUIRE(aligned16(pre) && aligned16(workspace), "gated gemm: pointers must be 16-byte aligned");
  DG_REQUIRE(layout != 1 || (m_indices != nullptr && aligned_to(m_indices, 4)), "contiguous gated gemm: m_indices is null or misaligned");
  DG_REQUIRE(layout != 2 || (masked_m != nullptr && aligned_to(masked_m, 4)), "masked gated gemm: masked_m is null or misaligned");
  const int cus = effective_cus();
  if (cus < 0) return cus;
  return launch_gemm_gated(layout, a, sa, ld_sa, b, sb, act, d, q, s, ld_s, pre, m_indices, masked_m, groups, m, n, k,
                           workspace, workspace ? workspace_bytes : 0, static_cast<hipStream_t>(stream), cus);
}

int dg_gemm_fp8_gated_nt(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb, int act,
                         uint16_t* d, uint8_t* q, float* s, int64_t ld_s, uint16_t* pre, int64_t m, int64_t n, int64_t k,
                         void* workspace, size_t workspace_bytes, dg_stream_t stream) {
  return gemm_gated(0, a, sa, ld_sa, b, sb, act, d, q, s, ld_s, pre, nullptr, nullptr, 1, m, n, k, workspace,
                    workspace_bytes, stream);
}

int dg_gemm_fp8_gated_contiguous(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                                 const int32_t* m_indices, int64_t num_groups, int act, uint16_t* d, uint8_t* q, float* s,
                                 int64_t ld_s, uint16_t* pre, int64_t m_total, int64_t n, int64_t k, dg_stream_t stream) {
  return gemm_gated(1, a, sa, ld_sa, b, sb, act, d, q, s, ld_s, pre, m_indices, nullptr, num_groups, m_total, n, k,
                    nullptr, 0, stream);
}

int dg_gemm_fp8_gated_masked(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                             const int32_t* masked_m, int64_t num_groups, int act, uint16_t* d, uint8_t* q, float* s,
                             int64_t ld_s, uint16_t* pre, int64_t m_max, int64_t n, int64_t k, void* workspace,
                             size_t workspace_bytes, dg_stream_t stream) {
  return gemm_gated(2, a, sa, ld_sa, b, sb, act, d, q, s, ld_s, pre, nullptr, masked_m, num_groups, m_max, n, k, workspace,
                    workspace_bytes, stream);
}

size_t dg_gemm_fp8_gated_workspace_size(int64_t m, int64_t n, int64_t k, int64_t num_groups) {
  if (m <= 0 || n <= 0 || k <= 0 || k % kKAlign || num_groups <= 0 || num_groups > 1024 || m > kInt31 || n > kInt31 || k > kInt31)
    return 0;
  const int cus = effective_cus();
  return cus < 0 ? 0 : gemm_gated_workspace_size(m, n, k, num_groups, cus);
}

const char* dg_gemm_fp8_gated_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t num_groups) {
  static thread_local char buf[96];
  buf[0] = 0;
  if (layout < 0 || layout > 2 || m <= 0 || n <= 0 || k <= 0 || k % kKAlign || num_groups <= 0 || m > kInt31 || n > kInt31 ||
      k > kInt31 || (layout == 2 && num_groups > 1024))
    return buf;
  const int cus = effective_cus();
  if (cus < 0) return buf;
  gemm_gated_config_name(layout, m, n, k, num_groups, cus, buf, sizeof(buf));
  return buf;
}

// ---- gated activation ---------------------------------------------------------------------------
static int check_act(const char* what, int dtype, int act, int64_t rows, int64_t n) {
  DG_REQUIRE(known_dtype(dtype), "%s: unknown dtype %d", what, dtype);
  DG_REQUIRE(act == DG_ACT_SILU || act == DG_ACT_GELU, "%s: unknown activation %d", what, act);
  DG_REQUIRE(rows >= 0 && n > 0 && n % kKAlign == 0, "%s: need rows >= 0, n > 0, n %% 16 == 0 (rows=%lld n=%lld)", what,
             (long long)rows, (long long)n);
  DG_REQUIRE(n <= kInt31 / 64 && rows <= kInt31, "%s: dimension too large", what);
  return DG_OK;
}

static int gated_act(const char* what, int form, const void* pre, int dtype, int act, const int32_t* m_indices,
                     const int32_t* masked_m, int64_t rows_per_group, int64_t rows, int64_t n, void* h, float* s,
                     int64_t ld_s, dg_stream_t stream) {
  const int c = check_act(what, dtype, act, rows, n);
  if (c != DG_OK) return c;
  DG_REQUIRE(m_indices == nullptr || masked_m == nullptr, "%s: m_indices or masked_m, not both", what);
  DG_REQUIRE(masked_m != nullptr ? rows_per_group > 0 && rows % rows_per_group == 0 : rows_per_group == 0,
             "%s: rows_per_group goes with masked_m and divides rows (rows_per_group=%lld rows=%lld)", what,
             (long long)rows_per_group, (long long)rows);
  if (form == 1) {
    const int64_t need = masked_m != nullptr ? rows_per_group : rows;
    DG_REQUIRE(ld_s >= need && ld_s % 4 == 0, "%s: need ld_s >= %lld and ld_s %% 4 == 0 (ld_s=%lld)", what, (long long)need,
               (long long)ld_s);
  }
  if (rows == 0) return DG_OK;
  DG_REQUIRE(pre && h && (form == 0 || s), "%s: null pointer", what);
  DG_REQUIRE(aligned16(pre) && aligned16(h), "%s: row data must be 16-byte aligned", what);
  DG_REQUIRE(aligned_to(s, 4) && aligned_to(m_indices, 4) && aligned_to(masked_m, 4), "%s: misaligned pointer", what);
  return launch_gated_act(form, pre, dtype, act, m_indices, masked_m, rows_per_group, rows, n, h, s, ld_s,
                          static_cast<hipStream_t>(stream));
}

int dg_gated_act(const void* pre, int dtype, int act, const int32_t* m_indices, const int32_t* masked_m,
                 int64_t rows_per_group, int64_t rows, int64_t n, void* h, dg_stream_t stream) {
  return gated_act("gated_act", 0, pre, dtype, act, m_indices, masked_m, rows_per_group, rows, n, h, nullptr, 0, stream);
}

int dg_gated_act_fp8(const void* pre, int dtype, int act, const int32_t* m_indices, const int32_t* masked_m,
                     int64_t rows_per_group, int64_t rows, int64_t n, uint8_t* q, float* s, int64_t ld_s,
                     dg_stream_t stream) {
  return gated_act("gated_act_fp8", 1, pre, dtype, act, m_indices, masked_m, rows_per_group, rows, n, q, s, ld_s, stream);
}

int dg_gated_act_int8(const void* pre, int dtype, int act, const int32_t* m_indices, const int32_t* masked_m,
                      int64_t rows_per_group, int64_t rows, int64_t n, int8_t* q, float* s, dg_stream_t stream) {
  return gated_act("gated_act_int8", 2, pre, dtype, act, m_indices, masked_m, rows_per_group, rows, n, q, s, 0, stream);
}

int dg_gated_act_grad(const void* dh, const void* pre, int dtype, int act, int64_t rows, int64_t n, void* dpre,
                      dg_stream_t stream) {
  const int c = check_act("gated_act_grad", dtype, act, rows, n);
  if (c != DG_OK) return c;
  if (rows == 0) return DG_OK;
  DG_REQUIRE(dh && pre && dpre, "gated_act_grad: null pointer");
  DG_REQUIRE(aligned16(dh) && aligned16(pre) && aligned16(dpre), "gated_act_grad: row data must be 16-byte aligned");
  return launch_gated_act_grad(dh, pre, dtype, act, rows, n, dpre, static_cast<hipStream_t>(stream));
}

int dg_gated_act_grad_fp8(const void* dh, const void* pre, int dtype, int act, int64_t rows, int64_t n, uint8_t* q,
                          float* s, int64_t ld_s, uint8_t* qt, float* st, int64_t ld_st, uint8_t* ht, float* hst,
                          int64_t ld_hst, dg_stream_t stream) {
  const int c = check_act("gated_act_grad_fp8", dtype, act, rows, n);
  if (c != DG_OK) return c;
  DG_REQUIRE(n % kGroup == 0 && rows % kKAlign == 0, "gated_act_grad_fp8: need n %% 128 == 0 and rows %% 16 == 0 (rows=%lld n=%lld)",
             (long long)rows, (long long)n);
  if (rows == 0) return DG_OK;
  DG_REQUIRE(dh && pre && (q || qt || ht), "gated_act_grad_fp8: null pointer");
  DG_REQUIRE((q == nullptr) == (s == nullptr) && (qt == nullptr) == (st == nullptr) && (ht == nullptr) == (hst == nullptr),
             "gated_act_grad_fp8: codes and scales are given together");
  DG_REQUIRE((!q || (ld_s >= rows && ld_s % 4 == 0)) && (!qt || (ld_st >= 2 * n && ld_st % 4 == 0)) &&
                 (!ht || (ld_hst >= n && ld_hst % 4 == 0)),
             "gated_act_grad_fp8: need ld_s >= rows, ld_st >= 2n, ld_hst >= n, multiples of 4");
  DG_REQUIRE(aligned16(dh) && aligned16(pre) && aligned16(q) && aligned16(s) && aligned16(qt) && aligned16(st) &&
                 aligned16(ht) && aligned16(hst), "gated_act_grad_fp8: pointers must be 16-byte aligned");
  return launch_gated_act_grad_fp8(dh, pre, dtype, act, rows, n, q, s, ld_s, qt, st, ld_st, ht, hst, ld_hst,
                                   static_cast<hipStream_t>(stream));
}

// ---- residual norms -----------------------------------------------------------------------------
static int check_norm(const char* what, int dtype, int residual_dtype, const void* x, const float* weight, const void* gate,
                      int64_t gate_rows, int post_norm, const float* post_weight, float eps, int64_t rows, int64_t hidden) {
  DG_REQUIRE(known_dtype(dtype) && (residual_dtype == dtype || residual_dtype == DG_DTYPE_F32),
             "%s: unknown dtype %d, or residual_dtype %d neither that nor fp32", what, dtype, residual_dtype);
  DG_REQUIRE(rows >= 0 && hidden > 0 && hidden % kKAlign == 0, "%s: need rows >= 0, hidden > 0, hidden %% 16 == 0 "
             "(rows=%lld hidden=%lld)", what, (long long)rows, (long long)hidden);
  DG_REQUIRE((gate == nullptr) == (gate_rows == 0) && gate_rows >= 0 && (gate_rows == 0 || rows % gate_rows == 0),
             "%s: gate_rows must divide rows, 0 without a gate (gate_rows=%lld rows=%lld)", what, (long long)gate_rows,
             (long long)rows);
  DG_REQUIRE(x != nullptr || rows == 0 || (gate == nullptr && !post_norm), "%s: a gate or a first norm without x", what);
  DG_REQUIRE(post_norm || post_weight == nullptr, "%s: post_weight without post_norm", what);
  DG_REQUIRE(eps >= 0.0f && eps <= 3.0e38f, "%s: eps must be finite and not negative", what);
  DG_REQUIRE(aligned16(x) && aligned16(gate) && aligned16(weight) && aligned16(post_weight),
             "%s: pointers must be 16-byte aligned", what);
  return DG_OK;
}

static int residual_norm(const char* what, int out, const void* x, const void* residual, int dtype, int residual_dtype,
                         const float* weight, const void* gate, int64_t gate_rows, int post_norm,
                         const float* post_weight, float scale, float eps, int64_t rows, int64_t hidden, void* sum, void* y,
                         float* s, int64_t ld_s, dg_stream_t stream) {
  const int c = check_norm(what, dtype, residual_dtype, x, weight, gate, gate_rows, post_norm, post_weight, eps, rows, hidden);
  if (c != DG_OK) return c;
  DG_REQUIRE(out != 1 || (ld_s >= rows && ld_s % 4 == 0), "%s: need ld_s >= rows and ld_s %% 4 == 0 (ld_s=%lld)", what,
             (long long)ld_s);
  if (rows == 0) return DG_OK;
  DG_REQUIRE(residual && y && (out == 0 || s), "%s: null pointer", what);
  DG_REQUIRE(x != nullptr || sum == nullptr, "%s: without x the sum is the residual: sum must be null", what);
  DG_REQUIRE(aligned16(residual) && aligned16(sum) && aligned16(y), "%s: row data must be 16-byte aligned", what);
  DG_REQUIRE(aligned_to(s, 4), "%s: misaligned pointer", what);
  return launch_residual_norm(out, x, residual, dtype, residual_dtype, weight, gate, gate_rows, post_norm != 0, post_weight,
                              scale, eps, rows, hidden, sum, y, s, ld_s, static_cast<hipStream_t>(stream));
}

int dg_residual_norm(const void* x, const void* residual, int dtype, int residual_dtype, const float* weight,
                     const void* gate, int64_t gate_rows, int post_norm, const float* post_weight, float scale, float eps,
                     int64_t rows, int64_t hidden, void* sum, void* y, dg_stream_t stream) {
  return residual_norm("residual_norm", 0, x, residual, dtype, residual_dtype, weight, gate, gate_rows, post_norm,
                       post_weight, scale, eps, rows, hidden, sum, y, nullptr, 0, stream);
}

int dg_residual_norm_fp8(const void* x, const void* residual, int dtype, int residual_dtype, const float* weight,
                         const void* gate, int64_t gate_rows, int post_norm, const float* post_weight, float scale,
                         float eps, int64_t rows, int64_t hidden, void* sum, uint8_t* q, float* s, int64_t ld_s,
                         dg_stream_t stream) {
  return residual_norm("residual_norm_fp8", 1, x, residual, dtype, residual_dtype, weight, gate, gate_rows, post_norm,
                       post_weight, scale, eps, rows, hidden, sum, q, s, ld_s, stream);
}

int dg_residual_norm_int8(const void* x, const void* residual, int dtype, int residual_dtype, const float* weight,
                          const void* gate, int64_t gate_rows, int post_norm, const float* post_weight, float scale,
                          float eps, int64_t rows, int64_t hidden, void* sum, int8_t* q, float* s, dg_stream_t stream) {
  return residual_norm("residual_norm_int8", 2, x, residual, dtype, residual_dtype, weight, gate, gate_rows, post_norm,
                       post_weight, scale, eps, rows, hidden, sum, q, s, 0, stream);
}

size_t dg_residual_norm_grad_workspace_size(int64_t rows, int64_t hidden) {
  if (rows <= 0 || hidden <= 0 || hidden % kKAlign || rows > kInt31 || hidden > kInt31) return 0;
  return residual_norm_grad_workspace_size(rows, hidden);
}

int dg_residual_norm_grad(const void* dy, const void* dsum, const void* x, const void* sum, int dtype, int residual_dtype,
                          const float* weight, const void* gate, int64_t gate_rows, int post_norm,
                          const float* post_weight, float scale, float eps, int64_t rows, int64_t hidden, void* dx,
                          void* dresidual, float* dweight, void* dgate, float* dpost_weight, void* workspace,
                          size_t workspace_bytes, dg_stream_t stream) {
  const char* what = "residual_norm_grad";
  const int c = check_norm(what, dtype, residual_dtype, x, weight, gate, gate_rows, post_norm, post_weight, eps, rows, hidden);
  if (c != DG_OK) return c;
  DG_REQUIRE(rows == 0 || (dy && sum && dresidual && (x == nullptr) == (dx == nullptr)), "%s: null pointer", what);
  DG_REQUIRE(weight || !dweight, "%s: dweight without a weight", what);
  DG_REQUIRE(gate || !dgate, "%s: dgate without a gate", what);
  DG_REQUIRE(post_weight || !dpost_weight, "%s: dpost_weight without a post_weight", what);
  DG_REQUIRE(aligned16(dy) && aligned16(dsum) && aligned16(sum) && aligned16(dx) && aligned16(dresidual) &&
                 aligned16(dweight) && aligned16(dgate) && aligned16(dpost_weight) && aligned16(workspace),
             "%s: pointers must be 16-byte aligned", what);
  const size_t need = dweight || dgate || dpost_weight ? dg_residual_norm_grad_workspace_size(rows, hidden) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return set_error(kWorkspace, "%s: workspace of %zu bytes, %zu needed", what, workspace ? workspace_bytes : (size_t)0, need);
  return launch_residual_norm_grad(dy, dsum, x, sum, dtype, residual_dtype, weight, gate, gate_rows, post_norm != 0,
                                   post_weight, scale, eps, rows, hidden, dx, dresidual, dweight, dgate, dpost_weight,
                                   workspace, static_cast<hipStream_t>(stream));
}

int dg_get_debug_status(uint32_t* flags, int64_t* block, int clear) {
  DG_REQUIRE(flags != nullptr, "dg_get_debug_status: flags is null");
  unsigned w[4] = {0u, 0u, 0u, 0u};
  const int r = read_diag(w, clear != 0);
  if (r != kOk) return r;
  *flags = w[0];
  if (block) *block = (int64_t)w[1] - 1;
  return DG_OK;
}

const char* dg_gemm_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t num_groups) {
  static thread_local char buf[96];
  buf[0] = 0;
  if (layout < 0 || layout > 3 || m <= 0 || n <= 0 || k <= 0 || k % kKAlign || num_groups <= 0) return buf;
  const int cus = effective_cus();
  if (cus < 0) return buf;
  gemm_config_name(layout, m, n, k, num_groups, cus, buf, sizeof(buf));
  return buf;
}

const char* dg_gemm_int8_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t num_groups) {
  static thread_local char buf[96];
  buf[0] = 0;
  if (layout < 0 || layout > 2 || m <= 0 || m > kInt31 - 1024 || n <= 0 || n > kInt31 - 1024 || k <= 0 || k % kKAlign ||
      k > kInt8MaxK || num_groups <= 0 || num_groups > kInt31 || (layout == 2 && num_groups > 1024))
    return buf;
  const int cus = effective_cus();
  if (cus < 0) return buf;
  gemm_int8_config_name(layout, m, n, k, num_groups, cus, buf, sizeof(buf));
  return buf;
}

}  // extern "C"
