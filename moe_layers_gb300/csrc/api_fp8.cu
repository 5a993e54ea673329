// C ABI of the operators on 8-bit numbers: argument checks, workspaces, launches.
#include <cmath>

#include "internal.h"

using namespace dec;

namespace {

constexpr int kMaxRows = 1 << 20;
constexpr int kMaxWidth = 65536;
constexpr int64_t kMaxStride = (int64_t)1 << 31;
constexpr int kMaxExpertRows = 64;
constexpr int kMaxChoices = 16;
constexpr int kMaxExperts = 1024;
constexpr int kMaxExpertWidth = 16384;  // 8 rows and their sums fit in shared memory

inline bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline dec_status status(cudaError_t e) { return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA; }
inline int blocks_of(int n) { return (n + 127) / 128; }

bool rows_ok(const dec_fp8_rows* r, int K) {
  return r != nullptr && r->q != nullptr && r->scales != nullptr && al(r->q, 16) && al(r->scales, 4) && r->ldq >= K &&
         r->ldq % 16 == 0 && r->ldq <= kMaxStride && r->lds >= blocks_of(K) && r->lds <= kMaxStride;
}

bool weight_ok(const dec_fp8_weight& w) { return w.q != nullptr && w.scales != nullptr && al(w.q, 16) && al(w.scales, 4); }

bool bf16_rows_ok(const void* p, int64_t ld, int width) {
  return al(p, 16) && ld >= width && ld % 8 == 0 && ld <= kMaxStride;
}

bool linear_shape_ok(int M, int N, int K) {
  return M >= 1 && M <= kMaxRows && N >= 1 && N <= kMaxRows && K >= 16 && K <= kMaxWidth && K % 16 == 0;
}

// The streaming kernel up to 8 rows, and up to 16 with weights of at most 64 MB, where the tcgen05 kernel's
// ramp counts (16 rows, streaming / tcgen05: 4096 x 4096 8.5 / 9.1 us, 7168 x 8192 18.4 / 18.4, 12288 x 7168
// 25.2 / 21.2; 8 rows: 7.0 / 9.0, 13.3 / 18.4, 18.2 / 21.2); as forced where its shared memory holds the rows.
bool linear_streams(const dec_handle* h, int M, int N, int K) {
  if (h->force_variant == DEC_VARIANT_SPLIT_K || M > stream8_rows(K, false)) return false;
  return h->force_variant == DEC_VARIANT_SMALL_M || M <= 8 || (int64_t)N * K <= (int64_t)64 << 20;
}

bool experts_shape_ok(const dec_moe_fp8_weights* W, int M, int k) {
  return W != nullptr && M >= 1 && M <= kMaxExpertRows && k >= 1 && k <= kMaxChoices && W->E >= 1 &&
         W->E <= kMaxExperts && W->H >= 128 && W->H % 128 == 0 && W->H <= kMaxWidth && W->I >= 128 && W->I % 128 == 0 &&
         W->I <= kMaxWidth;
}

bool experts_width_ok(const dec_moe_fp8_weights* W) { return W->H <= kMaxExpertWidth && W->I <= kMaxExpertWidth; }

bool has_shared(const dec_moe_fp8_weights* W) { return W->gate_s.q != nullptr; }

// Workspace of the experts: the table, the experts' inner rows and their outputs.
struct ExpertsWs {
  size_t inner, y, bytes;
  ExpertsWs(const Experts8Plan& p, int H, int I) {
    auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
    inner = up((size_t)p.words * 4);
    y = inner + up((size_t)p.slots * I * 4);
    bytes = y + up((size_t)p.slots * H * 4);
  }
};

Stream8Bank bank(const dec_fp8_weight& a, const dec_fp8_weight& b) { return {{a.q, b.q}, {a.scales, b.scales}}; }

}  // namespace

extern "C" {

dec_status dec_rmsnorm_quant(dec_handle* h, const dec_bf16* x, int64_t ldx, const dec_bf16* residual, int64_t ldr,
                             const dec_bf16* gamma, float eps, dec_bf16* sum, int64_t lds, dec_bf16* y, int64_t ldy,
                             const dec_fp8_rows* out, int M, int H, cudaStream_t stream) {
  if (h == nullptr || x == nullptr || M < 1 || M > kMaxRows || H < 16 || H > kMaxWidth || H % 16 != 0)
    return DEC_ERR_INVALID_ARG;
  if (!rows_ok(out, H) || !bf16_rows_ok(x, ldx, H)) return DEC_ERR_INVALID_ARG;
  if (residual != nullptr && !bf16_rows_ok(residual, ldr, H)) return DEC_ERR_INVALID_ARG;
  if (sum != nullptr && (residual == nullptr || !bf16_rows_ok(sum, lds, H))) return DEC_ERR_INVALID_ARG;
  if (y != nullptr && (!bf16_rows_ok(y, ldy, H) || y == sum)) return DEC_ERR_INVALID_ARG;
  if (sum != nullptr && ((sum == x && lds != ldx) || (sum == residual && lds != ldr))) return DEC_ERR_INVALID_ARG;
  if (y != nullptr && ((y == x && ldy != ldx) || (y == residual && ldy != ldr))) return DEC_ERR_INVALID_ARG;
  if (gamma != nullptr && (!al(gamma, 16) || !(eps >= 0.f) || !std::isfinite(eps))) return DEC_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return DEC_ERR_CUDA;
  QuantRows P = {x, ldx, residual, ldr, gamma, eps, sum, lds, y, ldy, out->q, out->ldq, out->scales, out->lds, H};
  LaunchScope scope(h, "rmsnorm_quant", stream);
  return status(launch_norm_quant(h, P, M, stream));
}

dec_status dec_quant_weight(dec_handle* h, const dec_bf16* W, int64_t N, int K, dec_e4m3* q, float* scales,
                            cudaStream_t stream) {
  if (h == nullptr || W == nullptr || q == nullptr || scales == nullptr || !al(W, 16) || !al(q, 16) || !al(scales, 4))
    return DEC_ERR_INVALID_ARG;
  if (N < 1 || N > (int64_t)1 << 32 || K < 16 || K > kMaxWidth || K % 16 != 0) return DEC_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return DEC_ERR_CUDA;
  LaunchScope scope(h, "quant_weight", stream);
  return status(launch_weight_quant(h, W, N, K, q, scales, stream));
}

dec_status dec_linear_fp8_workspace_size(const dec_handle* h, int M, int N, int K, size_t* bytes) {
  if (h == nullptr || bytes == nullptr || !linear_shape_ok(M, N, K)) return DEC_ERR_INVALID_ARG;
  *bytes = linear_streams(h, M, N, K) ? 0 : gemm8_ws_bytes(h, M, N, K);
  return DEC_OK;
}

dec_status dec_linear_fp8(dec_handle* h, const dec_fp8_rows* x, const dec_fp8_weight* W, const dec_bf16* residual,
                          int64_t ldr, dec_bf16* y, int64_t ldy, int M, int N, int K, void* ws, size_t ws_bytes,
                          cudaStream_t stream) {
  if (h == nullptr || W == nullptr || y == nullptr || !linear_shape_ok(M, N, K)) return DEC_ERR_INVALID_ARG;
  if (!rows_ok(x, K) || !weight_ok(*W) || !al(y, 2) || ldy < N || ldy > kMaxStride) return DEC_ERR_INVALID_ARG;
  if (residual != nullptr && (!al(residual, 2) || ldr < N || ldr > kMaxStride || (residual == y && ldr != ldy)))
    return DEC_ERR_INVALID_ARG;
  const bool stream8 = linear_streams(h, M, N, K);
  const size_t need = stream8 ? 0 : gemm8_ws_bytes(h, M, N, K);
  if (need > 0 && (ws == nullptr || !al(ws, 16) || ws_bytes < need)) return DEC_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return DEC_ERR_CUDA;
  const Linear8 L = {x->q, x->ldq, x->scales, x->lds, W->q, W->scales, residual, ldr, y, ldy, M, N, K};
  h->last_variant = stream8 ? DEC_VARIANT_SMALL_M : DEC_VARIANT_SPLIT_K;
  LaunchScope scope(h, "linear_fp8", stream);
  return status(stream8 ? launch_stream8_linear(h, L, stream) : launch_gemm8(h, L, ws, stream));
}

dec_status moe_experts_fp8_workspace_size(const dec_handle* h, const dec_moe_fp8_weights* Wt, int M, int k,
                                          size_t* bytes) {
  if (h == nullptr || bytes == nullptr || !experts_shape_ok(Wt, M, k)) return DEC_ERR_INVALID_ARG;
  if (!experts_width_ok(Wt)) return DEC_ERR_UNSUPPORTED;
  const Experts8Plan p = experts8_plan(M, k, Wt->E, Wt->H, Wt->I, has_shared(Wt));
  *bytes = ExpertsWs(p, Wt->H, Wt->I).bytes;
  return DEC_OK;
}

dec_status moe_experts_fp8(dec_handle* h, const dec_fp8_rows* x, const int32_t* idx, const float* w, int M, int k,
                           const dec_moe_fp8_weights* Wt, const dec_bf16* residual, dec_bf16* out, void* ws,
                           size_t ws_bytes, cudaStream_t stream) {
  if (h == nullptr || idx == nullptr || w == nullptr || out == nullptr || !experts_shape_ok(Wt, M, k))
    return DEC_ERR_INVALID_ARG;
  if (!rows_ok(x, Wt->H) || !weight_ok(Wt->gate) || !weight_ok(Wt->up) || !weight_ok(Wt->down))
    return DEC_ERR_INVALID_ARG;
  if (has_shared(Wt) || Wt->up_s.q || Wt->down_s.q || Wt->gate_s.scales || Wt->up_s.scales || Wt->down_s.scales)
    if (!weight_ok(Wt->gate_s) || !weight_ok(Wt->up_s) || !weight_ok(Wt->down_s)) return DEC_ERR_INVALID_ARG;
  if (!al(idx, 4) || !al(w, 4) || !al(out, 16) || !al(residual, 16) || !al(ws, 16)) return DEC_ERR_INVALID_ARG;
  if (!experts_width_ok(Wt)) return DEC_ERR_UNSUPPORTED;
  const Experts8Plan p = experts8_plan(M, k, Wt->E, Wt->H, Wt->I, has_shared(Wt));
  const ExpertsWs at(p, Wt->H, Wt->I);
  if (ws == nullptr || ws_bytes < at.bytes) return DEC_ERR_INVALID_ARG;
  DeviceGuard dev(h->device);
  if (!dev.ok) return DEC_ERR_CUDA;
  Experts8 X = {x->q, x->ldq, x->scales, x->lds, idx, w, M, k, Wt->E, Wt->H, Wt->I, bank(Wt->gate, Wt->up),
                bank(Wt->down, Wt->down), bank(Wt->gate_s, Wt->up_s), bank(Wt->down_s, Wt->down_s), residual, out};
  uint8_t* b = static_cast<uint8_t*>(ws);
  return status(launch_experts8(h, X, p, reinterpret_cast<int*>(b), reinterpret_cast<float*>(b + at.inner),
                                reinterpret_cast<float*>(b + at.y), stream));
}

}  // extern "C"
