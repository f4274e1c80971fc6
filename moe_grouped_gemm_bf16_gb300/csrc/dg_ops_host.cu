// Entry points of the operators around the FP8 GEMMs (include/dg.h): the
// root-mean-square norm, the gated activation with its 8-bit checkpoint and the
// ragged bf16 products.  Validation on the host, then one launch (the norm's
// gradient of many rows: two); errors as in dg_host.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "dg.h"
#include "dg_bf16.h"
#include "dg_host.h"
#include "dg_norm.h"
#include "dg_swiglu.h"

namespace {

using dgk::host_fail;
using dgk::host_ok;

dg_status cuda_fail(cudaError_t e, const char* what) {
  return host_fail(DG_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// dg_debug_force_ragged_plan: pair, lanes, rows, split packed; 0: the heuristic.
std::atomic<unsigned long long> g_ragged_plan{0};

// Opts an operator's kernels into their shared memory, once per device.
template <cudaError_t (*SET_UP)()>
dg_status set_up_once(int device) {
  static std::atomic<bool> done[dgk::kHostMaxDevices];
  if (done[device].load(std::memory_order_acquire)) return DG_OK;
  const cudaError_t e = SET_UP();
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(max dynamic shared memory)");
  done[device].store(true, std::memory_order_release);
  return DG_OK;
}

dg_status rms_norm(const dgk::NormFwd& a0, void* stream, bool ue8m0) {
  dgk::NormFwd a = a0;
  const char* name = "dg_rms_norm_quantize_fp8_1x128";
  if (!a.X || !a.W || (!a.Y && !a.Q) || (a.Q && !a.sa))
    return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer (X, W, one of Y and Q, sa with Q)", name);
  if (a.H && !a.R) return host_fail(DG_ERR_INVALID_ARG, "%s: H without a residual R", name);
  if (a.M < 0 || (a.Q && a.ld_sa < a.M) || !(a.eps >= 0.f))
    return host_fail(DG_ERR_INVALID_ARG, "%s: M=%d ld_sa=%d eps=%g", name, a.M, a.ld_sa, a.eps);
  if (a.K < 128 || a.K % 128 != 0 || a.K > dgk::kNormMaxK)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: K=%d (a multiple of 128 in [128, %d])", name, a.K,
                dgk::kNormMaxK);
  if ((a.Q && a.ld_sa % 4 != 0) || !aligned16(a.X) || !aligned16(a.R) || !aligned16(a.W) ||
      !aligned16(a.H) || !aligned16(a.Y) || !aligned16(a.Q) || !aligned16(a.sa) ||
      !aligned(a.rstd, 4))
    return host_fail(DG_ERR_MISALIGNED,
                "%s: ld_sa a multiple of 4; rstd 4-byte, the other tensors 16-byte aligned", name);
  if (a.M == 0) return host_ok();
  dgk::HostState st;
  dg_status s = dgk::host_state(&st);
  if (s == DG_OK) s = set_up_once<dgk::norm_set_up>(st.device);
  if (s != DG_OK) return s;
  a.status = st.status;
  a.timeout_ns = st.timeout_ns;
  a.debug_flags = st.debug_flags;
  const cudaError_t e =
      dgk::launch_rms_norm(a, ue8m0, st.sms, st.sms < st.device_sms, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "norm launch") : host_ok();
}

dg_status swiglu(const dgk::SwigluFwd& a0, void* stream, bool ue8m0) {
  const char* name = "dg_swiglu_quantize_fp8_1x128";
  dgk::SwigluFwd a = a0;
  if (!a.GU || (!a.Y && !a.Q && !a.CQ) || (a.Q && !a.sa) || (!a.CQ != !a.csa))
    return host_fail(DG_ERR_INVALID_ARG,
                "%s: null pointer (GU, one of Y, Q and CQ, sa with Q, csa with CQ)", name);
  const bool scales = a.Q || a.CQ;
  if (a.G < 1 || a.M < 0 || (scales && a.ld < a.M))
    return host_fail(DG_ERR_INVALID_ARG, "%s: G=%d M=%d ld_sa=%d", name, a.G, a.M, a.ld);
  if (a.I < 128 || a.I % 128 != 0 || a.I / 128 > 32767 || a.G > 65535)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE,
                "%s: I=%d (a positive multiple of 128, I/128 <= 32767), num_groups=%d (<= 65535)",
                name, a.I, a.G);
  if ((scales && a.ld % 4 != 0) || !aligned16(a.GU) || !aligned16(a.Y) || !aligned16(a.Q) ||
      !aligned16(a.sa) || !aligned16(a.CQ) || !aligned16(a.csa) || !aligned(a.masked_m, 4))
    return host_fail(DG_ERR_MISALIGNED,
                "%s: ld_sa a multiple of 4; masked_m 4-byte, the other tensors 16-byte aligned",
                name);
  if (a.M == 0) return host_ok();
  dgk::HostState st;
  dg_status s = dgk::host_state(&st);
  if (s == DG_OK) s = set_up_once<dgk::swiglu_set_up>(st.device);
  if (s != DG_OK) return s;
  a.status = st.status;
  a.timeout_ns = st.timeout_ns;
  a.debug_flags = st.debug_flags;
  const cudaError_t e = dgk::launch_swiglu(a, ue8m0, st.sms, st.sms < st.device_sms,
                                           static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "swiglu launch") : host_ok();
}

// Shared path of the ragged bf16 products.  rows: rows of A over all groups
// (M_total; tn: K_total).  M: tn only.
dg_status bf16_ragged(dgk::BfForm form, const void* A, const void* B, const void* C, void* D,
                      const int32_t* sizes, int rows, int M, int N, int K, int G, void* stream) {
  const bool tn = form == dgk::kBfTN;
  if (rows < 0 || N < 0 || K < 0 || M < 0)
    return host_fail(DG_ERR_INVALID_ARG, "negative size (rows=%d, M=%d, N=%d, K=%d)", rows, M, N, K);
  if (G < 1 || G > dgk::kBfMaxGroups)
    return host_fail(DG_ERR_INVALID_ARG, "num_groups=%d outside [1, %d]", G, dgk::kBfMaxGroups);
  // rows of 16 bytes' multiples, for TMA
  if (N < 8 || N % 8 != 0 || (!tn && (K < 8 || K % 8 != 0)) || (tn && M % 8 != 0))
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "N=%d, %s=%d: need positive multiples of 8", N,
                tn ? "M" : "K", tn ? M : K);
  // (the kernels' 32-bit counters step past these extents by less than 8192)
  constexpr int kMostExtent = INT_MAX - 8192;
  if (std::max(std::max(rows, K), M) > kMostExtent || N >= (1 << 23) || (long long)N * K >= (1ll << 34) || (long long)N * M >= (1ll << 34) ||
      ((long long)rows / 16 + G) * (N / 64 + 1) >= (1ll << 31) ||
      (long long)G * (M / 16 + 1) * (N / 64 + 1) >= (1ll << 31) ||
      (long long)rows * std::max(std::max(N, K), M) >= (1ll << 38))
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "tensor too large");
  if (tn ? M == 0 : rows == 0) return host_ok();  // D is empty
  // (without rows, tn reads neither A nor B: D = C or 0)
  if (!D || !sizes || (rows > 0 && (!A || !B)))
    return host_fail(DG_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned16(A) || !aligned16(B) || !aligned16(C) || !aligned16(D) || !aligned(sizes, 4))
    return host_fail(DG_ERR_MISALIGNED, "A, B, C and D need 16-byte alignment, the sizes 4");
  dgk::HostState st;
  dg_status s = dgk::host_state(&st);
  if (s == DG_OK) s = set_up_once<dgk::bf16_set_up>(st.device);
  if (s != DG_OK) return s;
  dgk::BfCall c{};
  c.form = form;
  c.A = A ? A : D;
  c.B = B ? B : D;
  c.C = C;
  c.D = D;
  c.sizes = sizes;
  c.G = G;
  c.rows = rows;
  c.M = M;
  c.N = N;
  c.K = K;
  c.status = st.status;
  c.timeout_ns = st.timeout_ns;
  c.debug_flags = st.debug_flags;
  c.limited = st.sms < st.device_sms;
  if (const unsigned long long f = g_ragged_plan.load()) {
    c.forced = {(f >> 48) != 0, static_cast<int>(f >> 32 & 0xFFFF), static_cast<int>(f >> 16 & 0xFFFF),
                static_cast<int>(f & 0xFFFF)};
    // boxes of an MN-major operand are 64 wide (nn, tn: B's; tn: A's)
    if ((!c.forced.pair && ((form != dgk::kBfNT && c.forced.lanes % 64) || (tn && c.forced.bc % 64))) ||
        c.forced.split * (c.forced.pair ? 2 : 1) > st.sms ||
        (c.limited && dgk::bf16_grid(c, c.forced, st.sms) > st.sms))
      return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "no kernel for the forced plan");
  }
  // (few rows: a grid of many small blocks, not under a limit on the SMs)
  const cudaError_t e =
      dgk::bf16_few_rows(c) && !c.limited
          ? dgk::launch_bf16_few(c, st.sms, static_cast<cudaStream_t>(stream))
          : dgk::launch_bf16_grouped(c, st.encode, st.sms, static_cast<cudaStream_t>(stream));
  if (e == cudaErrorInvalidValue) {
    cudaGetLastError();
    return host_fail(DG_ERR_CUDA, "ragged bf16 product: tensor map or launch rejected");
  }
  return e != cudaSuccess ? cuda_fail(e, "ragged bf16 product launch") : host_ok();
}
}  // namespace

extern "C" {

dg_status dg_rms_norm_quantize_fp8_1x128(const void* X, const void* R, const void* W, void* H,
                                         void* Y, void* Q, float* sa, float* rstd, int M, int K,
                                         int ld_sa, float eps, void* stream) {
  return rms_norm(dgk::NormFwd{X, R, W, H, Y, Q, sa, rstd, M, K, ld_sa, eps, nullptr, 0, 0}, stream,
                  false);
}

dg_status dg_rms_norm_quantize_fp8_1x128_ue8m0(const void* X, const void* R, const void* W, void* H,
                                               void* Y, void* Q, int32_t* sfa, float* rstd, int M,
                                               int K, int ld_sfa, float eps, void* stream) {
  return rms_norm(dgk::NormFwd{X, R, W, H, Y, Q, sfa, rstd, M, K, ld_sfa, eps, nullptr, 0, 0}, stream,
                  true);
}

long long dg_rms_norm_backward_workspace_bytes(int M, int K) {
  if (M < 0 || K < 0) return -1;
  return (long long)std::min(M, dgk::kNormBwdBlocks) * K * 4;
}

dg_status dg_rms_norm_backward(const void* dY, const void* H, const float* rstd, const void* W,
                               const void* dR, void* dX, float* dW, void* workspace,
                               long long workspace_bytes, int M, int K, void* stream) {
  const char* name = "dg_rms_norm_backward";
  if (M < 0) return host_fail(DG_ERR_INVALID_ARG, "%s: M=%d", name, M);
  if (!dW || (M > 0 && (!dY || !H || !rstd || !W || !dX || !workspace)))
    return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer", name);
  if (K < 128 || K % 128 != 0 || K > dgk::kNormMaxK)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: K=%d (a multiple of 128 in [128, %d])", name, K,
                dgk::kNormMaxK);
  if (workspace_bytes < dg_rms_norm_backward_workspace_bytes(M, K))
    return host_fail(DG_ERR_INVALID_ARG, "%s: %lld bytes of workspace, %lld needed", name,
                workspace_bytes, dg_rms_norm_backward_workspace_bytes(M, K));
  if (!aligned16(dY) || !aligned16(H) || !aligned16(W) || !aligned16(dR) || !aligned16(dX) ||
      !aligned16(dW) || !aligned16(workspace) || !aligned(rstd, 4))
    return host_fail(DG_ERR_MISALIGNED, "%s: rstd 4-byte, the other tensors 16-byte aligned", name);
  dgk::HostState st;
  dg_status s = dgk::host_state(&st);
  if (s == DG_OK) s = set_up_once<dgk::norm_set_up>(st.device);
  if (s != DG_OK) return s;
  const cudaError_t e = dgk::launch_rms_norm_backward(
      dgk::NormBwd{dY, H, rstd, W, dR, dX, dW, static_cast<float*>(workspace), M, K, st.status,
                   st.timeout_ns, st.debug_flags},
      st.sms, st.sms < st.device_sms, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "norm gradient launch") : host_ok();
}

dg_status dg_swiglu_quantize_fp8_1x128(const void* GU, void* Y, void* Q, float* sa, void* CQ,
                                       float* csa, const int32_t* masked_m, int num_groups, int M,
                                       int I, int ld_sa, void* stream) {
  return swiglu(dgk::SwigluFwd{GU, Y, Q, sa, CQ, csa, masked_m, num_groups, M, I, ld_sa, nullptr, 0, 0},
                stream, false);
}

dg_status dg_swiglu_quantize_fp8_1x128_ue8m0(const void* GU, void* Y, void* Q, int32_t* sfa,
                                             void* CQ, float* csa, const int32_t* masked_m,
                                             int num_groups, int M, int I, int ld_sfa,
                                             void* stream) {
  return swiglu(dgk::SwigluFwd{GU, Y, Q, sfa, CQ, csa, masked_m, num_groups, M, I, ld_sfa, nullptr, 0, 0},
                stream, true);
}

dg_status dg_swiglu_backward_fp8_1x128(const void* CQ, const float* csa, const void* dY, void* dGU,
                                       void* Y, const int32_t* masked_m, int num_groups, int M,
                                       int I, int ld_csa, void* stream) {
  const char* name = "dg_swiglu_backward_fp8_1x128";
  if (!CQ || !csa || !dY || !dGU) return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer", name);
  if (num_groups < 1 || M < 0 || ld_csa < M)
    return host_fail(DG_ERR_INVALID_ARG, "%s: G=%d M=%d ld_csa=%d", name, num_groups, M, ld_csa);
  if (I < 128 || I % 128 != 0 || I / 128 > 32767 || num_groups > 65535)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE,
                "%s: I=%d (a positive multiple of 128, I/128 <= 32767), num_groups=%d (<= 65535)",
                name, I, num_groups);
  if (ld_csa % 4 != 0 || !aligned16(CQ) || !aligned16(csa) || !aligned16(dY) || !aligned16(dGU) ||
      !aligned16(Y) || !aligned(masked_m, 4))
    return host_fail(DG_ERR_MISALIGNED,
                "%s: ld_csa a multiple of 4; masked_m 4-byte, the other tensors 16-byte aligned",
                name);
  if (M == 0) return host_ok();
  dgk::HostState st;
  const dg_status s = dgk::host_state(&st);
  if (s != DG_OK) return s;
  const cudaError_t e = dgk::launch_swiglu_backward(
      dgk::SwigluBwd{CQ, csa, dY, dGU, Y, masked_m, num_groups, M, I, ld_csa, st.status},
      st.sms, st.sms < st.device_sms, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "swiglu gradient launch") : host_ok();
}

dg_status dg_m_grouped_gemm_bf16_nt_ragged(const void* A, const void* B, void* D, const int32_t* ms,
                                           int M_total, int N, int K, int num_groups,
                                           void* stream) {
  return bf16_ragged(dgk::kBfNT, A, B, nullptr, D, ms, M_total, 0, N, K, num_groups, stream);
}

dg_status dg_m_grouped_gemm_bf16_nn_ragged(const void* A, const void* B, void* D, const int32_t* ms,
                                           int M_total, int N, int K, int num_groups,
                                           void* stream) {
  return bf16_ragged(dgk::kBfNN, A, B, nullptr, D, ms, M_total, 0, N, K, num_groups, stream);
}

dg_status dg_k_grouped_gemm_bf16_tn_ragged(const void* A, const void* B, const void* C, void* D,
                                           const int32_t* ks, int num_groups, int M, int N,
                                           int K_total, void* stream) {
  return bf16_ragged(dgk::kBfTN, A, B, C, D, ks, K_total, M, N, 0, num_groups, stream);
}

dg_status dg_debug_force_ragged_plan(int pair, int lanes, int rows, int split) {
  if (lanes == 0) {
    g_ragged_plan.store(0);
    return host_ok();
  }
  const bool ok = pair ? lanes == 256 && rows == 256 && (split == 1 || split == 2 || split == 4)
                       : lanes >= 64 && lanes <= 256 && lanes % 16 == 0 && rows >= 16 && rows <= 128 &&
                             rows % 16 == 0 && split >= 1 && split <= 8;
  if (!ok)
    return host_fail(DG_ERR_INVALID_ARG, "ragged plan pair=%d lanes=%d rows=%d split=%d", pair, lanes,
                     rows, split);
  g_ragged_plan.store(static_cast<unsigned long long>(pair ? 1 : 0) << 48 |
                      static_cast<unsigned long long>(lanes) << 32 |
                      static_cast<unsigned long long>(rows) << 16 | static_cast<unsigned>(split));
  return host_ok();
}

}  // extern "C"
