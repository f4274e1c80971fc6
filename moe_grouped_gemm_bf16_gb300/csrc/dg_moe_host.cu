// Entry points of the operators between the products of an expert layer, and of
// the loss (include/dg.h): routing, the experts' rows, dispatch, combine, softmax
// cross entropy.  Validation on the host, then one launch (the loss: two, or three
// per piece of the vocabulary); errors as in dg_host.cu.
#include <cuda_runtime.h>

#include <climits>

#include <algorithm>

#include "dg.h"
#include "dg_bf16.h"
#include "dg_loss.h"
#include "dg_ops_util.h"
#include "dg_route.h"
#include "dg_rows.h"

namespace {

using dgk::aligned;
using dgk::aligned16;
using dgk::cuda_fail;
using dgk::host_fail;
using dgk::host_ok;

constexpr long long kMostPairs = 1ll << 30;   // tokens x choices

// T tokens of top_k choices among num_experts experts.
dg_status check_choices(const char* name, int T, int top_k, int num_experts) {
  if (T < 0 || top_k < 1 || num_experts < 1)
    return host_fail(DG_ERR_INVALID_ARG, "%s: T=%d top_k=%d num_experts=%d", name, T, top_k, num_experts);
  if (top_k > dgk::kRouteMaxTopK || num_experts > dgk::kRouteMaxExperts ||
      static_cast<long long>(T) * top_k >= kMostPairs)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: T=%d top_k=%d (at most %d) num_experts=%d (at most %d)",
                     name, T, top_k, dgk::kRouteMaxTopK, num_experts, dgk::kRouteMaxExperts);
  return DG_OK;
}

dg_status route(dgk::RouteFwd a, bool bf16, void* stream) {
  const char* name = "dg_route_top_k";
  const dg_status bad = check_choices(name, a.T, a.k, a.G);
  if (bad != DG_OK) return bad;
  if (a.groups < 1 || a.top_groups < 1 || a.top_groups > a.groups || a.G % a.groups != 0 ||
      (a.best != 1 && a.best != 2) || a.k > a.G / a.groups * a.top_groups)
    return host_fail(DG_ERR_INVALID_ARG,
                     "%s: %d experts in %d groups, %d of them kept by their %d best, %d chosen", name, a.G,
                     a.groups, a.top_groups, a.best, a.k);
  if (a.groups > dgk::kRouteMaxGroups)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: num_groups=%d (at most %d)", name, a.groups,
                     dgk::kRouteMaxGroups);
  if (a.T == 0) return host_ok();
  if (!a.logits || !a.experts || !a.weights)
    return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(a.logits, bf16 ? 2 : 4) || !aligned(a.bias, 4) || !aligned(a.experts, 4) ||
      !aligned(a.weights, 4))
    return host_fail(DG_ERR_MISALIGNED, "%s: tensors aligned to their elements", name);
  dgk::HostState st;
  const dg_status s = dgk::host_state(&st);
  if (s != DG_OK) return s;
  a.status = st.status;
  const cudaError_t e =
      dgk::launch_route(a, bf16, st.sms, st.sms < st.device_sms, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "routing launch") : host_ok();
}

dg_status route_backward(dgk::RouteBwd a, bool bf16, void* stream) {
  const char* name = "dg_route_top_k_backward";
  const dg_status bad = check_choices(name, a.T, a.k, a.G);
  if (bad != DG_OK) return bad;
  if (a.T == 0) return host_ok();
  if (!a.logits || !a.experts || !a.d_weights || !a.d_logits)
    return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(a.logits, bf16 ? 2 : 4) || !aligned(a.d_logits, bf16 ? 2 : 4) || !aligned(a.experts, 4) ||
      !aligned(a.d_weights, 4))
    return host_fail(DG_ERR_MISALIGNED, "%s: tensors aligned to their elements", name);
  dgk::HostState st;
  const dg_status s = dgk::host_state(&st);
  if (s != DG_OK) return s;
  a.status = st.status;
  const cudaError_t e = dgk::launch_route_backward(a, bf16, st.sms, st.sms < st.device_sms,
                                                   static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "routing gradient launch") : host_ok();
}

// room: contiguous: M_total; masked: max_m.
dg_status expert_rows(dgk::RowsLayout layout, const int32_t* experts, int32_t* sizes, int32_t* rows,
                      int32_t* m_indices, int T, int top_k, int G, int room, void* stream) {
  const char* name = "dg_expert_rows";
  const dg_status bad = check_choices(name, T, top_k, G);
  if (bad != DG_OK) return bad;
  if (room < 0) return host_fail(DG_ERR_INVALID_ARG, "%s: %d rows", name, room);
  if (layout == dgk::kRowsContiguous && room % 128 != 0)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: M_total=%d (a multiple of 128)", name, room);
  if (layout == dgk::kRowsMasked && static_cast<long long>(G) * room > INT_MAX)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: %d experts of %d rows", name, G, room);
  // (without tokens the sizes are still written)
  if (!sizes || (T > 0 && (!experts || !rows)) ||
      (layout == dgk::kRowsContiguous && room > 0 && !m_indices))
    return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(experts, 4) || !aligned(sizes, 4) || !aligned(rows, 4) || !aligned(m_indices, 4))
    return host_fail(DG_ERR_MISALIGNED, "%s: tensors aligned to 4 bytes", name);
  dgk::HostState st;
  dg_status s = dgk::host_state(&st);
  if (s == DG_OK) s = dgk::set_up_once<dgk::rows_set_up>(st.device);
  if (s != DG_OK) return s;
  const cudaError_t e = dgk::launch_rows(
      dgk::RowsCall{experts, sizes, rows, m_indices, T * top_k, G, room, st.status}, layout, st.sms,
      static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "expert rows launch") : host_ok();
}

dg_status dispatch(const char* name, dgk::DispatchCall a, void* stream) {
  if (a.T == 0) return host_ok();
  if (!a.X || !a.rows || (a.num_rows > 0 && !a.D)) return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned16(a.X) || !aligned16(a.D) || !aligned16(a.sa) || !aligned16(a.sa_out) || !aligned(a.rows, 4))
    return host_fail(DG_ERR_MISALIGNED, "%s: rows 4-byte, the other tensors 16-byte aligned", name);
  dgk::HostState st;
  const dg_status s = dgk::host_state(&st);
  if (s != DG_OK) return s;
  a.status = st.status;
  const cudaError_t e =
      dgk::launch_dispatch(a, st.sms, st.sms < st.device_sms, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "dispatch launch") : host_ok();
}

// kb: words of scales per row.
dg_status dispatch_fp8(const char* name, const void* Q, const void* sa, int ld_sa, const int32_t* rows,
                       void* A, void* sa_out, int ld_out, int T, int K, int top_k, int G, int max_m,
                       int kb, void* stream) {
  const dg_status bad = check_choices(name, T, top_k, 1);
  if (bad != DG_OK) return bad;
  if (G < 1 || max_m < 0 || ld_sa < T || ld_out < max_m)
    return host_fail(DG_ERR_INVALID_ARG, "%s: T=%d ld_sa=%d num_groups=%d max_m=%d ld_out=%d", name, T,
                     ld_sa, G, max_m, ld_out);
  if (K < 128 || K % 128 != 0 || static_cast<long long>(G) * max_m > INT_MAX)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE,
                     "%s: K=%d (a positive multiple of 128), %d groups of %d rows", name, K, G, max_m);
  if (ld_sa % 4 != 0 || ld_out % 4 != 0)
    return host_fail(DG_ERR_MISALIGNED, "%s: ld_sa=%d, ld_out=%d (multiples of 4)", name, ld_sa, ld_out);
  if (T > 0 && (!sa || !sa_out)) return host_fail(DG_ERR_INVALID_ARG, "%s: null scales", name);
  return dispatch(name,
                  dgk::DispatchCall{Q, rows, A, T, top_k, K / 16, G * max_m,
                                    static_cast<const uint32_t*>(sa), static_cast<uint32_t*>(sa_out), kb,
                                    ld_sa, ld_out, max_m > 0 ? max_m : 1, nullptr},
                  stream);
}

// What combine and its gradient ask of their sizes.
dg_status check_rows(const char* name, int T, int K, int top_k, int num_rows) {
  const dg_status bad = check_choices(name, T, top_k, 1);
  if (bad != DG_OK) return bad;
  if (num_rows < 0) return host_fail(DG_ERR_INVALID_ARG, "%s: num_rows=%d", name, num_rows);
  if (K < 8 || K % 8 != 0)
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: K=%d (a positive multiple of 8)", name, K);
  return DG_OK;
}

// T tokens, V words, K columns: the limits of the bf16 products' kernel.
dg_status check_vocabulary(const char* name, int T, int V, int K) {
  if (T < 0 || V < 1 || K < 1) return host_fail(DG_ERR_INVALID_ARG, "%s: T=%d V=%d K=%d", name, T, V, K);
  if (K % 8 != 0) return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: K=%d (a multiple of 8)", name, K);
  const long long t = T, v = V, k = K;
  // (V: the tiles' decoding divides numbers of lane blocks in fp32)
  if (v >= (1 << 29) || T >= (1 << 23) || K >= (1 << 23) || v * k >= (1ll << 34) || t * k >= (1ll << 34) ||
      t * v >= (1ll << 38) || (v / 16 + 1) * (t / 64 + 1) >= (1ll << 31))
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "%s: T=%d V=%d K=%d: too large", name, T, V, K);
  return DG_OK;
}

dg_status check_workspace(const char* name, const void* workspace, long long bytes, long long need) {
  if (!workspace || bytes < need)
    return host_fail(DG_ERR_INVALID_ARG, "%s: %lld bytes of workspace, %lld needed", name,
                     workspace ? bytes : 0ll, need);
  return DG_OK;
}

dg_status loss_state(dgk::LossCall* a, int* sms) {
  dgk::HostState st;
  dg_status s = dgk::host_state(&st);
  if (s == DG_OK) s = dgk::set_up_once<dgk::loss_set_up>(st.device);
  if (s != DG_OK) return s;
  a->status = st.status;
  a->timeout_ns = st.timeout_ns;
  a->debug_flags = st.debug_flags;
  a->limited = st.sms < st.device_sms;
  a->encode = st.encode;
  a->forced = dgk::bf16_forced_plan();
  // (dW reads 64-wide boxes along the columns; words on the lanes are taken 32 at a time)
  if (a->forced.lanes > 0 && !a->forced.pair &&
      (a->forced.lanes % (dgk::loss_words_on_lanes(a->T) ? 32 : 64) != 0 || a->forced.bc % 64 != 0))
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "cross entropy: no kernel for the forced plan");
  if (a->forced.split * (a->forced.pair ? 2 : 1) > st.sms || (a->limited && a->forced.split > 1))
    return host_fail(DG_ERR_UNSUPPORTED_SHAPE, "cross entropy: forced plan past the limit on the SMs");
  *sms = st.sms;
  return DG_OK;
}

dg_status loss_result(cudaError_t e) {
  if (e == cudaErrorInvalidValue) {
    cudaGetLastError();
    return host_fail(DG_ERR_CUDA, "cross entropy: tensor map or launch rejected");
  }
  return e != cudaSuccess ? cuda_fail(e, "cross entropy launch") : host_ok();
}

}  // namespace

extern "C" {

dg_status dg_route_top_k_fp32(const float* logits, const float* bias, int32_t* experts, float* weights,
                              int T, int num_experts, int top_k, int sigmoid, int num_groups,
                              int top_groups, int group_best, int renormalize, float scale,
                              void* stream) {
  return route(dgk::RouteFwd{logits, bias, experts, weights, T, num_experts, top_k, sigmoid != 0,
                             num_groups, top_groups, group_best, renormalize != 0, scale, nullptr},
               false, stream);
}

dg_status dg_route_top_k_bf16(const void* logits, const float* bias, int32_t* experts, float* weights,
                              int T, int num_experts, int top_k, int sigmoid, int num_groups,
                              int top_groups, int group_best, int renormalize, float scale,
                              void* stream) {
  return route(dgk::RouteFwd{logits, bias, experts, weights, T, num_experts, top_k, sigmoid != 0,
                             num_groups, top_groups, group_best, renormalize != 0, scale, nullptr},
               true, stream);
}

dg_status dg_route_top_k_backward_fp32(const float* logits, const int32_t* experts,
                                       const float* d_weights, float* d_logits, int T,
                                       int num_experts, int top_k, int sigmoid, int renormalize,
                                       float scale, void* stream) {
  return route_backward(dgk::RouteBwd{logits, experts, d_weights, d_logits, T, num_experts, top_k,
                                      sigmoid != 0, renormalize != 0, scale, nullptr},
                        false, stream);
}

dg_status dg_route_top_k_backward_bf16(const void* logits, const int32_t* experts,
                                       const float* d_weights, void* d_logits, int T,
                                       int num_experts, int top_k, int sigmoid, int renormalize,
                                       float scale, void* stream) {
  return route_backward(dgk::RouteBwd{logits, experts, d_weights, d_logits, T, num_experts, top_k,
                                      sigmoid != 0, renormalize != 0, scale, nullptr},
                        true, stream);
}

dg_status dg_expert_rows_ragged(const int32_t* experts, int32_t* ms, int32_t* rows, int T, int top_k,
                                int num_groups, void* stream) {
  return expert_rows(dgk::kRowsRagged, experts, ms, rows, nullptr, T, top_k, num_groups, 0, stream);
}

dg_status dg_expert_rows_contiguous(const int32_t* experts, int32_t* ms, int32_t* rows,
                                    int32_t* m_indices, int T, int top_k, int num_groups, int M_total,
                                    void* stream) {
  return expert_rows(dgk::kRowsContiguous, experts, ms, rows, m_indices, T, top_k, num_groups, M_total,
                     stream);
}

dg_status dg_expert_rows_masked(const int32_t* experts, int32_t* masked_m, int32_t* rows, int T,
                                int top_k, int num_groups, int max_m, void* stream) {
  return expert_rows(dgk::kRowsMasked, experts, masked_m, rows, nullptr, T, top_k, num_groups, max_m,
                     stream);
}

dg_status dg_dispatch_rows_bf16(const void* X, const int32_t* rows, void* D, int T, int K, int top_k,
                                int num_rows, void* stream) {
  const char* name = "dg_dispatch_rows_bf16";
  const dg_status bad = check_rows(name, T, K, top_k, num_rows);
  if (bad != DG_OK) return bad;
  return dispatch(name,
                  dgk::DispatchCall{X, rows, D, T, top_k, K / 8, num_rows, nullptr, nullptr, 0, 0, 0, 1,
                                    nullptr},
                  stream);
}

dg_status dg_dispatch_rows_fp8_1x128(const void* Q, const float* sa, int ld_sa, const int32_t* rows,
                                     void* A, float* sa_out, int ld_out, int T, int K, int top_k,
                                     int num_groups, int max_m, void* stream) {
  return dispatch_fp8("dg_dispatch_rows_fp8_1x128", Q, sa, ld_sa, rows, A, sa_out, ld_out, T, K, top_k,
                      num_groups, max_m, K / 128, stream);
}

dg_status dg_dispatch_rows_fp8_1x128_ue8m0(const void* Q, const int32_t* sfa, int ld_sfa,
                                           const int32_t* rows, void* A, int32_t* sfa_out, int ld_out,
                                           int T, int K, int top_k, int num_groups, int max_m,
                                           void* stream) {
  return dispatch_fp8("dg_dispatch_rows_fp8_1x128_ue8m0", Q, sfa, ld_sfa, rows, A, sfa_out, ld_out, T, K,
                      top_k, num_groups, max_m, (K / 128 + 3) / 4, stream);
}

dg_status dg_combine_rows(const void* Y, const int32_t* rows, const float* weights, const void* R,
                          void* out, int T, int K, int top_k, int num_rows, void* stream) {
  const char* name = "dg_combine_rows";
  const dg_status bad = check_rows(name, T, K, top_k, num_rows);
  if (bad != DG_OK) return bad;
  if (T == 0) return host_ok();
  if (!rows || !out || (num_rows > 0 && !Y))
    return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned16(Y) || !aligned16(R) || !aligned16(out) || !aligned(rows, 4) || !aligned(weights, 4))
    return host_fail(DG_ERR_MISALIGNED, "%s: Y, R and out 16-byte, rows and weights 4-byte aligned", name);
  dgk::HostState st;
  const dg_status s = dgk::host_state(&st);
  if (s != DG_OK) return s;
  const cudaError_t e =
      dgk::launch_combine(dgk::CombineCall{Y, rows, weights, R, out, T, K, top_k, num_rows, st.status},
                          st.sms, st.sms < st.device_sms, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "combine launch") : host_ok();
}

dg_status dg_combine_rows_backward(const void* dO, const void* Y, const int32_t* rows,
                                   const float* weights, void* dY, float* d_weights, int T, int K,
                                   int top_k, int num_rows, void* stream) {
  const char* name = "dg_combine_rows_backward";
  const dg_status bad = check_rows(name, T, K, top_k, num_rows);
  if (bad != DG_OK) return bad;
  if (T == 0) return host_ok();
  if (!dO || !rows || (num_rows > 0 && (!dY || (d_weights && !Y))))
    return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer (dO, rows, dY, Y with d_weights)", name);
  if (!aligned16(dO) || !aligned16(Y) || !aligned16(dY) || !aligned(rows, 4) || !aligned(weights, 4) ||
      !aligned(d_weights, 4))
    return host_fail(DG_ERR_MISALIGNED,
                     "%s: dO, Y and dY 16-byte, rows and the weights 4-byte aligned", name);
  dgk::HostState st;
  const dg_status s = dgk::host_state(&st);
  if (s != DG_OK) return s;
  const cudaError_t e = dgk::launch_combine_backward(
      dgk::CombineBwd{dO, Y, rows, weights, dY, d_weights, T, K, top_k, num_rows, st.status}, st.sms,
      st.device_sms, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(e, "combine gradient launch") : host_ok();
}

long long dg_linear_cross_entropy_workspace_bytes(int T, int V, int K) {
  return T < 0 || V < 0 || K < 0 ? -1 : dgk::loss_workspace(T, V);
}

dg_status dg_linear_cross_entropy(const void* X, const void* W, const int32_t* targets, float* loss,
                                  float* lse, void* workspace, long long workspace_bytes, int T, int V,
                                  int K, void* stream) {
  const char* name = "dg_linear_cross_entropy";
  dg_status s = check_vocabulary(name, T, V, K);
  if (s != DG_OK) return s;
  if (T == 0) return host_ok();
  if (!X || !W || !targets || (!loss && !lse))
    return host_fail(DG_ERR_INVALID_ARG, "%s: null pointer (X, W, targets, one of loss and lse)", name);
  s = check_workspace(name, workspace, workspace_bytes, dgk::loss_workspace(T, V));
  if (s != DG_OK) return s;
  if (!aligned16(X) || !aligned16(W) || !aligned16(workspace) || !aligned(targets, 4) || !aligned(loss, 4) ||
      !aligned(lse, 4))
    return host_fail(DG_ERR_MISALIGNED, "%s: X, W and workspace 16-byte, the others 4-byte aligned", name);
  dgk::LossCall a{};
  a.X = X;
  a.W = W;
  a.targets = targets;
  a.loss = loss;
  a.lse = lse;
  a.workspace = workspace;
  a.T = T;
  a.V = V;
  a.K = K;
  int sms = 0;
  s = loss_state(&a, &sms);
  if (s != DG_OK) return s;
  return loss_result(dgk::launch_loss(a, sms, static_cast<cudaStream_t>(stream)));
}

long long dg_linear_cross_entropy_backward_workspace_bytes(int T, int V, int K) {
  return T < 0 || V < 0 || K < 0 ? -1 : dgk::loss_backward_workspace(T, V, K);
}

dg_status dg_linear_cross_entropy_backward(const void* X, const void* W, const int32_t* targets,
                                           const float* lse, const float* d_loss, void* dX, void* dW,
                                           void* workspace, long long workspace_bytes, int T, int V,
                                           int K, void* stream) {
  const char* name = "dg_linear_cross_entropy_backward";
  dg_status s = check_vocabulary(name, T, V, K);
  if (s != DG_OK) return s;
  if ((!dX && !dW) || (T > 0 && (!X || !W || !targets || !lse || !d_loss)))
    return host_fail(DG_ERR_INVALID_ARG,
                     "%s: null pointer (X, W, targets, lse, d_loss, one of dX and dW)", name);
  if (T > 0) {
    s = check_workspace(name, workspace, workspace_bytes, dgk::loss_backward_workspace(T, V, K));
    if (s != DG_OK) return s;
  }
  if (!aligned16(X) || !aligned16(W) || !aligned16(dX) || !aligned16(dW) || !aligned16(workspace) ||
      !aligned(targets, 4) || !aligned(lse, 4) || !aligned(d_loss, 4))
    return host_fail(DG_ERR_MISALIGNED,
                     "%s: X, W, dX, dW and workspace 16-byte, the others 4-byte aligned", name);
  if (T == 0 && !dW) return host_ok();
  dgk::LossCall a{};
  a.X = X;
  a.W = W;
  a.targets = targets;
  a.lse = const_cast<float*>(lse);
  a.d_loss = d_loss;
  a.dX = dX;
  a.dW = dW;
  a.workspace = workspace;
  a.T = T;
  a.V = V;
  a.K = K;
  int sms = 0;
  s = loss_state(&a, &sms);
  if (s != DG_OK) return s;
  if (T == 0) {   // no tokens: dW is 0
    const cudaError_t e = cudaMemsetAsync(dW, 0, 2ull * V * K, static_cast<cudaStream_t>(stream));
    return e != cudaSuccess ? cuda_fail(e, "cross entropy: clearing dW") : host_ok();
  }
  return loss_result(dgk::launch_loss_backward(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
