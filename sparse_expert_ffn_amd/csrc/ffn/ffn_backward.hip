// The dense gated feed-forward block, backward (include/moe_ffn.h), as four
// products: dh = dO W_down^T, whose epilogue forms dU, dG and h; dX over the two
// pairs (dU, W_up) and (dG, W_gate) in one sum; X^T (dU | dG) as one product of
// two panels; h^T dO.
#include "ffn_plan.h"

namespace moe {
namespace {

moe_status check_backward(const moe_ffn_shape* s) {
  const moe_status st = check_ffn(s);
  if (st != MOE_OK) return st;
  // the weight gradients' tiles run over H x D
  return (s->H + 63) / 64 * (s->D / 64 + 1) >= (1 << 23) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

struct BwdPlan {
  GemmPlan dh, dx, dw, dwd;
  size_t du, dg, h, part, total;
};
BwdPlan plan_backward(const moe_ffn_shape* s) {
  BwdPlan p;
  const bool f32 = s->dtype == MOE_F32;
  p.dh = plan_gemm(f32, tile_mask<false, true, true>(f32), false, s->S, s->D, s->H, 1);
  p.dx = plan_gemm(f32, tile_mask<false, true, true>(f32), false, s->S, s->H, s->D, 2);
  p.dw = plan_gemm(f32, tile_mask<true, false, false>(f32), true, s->H, s->D, s->S, 1);
  p.dwd = plan_gemm(f32, tile_mask<false, false, false>(f32), false, s->D, s->H, s->S, 1);
  const size_t n = ffn_round_up((size_t)s->S * s->D * (f32 ? 4 : 2), 256);
  p.du = 0;
  p.dg = n;
  p.h = 2 * n;
  p.part = 3 * n;
  size_t q = 0;
  for (const GemmPlan* g : {&p.dh, &p.dx, &p.dw, &p.dwd})
    if (g->part_bytes > q) q = g->part_bytes;
  p.total = p.part + ffn_round_up(q, 256);
  if (p.total == 0) p.total = 256;
  return p;
}

template <typename T, typename TW>
void backward_t(const moe_ffn_shape* s, const BwdPlan& p, const void* dO, const void* X,
                const void* Wu, const void* Wg, const void* Wd, const void* U, const void* G,
                void* dX, void* dWu, void* dWg, void* dWd, char* ws, hipStream_t st) {
  T* du = (T*)(ws + p.du);
  T* dg = (T*)(ws + p.dg);
  T* h = dWu != nullptr ? (T*)(ws + p.h) : nullptr;
  GemmArgs g = {};
  g.pairs = 1;
  g.A[0] = dO;
  g.B[0][0] = Wd;
  g.lda = g.ldb = s->H;
  g.M = s->S;
  g.N = s->D;
  g.K[0] = s->H;
  apply_plan(p.dh, &g, ws + p.part);
  launch_gemm<T, false, true, true>(
      p.dh, g, EpSwigluBwd<T>{(const T*)U, (const T*)G, du, dg, h, s->D}, st);
  if (dX != nullptr) {
    g.pairs = 2;
    g.A[0] = du;
    g.A[1] = dg;
    g.B[0][0] = Wu;
    g.B[1][0] = Wg;
    g.lda = g.ldb = s->D;
    g.N = s->H;
    g.K[0] = g.K[1] = s->D;
    apply_plan(p.dx, &g, ws + p.part);
    launch_gemm<T, false, true, true>(p.dx, g, EpStore<T>{(T*)dX, nullptr, s->H}, st);
  }
  if (dWu != nullptr) {
    g = GemmArgs{};
    g.pairs = 1;
    g.A[0] = X;
    g.B[0][0] = du;
    g.B[0][1] = dg;
    g.lda = s->H;
    g.ldb = s->D;
    g.M = s->H;
    g.N = s->D;
    g.K[0] = s->S;
    apply_plan(p.dw, &g, ws + p.part);
    launch_gemm<T, true, false, false>(p.dw, g, EpStore<TW, true>{(TW*)dWu, (TW*)dWg, s->D}, st);
    g.A[0] = h;
    g.B[0][0] = dO;
    g.lda = s->D;
    g.ldb = s->H;
    g.M = s->D;
    g.N = s->H;
    apply_plan(p.dwd, &g, ws + p.part);
    launch_gemm<T, false, false, false>(p.dwd, g, EpStore<TW>{(TW*)dWd, nullptr, s->H}, st);
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_ffn_backward_workspace_bytes(const moe_ffn_shape* shape) {
  return check_backward(shape) == MOE_OK ? plan_backward(shape).total : 0;
}

extern "C" moe_status moe_ffn_backward(const moe_ffn_shape* s, const void* dO, const void* X,
                                       const void* W_up, const void* W_gate, const void* W_down,
                                       const void* U, const void* G, void* dX, void* dW_up,
                                       void* dW_gate, void* dW_down, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  const moe_status st = check_backward(s);
  if (st != MOE_OK) return st;
  if ((dW_up == nullptr) != (dW_gate == nullptr) || (dW_up == nullptr) != (dW_down == nullptr) ||
      (dX == nullptr && dW_up == nullptr && s->S > 0))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ffn_shared({dX, dW_up, dW_gate, dW_down, workspace}, {dO, X, W_up, W_gate, W_down, U, G}))
    return MOE_ERR_INVALID_ARGUMENT;
  for (const void* q : {dO, X, W_up, W_gate, W_down, U, G}) {
    if (q == nullptr && s->S > 0) return MOE_ERR_INVALID_ARGUMENT;
    if (!ffn_aligned16(q)) return MOE_ERR_UNSUPPORTED;
  }
  for (const void* q : {dX, dW_up, dW_gate, dW_down, workspace})
    if (!ffn_aligned16(q)) return MOE_ERR_UNSUPPORTED;
  hipStream_t q = (hipStream_t)stream;
  const bool wf32 = s->dtype == MOE_F32 || (s->flags & MOE_OUTPUT_F32) != 0;
  if (s->S == 0) {
    if (dW_up == nullptr) return MOE_OK;
    const size_t n = (size_t)(s->H * s->D) * (wf32 ? 4 : 2);
    for (void* w : {dW_up, dW_gate, dW_down})
      if (launch_zero(w, n, q) != hipSuccess) return MOE_ERR_HIP;
    return MOE_OK;
  }
  const BwdPlan p = plan_backward(s);
  if (workspace == nullptr || workspace_bytes < p.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  char* ws = (char*)workspace;
  if (s->dtype == MOE_F32)
    backward_t<float, float>(s, p, dO, X, W_up, W_gate, W_down, U, G, dX, dW_up, dW_gate,
                             dW_down, ws, q);
  else if (wf32)
    backward_t<bf16_t, float>(s, p, dO, X, W_up, W_gate, W_down, U, G, dX, dW_up, dW_gate,
                              dW_down, ws, q);
  else
    backward_t<bf16_t, bf16_t>(s, p, dO, X, W_up, W_gate, W_down, U, G, dX, dW_up, dW_gate,
                               dW_down, ws, q);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
