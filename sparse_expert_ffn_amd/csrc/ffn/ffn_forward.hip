// The dense gated feed-forward block, forward (include/moe_ffn.h): X W_up and X
// W_gate as one product of two panels whose epilogue forms h in registers, then
// h W_down.
#include "ffn_plan.h"

namespace moe {

namespace {
__global__ void ffn_zero_kernel(uint32_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0;
}

struct FwdPlan {
  GemmPlan up, down;
  size_t h, part, total;
};
FwdPlan plan_forward(const moe_ffn_shape* s) {
  FwdPlan p;
  const bool f32 = s->dtype == MOE_F32;
  p.up = plan_gemm(f32, tile_mask<true, true, false>(f32), true, s->S, s->D, s->H, 1);
  p.down = plan_gemm(f32, tile_mask<false, true, false>(f32), false, s->S, s->H, s->D, 1);
  p.h = 0;
  p.part = ffn_round_up((size_t)s->S * s->D * (f32 ? 4 : 2), 256);
  const size_t q = p.up.part_bytes > p.down.part_bytes ? p.up.part_bytes : p.down.part_bytes;
  p.total = p.part + ffn_round_up(q, 256);
  if (p.total == 0) p.total = 256;
  return p;
}

template <typename T>
void forward_t(const moe_ffn_shape* s, const FwdPlan& p, const void* X, const void* Wu,
               const void* Wg, const void* Wd, void* U, void* G, void* O, char* ws,
               hipStream_t st) {
  GemmArgs g = {};
  g.A[0] = X;
  g.B[0][0] = Wu;
  g.B[0][1] = Wg;
  g.lda = s->H;
  g.ldb = s->D;
  g.M = s->S;
  g.N = s->D;
  g.K[0] = s->H;
  g.pairs = 1;
  apply_plan(p.up, &g, ws + p.part);
  launch_gemm<T, true, true, false>(p.up, g, EpSwiglu<T>{(T*)(ws + p.h), (T*)U, (T*)G, s->D}, st);
  g.A[0] = ws + p.h;
  g.B[0][0] = Wd;
  g.lda = s->D;
  g.ldb = s->H;
  g.N = s->H;
  g.K[0] = s->D;
  apply_plan(p.down, &g, ws + p.part);
  if (s->flags & MOE_OUTPUT_F32)
    launch_gemm<T, false, true, false>(p.down, g, EpStore<float>{(float*)O, nullptr, s->H}, st);
  else
    launch_gemm<T, false, true, false>(p.down, g, EpStore<T>{(T*)O, nullptr, s->H}, st);
}
}  // namespace

hipError_t launch_zero(void* p, size_t bytes, hipStream_t st) {
  const int64_t n = (int64_t)(bytes / 4);
  if (n == 0) return hipSuccess;
  const int64_t b = (n + 255) / 256;
  ffn_zero_kernel<<<(unsigned)(b < 8192 ? b : 8192), 256, 0, st>>>((uint32_t*)p, n);
  return hipGetLastError();
}

moe_status check_ffn(const moe_ffn_shape* s) {
  if (s == nullptr || s->S < 0 || s->H < 1 || s->D < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16 && s->dtype != MOE_MXFP8)
    return MOE_ERR_INVALID_ARGUMENT;
  if (s->flags & ~MOE_OUTPUT_F32) return MOE_ERR_INVALID_ARGUMENT;
  if (s->dtype == MOE_MXFP8 || s->H % 8 || s->D % 8 || s->H >= (1 << 22) || s->D >= (1 << 22) ||
      s->S >= INT32_MAX - 256)
    return MOE_ERR_UNSUPPORTED;
  // a launch's workgroups, in tiles of 64 x 64 (see kMaxGroups)
  if ((s->S + 63) / 64 * ((s->H > s->D ? s->H : s->D) / 64 + 1) >= (1 << 23))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_ffn_forward_workspace_bytes(const moe_ffn_shape* shape) {
  return check_ffn(shape) == MOE_OK ? plan_forward(shape).total : 0;
}

extern "C" moe_status moe_ffn_forward(const moe_ffn_shape* s, const void* X, const void* W_up,
                                      const void* W_gate, const void* W_down, void* U, void* G,
                                      void* O, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  const moe_status st = check_ffn(s);
  if (st != MOE_OK) return st;
  if ((U == nullptr) != (G == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (s->S == 0) return MOE_OK;
  if (X == nullptr || W_up == nullptr || W_gate == nullptr || W_down == nullptr || O == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (ffn_shared({O, U, G, workspace}, {X, W_up, W_gate, W_down}))
    return MOE_ERR_INVALID_ARGUMENT;
  for (const void* q : {X, W_up, W_gate, W_down, (const void*)O, (const void*)U, (const void*)G,
                        (const void*)workspace})
    if (!ffn_aligned16(q)) return MOE_ERR_UNSUPPORTED;
  const FwdPlan p = plan_forward(s);
  if (workspace == nullptr || workspace_bytes < p.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (s->dtype == MOE_F32)
    forward_t<float>(s, p, X, W_up, W_gate, W_down, U, G, O, (char*)workspace,
                     (hipStream_t)stream);
  else
    forward_t<bf16_t>(s, p, X, W_up, W_gate, W_down, U, G, O, (char*)workspace,
                      (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
