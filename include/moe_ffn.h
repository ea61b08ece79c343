/*
 * sparse_expert_ffn_amd — C ABI of the operators around the MoE layer on one
 * MI355X (gfx950) GPU: layer norm, the dense gated feed-forward block with its
 * backward pass, products with 4-bit weights for decode, products in 8-bit
 * integers, and the whole MoE layer for a few tokens.
 *
 * The conventions are those of moe.h: device pointers to dense row-major
 * arrays, every call validates on the host, enqueues kernels on `stream` (of
 * the current device) and returns a moe_status; nothing synchronises,
 * allocates, aborts or throws, no pointer is kept. In addition:
 *  - Workspaces may hold anything before a call. Calls that may run at the
 *    same time (other streams, graphs replayed at once) need workspaces and
 *    outputs of their own. Everything can be captured in a HIP graph.
 *  - No output and no workspace in use may overlap an input or another output
 *    (MOE_ERR_INVALID_ARGUMENT where the overlap is two equal pointers; other
 *    overlaps are not looked for).
 *  - Results are bit-reproducible: every sum runs in a fixed order for a given
 *    shape, none through atomics.
 *  - NaN and infinity in an input reach the outputs that depend on it, and no
 *    others.
 */
#ifndef SPARSE_EXPERT_FFN_AMD_MOE_FFN_H
#define SPARSE_EXPERT_FFN_AMD_MOE_FFN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm over rows of X [S][H]:
 *   m_s = (1/H) sum_h X_sh,  v_s = (1/H) sum_h (X_sh - m_s)^2,  r_s = 1 / sqrt(v_s + eps)
 *   Y_sh = (X_sh - m_s) r_s gamma_h + beta_h
 * dtype MOE_F32 or MOE_BF16 (X, gamma, beta, Y); statistics and sums are fp32
 * (those over a row longer than 16384 compensated), Y is rounded once. Any S from 0 and H from 1 on, S below 2^31 - 1, H below 2^27
 * (else MOE_ERR_UNSUPPORTED, as for arrays off their element's alignment or a
 * workspace off 16 bytes); arrays whose rows are whole 16-byte vectors
 * and aligned to them are fastest.
 *   gamma, beta  [H] dtype, each may be NULL (1 and 0)
 *   mean, rstd   [S] fp32 out, both or neither NULL (kept for the backward pass)
 * eps must be finite and >= 0.
 */
moe_status moe_layernorm_forward(int64_t S, int64_t H, int32_t dtype, const void* X,
                                 const void* gamma, const void* beta, float eps, void* Y,
                                 float* mean, float* rstd, void* stream);

/* Bytes of workspace of moe_layernorm_backward (0 on invalid sizes). */
size_t moe_layernorm_backward_workspace_bytes(int64_t S, int64_t H, int32_t dtype);

/*
 * Its backward pass: with n_sh = (X_sh - m_s) r_s and d_sh = dY_sh gamma_h,
 *   dX_sh   = r_s (d_sh - (1/H) sum_h d_sh - n_sh (1/H) sum_h d_sh n_sh)
 *   dgamma_h = sum_s dY_sh n_sh,  dbeta_h = sum_s dY_sh
 *   dY, X  [S][H] dtype;  gamma [H] dtype or NULL (1);  mean, rstd [S] fp32 as the
 *   forward pass left them;  dX [S][H] dtype out;  dgamma, dbeta [H] fp32 out, both
 *   or neither NULL (frozen weights). With S = 0, dgamma and dbeta are set to 0.
 */
moe_status moe_layernorm_backward(int64_t S, int64_t H, int32_t dtype, const void* dY,
                                  const void* X, const void* gamma, const float* mean,
                                  const float* rstd, void* dX, float* dgamma, float* dbeta,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Shape of a dense gated feed-forward block. */
typedef struct {
  int64_t S;      /* tokens; 0 is a valid empty call                             */
  int64_t H;      /* hidden size, a multiple of 8                                */
  int64_t D;      /* intermediate size, a multiple of 8                          */
  int32_t dtype;  /* MOE_F32 or MOE_BF16: activations, weights, gradients        */
  int32_t flags;  /* 0 or MOE_OUTPUT_F32: moe_ffn_forward writes O, and
                     moe_ffn_backward the three weight gradients, as fp32       */
} moe_ffn_shape;

/*
 * The dense gated feed-forward block (the shared expert's equation of moe.h on
 * its own):
 *   U = X W_up,  G = X W_gate,  h = SiLU(U) * G,  O = h W_down
 *   X [S][H];  W_up, W_gate [H][D];  W_down [D][H];  O [S][H] out
 *   U, G [S][D] dtype out, both or neither NULL: the pre-activations that
 *   moe_ffn_backward takes
 * Accumulation is fp32 and the activation is computed on the fp32 sums; in bf16
 * mode h is rounded once to bf16 as the second product's operand, U, G and O
 * once as outputs.
 * Requires H, D multiples of 8 and below 2^22, S < 2^31, 16-byte aligned
 * arrays (else MOE_ERR_UNSUPPORTED). Arrays may exceed 4 GiB.
 */
size_t moe_ffn_forward_workspace_bytes(const moe_ffn_shape* shape); /* 0 if unsupported */
moe_status moe_ffn_forward(const moe_ffn_shape* shape, const void* X, const void* W_up,
                           const void* W_gate, const void* W_down, void* U, void* G, void* O,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Its backward pass from dO [S][H] and the kept U, G:
 *   dh = dO W_down^T,  h = SiLU(U) * G,  s = 1 / (1 + exp(-U))
 *   dG = dh * U s,  dU = dh * G s (1 + U (1 - s))
 *   dX = dU W_up^T + dG W_gate^T                                    [S][H] dtype
 *   dW_up = X^T dU,  dW_gate = X^T dG  [H][D],  dW_down = h^T dO  [D][H]
 * The weight gradients are dtype, or fp32 with MOE_OUTPUT_F32, and are
 * overwritten (S = 0 sets them to 0). dX may be NULL (nothing before the block
 * is trained); the three weight gradients may be NULL together (frozen
 * weights). Sums are fp32; in bf16 mode dU, dG and h are rounded once to bf16
 * as operands of the products, whose results are rounded once.
 * Requirements as moe_ffn_forward; H / 64 times D / 64 stays below 2^23 too.
 */
size_t moe_ffn_backward_workspace_bytes(const moe_ffn_shape* shape); /* 0 if unsupported */
moe_status moe_ffn_backward(const moe_ffn_shape* shape, const void* dO, const void* X,
                            const void* W_up, const void* W_gate, const void* W_down,
                            const void* U, const void* G, void* dX, void* dW_up, void* dW_gate,
                            void* dW_down, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * 4-bit weights. A weight matrix W [K][N] is held as codes 0..15 and one bf16
 * scale per column and group of `group` (32, 64 or 128) consecutive rows:
 *   W_kn = (code_kn - 8) * scale_{k / group, n}
 * The last group may be shorter. E matrices lie one after another.
 *
 * moe_quantize_w4 gives the codes [E][K][N] (one byte each) and scales
 * [E][ceil(K/group)][N] (bf16) of a bf16 or fp32 tensor W [E][K][N]: a group's
 * scale is max |w| / 7 rounded to bf16 (0 for an all-zero group), its codes are
 * w / scale rounded to the nearest integer, ties to even, clamped to [-8, 7],
 * plus 8 (8 where the scale is 0). Values are expected to be finite.
 *
 * moe_pack_w4_weights lays codes and scales, of whatever quantiser, out for the
 * products below: moe_w4_weight_bytes(E, K, N, group) bytes at `packed` (16-byte
 * aligned). Only the low 4 bits of a code byte are taken. Rows and columns that
 * fill up a tile are given a scale of 0. Layout, for each matrix: tiles of 16
 * columns n by 128 rows k, column tile by column tile, k ascending. A tile holds
 * 1024 bytes of codes: 16 bytes for each lane l = 16 q + c (column c), dword i
 * of which holds the 8 rows 32 i + 8 q + j, row j in bits 4 (j / 2) + 16 (j % 2)
 * to + 3, the whole dword then rotated left by 3 bits; then its scales
 * [16][128 / group] bf16. Both calls are one-time steps, at weight load. K and
 * N multiples of 8, below 2^22.
 */
size_t moe_w4_weight_bytes(int64_t E, int64_t K, int64_t N, int32_t group); /* 0 if unsupported */
moe_status moe_quantize_w4(const void* W, int64_t E, int64_t K, int64_t N, int32_t dtype,
                           int32_t group, uint8_t* codes, void* scales, void* stream);
moe_status moe_pack_w4_weights(const uint8_t* codes, const void* scales, int64_t E, int64_t K,
                               int64_t N, int32_t group, void* packed, void* stream);

/*
 * Y = X W for few rows (decode): X [S][K] bf16, W packed with E matrices, Y
 * [S][N] bf16, or fp32 with flags = MOE_OUTPUT_F32. The weights are read once
 * per 16 rows; made for S up to a few tens, S <= 4096 and X below 2 GiB.
 *   expert_ids  [S] int32 or NULL. NULL: every row takes matrix 0. Else row s
 *               takes matrix expert_ids[s] (rows may share one, and its weights
 *               are then read once for 16 of them); an id outside [0, E) gives
 *               a row of zeros.
 * A group's sum is formed as sum X (code + 16) - 24 sum X, products exact and
 * sums fp32, then scaled; so an infinite X gives NaN, and |X| has to stay below
 * 2^120. Y is rounded once.
 */
moe_status moe_w4_matvec(int64_t S, int64_t K, int64_t N, int64_t E, int32_t group,
                         int32_t flags, const void* X, const void* W, const int32_t* expert_ids,
                         void* Y, void* stream);

/*
 * The MoE layer's expert computation and combine (moe_forward's formulas) with
 * 4-bit expert weights, for few tokens: takes moe_gate_topk's topk_ids and
 * topk_weights as they are, without moe_align_block_size.
 *   O_t = sum_j topk_weights[t][j] FFN_{topk_ids[t][j]}(A_t)  (+ FFN_shared(A_t))
 * in slot order, then the shared expert; an id outside [0, E) is a slot
 * without an expert (it contributes nothing, whatever its weight), a token
 * whose slots are all empty (padding) and no shared expert gives a row of
 * zeros. An expert's weights are read once per 16 of its rows.
 *   shape     dtype MOE_BF16, capacity 0, flags 0 or MOE_OUTPUT_F32, E at most 1024,
 *             k at most 32, S * k and S at most 4096, A and the h rows below 2 GiB;
 *             block_size and renormalize are not looked at
 *   A         [S][H] bf16;  W_up, W_gate: packed [E][H][D];  W_down: packed [E][D][H];
 *   Ws_*      packed with E = 1 ([H][D_shared] twice, [D_shared][H]), NULL iff D_shared = 0
 *   O         [S][H] bf16, or fp32 with MOE_OUTPUT_F32
 * Sums are as in moe_w4_matvec; h is rounded once to bf16 as the second product's
 * operand. H, D, D_shared multiples of 8.
 */
size_t moe_w4_forward_workspace_bytes(const moe_shape* shape); /* 0 if unsupported */
moe_status moe_w4_forward(const moe_shape* shape, int32_t group, const void* A,
                          const void* W_up, const void* W_gate, const void* W_down,
                          const void* Ws_up, const void* Ws_gate, const void* Ws_down,
                          const int32_t* topk_ids, const float* topk_weights, void* O,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * 8-bit integers with a scale for each token and channel. A weight matrix W [K][N] is
 * held as codes -127..127 and one fp32 scale per column, W_kn = code_kn scale_n; a row
 * of activations as codes and one scale. A vector x (a column of W, a row of X) has
 *   scale = max |x| / 127 rounded to fp32,  code = x / scale rounded to the nearest
 *   integer, ties to even (0 where the scale is 0, clamped to [-127, 127])
 * decided exactly, both of them (max |x| times the rounded 1 / 127 is another scale in 3 to 6%
 * of the vectors). A vector that holds an infinity or NaN gets a scale of NaN and
 * codes 0: every product with it is NaN.
 *
 * moe_quantize_i8 gives the codes [E][K][N] and scales [E][N] of a bf16 or fp32
 * tensor W [E][K][N]. moe_pack_i8_weights lays codes and scales, of whatever
 * quantiser (codes of -128 and scales below 0 are allowed), out for the products below:
 * moe_i8_weight_bytes(E, K, N) bytes at `packed`. Layout, matrix by matrix: tiles of
 * 16 columns n by 64 rows k, column tile by column tile, k ascending, 1024 bytes each:
 * 16 bytes for each lane l = 16 q + c, rows 16 q .. + 15 of column c; then the scales,
 * one for each column of the tiles. What fills up a tile is 0. Both calls are one-time
 * steps, at weight load. moe_quantize_i8_rows gives the codes [S][K] and scales [S] of
 * the rows of X [S][K].
 *
 * K a multiple of 16 up to 131072 (sums of products of codes stay exact in 32 bits;
 * for codes of -128 on both sides below that), N a multiple of 8 below 2^22, 16-byte
 * aligned arrays (scales: 4), else MOE_ERR_UNSUPPORTED.
 */
size_t moe_i8_weight_bytes(int64_t E, int64_t K, int64_t N); /* 0 if unsupported */
moe_status moe_quantize_i8(const void* W, int64_t E, int64_t K, int64_t N, int32_t dtype,
                           int8_t* codes, float* scales, void* stream);
moe_status moe_pack_i8_weights(const int8_t* codes, const float* scales, int64_t E, int64_t K,
                               int64_t N, void* packed, void* stream);
moe_status moe_quantize_i8_rows(const void* X, int64_t S, int64_t K, int32_t dtype,
                                int8_t* codes, float* scales, void* stream);

/*
 * Y = X W in that arithmetic: Y_sn = (sum_k xcode_sk wcode_kn) xscale_s wscale_n, the
 * sum exact in integers, scaled in fp32 (the scale nearer to 0 first), rounded once. Any S:
 * one token to a prompt; a row's result does not depend on S.
 *   row_scales  NULL: X is [S][K] of `dtype` (MOE_F32 or MOE_BF16), quantised by the
 *               call as moe_quantize_i8_rows does.
 *               [S] fp32: X holds [S][K] codes (int8) with these scales
 *   W           packed with E = 1;  Y [S][N] of `dtype`, fp32 with flags = MOE_OUTPUT_F32
 * A NaN or infinity in a row of X gives a row of NaN.
 */
size_t moe_i8_matmul_workspace_bytes(int64_t S, int64_t K, int64_t N); /* 0 if unsupported */
moe_status moe_i8_matmul(int64_t S, int64_t K, int64_t N, int32_t dtype, int32_t flags,
                         const void* X, const float* row_scales, const void* W, void* Y,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * The dense gated feed-forward block (moe_ffn_forward's) in that arithmetic:
 *   U = X W_up,  G = X W_gate,  h = SiLU(U) * G,  O = h W_down,
 * each product as in moe_i8_matmul: the rows of X and those of h (kept in fp32, not
 * rounded before) are quantised.
 *   X [S][H] dtype;  W_up, W_gate packed [H][D], W_down packed [D][H];  O [S][H] dtype, or
 *   fp32 with MOE_OUTPUT_F32
 * H and D multiples of 16 up to 131072.
 */
size_t moe_i8_ffn_workspace_bytes(const moe_ffn_shape* shape); /* 0 if unsupported */
moe_status moe_i8_ffn_forward(const moe_ffn_shape* shape, const void* X, const void* W_up,
                              const void* W_gate, const void* W_down, void* O, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * The whole MoE layer for a few tokens (decode): gate scores, softmax top-k, the
 * experts, the shared expert and the combine, in three launches (four beyond 8 tokens or
 * 256 assignments).
 *   G = A W_router (+ router_bias); topk_ids, topk_weights from G as moe_gate_topk's
 *   O_t = sum_j topk_weights[t][j] FFN_{topk_ids[t][j]}(A_t)  (+ FFN_shared(A_t))
 * in slot order, then the shared expert. An expert's weights are read once per 16 of
 * its rows.
 *   shape        dtype MOE_F32 or MOE_BF16, capacity 0, flags 0 or MOE_OUTPUT_F32, S at
 *                most 128, E at most 1024, k at most 32; block_size is not looked at
 *   A            [S][H];  W_router [H][E];  router_bias [E] fp32 or NULL
 *   W_up, W_gate [E][H][D];  W_down [E][D][H];  Ws_up, Ws_gate [H][D_shared], Ws_down
 *                [D_shared][H], NULL iff D_shared = 0
 *   topk_ids     [S][k] int32, topk_weights [S][k] fp32. Outputs; with W_router NULL (and
 *                then router_bias) inputs: the routing is given, an id outside [0, E) is
 *                a slot without an expert (it contributes nothing, whatever its weight)
 *   O            [S][H] dtype, or fp32 with MOE_OUTPUT_F32
 * Scores are summed in fp32 over up to 512 values of H, these sums in double, and
 * rounded to fp32; a NaN score ranks as -inf. Sums of the products are fp32, in an order
 * that the shape alone fixes; in bf16 mode h is rounded once to bf16. Workgroups count each
 * other's arrivals and never wait for one another.
 * H, D, D_shared multiples of 8 up to 65536, one matrix (with 64 rows and columns more)
 * below 0x7F000000 bytes, 16-byte aligned arrays (else MOE_ERR_UNSUPPORTED).
 *
 * moe_few_i8_forward takes expert weights packed by moe_pack_i8_weights (E matrices; the
 * shared expert's with E = 1) and computes each expert as moe_i8_ffn_forward does; dtype
 * MOE_BF16 (A, W_router), H, D, D_shared multiples of 16. It is the one MoE call that takes
 * such experts: above 128 tokens moe_forward does the layer, with weights in its own types.
 */
size_t moe_few_workspace_bytes(const moe_shape* shape);    /* 0 if unsupported */
moe_status moe_few_forward(const moe_shape* shape, const void* A, const void* W_router,
                           const float* router_bias, const void* W_up, const void* W_gate,
                           const void* W_down, const void* Ws_up, const void* Ws_gate,
                           const void* Ws_down, int32_t* topk_ids, float* topk_weights, void* O,
                           void* workspace, size_t workspace_bytes, void* stream);
size_t moe_few_i8_workspace_bytes(const moe_shape* shape); /* 0 if unsupported */
moe_status moe_few_i8_forward(const moe_shape* shape, const void* A, const void* W_router,
                              const float* router_bias, const void* W_up, const void* W_gate,
                              const void* W_down, const void* Ws_up, const void* Ws_gate,
                              const void* Ws_down, int32_t* topk_ids, float* topk_weights,
                              void* O, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_EXPERT_FFN_AMD_MOE_FFN_H */
