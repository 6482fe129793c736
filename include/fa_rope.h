/*
 * fa_rope.h — per-head norm of queries and keys with the position rotation,
 * in one pass over the projection's output (C ABI, companion of fa.h).
 *
 * What is computed, for every row x = x[b, h, n, :] of D values of q (weights
 * q_weight) and of k (weights k_weight), at position p = positions[b, n]:
 *     r = (mean_d x_d^2 + eps)^(-1/2),   u_d = x_d r w_d
 *     a_i = p * inv_freq[i],             i < rotary_dim / 2
 *     (y_lo, y_hi) = (u_lo cos a_i - u_hi sin a_i,  u_hi cos a_i + u_lo sin a_i)
 * for the pairs (lo, hi) = (i, i + rotary_dim / 2), or (2i, 2i + 1) when
 * interleaved != 0.  y_d = u_d for d >= rotary_dim.  The rows are read from
 * strided views (the [B, N, heads, D] output of the projection, packed or
 * not) and written in the contiguous [B, H, N, D] layout that fa_fwd,
 * fa_decode and the cache take.
 *
 * The backward takes dy in that layout and returns
 *     g = R(a)^T dy,   dw_d = sum over b, h, n of g_d x_d r,
 *     h = g w,         dx_d = r (h_d - x_d r mean(h x r)),
 * with x read again and r recomputed from it.
 *
 * Sums and norms are in fp32.  An angle is reduced modulo a turn in 64-bit
 * integers, to within 2^-31 + 2^-106 |position * inv_freq| of a turn whatever
 * the position, and its cos and sin are fp32's (of the angle rounded to fp32:
 * about 1e-7 rad).  Results are rounded to bf16 once, dw stays fp32.  A row
 * whose sum of squares is beyond fp32 (values above about 1e18) is out of range.
 * dw is summed in a fixed order: repeated calls are bitwise equal.
 *
 * Ownership, streams, errors: as in fa.h.  Calls are asynchronous on
 * `stream`, allocate nothing and can be captured into a CUDA graph.
 */
#ifndef TILED_ATTENTION_FA_ROPE_H
#define TILED_ATTENTION_FA_ROPE_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bf16 rows x[b, h, n, 0..D): the D values of a row are contiguous, the
 * strides (in elements) are free.  data 16-byte aligned; the strides of
 * dimensions larger than 1 are >= 0 and multiples of 8.  Views that are
 * written must not overlap themselves, nor anything that the call reads or
 * writes. */
typedef struct {
    void* data;
    long long stride_b, stride_h, stride_n;
} fa_rows;

/* D = 64 or 128 (FA_ERR_UNSUPPORTED otherwise); Hq and Hkv are free of each
 * other, Hq + Hkv <= 65535; B * N <= 2^31 - 1; 0 <= rotary_dim <= D, a multiple
 * of 8; eps finite and > 0; weight_bf16: the weights are bf16, else fp32. */
typedef struct {
    int B, Hq, Hkv, N, D;
    int rotary_dim, interleaved;
    float eps;
    int weight_bf16;
} fa_rope_shape;

/* q [B,Hq,N,D], k [B,Hkv,N,D] bf16 views; q_weight, k_weight [D];
 * inv_freq fp32 [rotary_dim / 2], finite (NULL allowed when rotary_dim is 0);
 * positions int32 [B,N], or NULL: token n of each sequence is at position n.
 * q_out [B,Hq,N,D], k_out [B,Hkv,N,D] bf16 contiguous, apart from the inputs.
 * Outputs 16-byte aligned, weights, inv_freq and positions 4-byte. */
FA_API fa_status fa_qk_norm_rope(const fa_rope_shape* shape, const fa_rows* q, const fa_rows* k, const void* q_weight,
                                 const void* k_weight, const float* inv_freq, const int* positions, void* q_out,
                                 void* k_out, void* stream);

/* Bytes of device workspace the backward needs (0 if the shape is invalid or
 * there is no CUDA device): partial sums of the weights' gradients, one pair
 * of rows for each CTA, whatever the number of tokens. */
FA_API size_t fa_qk_norm_rope_bwd_workspace_bytes(const fa_rope_shape* shape);

/* dq_out, dk_out: gradients of q_out and k_out (bf16, contiguous).  Writes
 * dq [B,Hq,N,D] and dk [B,Hkv,N,D] (bf16 views) and dq_weight, dk_weight
 * (fp32 [D]).  workspace: 256-byte aligned, contents on entry do not matter.
 * Calls that may overlap need workspaces of their own. */
FA_API fa_status fa_qk_norm_rope_bwd(const fa_rope_shape* shape, const void* dq_out, const void* dk_out,
                                     const fa_rows* q, const fa_rows* k, const void* q_weight, const void* k_weight,
                                     const float* inv_freq, const int* positions, const fa_rows* dq,
                                     const fa_rows* dk, float* dq_weight, float* dk_weight, void* workspace,
                                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TILED_ATTENTION_FA_ROPE_H */
