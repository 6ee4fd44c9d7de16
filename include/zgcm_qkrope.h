/*
 * zgcm_qkrope.h — C ABI of the layer's query/key preparation as an operator of its own
 * (sm_100a): per-head RMSNorm and partial rotation of q and k in one pass, forward and
 * backward.
 *
 * The attention calls of zgcm_attn.h form these values inside their kernels.  This operator
 * hands them to the caller: the keys a KV cache holds (the prompt's rows of zgcm_attn_decode's
 * k_cache, the blocks of zgcm_kv8.h), the queries of zgcm_attn_decode_kv8 and
 * zgcm_kv8_select, or the inputs of an attention that takes them prepared.  (QK-RMSNorm and the RoPE ratio 0.33:
 * shibing624 review of ZGCM-1, section "架构".)
 *
 *   forward   r = 1 / sqrt(mean_d x^2 + eps);  y = RoPE(gamma * x * r) at position pos[t],
 *             for every row x of q (gamma_q) and of k (gamma_k); RoPE as in zgcm_attn.h
 *             (pairs (i, i + rope_dims/2), angle pos * rope_base^(-2i/rope_dims))
 *   backward  u = RoPE^T(dy);  dgamma = sum over rows of u * x * r;
 *             dx = r * (gamma*u - x*r * mean_d(gamma * u * x * r))
 *
 * Conventions: T tokens of any packing (batches of sequences, ragged or padded: every token
 * brings its own position, pos int32 [T] on the device, any value).  Rows are given by
 * zgcm_rows: element (t, h, d) of a tensor is at ptr + (t * t_stride + h * h_stride + d)
 * elements, so the parts of a packed projection [T, (Hq + 2 Hkv + ...) * D] are read and
 * written in place; strides are multiples of 8 elements from 0 to 2^32 - 1 (larger or negative
 * ones: ZGCM_ERR_UNSUPPORTED) and pointers 16-byte aligned.
 * Rows of one tensor must not overlap in an output, and outputs must not alias inputs.
 * Types (zgcm_dtype): q, k, dq, dk have x_type; qr, kr, dqr, dkr have y_type; gamma fp32 [D].
 * Arithmetic is fp32 (angles are formed and reduced in fp64); each output element is
 * rounded once.  The sums of dgamma run in a fixed order: results repeat bit for bit.
 * A non-finite x makes its own row non-finite and no other.
 * The sum of a row's squares has to stay within fp32 (elements below 2^60), and above its smallest numbers where eps is 0.
 * Shapes: D == 128; Hq, Hkv >= 1; rope_dims even, 0 .. 128; T >= 0 (0: nothing is computed,
 * the backward zeroes dgamma_q and dgamma_k).
 * Errors and streams as in zgcm_attn.h: checks before any launch, asynchronous on
 * `cuda_stream`, nothing allocated.
 */
#ifndef ZGCM_QKROPE_H
#define ZGCM_QKROPE_H

#include "zgcm_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ZGCM_BF16 = 0, ZGCM_FP16 = 1, ZGCM_FP32 = 2 } zgcm_dtype;

typedef struct {
    void* ptr;
    long long t_stride, h_stride; /* elements between tokens, between heads */
} zgcm_rows;

int zgcm_qk_norm_rope_fwd(zgcm_rows q, zgcm_rows k, const float* gamma_q, const float* gamma_k, const int* pos, int T,
                          int Hq, int Hkv, int D, int x_type, int y_type, int rope_dims, double rope_base, float eps,
                          zgcm_rows qr, zgcm_rows kr, void* cuda_stream);

/* Workspace of the backward (partial sums of dgamma): at least
 * zgcm_qk_norm_rope_bwd_workspace_size(T) bytes, 16-byte aligned, not used by a concurrent call. */
size_t zgcm_qk_norm_rope_bwd_workspace_size(int T);

int zgcm_qk_norm_rope_bwd(zgcm_rows q, zgcm_rows k, const float* gamma_q, const float* gamma_k, const int* pos,
                          zgcm_rows dqr, zgcm_rows dkr, int T, int Hq, int Hkv, int D, int x_type, int y_type,
                          int rope_dims, double rope_base, float eps, zgcm_rows dq, zgcm_rows dk, float* dgamma_q,
                          float* dgamma_k, void* workspace, size_t workspace_bytes, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* ZGCM_QKROPE_H */
