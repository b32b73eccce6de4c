/*
 * gdn_qk_norm.h -- norms of the queries and keys of each head, with the
 * position rotation in the same pass (sm_100a).
 *
 * gdn_cpr_forward, gdn_cpr_decode_step and the other layouts take q and k
 * that are already normalised for each head; these entry points make them
 * from a layer's raw projections, and take the gradients that
 * gdn_cpr_backward returns back to the projections.  (The pages leave this
 * step to the caller; it has no counterpart there.)  For one head x[0..d):
 *
 *     r = (sum x^2 + eps)^(-1/2)       GDN_QK_NORM_L2
 *     r = (sum x^2 / d + eps)^(-1/2)   GDN_QK_NORM_RMS
 *     n = x r w                        (w = 1 when no weight is given)
 *     y = n rotated: for j < F = rot_dim / 2 with the angle
 *         t_j = positions[token] inv_freq[j] and the pair (i, i') =
 *         (j, j + F), or (2j, 2j + 1) when interleaved,
 *         y_i = n_i cos t_j - n_i' sin t_j
 *         y_i' = n_i' cos t_j + n_i sin t_j
 *         and y = n for the channels from rot_dim on.
 *
 * Sums are fp32 in a fixed order for each head, so a head's bits depend on
 * that head, its position and the weights alone: prefill, training and
 * decode agree bit for bit whatever the batch.  (Another rotation of the same
 * head may give its norm's sum another order.)  Angles are reduced in 64 bits
 * before the fp32 sine and cosine.
 *
 * Conventions are those of gdn_cpr.h.  q and k are [tokens, heads, d] with
 * heads and channels contiguous and a token stride (ld*, in elements,
 * >= heads d), so that they can be slices of one fused projection.  Pointers
 * are 16-byte aligned, and strides are multiples of 16 bytes.
 * Supported: d in {64, 128, 256}, bf16 or fp32 data, rot_dim a multiple of
 * 16 from 0 to d, eps > 0, any Hq, Hk >= 0 with Hq + Hk from 1 to 65535.
 */
#ifndef GDN_QK_NORM_H
#define GDN_QK_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "gdn_cpr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GDN_QK_NORM_L2 = 0, GDN_QK_NORM_RMS = 1 } gdn_qk_norm_kind;

/*
 * gdn_qk_norm_forward
 *
 * q, k       [T, Hq, d], [T, Hk, d] in_dtype, token strides ldq, ldk
 *            (q may be NULL when Hq == 0, k when Hk == 0)
 * wq, wk     [d] fp32 weights, or NULL for ones
 * positions  [T] int32 on the device (any sign), and
 * inv_freq   [rot_dim / 2] fp32; both unused (may be NULL) when rot_dim == 0
 * oq, ok     [T, Hq, d], [T, Hk, d] out_dtype, token strides ldoq, ldok.
 *            oq may be q and ok may be k (in place: same pointer, stride and
 *            dtype); any other overlap is an error that is not detected.
 * T may be 0.
 */
int gdn_qk_norm_forward(const void* q, int64_t ldq, const void* k, int64_t ldk, int in_dtype,
                        int64_t T, int Hq, int Hk, int d, int norm, float eps, const float* wq,
                        const float* wk, const int32_t* positions, const float* inv_freq,
                        int rot_dim, int interleaved, void* oq, int64_t ldoq, void* ok,
                        int64_t ldok, int out_dtype, void* stream);

/* Bytes of device workspace gdn_qk_norm_backward needs when it returns d_wq or
 * d_wk (it needs none otherwise); 0 for arguments it would reject. */
size_t gdn_qk_norm_backward_workspace_bytes(int64_t T, int Hq, int Hk, int d);

/*
 * gdn_qk_norm_backward -- with dn = dL/dy rotated back and e = dn w,
 *     dx = r (e - x r^2 m(x e)),  m = sum (L2) or mean (RMS) over the head
 *     dw = sum over tokens and heads of dn x r   (fixed order, fp32)
 *
 * q .. interleaved  as for the forward (q and k are the forward's inputs)
 * d_oq, d_ok  [T, Hq, d], [T, Hk, d] grad_dtype (GDN_F32 is what
 *             gdn_cpr_backward returns), token strides lddoq, lddok
 * d_q, d_k    [T, Hq, d], [T, Hk, d] in_dtype, token strides lddq, lddk
 * d_wq, d_wk  [d] fp32 or NULL (gradient not wanted; must be NULL where the
 *             weight is NULL).  T == 0 sets them to zero.
 * workspace   gdn_qk_norm_backward_workspace_bytes bytes, 16-byte aligned, or
 *             NULL when neither d_wq nor d_wk is wanted
 * Outputs must not overlap the inputs.
 */
int gdn_qk_norm_backward(const void* q, int64_t ldq, const void* k, int64_t ldk, int in_dtype,
                         int64_t T, int Hq, int Hk, int d, int norm, float eps, const float* wq,
                         const float* wk, const int32_t* positions, const float* inv_freq,
                         int rot_dim, int interleaved, const void* d_oq, int64_t lddoq,
                         const void* d_ok, int64_t lddok, int grad_dtype, void* d_q,
                         int64_t lddq, void* d_k, int64_t lddk, float* d_wq, float* d_wk,
                         void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_QK_NORM_H */
