/*
 * moe_ffn_ops.h -- C ABI of the operators around the layer and the block
 * (sm_103a): the norm in front of them with the residual's addition, the
 * router's losses and its gradient, and low-rank adapters beside a projection.
 *
 * Conventions as in moe_ffn.h: device pointers of the current device,
 * caller-owned buffers, no allocation, no synchronisation (every call can be
 * captured in a CUDA graph), MOE_OK or an error status, results deterministic,
 * m == 0 launches nothing.  bf16 rows (and e4m3 codes) are 16-byte aligned with
 * strides in elements, multiples of 8 and at least the row; fp32 and int32
 * tensors are dense and aligned to their elements where nothing else is said.
 * Outputs share no memory with inputs or with each other but where it is said
 * (rows of one buffer whose columns do not meet share none).  Refused for it are
 * the norm's rows, codes and scales, dx with dout, r and dresidual, dlogits with
 * logits, and the adapters' out with x and y; other pointers (weights, ids, counts,
 * losses, workspaces) are not compared.  Up to 2^31 / 64 tokens.
 */
#ifndef MOE_FFN_OPS_GB300_H
#define MOE_FFN_OPS_GB300_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* RMSNorm of x, or of its sum with a residual:
 *   r[t,:]   = bf16(x[t,:] + residual[t,:])      (x itself where residual is NULL)
 *   out[t,:] = r[t,:] / sqrt(sum_h r[t,h]^2 / h + eps) * weight
 *   x bf16 [m, h] (row stride ldx); residual bf16 [m, h] (ldr) or NULL, with it
 *   residual_out (ldo), which receives r and may be residual (with the same
 *   stride); weight fp32 [h], 16-byte aligned; eps finite, >= 0.
 *   out bf16 [m, h] or NULL; it may be x (ldx == h).
 *   codes uint8 [m, h] (e4m3) and scales fp32 [m, ceil(h / 128)], both or
 *   neither: out in 8 bits as moe_act_quant_fp8 makes them, s = amax / 448 per
 *   128 columns (the last block may be shorter; s = 1 and codes 0 also where
 *   amax / 448 is below fp32's numbers), but of out before it is rounded to
 *   bf16.  A row that holds an infinity or a NaN has NaN codes, at the NaN of
 *   out.  One of out and codes is wanted at least.
 *   h a multiple of 8, up to 24576.
 * The norm is taken of the rounded r, as moe_forward_residual_rmsnorm takes it.
 * Sums are fp32: a row whose squares pass its range (|r| from about 1e19 on)
 * comes out as zeros, and one whose squares fall below it counts as one of zeros,
 * which only an eps of 0 shows (|r| below about 1e-19 loses bits, below 1e-23 out is
 * infinite). */
MOE_API int moe_add_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t m, int64_t h,
                            const float* weight, float eps, void* residual_out, int64_t ldo, void* out, uint8_t* codes,
                            float* scales, void* stream);

/* Its gradients, given dout = dL/dout and the r that was normalised: with
 * rstd = 1 / sqrt(sum r^2 / h + eps), n = r rstd, g = dout weight,
 *   dx      = rstd (g - n sum_h(g n) / h) + dresidual
 *   dweight = sum_t dout n                          (fp32 [h])
 *   dout, r bf16 [m, h] (ldd, ldr); dresidual bf16 [m, h] (ldq) or NULL: what
 *   else flows into r; dx bf16 [m, h], the gradient of x and of the residual
 *   alike; it may be dout (ldd == h) or dresidual (ldq == h).  dweight may be
 *   NULL (not wanted).  m == 0 leaves dweight as it is.
 * workspace: moe_add_rmsnorm_backward_workspace_size bytes, 256-byte aligned
 * (NULL where dweight is NULL); it has no header and keeps nothing. */
MOE_API int moe_add_rmsnorm_backward_workspace_size(int64_t m, int64_t h, size_t* bytes);
MOE_API int moe_add_rmsnorm_backward(const void* dout, int64_t ldd, const void* r, int64_t ldr, int64_t m, int64_t h,
                                     const float* weight, float eps, const void* dresidual, int64_t ldq, void* dx,
                                     float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/* What keeps a router's experts in use.  logits fp32 [m, e] and topk_ids int32
 * [m, k] as moe_route gives them; sequences of tokens [seq_offsets[s],
 * seq_offsets[s + 1]), s < seqs, int32 and not falling, from 0 to at most m
 * (NULL: one sequence of all m tokens, seqs == 1).  Tokens in no sequence are
 * padding.  For a sequence of T tokens:
 *   counts[s,i] = its pairs (t, j) with topk_ids[t,j] == i; ids outside [0, e)
 *                 count nowhere (-1 marks a dropped pair)
 *   p[t,:]      = softmax(logits[t,:]), or for MOE_SCORING_SIGMOID
 *                 sigmoid(logits[t,:]) over its sum
 *   balance[s]  = e / (k T^2) sum_i counts[s,i] sum_t p[t,i]
 *   z[s]        = 1 / T sum_t log(sum_i exp(logits[t,i]))^2
 * An empty sequence has zeros.  A token whose logits are all -inf has p = 0 and
 * no part in z; one with a NaN makes its sequence's losses NaN, one with a +inf its
 * z and, of softmax, its balance.
 * counts int32 [seqs, e]; balance, z fp32 [seqs].  e in 1..1024,
 * k in 1..min(e, 32), seqs in 1..2^24.  Offsets that fall or leave [0, m] give
 * unspecified values, and touch nothing outside the tensors.
 * workspace: moe_balance_loss_workspace_size bytes, 256-byte aligned; it has no
 * header and keeps nothing. */
MOE_API int moe_balance_loss_workspace_size(int64_t m, int64_t seqs, size_t* bytes);
MOE_API int moe_balance_loss(const float* logits, const int32_t* topk_ids, int64_t m, int32_t e, int32_t k,
                             const int32_t* seq_offsets, int64_t seqs, int scoring, float* balance, float* z,
                             int32_t* counts, void* workspace, size_t workspace_bytes, void* stream);

/* The gradient of the logits, dlogits fp32 [m, e], all of it written: what
 * flows back through the routing weights and through the two losses.
 *   dtopk_w fp32 [m, k] or NULL: gradient of moe_route's topk_w (softmax over
 *     the picks; sigmoid: renormalised where norm_topk_prob is 1, times
 *     routed_scaling_factor).  Ids outside [0, e) have none and are left out of
 *     the sum that renormalises; picks that name one expert twice add up.
 *   dbalance, dz fp32 [seqs] or NULL: gradients of balance[s] and z[s]; counts
 *     int32 [seqs, e] as moe_balance_loss gave them (needed with dbalance; the
 *     counts are constants).
 * seq_offsets and seqs as above; padding tokens have the first part alone.  The
 * gradients of the router's operands are then products with dlogits:
 * drouter_w = dlogits^T x, dx = dlogits router_w. */
MOE_API int moe_route_backward(const float* logits, const int32_t* topk_ids, int64_t m, int32_t e, int32_t k,
                               int scoring, int norm_topk_prob, float routed_scaling_factor, const float* dtopk_w,
                               const int32_t* seq_offsets, int64_t seqs, const int32_t* counts, const float* dbalance,
                               const float* dz, float* dlogits, void* stream);

/* Low-rank adapters of many requests beside a projection they share:
 *   out[t,:] = y[t,:] + scale[i] B_i (A_i x[t,:]),  i = ids[t]
 * in fp32 sums, out rounded once.  ids int32 [m]; -1: no adapter (out[t,:] is
 * y[t,:], bit for bit); any other id outside [0, n) sets the device error word and
 * counts as -1.
 * By tiles of 128 tokens (above MOE_LORA_BY_TOKEN tokens, sooner or later by r and
 * n) scale[i] A_i x[t] goes into the second product as two bf16 parts, 16 bits of
 * it, and infinities in b may then make NaN.  Which way and in which slices of k
 * depends on m, k, n and r alone: for the same sizes a token's result does not
 * depend on the others' adapters, bit for bit.
 *   x bf16 [m, k] (ldx); y bf16 [m, d] (ldy), the projection's output; out bf16
 *   [m, d] (ldo), which may be y (with the same stride); a bf16 [n, r, k], b
 *   bf16 [n, d, r]: the adapters stacked, smaller ranks padded with zeros; scale
 *   fp32 [n] or NULL (1).
 *   r a multiple of 8 up to 128; k and d multiples of 8 up to 2^20; n r up to
 *   2^30.
 * workspace: moe_lora_add_workspace_size bytes, 256-byte aligned, its first 256
 * bytes (the header of moe_ffn.h) zero before its first use.  Every wait of the
 * kernels is bounded (moe_lora_set_wait_limit): moe_device_status. */
#define MOE_LORA_BY_TOKEN 64 /* up to so many tokens it is the header alone */
MOE_API int moe_lora_add_workspace_size(int64_t m, int64_t k, int64_t r, size_t* bytes);
MOE_API int moe_lora_add(const void* x, int64_t ldx, int64_t m, int64_t k, const void* y, int64_t ldy, int64_t d,
                         const void* a, const void* b, int64_t n, int64_t r, const int32_t* ids, const float* scale,
                         void* out, int64_t ldo, void* workspace, size_t workspace_bytes, void* stream);

/* As moe_layer_set_wait_limit and moe_layer_stall_test, of every moe_lora_add of
 * the process from then on, as adapters have no handle: the limit (ns; 0: 2 s) of
 * each bounded wait in the kernels that take many tokens, and the test of their
 * failure path, in which the tensor-core issuer of the first (1: A x) or second
 * (2: B times it) first waits on a barrier that nothing completes (0: neither).  A
 * wait that runs out leaves DEV_ERR_TIMEOUT (2) in the workspace's error word, and
 * that call's out unspecified. */
MOE_API int moe_lora_set_wait_limit(uint64_t ns);
MOE_API int moe_lora_stall_test(int kernel);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FFN_OPS_GB300_H */
