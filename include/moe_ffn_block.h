/*
 * moe_ffn_block.h -- C ABI of the dense gated feed-forward block and of the
 * MXFP4 operators (sm_103a).
 *
 * The block is the FFN that stands between MoE layers and beside their routed
 * experts:  out = (act(x W1^T) * (x W3^T)) W2^T  for m tokens, with
 *   x [m, H], W1, W3 [I, H], W2 [H, I] (out, in), bf16 or MXFP4 weights, and
 *   for bf16 weights its backward pass.
 * Conventions as in moe_ffn.h: device pointers, caller-owned buffers, no
 * allocation, no synchronisation (every call can be captured in a CUDA
 * graph), MOE_OK or an error status, m == 0 launches nothing, results
 * deterministic.  Pointers are 16-byte aligned.  Outputs share no memory with
 * inputs, but out may be x (or lie in it) in moe_ffn_forward and moe_mxfp4_linear.
 *
 * MXFP4 (OCP Microscaling Formats v1.0): e2m1 codes (magnitudes 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6), two per byte, element 2j in the low nibble of byte j; one
 * e8m0 scale 2^(s - 127) per 32 contiguous elements of a row (s = 255: NaN).
 * Quantisation of a block with largest magnitude a:
 *   s = max(floor(log2 a) - 2 + 127, 0);  code = e2m1(v / 2^(s - 127)), round
 *   to nearest even, saturating at +-6; all-zero blocks get s = 0; a block
 *   that holds an infinity or a NaN gets s = 255 and zero codes.
 * The scales of a [rows, n] matrix are kept in the order the tensor core's
 * scale copies read them: tiles of 128 rows x 4 blocks, 512 bytes each, tile
 * (r / 128, b / 4) after tile in row-major order, and inside a tile the scale of
 * row r, block b at byte (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4:
 * moe_mxfp4_scales_size bytes.  The blocks that pad a row to a multiple of 4
 * must hold 0; what pads the rows to a multiple of 128 is never used.
 */
#ifndef MOE_FFN_BLOCK_GB300_H
#define MOE_FFN_BLOCK_GB300_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- activations: act(g) = g s(t(g)), s(t) = 1 / (1 + exp(-t)) */
#define MOE_ACT_SILU 0      /* t = g */
#define MOE_ACT_GELU_TANH 1 /* t = 2 sqrt(2/pi) (g + 0.044715 g^3): gelu, tanh form */

/* Block weight format besides MOE_WEIGHTS_BF16: codes uint8 [rows, n/2] and
 * packed scales as above. */
#define MOE_WEIGHTS_MXFP4 3

typedef struct moe_ffn_config {
    int32_t hidden;     /* H: multiple of 8 (bf16) or 32 (MXFP4), 8 .. 2^20 */
    int32_t inter;      /* I: the same */
    int32_t activation; /* MOE_ACT_* */
    int32_t weights;    /* MOE_WEIGHTS_BF16 or MOE_WEIGHTS_MXFP4 */
} moe_ffn_config;

/* s1, s3, s2: packed scales of MXFP4 weights, NULL for bf16.  The weights
 * must outlive the handle; they may be rewritten in place between calls. */
typedef struct moe_ffn_weights {
    const void* w1;
    const void* w3;
    const void* w2;
    const uint8_t* s1;
    const uint8_t* s3;
    const uint8_t* s2;
} moe_ffn_weights;

typedef struct moe_ffn moe_ffn;

/* A handle on the current device: the config, the weight pointers and their
 * TMA descriptors.  It owns no device memory. */
MOE_API int moe_ffn_create(const moe_ffn_config* cfg, const moe_ffn_weights* weights, moe_ffn** out);
MOE_API int moe_ffn_destroy(moe_ffn* ffn);

/* Workspace bytes a forward (backward = 0) or backward (1) call on m tokens
 * needs, never fewer for more tokens; 256-byte aligned.  Its first 256 bytes are the header of moe_ffn.h,
 * read and cleared by moe_device_status; a handle zeroes it when a call
 * passes a workspace other than its previous call's, as in moe_ffn.h. */
MOE_API int moe_ffn_workspace_size(const moe_ffn* ffn, int64_t m, int backward, size_t* bytes);

/* Bytes that a forward pass on m tokens saves for the backward pass: 10 for each
 * element of [m, I] (two fp32 and one bf16), m and I rounded up to 32 in the fp32
 * parts. */
MOE_API int moe_ffn_saved_size(const moe_ffn* ffn, int64_t m, size_t* bytes);

/* out[t, :] = the block applied to x[t, :].
 *   x bf16 [m, H] with row stride ldx >= H (a multiple of 8); out bf16 [m, H].
 *   saved (bf16 weights only, else NULL): NULL, or moe_ffn_saved_size bytes,
 *   32-byte aligned, that receive what moe_ffn_backward needs: with g = x W1^T
 *   and u = x W3^T, act(g) and u act'(g) in fp32 (rounded to bf16 they would be
 *   the largest error of the gradients), each [ceil(m / 32), ceil(I / 32), 4, 32, 8]
 *   with row r, column c at [r / 32, c / 32, c % 32 / 8, r % 32, c % 8] (what pads
 *   m and I is left as it is), then h = act(g) u, bf16 [m, I].
 * Sums are fp32.  h, an operand of the down product, is rounded to bf16, which is
 * what the tensor core multiplies; up to 8 tokens whose h is not saved go on in
 * two bf16 parts (16 bits), which the tensor core has columns to spare for.  So up
 * to 8 tokens a call that saves and one that does not differ by h's rounding, and
 * from 9 on a result's error against exact arithmetic is 2.3e-3 of it (relative
 * L2) where rounding the result alone makes 1.7e-3.  dg and du are rounded to bf16
 * alike.  MXFP4: x and h are rounded to MXFP4, h straight from the fp32 sums. */
MOE_API int moe_ffn_forward(const moe_ffn* ffn, const void* x, int64_t ldx, int64_t m, void* out, void* saved,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of the block, given dout = dL/dout and what forward saved:
 *   dh = dout W2 (fp32), dg = dh u act'(g), du = dh act(g) (bf16)
 *   dx = dg W1 + du W3   dw1 = dg^T x   dw3 = du^T x   dw2 = dout^T h
 *   dout bf16 [m, H] with row stride ldd, x as in forward; dx bf16 [m, H];
 *   dw1, dw3 bf16 [I, H]; dw2 bf16 [H, I], all overwritten.  dx may be NULL,
 *   and dw1, dw3, dw2 may all three be NULL (gradients not wanted).
 * bf16 weights only (MOE_ERR_UNSUPPORTED otherwise).  m == 0 writes nothing:
 * weight gradients are then left as they are. */
MOE_API int moe_ffn_backward(const moe_ffn* ffn, const void* dout, int64_t ldd, const void* x, int64_t ldx,
                             const void* saved, int64_t m, void* dx, void* dw1, void* dw3, void* dw2,
                             void* workspace, size_t workspace_bytes, void* stream);

/* As moe_layer_set_wait_limit and moe_layer_stall_test: the limit (ns; 0: 2 s)
 * of every bounded wait in the handle's kernels, and the test of the failure
 * path, in which their tensor-core issuers first wait on a barrier that nothing
 * completes.  A wait that runs out leaves DEV_ERR_TIMEOUT (2) in the workspace's
 * error word, and that call's outputs unspecified. */
MOE_API int moe_ffn_set_wait_limit(moe_ffn* ffn, uint64_t ns);
MOE_API int moe_ffn_stall_test(moe_ffn* ffn, int enable);

/* Kernels the last successful call on `ffn` launched. */
MOE_API int moe_ffn_last_launch_count(const moe_ffn* ffn);

/* Bytes of the packed scales of a [rows, n] matrix; n a multiple of 32. */
MOE_API int moe_mxfp4_scales_size(int64_t rows, int64_t n, size_t* bytes);

/* x [rows, n] (bf16, or fp32 for _f32; row stride ldx >= n elements, rows
 * 16-byte aligned) to MXFP4: codes uint8 [rows, n/2], scales packed.  At most
 * 2^26 pieces of 512 elements of a row (2^35 elements in full pieces), here and
 * in moe_mxfp4_dequant. */
MOE_API int moe_mxfp4_quant(const void* x, int64_t ldx, int64_t rows, int64_t n, uint8_t* codes, uint8_t* scales,
                            void* stream);
MOE_API int moe_mxfp4_quant_f32(const float* x, int64_t ldx, int64_t rows, int64_t n, uint8_t* codes,
                                uint8_t* scales, void* stream);

/* The values codes and scales stand for, bf16 [rows, n]: exact but for those past
 * bf16's range, which are infinite (scale 253 with a code of 4 or 6, 254 with one
 * of 2 or more). */
MOE_API int moe_mxfp4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t n, void* out,
                              void* stream);

/* out[t, j] = sum_k A[t, k] B[j, k], fp32 sums rounded once to bf16:
 *   A [m, k] and B [n, k] in MXFP4 (codes and packed scales), out bf16 [m, n];
 *   k a multiple of 32, n a multiple of 8.
 * workspace: moe_mxfp4_gemm_workspace_size bytes, 256-byte aligned, its first
 * 256 bytes (the header) zero before its first use. */
MOE_API int moe_mxfp4_gemm_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes);
MOE_API int moe_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, const uint8_t* b_codes,
                           const uint8_t* b_scales, int64_t n, int64_t k, void* out, void* workspace,
                           size_t workspace_bytes, void* stream);

/* moe_mxfp4_quant of x [m, k] (bf16, or fp32 for _f32; row stride ldx), kept in
 * the workspace, then moe_mxfp4_gemm of it with W [n, k]: out bf16 [m, n].
 * Workspace as for moe_mxfp4_gemm, moe_mxfp4_linear_workspace_size bytes. */
MOE_API int moe_mxfp4_linear_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes);
MOE_API int moe_mxfp4_linear(const void* x, int64_t ldx, int64_t m, const uint8_t* w_codes, const uint8_t* w_scales,
                             int64_t n, int64_t k, void* out, void* workspace, size_t workspace_bytes, void* stream);
MOE_API int moe_mxfp4_linear_f32(const float* x, int64_t ldx, int64_t m, const uint8_t* w_codes,
                                 const uint8_t* w_scales, int64_t n, int64_t k, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FFN_BLOCK_GB300_H */
