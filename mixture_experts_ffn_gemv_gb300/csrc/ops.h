// Operators around the layer and the block (include/moe_ffn_ops.h): host
// interface of their kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ffn_ops.h"

namespace moe {

struct WsHeader;

constexpr int kNormMaxH = 24576;  // widest row of the norm kernels: 1024 threads x 3 x 8 columns

// r = bf16(x + res), out = r rstd w, codes and scales of out; res, out, codes null: not wanted.
struct NormArgs {
    const uint16_t *x, *res;
    int64_t ldx, ldr, ldo;  // row strides of x, res, res_out (elements)
    const float* w;
    float eps;
    uint16_t *res_out, *out;
    uint8_t* codes;
    float* scales;
    int m, H;
};
cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t st);

// dx = rstd (g - n mean(g n)) + dres, dw = sum over rows of dout n; dres, dw null: none.
struct NormGradArgs {
    const uint16_t *dout, *r, *dres;
    int64_t ldd, ldr, ldq;  // row strides of dout, r, dres
    const float* w;
    float eps;
    uint16_t* dx;
    float* dw;
    float* part;  // [norm_grad_blocks(m, H), H] when dw is wanted
    int m, H;
};
int norm_grad_blocks(int m, int H);
cudaError_t launch_add_rmsnorm_backward(const NormGradArgs& a, cudaStream_t st);

// Router losses of sequences of tokens, [off[s], off[s + 1]) of m (off null: one sequence, all m).
struct RouterArgs {
    const float* logits;   // [m, E]
    const int32_t* ids;    // [m, k], outside [0, E): no pair
    const int32_t* off;    // [S + 1] or null
    int m, E, k, S;
    int sigmoid;
    int32_t* counts;       // [S, E]: written by launch_balance_loss, read by launch_route_backward
    // losses
    float *balance, *z;    // [S]
    float2* part;          // [balance_slots(m, S)]: sums of a chunk's tokens of a sequence
    int* ticket;           // [S]: chunks of a sequence that are summed
    // gradients; null: that part is not wanted
    const float *dtopk_w;  // [m, k]
    const float *dbalance, *dz;  // [S]
    int norm;              // sigmoid scoring: the weights are renormalised
    float scale;           // ... and multiplied by this
    float* dlogits;        // [m, E]
    int chunk;             // tokens of a block; set by the launches
};
int64_t balance_slots(int64_t m, int64_t S);
cudaError_t launch_balance_loss(RouterArgs a, cudaStream_t st);
cudaError_t launch_route_backward(RouterArgs a, cudaStream_t st);

// out[t] = y[t] + scale[i] B_i A_i x[t], i = ids[t] (-1: out[t] = y[t]).
struct LoraArgs {
    const uint16_t *x, *y, *a, *b;  // A [n, r, K], B [n, N, r]
    uint16_t* out;
    const float* scale;             // [n] or null: 1
    const int32_t* ids;
    int64_t ldx, ldy, ldo;
    int m, K, N, r, n;
    WsHeader* hdr;
    uint64_t wait_ns;  // limit of every protocol wait
    int stall;         // 1, 2: the issuer of lora_shrink, lora_expand first waits on a barrier nothing completes
    // tiles of tokens: set by launch_lora_tiles
    float* part;       // [splits, m, r]: A x by slices of K
    int splits, kblocks, split_blocks;
    int group;         // adapters whose products share a pass over x
    int n_tiles, n_ctas;  // expand: tiles of N, blocks that share them
    int stages;           // ... stages of B
    CUtensorMap mx, ma, mb, my, mo;
};
constexpr int kLoraMaxRank = 128;
constexpr int kLoraByToken = MOE_LORA_BY_TOKEN;  // up to so many tokens always a cluster each
bool lora_by_token(int m, int n, int r);  // which of the two kernels
int64_t lora_part_floats(int64_t m, int64_t r);  // never fewer for more tokens
cudaError_t launch_lora_tokens(const LoraArgs& a, cudaStream_t st);
cudaError_t launch_lora_tiles(LoraArgs& a, cudaStream_t st);

}  // namespace moe
