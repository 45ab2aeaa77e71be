// Dense gated feed-forward block and MXFP4 operators: host interface of their
// kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ffn_block.h"

namespace moe {

struct WsHeader;

// What a product's epilogue makes of its fp32 sums.
enum FfnEpilogue : int {
    EPI_STORE = 0,    // out = D
    EPI_GATEUP,       // D = (g, u) side by side: out = act(g) u
    EPI_GATEUP_SAVE,  // ... and a = act(g), d = u act'(g) for the backward pass
    EPI_DACT,         // D = dh: out = dg = dh d, du = dh a
};

// How an operand lies in memory: along K; along M (N), as boxes of 64 x 64, or
// (multiples of 64) two of these at a time.
enum FfnOrder : int { K_MAJOR = 0, MN_ROWS, MN_BLOCKS };

// One product D[M, N] = sum over one or two sources of A B^T, as a work list
// of 256 x 256 tiles (gate/up: 256 rows x 128 columns of g and of u).
struct FfnProduct {
    CUtensorMap a[2], b[2];  // per source (gate/up: b = W1, W3, one source)
    int a_mn, b_mn;          // FfnOrder of the operands
    int kblocks;             // 64-wide K blocks per source
    int sources;
    int m_tiles, n_tiles;
    int M, N;
    uint16_t* out;           // [M, N], row stride N
    CUtensorMap o;           // ... of a plain product, in boxes of 64 columns x 32 rows (set by launch_ffn_products)
};
constexpr int kMaxProducts = 4;
struct FfnProducts {
    FfnProduct p[kMaxProducts];  // longest reductions (sources * kblocks) first
    int count;
    int first[kMaxProducts + 1];  // first work item of each product; set by launch_ffn_products, as are
    int dear, fill;               // ... the order of the items (ffn_wide.cu, Turns)
    int act;
    // a = act(g) and d = u act'(g), fp32, in the order of saved_at: written by EPI_GATEUP_SAVE, read by EPI_DACT
    float *a, *d;
    uint16_t* out_du;       // EPI_DACT (out: dg)
    WsHeader* hdr;
    uint64_t wait_ns;  // limit of every protocol wait
    int stall;         // 1: the issuer first waits on a barrier nothing completes
};

// Maps of a bf16 operand [rows, cols] (row stride ld elements), all even, as
// 32-bit words in three dimensions.  K-major: (word, row, 0), boxes of 64 of K
// x box_rows rows.  ffn_map_mn: MN-major, 64 of M x 64 rows of K; returns the
// order it chose (K_MAJOR: an error).
bool ffn_map(CUtensorMap* m, const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows);
int ffn_map_mn(CUtensorMap* m, const void* p, uint64_t rows, uint64_t cols, uint64_t ld);

cudaError_t launch_ffn_products(FfnProducts& p, int epilogue, cudaStream_t st);

// One MXFP4 product (codes and packed scales of both sides).
struct MxProduct {
    CUtensorMap a, as;        // codes [M, K/2], scale tiles
    CUtensorMap b[2], bs[2];  // one matrix, or W1 and W3 (gate/up)
    int kblocks;              // ceil(K / 256)
    int m_tiles, n_tiles;
    int M, N;
    int act;
    uint16_t* out;            // plain: bf16 [M, N]
    CUtensorMap o;            // ... its map (set by launch_mx_product)
    uint8_t *codes, *scales;  // gate/up: h as MXFP4, [M, N/2] and packed scales
    int nkt;                  // ... scale tiles per row of it
    WsHeader* hdr;
    uint64_t wait_ns;  // limit of every protocol wait
    int stall;         // 1: the issuer first waits on a barrier nothing completes
};
bool mx_code_map(CUtensorMap* m, const void* codes, uint64_t rows, uint64_t k, uint32_t box_rows);
bool mx_scale_map(CUtensorMap* m, const void* scales, uint64_t rows, uint64_t k);
cudaError_t launch_mx_product(MxProduct& p, bool gateup, cudaStream_t st);

// One product for few tokens, out[T, R] = tokens W^T, weights as the MMA's M
// operand.
enum NarrowKind : int {
    NARROW_PLAIN = 0,
    NARROW_GATEUP,  // W1 and W3: h
    NARROW_DACT,    // dout W2, W2 along M: dg and du
    NARROW_DX,      // dg W1 + du W3, both along M
    // at most kNarrowParts tokens: h written, and read, in two bf16 parts, rows t and 8 + t
    NARROW_GATEUP_PARTS,
    NARROW_PLAIN_PARTS,
};
struct NarrowProduct {
    CUtensorMap a[2], as[2];  // weights (128-row boxes) and, MXFP4, their scales
    CUtensorMap b[2], bs;     // tokens (narrow_tokens(T)-row boxes; NARROW_DX: dg, du) and their scales
    const uint16_t* x;        // MXFP4 weights, at most kNarrowQuant tokens: bf16 tokens in place of b and bs,
    size_t ldx;               // ... quantised by the kernel itself; else null
    int a_mn;                 // FfnOrder of weights along M
    int T, R, K;
    int early;                // the preceding kernel wrote only the tokens: weights may be read before it ends
    int act;
    uint16_t *out, *du;       // bf16 [T, R]; gate/up of a bf16 block: h; NARROW_DACT: dg, du
    float *sa, *sd;           // act(g) and u act'(g) (saved_at): NARROW_GATEUP writes them unless null, NARROW_DACT reads
    uint8_t *codes, *scales;  // gate/up of an MXFP4 block: h
    int nkt;                  // ... scale tiles per row of it
    WsHeader* hdr;
    uint64_t wait_ns;  // limit of every protocol wait
    int stall;         // 1: the issuer first waits on a barrier nothing completes
    // set by launch_ffn_narrow
    int nt, kstages, slices, stages, ring_bytes, tmem_cols;
};
bool narrow_is_faster(int m, int R, bool mx);  // than the 256 x 256 tiles, for out [m, R]
constexpr int kNarrowQuant = 16, kNarrowParts = 8;
int narrow_tokens(int m);           // rows of a token tile
cudaError_t launch_ffn_narrow(NarrowProduct& p, bool mx, int kind, cudaStream_t st);

cudaError_t launch_mx_quant(const void* x, bool f32, size_t ldx, int rows, int n, uint8_t* codes, uint8_t* scales,
                            cudaStream_t st);
cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int rows, int n, uint16_t* out,
                              cudaStream_t st);

}  // namespace moe
