// Products of the gated feed-forward block for few tokens: every weight is read
// once, so the time is that of streaming the weights.
//
// Both products of a block of 7168 x 2048, weights from HBM: bf16 (88 MB) 24 us
// for 48 tokens (3.7 TB/s over all), 21 for one; MXFP4 (23 MB) 16 and 12 to 14.
// What is not streaming is the two kernels' start and end.
//
// The operands change places: 128 weight rows are the MMA's M, the tokens
// (16 .. 128, a multiple of 16) its N, so no tensor-core row is wasted and a
// CTA's shared memory holds almost nothing but weights in flight.  One CTA
// takes 128 rows (gate/up: 128 of W1 and the same 128 of W3) and one slice of
// K; the slices of a row tile are the CTAs of a cluster.  Each leaves its fp32
// sums in its own shared memory, and the cluster adds them up, slice by slice
// in a fixed order, through distributed shared memory: the split costs no
// global traffic and the result does not depend on who comes first.
//   warp 0     TMA producer; it fills the ring with weights before it waits
//              for the preceding kernel where that one wrote only the tokens,
//              so that the stream of weights starts while that kernel drains;
//   warp 1     MMA issuer (and, MXFP4, the scale copies to tensor memory);
//   warps 2..  where bf16 tokens meet MXFP4 weights (up to 16 tokens): quantise
//              each stage's piece of them straight into the ring, which saves
//              the quantiser's launch;
//   all warps  the sum over slices and the epilogue, a warp per token, four rows
//              per lane: eight lanes hold one block of an MXFP4 h.
// Up to 8 tokens' h goes from gate/up to down in two bf16 parts (h and what its
// rounding left, 16 bits together): 8 + 8 rows of the smallest token tile, so
// the second part costs four MMAs of 16 columns per K block and no bandwidth
// (they read past the tile: ring_margin).
// A stage holds two weight tiles of 128 bytes of K: W1 and W3 (which share the
// tokens); two neighbours along K; or a tile of each source, with its tokens,
// of dx = dg W1 + du W3.  The backward products read the weights as they lie,
// 64 of K x 128 of M.  Bounded waits as in ffn_wide.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "ffn_act.cuh"
#include "ffn_block.h"
#include "ffn_box.cuh"
#include "launch.cuh"
#include "mxfp4.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace moe {

namespace {

using namespace sm100;

constexpr int TILE = 128 * 128;  // 128 rows x 128 bytes of K
constexpr int WARPS = 10, THREADS = 32 * WARPS;
constexpr int MAX_STAGES = 8;
constexpr int MAX_SLICES = 8;  // the portable cluster size
constexpr uint64_t DRAIN_NS = 2000000000ull;

// bf16; MXFP4 on both sides; the same from bf16 tokens, quantised on the way.
enum : int { FMT_BF16 = 0, FMT_MXFP4, FMT_MXFP4_QUANT };
constexpr int QUANT_WARPS = WARPS - 2;

// Byte offsets inside a stage.
struct StageShape {
    int tok, sa, sb, bytes;
};
// tok: the token tile(s); sa, sb: scales of the weights and of the tokens.
__host__ __device__ inline StageShape stage_shape(bool mx, int kind, int nt) {
    const bool gateup = kind == NARROW_GATEUP || kind == NARROW_GATEUP_PARTS;
    StageShape s;
    s.tok = 2 * TILE;
    s.sa = s.tok + (gateup ? 1 : 2) * nt * 128;
    s.sb = s.sa + (mx ? 2048 : 0);
    s.bytes = s.sb + (mx ? (gateup ? 1024 : 2048) : 0);
    return s;
}
__host__ __device__ inline int stage_stride(const StageShape& s) { return (s.bytes + 1023) & ~1023; }

// The MMA of a second part starts kNarrowParts rows into a token tile and takes
// the smallest N, 16 columns: its last kNarrowParts rows lie past the tile.
// What they hold does not matter (they make columns of D that are never read),
// but they are read, so that this much shared memory has to follow the ring.
constexpr int PARTS_N = 16, ROW_BYTES = 128;
constexpr int PARTS_MARGIN = kNarrowParts * ROW_BYTES;
__host__ __device__ constexpr int ring_margin(int kind) { return kind == NARROW_PLAIN_PARTS ? PARTS_MARGIN : 0; }
static_assert((kNarrowParts + PARTS_N) * ROW_BYTES == PARTS_N * ROW_BYTES + PARTS_MARGIN,
              "a second part's MMA ends within the token tile and the margin behind it");
static_assert(2 * kNarrowParts <= PARTS_N, "both parts' rows fit a token tile");

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ void add4(float (&a)[4], const float4& v) {
    a[0] += v.x;
    a[1] += v.y;
    a[2] += v.z;
    a[3] += v.w;
}

// h's second part where hi is the first: 0 where that is infinite (or a NaN),
// since an infinity less itself would make the sum of both a NaN.
__device__ __forceinline__ float second_part(float h, float hi) {
    return fabsf(hi) < __int_as_float(0x7f800000) ? h - hi : 0.f;
}

template <int FMT, int KIND>
__global__ void __launch_bounds__(THREADS, 2) ffn_narrow(const __grid_constant__ NarrowProduct p) {
    constexpr bool MX = FMT != FMT_BF16, QUANT = FMT == FMT_MXFP4_QUANT;
    constexpr bool GATEUP = KIND == NARROW_GATEUP || KIND == NARROW_GATEUP_PARTS;  // two accumulators, one token tile
    constexpr bool PARTS = KIND == NARROW_GATEUP_PARTS || KIND == NARROW_PLAIN_PARTS;
    constexpr bool SOURCES = KIND == NARROW_DX;         // a stage's tiles: two sources, not two K blocks
    constexpr bool MN = KIND == NARROW_DACT || KIND == NARROW_DX;  // weights along M
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const StageShape ss = stage_shape(MX, KIND, p.nt);
    const int stride = stage_stride(ss);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.ring_bytes + ring_margin(KIND));
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + MAX_STAGES), done = smem_u32(bars + 2 * MAX_STAGES);
    const uint32_t never = smem_u32(bars + 2 * MAX_STAGES + 1);  // stall test: no thread ever arrives here
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * MAX_STAGES + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.slices;
    const uint32_t rank = cluster_ctarank();
    const int tile = blockIdx.x / S;
    const int row0 = tile * 128, tok0 = blockIdx.y * p.nt;
    const int k0 = (int)((int64_t)p.kstages * rank / S), k1 = (int)((int64_t)p.kstages * (rank + 1) / S);
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full0 + 8 * s, QUANT ? 1 + QUANT_WARPS : 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(done, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
        tmem_relinquish();
    }
    if (warp == 2 && lane < 2) {
        prefetch_tmap(&p.a[GATEUP || SOURCES ? lane : 0]);
        if (!QUANT) prefetch_tmap(&p.b[SOURCES ? lane : 0]);
        if (MX) prefetch_tmap(&p.as[GATEUP ? lane : 0]);
        if (MX && !QUANT) prefetch_tmap(&p.bs);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t sf0 = tmem_base + (GATEUP ? 2 : 1) * p.nt;  // scale columns, 32 per stage
    if (!p.early) pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        // the whole warp's loop, one lane's body: as in ffn_wide.cu
        const CUtensorMap *a0 = &p.a[0], *a1 = &p.a[GATEUP || SOURCES ? 1 : 0];
        const CUtensorMap *b0 = &p.b[0], *b1 = &p.b[SOURCES ? 1 : 0];
        const CUtensorMap *s0 = &p.as[0], *s1 = &p.as[GATEUP ? 1 : 0];
        const BoxWalk w(MN ? p.a_mn : K_MAJOR, row0);
        const auto weights = [&](int ks, uint32_t st, uint32_t bar) {
            // K blocks (128 bytes) of the stage's two tiles
            const int ka = GATEUP || SOURCES ? ks : 2 * ks, kb = GATEUP || SOURCES ? ks : 2 * ks + 1;
            mbar_arrive_expect_tx(bar, QUANT ? 2 * TILE + 2048 : ss.bytes);
            tma_load_3d(st, a0, w.c0 + ka * w.d0, w.c1 + ka * w.d1, w.c2, bar);
            tma_load_3d(st + TILE, a1, w.c0 + kb * w.d0, w.c1 + kb * w.d1, w.c2, bar);
            if (MN && w.two) {
                tma_load_3d(st + TILE / 2, a0, w.c0 + 32, w.c1 + ka * w.d1, 0, bar);
                tma_load_3d(st + TILE + TILE / 2, a1, w.c0 + 32, w.c1 + kb * w.d1, 0, bar);
            }
            if (MX) {
                const int kt = (GATEUP ? 2 : 4) * ks;
                tma_load_3d(st + ss.sa, s0, 0, kt, tile, bar);
                tma_load_3d(st + ss.sa + 1024, s1, 0, GATEUP ? kt : kt + 2, tile, bar);
            }
        };
        const auto tokens = [&](int ks, uint32_t st, uint32_t bar) {
            if (QUANT) return;
            const int kc = (GATEUP || SOURCES ? ks : 2 * ks) * 32;  // words along K: 128 bytes are 32
            tma_load_3d(st + ss.tok, b0, kc, tok0, 0, bar);
            if (!GATEUP) tma_load_3d(st + ss.tok + p.nt * 128, b1, SOURCES ? kc : kc + 32, tok0, 0, bar);
            if (MX) {
                const int kt = (GATEUP ? 2 : 4) * ks;
                tma_load_3d(st + ss.sb, &p.bs, 0, kt, tok0 >> 7, bar);
                if (!GATEUP) tma_load_3d(st + ss.sb + 1024, &p.bs, 0, kt + 2, tok0 >> 7, bar);
            }
        };
        const int n = k1 - k0, pre = min(n, p.stages);
        bool ok = true;
        if (elect_one())
            for (int i = 0; i < pre; ++i) weights(k0 + i, sbase + i * stride, full0 + 8 * i);
        __syncwarp();
        if (p.early) pdl_wait();
        if (elect_one())
            for (int i = 0; i < pre; ++i) tokens(k0 + i, sbase + i * stride, full0 + 8 * i);
        __syncwarp();
        int i = pre, s = 0;
        uint32_t ph = 0;
        for (; i < n; ++i) {
            if (!warp_wait(empty0 + 8 * s, ph, p.wait_ns)) {
                ok = false;
                break;
            }
            if (elect_one()) {
                weights(k0 + i, sbase + s * stride, full0 + 8 * s);
                tokens(k0 + i, sbase + s * stride, full0 + 8 * s);
            }
            __syncwarp();
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (!ok && lane == 0) {
            set_error(p.hdr, DEV_ERR_TIMEOUT, 41);
            *abort_flag = 1;
        }
        for (int j = max(0, i - p.stages); j < i; ++j)  // every issued copy has landed
            mbar_wait(full0 + 8 * (j % p.stages), (j / p.stages) & 1u, DRAIN_NS);
    } else if (warp == 1) {
        bool ok = !p.stall || warp_wait(never, 0, p.wait_ns);
        const uint32_t idesc = idesc_bf16(128, p.nt) | (MN ? kIdescAMn : 0u);
        int s = 0;
        uint32_t ph = 0;
        for (int i = 0; ok && i < k1 - k0; ++i) {
            if (warp_sees(abort_flag) || !warp_wait(full0 + 8 * s, ph, p.wait_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t st = sbase + s * stride;
            const uint32_t sf = sf0 + s * 32;
            if (elect_one()) {
                if (MX) {
                    // 8 columns per weight tile (two K tiles of 128), then 8 per token tile
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int kt = 0; kt < 2; ++kt) {
                            tmem_cp_scales(sf + 8 * h + 4 * kt, desc_scales(st + ss.sa + h * 1024 + kt * 512));
                            if (h == 0 || !GATEUP)
                                tmem_cp_scales(sf + 16 + 8 * h + 4 * kt, desc_scales(st + ss.sb + h * 1024 + kt * 512));
                        }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t ad = MN ? desc_sw128_mn(st + h * TILE) : desc_sw128(st + h * TILE);
                    const uint64_t bd = desc_sw128(st + ss.tok + (GATEUP ? 0 : h * p.nt * 128));
                    const uint32_t d = tmem_base + (GATEUP ? h * p.nt : 0);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t acc = (i | kk | (GATEUP ? 0 : h)) != 0;
                        if (MX)
                            mma_mxf4(d, ad + 2 * kk, bd + 2 * kk, idesc_mxf4(128, p.nt, 2 * (kk & 1)),
                                     sf + 8 * h + 4 * (kk >> 1), sf + 16 + (GATEUP ? 0 : 8 * h) + 4 * (kk >> 1), acc);
                        else
                            mma_bf16(d, ad + (MN ? 128 : 2) * kk, bd + 2 * kk, idesc, acc);
                        // tokens in two parts: the second one's rows, further on, onto the same columns
                        if (PARTS && !GATEUP)
                            mma_bf16(d, ad + 2 * kk, bd + kNarrowParts * ROW_BYTES / 16 + 2 * kk, idesc, 1u);
                    }
                }
                mma_commit(empty0 + 8 * s);
            }
            __syncwarp();
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (!ok && lane == 0) {
            set_error(p.hdr, DEV_ERR_TIMEOUT, 42);
            *abort_flag = 1;
        }
        if (elect_one()) mma_commit(done);
        __syncwarp();
    } else if (QUANT) {
        // Tokens warp - 2 and warp - 2 + 8, 256 of K per tile: eight elements a
        // lane, four lanes a block.  Two stages' loads are under way ahead of
        // the one being written.
        constexpr int TT = GATEUP ? 1 : 2;  // token tiles of a stage
        const int n = k1 - k0, ntok = min(p.nt, p.T - tok0);
        struct Piece {
            uint4 v[2][TT];
        };
        const auto load = [&](int i) {
            Piece q{};
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int h = 0; h < TT; ++h) {
                    const int j = warp - 2 + x * QUANT_WARPS, k = (TT * (k0 + i) + h) * 256 + lane * 8;
                    if (i < n && j < ntok && k < p.K)
                        q.v[x][h] = *reinterpret_cast<const uint4*>(p.x + (size_t)(tok0 + j) * p.ldx + k);
                }
            return q;
        };
        Piece cur = load(0), next = load(1);
        int s = 0;
        uint32_t ph = 1;
        for (int i = 0; i < n; ++i) {
            const Piece after = load(i + 2);
            if (warp_sees(abort_flag) || !warp_wait(empty0 + 8 * s, ph, p.wait_ns)) {
                if (lane == 0) {
                    set_error(p.hdr, DEV_ERR_TIMEOUT, 44);
                    *abort_flag = 1;
                }
                break;
            }
            const uint32_t st = sbase + s * stride;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int h = 0; h < TT; ++h) {
                    const int j = warp - 2 + x * QUANT_WARPS;
                    if (j >= ntok) continue;  // a column of D that is never read
                    const uint4 q = cur.v[x][h];
                    const float v[8] = {bf16lo(q.x), bf16hi(q.x), bf16lo(q.y), bf16hi(q.y),
                                        bf16lo(q.z), bf16hi(q.z), bf16lo(q.w), bf16hi(q.w)};
                    uint32_t a = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(v[e]) & 0x7fffffffu);
                    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
                    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
                    const uint32_t sc = mx_scale(a);
                    const uint32_t w = sc == 255u ? 0u : mx_codes8(v, mx_inverse(sc));
                    sts32(st + ss.tok + h * p.nt * 128 + j * 128 + (((lane >> 2) ^ (j & 7)) << 4) + (lane & 3) * 4, w);
                    uint32_t sw = sc << (((lane >> 2) & 3) * 8);
                    sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
                    sw |= __shfl_xor_sync(0xffffffffu, sw, 8);
                    if ((lane & 15) == 0) sts32(st + ss.sb + h * 1024 + (lane >> 4) * 512 + j * 16, sw);
                }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full0 + 8 * s);
            cur = next;
            next = after;
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
    }
    // the sums to shared memory, over the ring (its copies have landed and its
    // MMAs have read them): part[h][token][row], fp32
    if (!mbar_wait(done, 0, DRAIN_NS) && threadIdx.x == 0) set_error(p.hdr, DEV_ERR_TIMEOUT, 43);
    __syncthreads();
    tc_fence_after();
    const int ntok = min(p.nt, p.T - tok0);
    float* part = reinterpret_cast<float*>(smem);
    if (warp >= 2) {
        const int q = warp & 3, half = (warp - 2) >> 2;
        for (int c = 16 * half; c < (GATEUP ? 2 : 1) * p.nt; c += 32) {
            uint32_t v[16];
            tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = __uint_as_float(v[j]);
        }
        tc_fence_before();
    }
    cluster_sync();
    // Tokens, dealt over the cluster's warps; the loads of all slices of a token
    // are on their way before the first is added.  One token at a time: this code
    // runs once or a few times per CTA, and its size costs more (instructions
    // fetched cold) than more loads under way would save.
    const uint32_t pbase = smem_u32(part) + lane * 16;
    const int r = row0 + lane * 4;  // this lane's output columns r .. r + 3
    for (int j = (int)rank + S * warp; j < ntok; j += S * WARPS) {
        float v0[4] = {}, v1[4] = {};
        float4 q0[MAX_SLICES], q1[MAX_SLICES];
#pragma unroll
        for (int s = 0; s < MAX_SLICES; ++s)
            if (s < S) {
                const uint32_t a = mapa(pbase + j * 512, s);
                q0[s] = ld_cluster4(a);
                if (GATEUP) q1[s] = ld_cluster4(a + p.nt * 512);
            }
#pragma unroll
        for (int s = 0; s < MAX_SLICES; ++s)
            if (s < S) {
                add4(v0, q0[s]);
                if (GATEUP) add4(v1, q1[s]);
            }
        const size_t t = (size_t)(tok0 + j);
        if (GATEUP && MX) {
            float h[4];
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[i] = r < p.R ? glu(v0[i], v1[i], p.act) : 0.f;
                a = max(a, __float_as_uint(h[i]) & 0x7fffffffu);
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
            const uint32_t sc = mx_scale(a);
            const uint32_t w = sc == 255u ? 0u : mx_codes4(h, mx_inverse(sc));
            if (r < p.R) *reinterpret_cast<uint16_t*>(p.codes + (t * p.R + r) / 2) = (uint16_t)w;
            if ((lane & 7) == 0) p.scales[mx_scale_at(t, (size_t)(tile * 4 + (lane >> 3)), p.nkt)] = (uint8_t)sc;
        } else if (r < p.R) {  // R is a multiple of 8: whole quads
            const size_t at = t * p.R + r;
            float o[4];
            if (KIND == NARROW_DACT) {  // dg = dh d; du = dh a
                const size_t sat = saved_at(t, r, p.R);
                const float4 a = *reinterpret_cast<const float4*>(p.sa + sat), d = *reinterpret_cast<const float4*>(p.sd + sat);
                const float* h = v0;
                *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(h[0] * d.x, h[1] * d.y), pack_bf16x2(h[2] * d.z, h[3] * d.w));
                *reinterpret_cast<uint2*>(p.du + at) = make_uint2(pack_bf16x2(h[0] * a.x, h[1] * a.y), pack_bf16x2(h[2] * a.z, h[3] * a.w));
                continue;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i] = v0[i];
                if (GATEUP) {
                    float a, slope;
                    act_slope(v0[i], p.act, a, slope);
                    o[i] = a * v1[i];
                    v0[i] = a;
                    v1[i] *= slope;
                }
            }
            if (GATEUP && p.sa) {
                const size_t sat = saved_at(t, r, p.R);
                *reinterpret_cast<float4*>(p.sa + sat) = make_float4(v0[0], v0[1], v0[2], v0[3]);
                *reinterpret_cast<float4*>(p.sd + sat) = make_float4(v1[0], v1[1], v1[2], v1[3]);
            }
            const uint2 hi = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
            *reinterpret_cast<uint2*>(p.out + at) = hi;
            if (GATEUP && PARTS)  // what rounding left of h, kNarrowParts rows further on
                *reinterpret_cast<uint2*>(p.out + at + kNarrowParts * (size_t)p.R) =
                    make_uint2(pack_bf16x2(second_part(o[0], bf16lo(hi.x)), second_part(o[1], bf16hi(hi.x))),
                               pack_bf16x2(second_part(o[2], bf16lo(hi.y)), second_part(o[3], bf16hi(hi.y))));
        }
    }
    cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, p.tmem_cols);
    }
}

int sms() {
    static int n = device_sm_count();
    return n;
}

// Clusters of `size` CTAs that the device holds at once with one CTA per SM
// (asked once, of one kernel: with 222 KB each, no kernel here has two CTAs on an
// SM, and what is left to decide is where SMs stand, not which kernel it is).
int clusters_resident(int size) {
    static std::atomic<int> known[MAX_SLICES + 1];
    std::atomic<int>& k = known[size];
    if (k.load() == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = 222 * 1024;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = size;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        int n = 0;
        if (allow_smem<ffn_narrow<FMT_BF16, NARROW_GATEUP>>(227 * 1024) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, ffn_narrow<FMT_BF16, NARROW_GATEUP>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = sms() / size * 3 / 4;
        }
        k.store(std::max(n, 1));
    }
    return k.load();
}

template <int FMT, int KIND>
cudaError_t launch(const NarrowProduct& p, int smem, cudaStream_t st) {
    const cudaError_t attr = allow_smem<ffn_narrow<FMT, KIND>>(227 * 1024);
    if (attr != cudaSuccess) return attr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ceil_div(p.R, 128) * p.slices, ceil_div(p.T, p.nt));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.slices;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, ffn_narrow<FMT, KIND>, p);
}

}  // namespace

// Measured as whole blocks, narrow / wide in us: bf16 7168 x 2048 at 256 tokens
// 35.6 / 48.8, at 384 54.2 / 50.1; 2048 x 8192 at 256 38.8 / 55.2, at 384 65.2 /
// 64.8; 2048 x 768 (few tiles) at 512 18.5 / 21.2, at 1024 22.6 / 21.5.
// MXFP4, weights from HBM, at 64, 128, 192 and 256 tokens: blocks of 7168 x 2048
// 17.6 / 21.3, 21.4 / 22.5, 22.3 / 23.0, 24.1 / 23.2; 2048 x 8192 18.5 / 23.3,
// 22.5 / 24.2, 26.5 / 24.4, 27.7 / 24.8; the product 7168 -> 7168 12.1 / 16.2,
// 14.2 / 17.1, 17.7 / 17.4, 18.1 / 17.8.  One border for all does not suit small
// blocks (2048 x 768: 12.8 / 12.9, 16.9 / 14.2) nor a long K with few rows (the
// product 7168 -> 2048 at 256: 12.1 / 16.6).
bool narrow_is_faster(int m, int R, bool mx) {
    if (mx) return m <= 128;
    return m <= 256 || (m <= 512 && ceil_div(m, 256) * ceil_div(R, 256) * 4 <= sms() / 2);
}

int narrow_tokens(int m) { return std::min(128, (m + 15) / 16 * 16); }

cudaError_t launch_ffn_narrow(NarrowProduct& p, bool mx, int kind, cudaStream_t st) {
    const bool gateup = kind == NARROW_GATEUP || kind == NARROW_GATEUP_PARTS;
    p.nt = narrow_tokens(p.T);
    p.kstages = ceil_div(p.K, (mx ? 256 : 64) * (gateup || kind == NARROW_DX ? 1 : 2));
    const StageShape ss = stage_shape(mx, kind, p.nt);
    const int stride = stage_stride(ss);
    // Two CTAs per SM for up to 16 tokens: the next kernel's weights then arrive
    // while this one drains (7168 x 2048, one token: 20.2 us, with one CTA of
    // twice the stages 21.2).  Above, two would have two or three stages each
    // (48 tokens: 27.4 us, with one of five 23.6).
    const int resident = p.nt <= 16 ? 2 : 1;
    const int budget = resident == 2 ? 110 * 1024 : 220 * 1024;
    p.stages = std::min(MAX_STAGES, budget / stride);
    if (mx) p.stages = std::min(p.stages, 4);  // 32 scale columns each
    const int acc = (gateup ? 2 : 1) * p.nt;
    p.ring_bytes = (std::max(p.stages * stride, acc * 512) + 1023) & ~1023;
    const int smem = 1024 + p.ring_bytes + ring_margin(kind) + 256;
    int cols = 32;
    while (cols < acc + (mx ? 32 * p.stages : 0)) cols *= 2;
    p.tmem_cols = cols;
    // Slices of K: as many as the device takes at once, with two stages or more
    // each.  At one CTA per SM that goes by the clusters that fit (eights do not
    // fill the SMs: 16 row tiles in 8 slices took 31.5 us, in 6 slices 23.6); at
    // two, where a few clusters may start late, by CTAs, an eighth of the slots
    // left free (56 tiles: 224 CTAs 20.2 us, 280 20.9, 168 21.4).
    const int tiles = ceil_div(p.R, 128) * ceil_div(p.T, p.nt);
    p.slices = 1;
    for (int s = std::min(MAX_SLICES, p.kstages / 2); s > 1; --s)
        if (resident == 2 ? 8 * tiles * s <= 7 * 2 * sms() : tiles <= clusters_resident(s)) {
            p.slices = s;
            break;
        }
    if (p.x) return gateup ? launch<FMT_MXFP4_QUANT, NARROW_GATEUP>(p, smem, st) : launch<FMT_MXFP4_QUANT, NARROW_PLAIN>(p, smem, st);
    if (mx) return gateup ? launch<FMT_MXFP4, NARROW_GATEUP>(p, smem, st) : launch<FMT_MXFP4, NARROW_PLAIN>(p, smem, st);
    switch (kind) {
        case NARROW_GATEUP: return launch<FMT_BF16, NARROW_GATEUP>(p, smem, st);
        case NARROW_GATEUP_PARTS: return launch<FMT_BF16, NARROW_GATEUP_PARTS>(p, smem, st);
        case NARROW_PLAIN_PARTS: return launch<FMT_BF16, NARROW_PLAIN_PARTS>(p, smem, st);
        case NARROW_DACT: return launch<FMT_BF16, NARROW_DACT>(p, smem, st);
        case NARROW_DX: return launch<FMT_BF16, NARROW_DX>(p, smem, st);
        default: return launch<FMT_BF16, NARROW_PLAIN>(p, smem, st);
    }
}

}  // namespace moe
