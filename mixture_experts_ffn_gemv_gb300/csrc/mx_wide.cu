// MXFP4 products for many tokens on the block-scaled fp4 MMA
// (tcgen05.mma kind::mxf4, K = 64, one e8m0 scale per 32).
//
// A persistent kernel on CTA pairs; tiles are 256 rows x 256 columns (gate/up:
// 128 columns of g and the same of u).  A stage is 256 of K: this CTA's 128
// rows of A codes (16 KB, 128-byte swizzle), its half of the 256 rows of B
// (16 KB), and the packed scales of its A rows (1 KB) and of all 256 B rows
// (2 KB), which each CTA needs whole.
// Scales: four warps, one per TMEM lane quarter, move a stage's scales to
// tensor memory -- a lane's 16 bytes of each 512-byte tile are its four
// columns as they lie -- with tcgen05.st, beside the running MMAs.  tcgen05.cp
// would need no warps, but copies and MMAs run in issue order and the six
// copies of a stage held the tensor core up for 175 ns of every 480 (4096 x
// 7168 x 7168; issuing them a stage ahead changed nothing).
// TMEM: one accumulator of 256 columns and 24 scale columns per stage.  One
// accumulator, not two: 256 x 256 tiles halve the operand bytes per product
// of the 128 x 128 tiles that would leave room for two, and the epilogue holds
// up the next tile only while it reads the accumulator into registers.
// Bound by the MMAs (tensor pipe active 73%, 60% of gate/up), which stand still
// while the one accumulator is read.  8192 x 7168 x 7168 in 117 us (7.2 PFLOP/s),
// in 124 over two seconds and 141 after a long load, when the power cap holds.
// Gate/up quantises h in its epilogue: a thread's 32 columns of a row are one
// MXFP4 block, so h never exists in wider form.
//   warp 0 producer, warp 1 (leader) issuer, then the epilogue warps (an
//   equal number per lane quarter) and four scale warps.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "ffn_act.cuh"
#include "ffn_block.h"
#include "launch.cuh"
#include "mxfp4.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace moe {

namespace {

using namespace sm100;

constexpr int BM = 128, BN = 256;
constexpr int BKB = 128;  // bytes of K per stage and row: 256 codes
constexpr int A_BYTES = BM * BKB, B_BYTES = 128 * BKB;
constexpr int SA_BYTES = 2 * 512, SB_BYTES = 2 * 2 * 512;  // two K tiles x one / two row tiles
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
constexpr int B_OFF = A_BYTES, SA_OFF = B_OFF + B_BYTES, SB_OFF = SA_OFF + SA_BYTES;
constexpr int STAGE_STRIDE = 35 * 1024;
static_assert(STAGE_BYTES == STAGE_STRIDE, "stages keep the swizzle's 1024-byte alignment");
constexpr int TMEM_COLS = 512;
constexpr int SF_COL0 = BN, SF_COLS = 24;  // per stage: 2 K tiles x (4 of A + 8 of B)
// Epilogue warps: gate/up has the activation and the quantisation of h to
// compute; a plain product only rounds, and more warps would only poll.
template <bool GATEUP>
struct Shape {
    static constexpr int EPI_WARPS = GATEUP ? 16 : 8;
    static constexpr int STAGES = GATEUP ? 6 : 5;  // a plain product also stages its output: 4 KB per epilogue warp
    static constexpr int STG_OFF = STAGES * STAGE_STRIDE;
    static constexpr int BAR_OFF = STG_OFF + (GATEUP ? 0 : EPI_WARPS * 4096);
    static constexpr int SMEM_BYTES = 1024 + BAR_OFF + 256;
    static_assert(SF_COL0 + STAGES * SF_COLS <= TMEM_COLS, "accumulator and scale columns fit tensor memory");
    static_assert(SMEM_BYTES <= 227 * 1024, "fits one SM's shared memory");
    static constexpr int SCALE0 = 2 + EPI_WARPS;
    static constexpr int THREADS = 32 * (SCALE0 + 4);
};
constexpr int SCALE_WARPS = 4;
constexpr uint64_t DRAIN_NS = 2000000000ull;

template <bool GATEUP>
__global__ void __launch_bounds__(Shape<GATEUP>::THREADS, 1) mx_product(const __grid_constant__ MxProduct p) {
    constexpr int EPI_WARPS = Shape<GATEUP>::EPI_WARPS, SCALE0 = Shape<GATEUP>::SCALE0;
    constexpr int STAGES = Shape<GATEUP>::STAGES, STG_OFF = Shape<GATEUP>::STG_OFF, BAR_OFF = Shape<GATEUP>::BAR_OFF;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
    const uint32_t tfull = smem_u32(bars + 2 * STAGES), tempty = smem_u32(bars + 2 * STAGES + 1);
    const uint32_t drain = smem_u32(bars + 2 * STAGES + 2);
    // scales of a stage: landed in this CTA's shared memory; in both CTAs' TMEM
    const uint32_t sland0 = smem_u32(bars + 2 * STAGES + 3), sfull0 = smem_u32(bars + 3 * STAGES + 3);
    const uint32_t never = smem_u32(bars + 4 * STAGES + 3);  // stall test: no thread ever arrives here
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * STAGES + 4);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
            mbar_init(sland0 + 8 * s, 1);
            mbar_init(sfull0 + 8 * s, 2 * SCALE_WARPS);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, 2 * EPI_WARPS);
        mbar_init(drain, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    if (warp == 2 && lane == 0) {
        prefetch_tmap(&p.a);
        prefetch_tmap(&p.as);
        prefetch_tmap(&p.b[GATEUP ? rank : 0]);
        prefetch_tmap(&p.bs[0]);
        if (GATEUP) prefetch_tmap(&p.bs[1]);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();  // all of the above ran beside the preceding kernel's end
    pdl_trigger();
    const int total = p.m_tiles * p.n_tiles;
    const int cl = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    const uint32_t lead_full0 = mapa(full0, 0), lead_tempty = mapa(tempty, 0);

    if (warp == 0) {
        // the whole warp's loop, one lane's body: as in ffn_wide.cu
        uint32_t s = 0, ph = 1, n = 0;
        bool ok = true;
        for (int t = cl; t < total && ok; t += ncl) {
            if (warp_sees(abort_flag)) break;
            const int mt = t / p.n_tiles, nt = t % p.n_tiles;
            const int m0 = mt * 256 + (int)rank * BM, mt0 = m0 >> 7;
            const int n0 = GATEUP ? nt * 128 : nt * 256 + (int)rank * 128;
            const int bt0 = GATEUP ? nt : 2 * nt, bt1 = GATEUP ? nt : 2 * nt + 1;
            const CUtensorMap *mb = &p.b[GATEUP ? rank : 0], *ms1 = &p.bs[GATEUP ? 1 : 0];
            for (int kb = 0; kb < p.kblocks; ++kb) {
                if (!warp_wait_cluster(empty0 + 8 * s, ph, p.wait_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = sbase + s * STAGE_STRIDE, bar = lead_full0 + 8 * s, sl = sland0 + 8 * s;
                if (elect_one()) {
                    mbar_arrive_expect_tx(sl, SA_BYTES + SB_BYTES);
                    tma_load_3d(sa + SA_OFF, &p.as, 0, 2 * kb, mt0, sl);
                    tma_load_3d(sa + SB_OFF, &p.bs[0], 0, 2 * kb, bt0, sl);
                    tma_load_3d(sa + SB_OFF + 1024, ms1, 0, 2 * kb, bt1, sl);
                    if (leader) mbar_arrive_expect_tx(full0 + 8 * s, 2 * (A_BYTES + B_BYTES));
                    tma_load_3d_pair(sa, &p.a, kb * (BKB / 4), m0, 0, bar);
                    tma_load_3d_pair(sa + B_OFF, mb, kb * (BKB / 4), n0, 0, bar);
                }
                __syncwarp();
                ++n;
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {
            set_error(p.hdr, DEV_ERR_TIMEOUT, 31);
            *abort_flag = 1;
        }
        const uint32_t first = n > (uint32_t)STAGES ? n - STAGES : 0;
        for (uint32_t i = first; i < n; ++i) mbar_wait(sland0 + 8 * (i % STAGES), (i / STAGES) & 1u, DRAIN_NS);
        if (leader) {
            for (uint32_t i = first; i < n; ++i)
                mbar_wait_cluster(full0 + 8 * (i % STAGES), (i / STAGES) & 1u, DRAIN_NS);
        } else if (!ok || *abort_flag) {
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 50000ull) __nanosleep(1000);
        }
    } else if (warp == 1) {
        // The whole warp walks the loop and one lane issues: the addresses are
        // then warp-uniform values.  (One lane looping alone took 310 ns for a
        // stage's four MMAs, more than the tensor core does.)
        if (leader) {
            uint32_t s = 0, ph = 0, tc = 0;
            bool ok = !p.stall || warp_wait(never, 0, p.wait_ns);
            for (int t = cl; t < total && ok; t += ncl, ++tc) {
                if (warp_sees(abort_flag)) break;
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if ((kb == 0 && !warp_wait_cluster(tempty, (tc & 1u) ^ 1u, p.wait_ns)) ||
                        !warp_wait_cluster(full0 + 8 * s, ph, p.wait_ns) ||
                        !warp_wait_cluster(sfull0 + 8 * s, ph, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = sbase + s * STAGE_STRIDE;
                    const uint32_t sf = tmem_base + SF_COL0 + s * SF_COLS;
                    const uint64_t ad = desc_sw128(sa), bd = desc_sw128(sa + B_OFF);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_mxf4_pair(tmem_base, ad + 2 * kk, bd + 2 * kk, idesc_mxf4(2 * BM, BN, 2 * (kk & 1)),
                                          sf + 4 * (kk >> 1), sf + 8 + 8 * (kk >> 1), (kb | kk) != 0);
                        mma_commit_pair(empty0 + 8 * s);
                        if (kb == p.kblocks - 1) mma_commit_pair(tfull);
                    }
                    __syncwarp();
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok && lane == 0) {
                set_error(p.hdr, DEV_ERR_TIMEOUT, 32);
                *abort_flag = 1;
            }
            if (elect_one()) mma_commit_pair(drain);
            mbar_wait_cluster(drain, 0, DRAIN_NS);
        }
        __syncwarp();
    } else if (warp >= SCALE0) {
        // columns: A tiles of K 0..127, 128..255; then per K tile the two B row tiles
        const uint32_t lane_base = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + SF_COL0;
        const uint32_t lead_sfull0 = mapa(sfull0, 0);
        const uint32_t n = total > cl ? (uint32_t)((total - cl + ncl - 1) / ncl) * p.kblocks : 0;
        uint32_t s = 0, ph = 0;
        for (uint32_t it = 0; it < n; ++it) {
            if (warp_sees(abort_flag) || !warp_wait(sland0 + 8 * s, ph, p.wait_ns)) {
                set_error(p.hdr, DEV_ERR_TIMEOUT, 34);
                *abort_flag = 1;
                break;
            }
            const uint32_t src = sbase + s * STAGE_STRIDE + SA_OFF + lane * 16;
            uint4 w[6];
#pragma unroll
            for (int i = 0; i < 2; ++i) w[i] = lds128(src + i * 512);
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[2 + 2 * kt + h] = lds128(src + SB_OFF - SA_OFF + h * 1024 + kt * 512);
            const uint32_t d = lane_base + s * SF_COLS;
            tmem_st8(d, w[0], w[1]);
            tmem_st8(d + 8, w[2], w[3]);
            tmem_st8(d + 16, w[4], w[5]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(lead_sfull0 + 8 * s);
            if (++s == STAGES) {
                s = 0;
                ph ^= 1u;
            }
        }
    } else {
        const int q4 = warp & 3, part = (warp - 2) >> 2;  // lane quarter, share of the columns
        uint32_t tc = 0;
        for (int t = cl; t < total; t += ncl, ++tc) {
            if (warp_sees(abort_flag)) break;
            const int mt = t / p.n_tiles, nt = t % p.n_tiles;
            const int r = mt * 256 + (int)rank * BM + q4 * 32 + lane;
            const bool ok = r < p.M, any = r - lane < p.M;
            if (!warp_wait_cluster(tfull, tc & 1u, p.wait_ns)) {
                set_error(p.hdr, DEV_ERR_TIMEOUT, 33);
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q4 * 32) << 16);
            // the accumulator is read whole and handed back before anything is
            // computed from it or stored: the next tile's MMAs wait for no more
            uint32_t v[2][32];            // gate/up: a block of g and of u; else two chunks of D on their way to o
            uint32_t o[GATEUP ? 1 : 2][32];  // bf16 pairs of 64 columns each
            if (any) {
                if (GATEUP) {
                    tmem_ld32(taddr + 32 * part, v[0]);
                    tmem_ld32(taddr + 128 + 32 * part, v[1]);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tmem_ld32(taddr + 128 * part + 64 * c, v[0]);
                        tmem_ld32(taddr + 128 * part + 64 * c + 32, v[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[GATEUP ? 0 : c][i] = pack_bf16x2(__uint_as_float(v[i >> 4][(2 * i) & 31]),
                                                               __uint_as_float(v[i >> 4][(2 * i + 1) & 31]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(lead_tempty);
            if (!any) continue;
            if (GATEUP) {
                if (!ok) continue;
                const int col = nt * 128 + part * 32;
                uint32_t s = 0;  // blocks past the last column: 0
                if (col < p.N) {
                    glu32(v[0], v[1], p.act);
                    const float* h = reinterpret_cast<const float*>(v[0]);
                    float a = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) a = max_nan(a, fabsf(h[i]));
                    s = mx_scale(__float_as_uint(a));
                    const float inv = mx_inverse(s);
                    uint4 w = make_uint4(mx_codes8(h, inv), mx_codes8(h + 8, inv), mx_codes8(h + 16, inv), mx_codes8(h + 24, inv));
                    if (s == 255u) w = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(p.codes + ((size_t)r * p.N + col) / 2) = w;
                }
                p.scales[mx_scale_at(r, (size_t)nt * 4 + part, p.nkt)] = (uint8_t)s;
            } else {
                // 32 rows x 64 columns at a time through this warp's staging
                // and out by TMA: whole lines, clipped at M and N
                const uint32_t stg = sbase + STG_OFF + (warp - 2) * 4096;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = nt * 256 + part * 128 + 64 * c;
                    if (col >= p.N) break;
                    if (lane == 0) tma_store_wait_read();
                    __syncwarp();
                    stage_row128(stg, o[GATEUP ? 0 : c], lane);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store_3d(&p.o, col / 2, r, 0, stg);
                }
            }
        }
        if (!GATEUP && lane == 0) tma_store_wait();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

int sms() {
    static int n = device_sm_count();
    return n;
}

template <bool GATEUP>
cudaError_t launch(const MxProduct& p, cudaStream_t st) {
    const cudaError_t attr = allow_smem<mx_product<GATEUP>>(Shape<GATEUP>::SMEM_BYTES);
    if (attr != cudaSuccess) return attr;
    const int pairs = std::max(1, std::min(sms() / 2, p.m_tiles * p.n_tiles));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(Shape<GATEUP>::THREADS);
    cfg.dynamicSmemBytes = Shape<GATEUP>::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mx_product<GATEUP>, p);
}

}  // namespace

// Codes [rows, k/2 bytes]: boxes of 128 bytes x box_rows rows, as bf16 rows of k/4.
bool mx_code_map(CUtensorMap* m, const void* codes, uint64_t rows, uint64_t k, uint32_t box_rows) {
    return ffn_map(m, codes, rows, k / 4, k / 4, box_rows);
}
// Packed scales as [row tiles][K tiles][128 words]: boxes of two K tiles of
// one row tile (tiles past the end read as zero: scale 2^-127 on zero codes).
bool mx_scale_map(CUtensorMap* m, const void* scales, uint64_t rows, uint64_t k) {
    const uint64_t dims[3] = {128, (k + 127) / 128, (rows + 127) / 128};
    return tmap_encode(m, scales, 3, dims, 4, 128, 2, false);
}

cudaError_t launch_mx_product(MxProduct& p, bool gateup, cudaStream_t st) {
    p.m_tiles = ceil_div(p.M, 256);
    p.n_tiles = ceil_div(p.N, gateup ? 128 : 256);
    if (!gateup) {
        if (!ffn_map(&p.o, p.out, p.M, p.N, p.N, 32)) return cudaErrorUnknown;
    }
    return gateup ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace moe
