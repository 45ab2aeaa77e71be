// Products of the gated feed-forward block for few tokens: every weight is read
// once, so the time is that of streaming the weights.
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
//   all warps  the sum over slices and the epilogue, a warp per (token, 32 rows):
//              of an MXFP4 h exactly one block.
// A stage holds two weight tiles of 128 bytes of K: W1 and W3, or (one matrix)
// two neighbours along K.  Bounded waits as in ffn_wide.cu.
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

constexpr int TILE = 128 * 128;  // 128 rows x 128 bytes of K
constexpr int WARPS = 10, THREADS = 32 * WARPS;
constexpr int MAX_STAGES = 8;
constexpr uint64_t DRAIN_NS = 2000000000ull;

// Byte offsets inside a stage.
struct StageShape {
    int tok, sa, sb, bytes;
};
// tok: the token tile(s); sa, sb: scales of the weights and of the tokens.
__host__ __device__ inline StageShape stage_shape(bool mx, bool gateup, int nt) {
    StageShape s;
    s.tok = 2 * TILE;
    s.sa = s.tok + (gateup ? 1 : 2) * nt * 128;
    s.sb = s.sa + (mx ? 2048 : 0);
    s.bytes = s.sb + (mx ? (gateup ? 1024 : 2048) : 0);
    return s;
}
__host__ __device__ inline int stage_stride(const StageShape& s) { return (s.bytes + 1023) & ~1023; }

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

template <bool MX, bool GATEUP>
__global__ void __launch_bounds__(THREADS, 1) ffn_narrow(const __grid_constant__ NarrowProduct p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const StageShape ss = stage_shape(MX, GATEUP, p.nt);
    const int stride = stage_stride(ss);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.ring_bytes);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + MAX_STAGES), done = smem_u32(bars + 2 * MAX_STAGES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * MAX_STAGES + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.slices;
    const uint32_t rank = cluster_ctarank();
    const int tile = blockIdx.x / S;
    const int row0 = tile * 128, tok0 = blockIdx.y * p.nt;
    const int k0 = (int)((int64_t)p.kstages * rank / S), k1 = (int)((int64_t)p.kstages * (rank + 1) / S);
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
        tmem_relinquish();
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
        const CUtensorMap *a0 = &p.a[0], *a1 = &p.a[GATEUP ? 1 : 0], *s0 = &p.as[0], *s1 = &p.as[GATEUP ? 1 : 0];
        const auto weights = [&](int ks, uint32_t st, uint32_t bar) {
            const int kc = (GATEUP ? ks : 2 * ks) * 32;  // words along K: 128 bytes are 32
            mbar_arrive_expect_tx(bar, ss.bytes);
            tma_load_3d(st, a0, kc, row0, 0, bar);
            tma_load_3d(st + TILE, a1, GATEUP ? kc : kc + 32, row0, 0, bar);
            if (MX) {
                const int kt = (GATEUP ? 2 : 4) * ks;
                tma_load_3d(st + ss.sa, s0, 0, kt, tile, bar);
                tma_load_3d(st + ss.sa + 1024, s1, 0, GATEUP ? kt : kt + 2, tile, bar);
            }
        };
        const auto tokens = [&](int ks, uint32_t st, uint32_t bar) {
            const int kc = (GATEUP ? ks : 2 * ks) * 32;
            tma_load_3d(st + ss.tok, &p.b, kc, tok0, 0, bar);
            if (!GATEUP) tma_load_3d(st + ss.tok + p.nt * 128, &p.b, kc + 32, tok0, 0, bar);
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
            if (!mbar_wait(empty0 + 8 * s, ph, p.wait_ns)) {
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
        bool ok = true;
        const uint32_t idesc = idesc_bf16(128, p.nt);
        int s = 0;
        uint32_t ph = 0;
        for (int i = 0; i < k1 - k0; ++i) {
            if (*abort_flag || !mbar_wait(full0 + 8 * s, ph, p.wait_ns)) {
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
                    const uint64_t ad = desc_sw128(st + h * TILE);
                    const uint64_t bd = desc_sw128(st + ss.tok + (GATEUP ? 0 : h * p.nt * 128));
                    const uint32_t d = tmem_base + (GATEUP ? h * p.nt : 0);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t acc = (i | kk | (GATEUP ? 0 : h)) != 0;
                        if (MX)
                            mma_mxf4(d, ad + 2 * kk, bd + 2 * kk, idesc_mxf4(128, p.nt, 2 * (kk & 1)),
                                     sf + 8 * h + 4 * (kk >> 1), sf + 16 + (GATEUP ? 0 : 8 * h) + 4 * (kk >> 1), acc);
                        else
                            mma_bf16(d, ad + 2 * kk, bd + 2 * kk, idesc, acc);
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
    // units of (token, 32 rows), dealt over the cluster's warps
    const uint32_t pbase = smem_u32(part);
    for (int u = (int)rank + S * warp; u < ntok * 4; u += S * WARPS) {
        const int j = u >> 2, q = u & 3;
        const int r = row0 + q * 32 + lane;  // output column of this lane
        if (row0 + q * 32 >= p.R && !(MX && GATEUP)) continue;
        const uint32_t off = pbase + (uint32_t)(j * 128 + q * 32 + lane) * 4;
        float v0 = 0.f, v1 = 0.f;
#pragma unroll 8
        for (int s = 0; s < S; ++s) {
            const uint32_t a = mapa(off, s);
            v0 += ld_cluster(a);
            if (GATEUP) v1 += ld_cluster(a + p.nt * 512);
        }
        const size_t t = (size_t)(tok0 + j);
        if (GATEUP && MX) {
            const float h = r < p.R ? glu(v0, v1, p.act) : 0.f;
            const uint32_t sc = mx_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu));
            uint32_t w = sc == 255u ? 0u : mx_code(h * mx_inverse(sc)) << (4 * (lane & 7));
            w |= __shfl_xor_sync(0xffffffffu, w, 1);
            w |= __shfl_xor_sync(0xffffffffu, w, 2);
            w |= __shfl_xor_sync(0xffffffffu, w, 4);
            if ((lane & 7) == 0 && r < p.R) *reinterpret_cast<uint32_t*>(p.codes + (t * p.R + r) / 2) = w;
            if (lane == 0) p.scales[mx_scale_at(t, (size_t)(tile * 4 + q), p.nkt)] = (uint8_t)sc;
        } else if (r < p.R) {
            const size_t at = t * p.R + r;
            if (GATEUP) {
                float a, slope;
                act_slope(v0, p.act, a, slope);
                p.out[at] = f32_to_bf16(a * v1);
                if (p.sa) {
                    p.sa[at] = a;
                    p.sd[at] = v1 * slope;
                }
            } else {
                p.out[at] = f32_to_bf16(v0);
            }
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

template <bool MX, bool GATEUP>
cudaError_t launch(const NarrowProduct& p, int smem, cudaStream_t st) {
    static cudaError_t attr =
        cudaFuncSetAttribute(ffn_narrow<MX, GATEUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
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
    return cudaLaunchKernelEx(&cfg, ffn_narrow<MX, GATEUP>, p);
}

}  // namespace

int narrow_tokens(int m) { return std::min(128, (m + 15) / 16 * 16); }

cudaError_t launch_ffn_narrow(NarrowProduct& p, bool mx, bool gateup, cudaStream_t st) {
    p.nt = narrow_tokens(p.T);
    p.kstages = ceil_div(p.K, (mx ? 256 : 64) * (gateup ? 1 : 2));
    const StageShape ss = stage_shape(mx, gateup, p.nt);
    const int stride = stage_stride(ss);
    // two CTAs per SM while the token tiles are small: the second one's stream
    // covers the first one's start and end
    const int budget = p.nt <= 48 ? 110 * 1024 : 220 * 1024;
    p.stages = std::min(MAX_STAGES, budget / stride);
    if (mx) p.stages = std::min(p.stages, 4);  // 32 scale columns each
    const int acc = (gateup ? 2 : 1) * p.nt;
    p.ring_bytes = (std::max(p.stages * stride, acc * 512) + 1023) & ~1023;
    const int smem = 1024 + p.ring_bytes + 256;
    int cols = 32;
    while (cols < acc + (mx ? 32 * p.stages : 0)) cols *= 2;
    p.tmem_cols = cols;
    // slices of K: the count (at most 8, the portable cluster size, and a stage
    // each) that spreads the row tiles most evenly over two CTAs per SM
    const int tiles = ceil_div(p.R, 128) * ceil_div(p.T, p.nt);
    int best = 1;
    double eff = 0.0;
    for (int s = 1; s <= std::min(8, p.kstages); ++s) {
        const int ctas = tiles * s;
        if (s > 1 && ctas > 2 * sms()) break;
        const double e = (double)ctas / ((double)sms() * ceil_div(ctas, sms()));
        if (e > eff + 1e-9) {
            eff = e;
            best = s;
        }
    }
    p.slices = best;
    if (mx) return gateup ? launch<true, true>(p, smem, st) : launch<true, false>(p, smem, st);
    return gateup ? launch<false, true>(p, smem, st) : launch<false, false>(p, smem, st);
}

}  // namespace moe
