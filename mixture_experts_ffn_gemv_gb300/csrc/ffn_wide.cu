// bf16 products of the gated feed-forward block and of its backward pass on
// the tensor cores, for many tokens.
//
// One persistent kernel on CTA pairs (a cluster of two, cta_group::2) works
// through the 256 x 256 tiles of up to four products D = A B^T; a product's
// reduction runs over one or two sources (dx = dg W1 + du W3 is one sum of
// length 2 I), and either operand may be stored along K or along M (N): the
// backward products read W, x, dg and h as they lie, through MN-major
// descriptors, so nothing is transposed in memory.
//   warp 0      TMA producer: this CTA's 128 rows of A and half of the tile's
//               256 rows of B, 64 of K per stage of 32 KB, 6 or 7 stages;
//   warp 1      (leader) MMA issuer: M = 256, N = 256, fp32 accumulators in
//               TMEM, two buffers of 256 columns; the whole warp walks the
//               loop and one lane issues, so addresses are warp-uniform;
//   warps 2..   epilogue, 8 (plain products) or 16 (where there is an
//               activation or its gradient to compute), an equal share of each
//               TMEM lane quarter's columns.  A plain product's output leaves
//               through staging in shared memory and TMA stores, which write
//               whole lines and clip at the matrix's edges; the others store
//               32 bytes at a time from the lanes and keep the seventh stage.
// A forward pass that is to be differentiated saves a = act(g), d = u act'(g) in
// fp32 and h = a u in bf16, so that the backward pass multiplies (du = dh a,
// dg = dh d) where it would recompute: its epilogue, with the activation in it,
// took 202 us for 4096 x 8192 x 2048, three times the MMAs' time.
// Gate/up: the leader's half of B is 128 rows of W1, the peer's the same rows
// of W3, so a thread finds g and u of one element in its own lane.
// Bound by the MMAs (tensor pipe active 78% of gate/up, 86% of the weight
// gradients) and by how full the last round of tiles is; 256 x 256 over two SMs
// because a smaller tile loads more per product.  A block's forward pass, 7168 x
// 2048: 4096 tokens 200 us (1.80 PFLOP/s), 16384 825 (1.75, under the power cap);
// its backward pass, 4096 tokens, 2048 x 8192: 506 us (1.63).
// Every wait is bounded; on expiry the CTA records DEV_ERR_TIMEOUT, stops
// issuing, waits (2 s at most) for its copies and MMAs in flight, frees TMEM
// and returns.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "ffn_act.cuh"
#include "ffn_block.h"
#include "ffn_box.cuh"
#include "launch.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace moe {

namespace {

using namespace sm100;

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = 128 * BK * 2;  // per CTA
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int TMEM_COLS = 2 * BN;
constexpr uint64_t DRAIN_NS = 2000000000ull;
template <int EPI>
struct Shape {
    static constexpr int EPI_WARPS = EPI == EPI_STORE ? 8 : 16;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int STAGES = EPI == EPI_STORE ? 6 : 7;
    static constexpr int STG_OFF = STAGES * STAGE_BYTES;  // staging of a plain product: 4 KB per epilogue warp
    static constexpr int BAR_OFF = STG_OFF + (EPI == EPI_STORE ? EPI_WARPS * 4096 : 0);
    static constexpr int SMEM_BYTES = 1024 + BAR_OFF + 256;
    static_assert(SMEM_BYTES <= 227 * 1024, "fits one SM's shared memory");
};

// A lane's row of a saved block (ffn_box.cuh, saved_at): 32 values, n of them in
// the matrix (n a multiple of 8; the rest zero); a warp moves 1 KB at a time.
__device__ __forceinline__ void load_saved(const float* p, int n, float (&f)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[8] = {};
        if (8 * i < n) ld_global_v8(p + 256 * i, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[8 * i + k] = __uint_as_float(w[k]);
    }
}
__device__ __forceinline__ void store_saved(float* p, int n, const uint32_t (&f)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = f[8 * i + k];
        if (8 * i < n) st_global_v8(p + 256 * i, w);
    }
}

struct Item {
    int op, mt, nt;
};
__device__ __forceinline__ Item item_of(const FfnProducts& p, int t) {
    Item it;
    it.op = 0;
#pragma unroll
    for (int i = 1; i < kMaxProducts; ++i)
        if (i < p.count && t >= p.first[i]) it.op = i;
    const int r = t - p.first[it.op];
    it.mt = r / p.p[it.op].n_tiles;
    it.nt = r % p.p[it.op].n_tiles;
    return it;
}

// The work items of CTA pair c of n, in order.  The first `dear` items (the
// products with the longest reductions come first) go round; the pairs that
// then have one fewer take `fill` of the others each instead, and the rest go
// round again, from those pairs on.  (dx and three weight gradients of 4096 x
// 2048 x 8192: 1152 K blocks on the fullest pair by plain turns, 1088 so, 1078 on
// the average.)
struct Turns {
    int a, b, c0, n, pairs, total, dear, rest;
    __device__ __forceinline__ Turns(const FfnProducts& p, int pair, int pairs_)
        : c0(pair), pairs(pairs_), total(p.first[p.count]), dear(p.dear) {
        const int r = dear % pairs;
        a = pair < dear ? (dear - pair + pairs - 1) / pairs : 0;
        b = r && pair >= r ? p.fill : 0;
        n = pairs - r;
        rest = dear + (r ? n * p.fill : 0);
    }
    __device__ __forceinline__ int item(int i) const {  // -1: no more
        if (i < a) return c0 + i * pairs;
        if (i < a + b) return dear + (i - a) * n + c0 - (pairs - n);
        const int t = rest + (c0 + n) % pairs + (i - a - b) * pairs;
        return t < total ? t : -1;
    }
};

template <int EPI>
__global__ void __launch_bounds__(Shape<EPI>::THREADS, 1) ffn_products(const __grid_constant__ FfnProducts p) {
    constexpr int EPI_WARPS = Shape<EPI>::EPI_WARPS, STAGES = Shape<EPI>::STAGES, BAR_OFF = Shape<EPI>::BAR_OFF;
    constexpr bool GATEUP = EPI == EPI_GATEUP || EPI == EPI_GATEUP_SAVE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
    const uint32_t tfull0 = smem_u32(bars + 2 * STAGES), tempty0 = smem_u32(bars + 2 * STAGES + 2);
    const uint32_t drain = smem_u32(bars + 2 * STAGES + 4);
    const uint32_t never = smem_u32(bars + 2 * STAGES + 5);  // stall test: no thread ever arrives here
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 6);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tempty0 + 8 * a, 2 * EPI_WARPS);
        }
        mbar_init(drain, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    if (warp == 2 && lane < 2 * p.count) {
        const FfnProduct& q = p.p[lane >> 1];
        prefetch_tmap(&q.a[lane & 1 & (q.sources - 1)]);
        prefetch_tmap(&q.b[GATEUP ? rank : lane & 1 & (q.sources - 1)]);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();  // all of the above ran beside the preceding kernel's end
    pdl_trigger();
    const Turns turns(p, blockIdx.x >> 1, gridDim.x >> 1);
    const uint32_t lead_full0 = mapa(full0, 0), lead_tempty0 = mapa(tempty0, 0);

    if (warp == 0) {
        // Like the issuer's, this loop is the whole warp's, its body one lane's
        // and free of choices: every map has three dimensions, and a box moves
        // by (w, r) along the first two per K block.  (One lane alone, choosing
        // by order, took 620 to 790 cycles a stage: more than the MMAs.)
        uint32_t s = 0, ph = 1, n = 0;
        bool ok = true;
        for (int i = 0, t; ok && (t = turns.item(i)) >= 0; ++i) {
            if (warp_sees(abort_flag)) break;
            const Item w = item_of(p, t);
            const FfnProduct& q = p.p[w.op];
            const int m0 = w.mt * 256 + (int)rank * BM;
            const int n0 = GATEUP ? w.nt * 128 : w.nt * 256 + (int)rank * 128;
            const BoxWalk a(q.a_mn, m0), b(q.b_mn, n0);
            for (int src = 0; src < q.sources && ok; ++src) {
                const CUtensorMap* ma = &q.a[src];
                const CUtensorMap* mb = &q.b[GATEUP ? rank : src];
                for (int kb = 0; kb < q.kblocks; ++kb) {
                    if (!warp_wait_cluster(empty0 + 8 * s, ph, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = sbase + s * STAGE_BYTES, sb = sa + A_BYTES, bar = lead_full0 + 8 * s;
                    if (elect_one()) {
                        if (leader) mbar_arrive_expect_tx(full0 + 8 * s, 2 * STAGE_BYTES);
                        tma_load_3d_pair(sa, ma, a.c0 + kb * a.d0, a.c1 + kb * a.d1, a.c2, bar);
                        if (a.two) tma_load_3d_pair(sa + A_BYTES / 2, ma, a.c0 + 32, a.c1 + kb * a.d1, 0, bar);
                        tma_load_3d_pair(sb, mb, b.c0 + kb * b.d0, b.c1 + kb * b.d1, b.c2, bar);
                        if (b.two) tma_load_3d_pair(sb + B_BYTES / 2, mb, b.c0 + 32, b.c1 + kb * b.d1, 0, bar);
                    }
                    __syncwarp();
                    ++n;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
        if (!ok && lane == 0) {
            set_error(p.hdr, DEV_ERR_TIMEOUT, 21);
            *abort_flag = 1;
        }
        if (leader) {
            // every issued copy of both CTAs has landed before either can exit
            for (uint32_t i = n > (uint32_t)STAGES ? n - STAGES : 0; i < n; ++i)
                mbar_wait_cluster(full0 + 8 * (i % STAGES), (i / STAGES) & 1u, DRAIN_NS);
        } else if (!ok || *abort_flag) {
            // the peer's copies complete on the leader's barriers: after an
            // abort, give any still in flight time to land
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 50000ull) __nanosleep(1000);
        }
    } else if (warp == 1) {
        if (leader) {
            uint32_t s = 0, ph = 0, tc = 0;
            bool ok = !p.stall || warp_wait(never, 0, p.wait_ns);
            for (int t; ok && (t = turns.item((int)tc)) >= 0; ++tc) {
                if (warp_sees(abort_flag)) break;
                const FfnProduct& q = p.p[item_of(p, t).op];
                const uint32_t idesc = idesc_bf16(2 * BM, BN) | (q.a_mn ? kIdescAMn : 0u) | (q.b_mn ? kIdescBMn : 0u);
                // 16 of K further: 32 bytes along a swizzled row, or 16 rows of 128
                const uint32_t sta = q.a_mn ? 128 : 2, stb = q.b_mn ? 128 : 2;
                const uint32_t acc = tc & 1u, aph = (tc >> 1) & 1u;
                if (!warp_wait_cluster(tempty0 + 8 * acc, aph ^ 1u, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + acc * BN;
                const int kbs = q.kblocks * q.sources;
                const uint64_t ad0 = q.a_mn ? desc_sw128_mn(sbase) : desc_sw128(sbase);
                const uint64_t bd0 = q.b_mn ? desc_sw128_mn(sbase + A_BYTES) : desc_sw128(sbase + A_BYTES);
                for (int kb = 0; kb < kbs; ++kb) {
                    if (!warp_wait_cluster(full0 + 8 * s, ph, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = ad0 + s * (STAGE_BYTES >> 4), bd = bd0 + s * (STAGE_BYTES >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            mma_bf16_pair(d, ad + sta * kk, bd + stb * kk, idesc, (kb | kk) != 0);
                        mma_commit_pair(empty0 + 8 * s);
                        if (kb == kbs - 1) mma_commit_pair(tfull0 + 8 * acc);
                    }
                    __syncwarp();
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok && lane == 0) {
                set_error(p.hdr, DEV_ERR_TIMEOUT, 22);
                *abort_flag = 1;
            }
            if (elect_one()) mma_commit_pair(drain);
            mbar_wait_cluster(drain, 0, DRAIN_NS);
        }
        __syncwarp();
    } else {
        const int q4 = warp & 3;           // the TMEM lane quarter this warp may read
        const int part = (warp - 2) >> 2;  // its share of the tile's columns
        const uint32_t stg = sbase + Shape<EPI>::STG_OFF + (warp - 2) * 4096;
        uint32_t tc = 0;
        for (int t; (t = turns.item((int)tc)) >= 0; ++tc) {
            if (warp_sees(abort_flag)) break;
            const Item w = item_of(p, t);
            const FfnProduct& q = p.p[w.op];
            const int row0 = w.mt * 256 + (int)rank * BM + q4 * 32;  // first of this warp's rows of D
            const int N = q.N;
            // first of its columns of the output
            const int col0 = GATEUP ? w.nt * 128 + part * 32 : w.nt * 256 + part * (1024 / EPI_WARPS);
            const bool ok = row0 + lane < q.M;
            const size_t at = (size_t)(row0 + lane) * N + col0;
            const uint32_t acc = tc & 1u, aph = (tc >> 1) & 1u;
            if (!warp_wait_cluster(tfull0 + 8 * acc, aph, p.wait_ns)) {
                set_error(p.hdr, DEV_ERR_TIMEOUT, 23);
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q4 * 32) << 16) + acc * BN;
            const uint32_t tempty = lead_tempty0 + 8 * acc;
            const auto release = [&] {  // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(tempty);
            };
            if (row0 >= q.M || col0 >= N) {  // nothing of the tile in the matrix
                release();
            } else if (GATEUP) {
                uint32_t gv[32], uv[32], o[16];
                tmem_ld32(taddr + 32 * part, gv);
                tmem_ld32(taddr + 128 + 32 * part, uv);
                tmem_wait_ld();
                release();
                if (EPI == EPI_GATEUP_SAVE) {
                    glu32_save(gv, uv, o, p.act);
                    if (ok) {
                        const size_t sat = saved_at(row0 + lane, col0, N);
                        store_saved(p.a + sat, N - col0, gv);
                        store_saved(p.d + sat, N - col0, uv);
                    }
                } else {
                    glu32(gv, uv, p.act);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = pack_bf16x2(__uint_as_float(gv[2 * i]), __uint_as_float(gv[2 * i + 1]));
                }
                if (ok) store_row32(q.out + at, N - col0, (N & 15) == 0, o);
            } else if (EPI == EPI_DACT) {
                uint32_t dv[2][32];
                tmem_ld32(taddr + 64 * part, dv[0]);
                tmem_ld32(taddr + 64 * part + 32, dv[1]);
                tmem_wait_ld();
                release();
                if (!ok) continue;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int n = N - col0 - 32 * e;
                        float f[32];
                        uint32_t o[16];
                        load_saved((x ? p.d : p.a) + saved_at(row0 + lane, col0, N) + 1024 * e, n, f);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = pack_bf16x2(__uint_as_float(dv[e][2 * i]) * f[2 * i],
                                               __uint_as_float(dv[e][2 * i + 1]) * f[2 * i + 1]);
                        store_row32((x ? q.out : p.out_du) + at + 32 * e, n, (N & 15) == 0, o);
                    }
            } else {
                uint32_t o[2][32];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t v[2][32];
                    tmem_ld32(taddr + 128 * part + 64 * j, v[0]);
                    tmem_ld32(taddr + 128 * part + 64 * j + 32, v[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[j][i] = pack_bf16x2(__uint_as_float(v[i >> 4][(2 * i) & 31]), __uint_as_float(v[i >> 4][(2 * i + 1) & 31]));
                }
                release();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (col0 + 64 * j >= N) break;
                    if (lane == 0) tma_store_wait_read();
                    __syncwarp();
                    stage_row128(stg, o[j], lane);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store_3d(&q.o, col0 / 2 + 32 * j, row0, 0, stg);
                }
            }
        }
        if (lane == 0) tma_store_wait();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still signal it or read its TMEM
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

int sms() {
    static int n = device_sm_count();
    return n;
}

template <int EPI>
cudaError_t launch(const FfnProducts& p, cudaStream_t st) {
    const cudaError_t attr = allow_smem<ffn_products<EPI>>(Shape<EPI>::SMEM_BYTES);
    if (attr != cudaSuccess) return attr;
    const int pairs = std::max(1, std::min(sms() / 2, p.first[p.count]));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(Shape<EPI>::THREADS);
    cfg.dynamicSmemBytes = Shape<EPI>::SMEM_BYTES;
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
    return cudaLaunchKernelEx(&cfg, ffn_products<EPI>, p);
}

}  // namespace

bool ffn_map(CUtensorMap* m, const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows) {
    const uint64_t dims[3] = {cols / 2, rows, 1}, strides[2] = {ld * 2, 128};
    const uint32_t box[3] = {BK / 2, box_rows, 1};
    return tmap_encode_words(m, p, 3, dims, strides, box);
}

int ffn_map_mn(CUtensorMap* m, const void* p, uint64_t rows, uint64_t cols, uint64_t ld) {
    if (cols % 64) return ffn_map(m, p, rows, cols, ld, 64) ? MN_ROWS : K_MAJOR;
    const uint64_t dims[3] = {32, rows, cols / 64}, strides[2] = {ld * 2, 128};
    const uint32_t box[3] = {32, 64, 2};
    return tmap_encode_words(m, p, 3, dims, strides, box) ? MN_BLOCKS : K_MAJOR;
}

cudaError_t launch_ffn_products(FfnProducts& p, int epilogue, cudaStream_t st) {
    const int bn = epilogue == EPI_GATEUP || epilogue == EPI_GATEUP_SAVE ? 128 : 256;
    p.first[0] = 0;
    for (int i = 0; i < p.count; ++i) {
        FfnProduct& q = p.p[i];
        q.m_tiles = ceil_div(q.M, 256);
        q.n_tiles = ceil_div(q.N, bn);
        p.first[i + 1] = p.first[i] + q.m_tiles * q.n_tiles;
        if (epilogue == EPI_STORE && !ffn_map(&q.o, q.out, q.M, q.N, q.N, 32)) return cudaErrorUnknown;
    }
    // items of the longest reduction, and how many of the others weigh as much
    // (an epilogue counted as 6 K blocks)
    const int total = p.first[p.count], pairs = std::min(sms() / 2, total);
    const auto cost = [&](int i) { return p.p[i].sources * p.p[i].kblocks + 6; };
    int k = 1;
    while (k < p.count && cost(k) == cost(0)) ++k;
    p.dear = p.first[k];
    p.fill = 0;
    if (k < p.count) p.fill = std::min(cost(0) / cost(p.count - 1), (total - p.dear) / (pairs - p.dear % pairs));
    switch (epilogue) {
        case EPI_GATEUP: return launch<EPI_GATEUP>(p, st);
        case EPI_GATEUP_SAVE: return launch<EPI_GATEUP_SAVE>(p, st);
        case EPI_DACT: return launch<EPI_DACT>(p, st);
        default: return launch<EPI_STORE>(p, st);
    }
}

}  // namespace moe
