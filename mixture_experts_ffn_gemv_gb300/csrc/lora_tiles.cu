// Low-rank adapters for many tokens: out[t] = y[t] + scale B (A x[t]) as two
// kernels over tiles of 128 tokens as they lie, whatever adapters they use.
//
// A tile's tokens are not sorted.  It lists the adapters that occur in it, in the
// order of their first tokens, and multiplies the whole tile by each; a row then
// takes the result of its own.  That spends products, which the tensor core has to
// spare (r is small and everything here is bound by x, y and out), and saves
// sorting, gathering and scattering: x, y and out move as TMA boxes.  Requests that
// lie together make one or two adapters a tile.  Where there are few tiles and many
// adapters, several blocks share a tile's adapters: each token is one block's own.
//
// lora_shrink: part[z, t, :] = A x[t] over slice z of K.  Up to 256 / r adapters
// share a pass over x: their rows of A are the MMA's N.
// lora_expand: T = scale * sum of the slices, as two bf16 parts (the second what
// the first's rounding left, so that T counts with 16 bits), in shared memory for
// all of a block's tiles of 128 outputs; D = T B^T per adapter and tile, the row's
// own added to y in shared memory, rounded once, and out by TMA.  y and the first
// B are loaded before the shrink kernel ends.
// Each: a thread of warp 0 loads by TMA, one of warp 1 issues the products, then the
// epilogue warps.  (With whole warps, their votes and joins at each wait were most of an
// adapter's turn: 950 cycles of the issuer at r = 16, now 770; 300 tokens of 64 adapters,
// 4096 -> 4096, 42.5 -> 35 us.)
//
// 8192 tokens, 7168 -> 7168, r = 64, 4 requests: 67 us for 360 MB (52.9 at the copy
// rate): shrink some 24 of them (17 at that rate), two launches' start and end and T's
// way between them 10, expand 30.  In one kernel, clusters handing T over through
// distributed shared memory, the same took 79 us: blocks wait for the slowest of their
// cluster (5 us), and the exchange itself takes 4.  A tile of many adapters pays for each
// about as much as for one: 2048 tokens of 64 adapters, 4096 -> 4096, r = 16, 110 us, of one 14.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "ffn_block.h"
#include "launch.cuh"
#include "ops.h"
#include "sm100.cuh"
#include "tmap.h"

namespace moe {

namespace {

using namespace sm100;

constexpr int BM = 128, BK = 64;
constexpr int X_BYTES = BM * BK * 2;  // a box of 128 rows x 64 columns, 128-byte swizzle
constexpr uint64_t DRAIN_NS = 2000000000ull;
constexpr int SHRINK_COLS = 256;  // of tensor memory: two blocks on an SM

// A role of one thread waits; what is there already costs no look at the others' flag.
__device__ __forceinline__ bool role_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, const volatile int* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    return !*abort_flag && mbar_wait(bar, parity, limit_ns);
}

// The adapters of a tile's tokens, or this block's share of them: every gridDim.z-th.
struct Tile {
    int id[BM];    // of each token, -1: none
    int list[BM];  // those that occur
    int slot[BM];  // a token's place in the list, -1: none, -2: in another block's list
    uint32_t firsts[4];
    int count;
};
// By all threads of the block (at least 128).
__device__ __forceinline__ void list_adapters(const LoraArgs& p, int m0, Tile& tl) {
    const int share = blockIdx.z, shares = gridDim.z;
    const int i = threadIdx.x;
    int id = -1;
    if (i < BM) {
        if (m0 + i < p.m) {
            id = __ldcg(p.ids + m0 + i);  // past L1: lora_expand reads them before it waits
            if (id < -1 || id >= p.n) {
                note_error(p.hdr, DEV_ERR_BAD_ID, m0 + i);
                id = -1;
            }
        }
        tl.id[i] = id;
    }
    __syncthreads();
    if (__syncthreads_and(i >= BM || m0 + i >= p.m || id == tl.id[0])) {  // one request's, as most tiles are
        if (i < BM) tl.slot[i] = id < 0 ? -1 : share ? -2 : 0;
        if (i == 0) {
            tl.list[0] = id;
            tl.count = id >= 0 && !share;
        }
        __syncthreads();
        return;
    }
    int first = i;
    if (i < BM) {
        for (int j = BM - 4; j >= 0; j -= 4) {
            const int4 q = *reinterpret_cast<const int4*>(tl.id + j);
            if (q.w == id) first = min(first, j + 3);
            if (q.z == id) first = min(first, j + 2);
            if (q.y == id) first = min(first, j + 1);
            if (q.x == id) first = min(first, j);
        }
        const uint32_t b = __ballot_sync(0xffffffffu, id >= 0 && first == i);
        if ((i & 31) == 0) tl.firsts[i >> 5] = b;
    }
    __syncthreads();
    if (i < BM) {
        int place = __popc(tl.firsts[first >> 5] & ((1u << (first & 31)) - 1u));
        for (int w = 0; w < first >> 5; ++w) place += __popc(tl.firsts[w]);
        const bool mine = place % shares == share;
        tl.slot[i] = id < 0 ? -1 : mine ? place / shares : -2;
        if (id >= 0 && first == i && mine) tl.list[place / shares] = id;
        if (i == 0) {
            int n = 0;
            for (int w = 0; w < 4; ++w) n += __popc(tl.firsts[w]);
            tl.count = (n + shares - 1 - share) / shares;
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- A x

constexpr int SHRINK_THREADS = 192;
constexpr int SHRINK_SMEM = 110 * 1024;  // two blocks on an SM

__global__ void __launch_bounds__(SHRINK_THREADS, 2) lora_shrink(const __grid_constant__ LoraArgs p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ alignas(16) Tile tl;
    __shared__ uint64_t bars[2 * 8 + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + 8), tfull = smem_u32(bars + 16),
                   tempty = smem_u32(bars + 17), drain = smem_u32(bars + 18),
                   never = smem_u32(bars + 19);  // stall test: no thread ever arrives here
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int z = blockIdx.y, m0 = blockIdx.x * BM;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 8; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, 4);
        mbar_init(drain, 1);
        mbar_init(never, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    list_adapters(p, m0, tl);
    if (tl.count == 0) return;  // the whole block: nothing is allocated yet
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), SHRINK_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // a stage holds a box of x and the rows of A of as many adapters as the tile has (or a pass takes)
    const uint32_t stride = X_BYTES + (min(tl.count, p.group) * p.r + 15) / 16 * (16 * BK * 2);
    const uint32_t stages = min(8u, (uint32_t)(SHRINK_SMEM - 1024) / stride);
    const int k0 = z * p.split_blocks, k1 = min(p.kblocks, k0 + p.split_blocks);
    const int passes = (tl.count + p.group - 1) / p.group;

    if (warp == 0) {
        if (elect_one()) {
            uint32_t s = 0, ph = 1, n = 0;
            const int count = tl.count;
            bool ok = true;
            for (int g = 0; g < passes && ok; ++g) {
                const int u0 = g * p.group, u1 = min(count, u0 + p.group);
                for (int kb = k0; kb < k1; ++kb) {
                    ok = role_wait(empty0 + 8 * s, ph, p.wait_ns, &abort_flag);
                    if (!ok) break;
                    const uint32_t sa = sbase + s * stride, bar = full0 + 8 * s;
                    mbar_arrive_expect_tx(bar, X_BYTES + (u1 - u0) * p.r * BK * 2);
                    tma_load_3d(sa, &p.mx, kb * (BK / 2), m0, 0, bar);
                    for (int u = u0; u < u1; ++u)
                        tma_load_3d(sa + X_BYTES + (u - u0) * p.r * BK * 2, &p.ma, kb * (BK / 2), tl.list[u] * p.r, 0, bar);
                    ++n;
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                note_error(p.hdr, DEV_ERR_TIMEOUT, 61);
                abort_flag = 1;
            }
            const uint32_t S = stages;
            for (uint32_t i = n > S ? n - S : 0; i < n; ++i) mbar_wait(full0 + 8 * (i % S), (i / S) & 1u, DRAIN_NS);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            uint32_t s = 0, ph = 0;
            const int count = tl.count;
            bool ok = p.stall != 1 || mbar_wait(never, 0, p.wait_ns);
            for (int g = 0; g < passes && ok; ++g) {
                const int u0 = g * p.group, u1 = min(count, u0 + p.group);
                const uint32_t idesc = idesc_bf16(BM, ((u1 - u0) * p.r + 15) / 16 * 16);
                ok = role_wait(tempty, (g & 1u) ^ 1u, p.wait_ns, &abort_flag);
                for (int kb = k0; kb < k1 && ok; ++kb) {
                    ok = role_wait(full0 + 8 * s, ph, p.wait_ns, &abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sa = sbase + s * stride;
                    const uint64_t ad = desc_sw128(sa), bd = desc_sw128(sa + X_BYTES);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma_bf16(tmem, ad + 2 * kk, bd + 2 * kk, idesc, kb != k0 || kk != 0);
                    mma_commit(empty0 + 8 * s);
                    if (kb == k1 - 1) mma_commit(tfull);
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                note_error(p.hdr, DEV_ERR_TIMEOUT, 62);
                abort_flag = 1;
            }
            mma_commit(drain);
            mbar_wait(drain, 0, DRAIN_NS);
        }
        __syncwarp();
    } else {
        const int row = (warp & 3) * 32 + lane, slot = tl.slot[row];
        float* dst = p.part + ((size_t)z * p.m + m0 + row) * p.r;
        const uint32_t taddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        for (int g = 0; g < passes; ++g) {
            if (!warp_wait(tfull, g & 1u, p.wait_ns) || warp_sees(&abort_flag)) {
                if (lane == 0) {
                    note_error(p.hdr, DEV_ERR_TIMEOUT, 63);
                    abort_flag = 1;
                }
                break;
            }
            tc_fence_after();
            const int u0 = g * p.group, u1 = min(tl.count, u0 + p.group);
            for (int u = u0; u < u1; ++u) {
                const bool own = slot == u;
                if (!__any_sync(0xffffffffu, own)) continue;
                for (int j = 0; j < p.r; j += 8) {
                    uint32_t v[8];
                    tmem_ld8(taddr + (u - u0) * p.r + j, v);
                    tmem_wait_ld();
                    if (own) {
                        *reinterpret_cast<uint4*>(dst + j) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4*>(dst + j + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, SHRINK_COLS);
    }
}

// ---------------------------------------------------------------- y + T B^T

constexpr int BN = 128;
// Epilogue warps.  The teams take tiles in turn or, where a tile has many adapters (from
// MANY on), every second adapter of each tile.
constexpr int TEAMS = 2, TEAM_WARPS = 8, MANY = 4;
constexpr int EPI_WARPS = TEAMS * TEAM_WARPS;
constexpr int EXPAND_THREADS = 32 * (2 + EPI_WARPS);
// Accumulators are each one team's own, and so are stages of y unless both teams take
// every tile: whoever waits for the phases of a barrier waits for each of them, one after
// another, which a parity alone tells apart.
constexpr int ND = 2 * TEAMS, EXPAND_COLS = ND * BN;
constexpr int YS = 2 * TEAMS, Y_BYTES = 2 * X_BYTES;  // two boxes of 64 columns
constexpr int MAX_B = 4;

template <bool SHARED>
__global__ void __launch_bounds__(EXPAND_THREADS, 1) lora_expand(const __grid_constant__ LoraArgs p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ alignas(16) Tile tl;
    __shared__ uint64_t bars[2 * YS + 2 * MAX_B + 2 * ND + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nb = (p.r + BK - 1) / BK;  // boxes along r
    // T's first parts, its second parts, y, B
    const uint32_t t_at = smem_u32(smem), y_at = t_at + 2 * nb * X_BYTES, b_at = y_at + YS * Y_BYTES;
    const uint32_t yfull0 = smem_u32(bars), yempty0 = yfull0 + 8 * YS, bfull0 = yempty0 + 8 * YS,
                   bempty0 = bfull0 + 8 * MAX_B, dfull0 = bempty0 + 8 * MAX_B, dempty0 = dfull0 + 8 * ND,
                   tready = dempty0 + 8 * ND, drain = tready + 8, tdone = drain + 8,
                   never = tdone + 8;  // stall test: no thread ever arrives here
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m0 = blockIdx.x * BM;
    if (threadIdx.x == 0) {
        for (int s = 0; s < YS; ++s) {
            mbar_init(yfull0 + 8 * s, 1);
            mbar_init(yempty0 + 8 * s, TEAM_WARPS);
        }
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bfull0 + 8 * s, 1);
            mbar_init(bempty0 + 8 * s, 1);
        }
        for (int s = 0; s < ND; ++s) {
            mbar_init(dfull0 + 8 * s, 1);
            mbar_init(dempty0 + 8 * s, TEAM_WARPS);
        }
        mbar_init(tready, EPI_WARPS);
        mbar_init(drain, 1);
        mbar_init(tdone, EPI_WARPS);
        mbar_init(never, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    list_adapters(p, m0, tl);  // ids, like y, are older than the shrink kernel, whose sums alone are waited for
    // nothing of this block's: what no adapter changes is the first share's
    if (tl.count == 0 && ((SHARED && blockIdx.z) || (p.out == p.y && p.ldo == p.ldy))) {
        pdl_wait();
        return;
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), EXPAND_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const bool both = tl.count >= MANY;  // teams take every tile, and every second adapter of it

    if (warp == 0) {
        if (elect_one()) {
            uint32_t ys = 0, yph = 1, yn = 0, bs = 0, bph = 1, bn = 0;
            const int count = tl.count;
            bool ok = true;
            // Room comes free once the shrink kernel is done: the limit of a wait for it starts there.
            bool shrunk = false;
            const auto room = [&](uint32_t bar, uint32_t parity) {
                if (mbar_try_wait(bar, parity)) return true;
                if (!shrunk) pdl_wait();
                shrunk = true;
                return role_wait(bar, parity, p.wait_ns, &abort_flag);
            };
            for (int nt = blockIdx.y; nt < p.n_tiles && ok; nt += p.n_ctas) {
                const auto load_b = [&](int u) {
                    for (int kb = 0; kb < nb; ++kb) {
                        ok = room(bempty0 + 8 * bs, bph);
                        if (!ok) break;
                        const uint32_t bar = bfull0 + 8 * bs;
                        mbar_arrive_expect_tx(bar, X_BYTES);
                        tma_load_3d(b_at + bs * X_BYTES, &p.mb, kb * (BK / 2), nt * BN, tl.list[u], bar);
                        ++bn;
                        if (++bs == (uint32_t)p.stages) {
                            bs = 0;
                            bph ^= 1u;
                        }
                    }
                };
                // the first adapter's B ahead of y: its product is to be there when y is.  No more of
                // them: products beyond the accumulators wait for the first ones' addition to y.
                if (count) load_b(0);
                ok = ok && room(yempty0 + 8 * ys, yph);
                if (!ok) break;
                const bool two = nt * BN + 64 < p.N;
                const uint32_t dst = y_at + ys * Y_BYTES, bar = yfull0 + 8 * ys;
                mbar_arrive_expect_tx(bar, two ? Y_BYTES : X_BYTES);
                tma_load_3d(dst, &p.my, nt * (BN / 2), m0, 0, bar);
                if (two) tma_load_3d(dst + X_BYTES, &p.my, nt * (BN / 2) + 32, m0, 0, bar);
                ++yn;
                if (++ys == YS) {
                    ys = 0;
                    yph ^= 1u;
                }
                for (int u = 1; u < count && ok; ++u) load_b(u);
            }
            if (!ok) {
                note_error(p.hdr, DEV_ERR_TIMEOUT, 64);
                abort_flag = 1;
            }
            const uint32_t S = p.stages;
            for (uint32_t i = yn > (uint32_t)YS ? yn - YS : 0; i < yn; ++i) mbar_wait(yfull0 + 8 * (i % YS), (i / YS) & 1u, DRAIN_NS);
            for (uint32_t i = bn > S ? bn - S : 0; i < bn; ++i) mbar_wait(bfull0 + 8 * (i % S), (i / S) & 1u, DRAIN_NS);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            uint32_t bs = 0, bph = 0, tile = 0;
            uint32_t turn0 = 0, turn1 = 0;  // products of each team so far
            pdl_wait();  // T comes after it: the waits' limit starts here
            bool ok = tl.count == 0 || (role_wait(tready, 0, p.wait_ns, &abort_flag) &&
                                        (p.stall != 2 || mbar_wait(never, 0, p.wait_ns)));
            tc_fence_after();
            const int count = tl.count, last = p.r - (nb - 1) * BK;
            const uint32_t idesc = idesc_bf16(BM, BN);
            const auto products = [&](uint32_t d, int kb, uint32_t b) {
                const uint64_t hi = desc_sw128(t_at + kb * X_BYTES), lo = desc_sw128(t_at + (nb + kb) * X_BYTES),
                               bd = desc_sw128(b_at + b * X_BYTES);
                const int steps = kb < nb - 1 ? 4 : (last + 15) / 16;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (kk >= steps) break;
                    mma_bf16(tmem + d * BN, hi + 2 * kk, bd + 2 * kk, idesc, (kb | kk) != 0);
                    mma_bf16(tmem + d * BN, lo + 2 * kk, bd + 2 * kk, idesc, 1);
                }
            };
            const auto next_stage = [&]() {
                if (++bs == (uint32_t)p.stages) {
                    bs = 0;
                    bph ^= 1u;
                }
            };
            if (both && nb == 1) {  // two adapters at a time, one of each team: 512 tokens of 64, r = 64, 61 -> 57 us
                for (int nt = blockIdx.y; nt < p.n_tiles && ok; nt += p.n_ctas)
                    for (int u = 0; u < count && ok; u += 2) {
                        const bool two = u + 1 < count;
                        const uint32_t d0 = turn0 & 1, d1 = 2 + (turn1 & 1), s0 = bs;
                        ok = role_wait(dempty0 + 8 * d0, ((turn0 >> 1) & 1u) ^ 1u, p.wait_ns, &abort_flag) &&
                             (!two || role_wait(dempty0 + 8 * d1, ((turn1 >> 1) & 1u) ^ 1u, p.wait_ns, &abort_flag)) &&
                             role_wait(bfull0 + 8 * bs, bph, p.wait_ns, &abort_flag);
                        next_stage();
                        const uint32_t s1 = bs;
                        if (two) {
                            ok = ok && role_wait(bfull0 + 8 * bs, bph, p.wait_ns, &abort_flag);
                            next_stage();
                        }
                        if (!ok) break;
                        tc_fence_after();
                        products(d0, 0, s0);
                        if (two) products(d1, 0, s1);
                        mma_commit(bempty0 + 8 * s0);
                        mma_commit(dfull0 + 8 * d0);
                        ++turn0;
                        if (two) {
                            mma_commit(bempty0 + 8 * s1);
                            mma_commit(dfull0 + 8 * d1);
                            ++turn1;
                        }
                    }
            } else {
                for (int nt = blockIdx.y; nt < p.n_tiles && ok; nt += p.n_ctas, ++tile)
                    for (int u = 0; u < count && ok; ++u) {
                        const uint32_t team = (both ? (uint32_t)u : tile) % TEAMS, turn = team ? turn1++ : turn0++;
                        const uint32_t d = team * 2 + (turn & 1);
                        ok = role_wait(dempty0 + 8 * d, ((turn >> 1) & 1u) ^ 1u, p.wait_ns, &abort_flag);
                        for (int kb = 0; kb < nb && ok; ++kb) {
                            ok = role_wait(bfull0 + 8 * bs, bph, p.wait_ns, &abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            products(d, kb, bs);
                            mma_commit(bempty0 + 8 * bs);
                            if (kb == nb - 1) mma_commit(dfull0 + 8 * d);
                            next_stage();
                        }
                    }
            }
            if (!ok) {
                note_error(p.hdr, DEV_ERR_TIMEOUT, 65);
                abort_flag = 1;
            }
            mma_commit(drain);
            mbar_wait(drain, 0, DRAIN_NS);
        }
        __syncwarp();
    } else {
        const int q4 = warp & 3, half = ((warp - 2) >> 2) & 1, team = (warp - 2) / TEAM_WARPS;  // lane quarter, which 64 columns
        const int row = q4 * 32 + lane, slot = tl.slot[row];
        pdl_wait();
        pdl_trigger();
        if (tl.count) {
            // T, a thread a piece of 8 of a row (zeros up to a multiple of 16): neighbouring lanes read
            // neighbouring pieces of the sums.  (With a row to a lane each load touched 32 lines, and
            // this took 6.7 us of a block's 29 at r = 64.)
            const int pieces = (p.r + 15) / 16 * 2;
            for (int q = (int)threadIdx.x - 64; q < BM * pieces; q += 32 * EPI_WARPS) {
                const int i = q / pieces, c = q % pieces;
                const bool own = tl.slot[i] >= 0;
                const float scale = own && p.scale ? p.scale[tl.id[i]] : 1.f;
                const float* src = p.part + (size_t)(m0 + i) * p.r + 8 * c;
                float v[8] = {};
                if (own && 8 * c < p.r) {
                    for (int z0 = 0; z0 < p.splits; z0 += 4) {
                        float4 f[4], g[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const bool in = z0 + z < p.splits;
                            const float4* at = reinterpret_cast<const float4*>(src + (size_t)(z0 + z) * p.m * p.r);
                            f[z] = in ? at[0] : make_float4(0.f, 0.f, 0.f, 0.f);
                            g[z] = in ? at[1] : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            v[0] += f[z].x; v[1] += f[z].y; v[2] += f[z].z; v[3] += f[z].w;
                            v[4] += g[z].x; v[5] += g[z].y; v[6] += g[z].z; v[7] += g[z].w;
                        }
                    }
                }
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = v[2 * e] * scale, b = v[2 * e + 1] * scale;
                    hi[e] = pack_bf16x2(a, b);
                    const float ah = bf16lo(hi[e]), bh = bf16hi(hi[e]);
                    // an infinite first part is all there is of it
                    lo[e] = pack_bf16x2(isinf(ah) ? 0.f : a - ah, isinf(bh) ? 0.f : b - bh);
                }
                const uint32_t at = t_at + (c >> 3) * X_BYTES + i * 128 + (((c & 7) ^ (i & 7)) << 4);
                sts128(at, hi[0], hi[1], hi[2], hi[3]);
                sts128(at + nb * X_BYTES, lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(tready);
        }
        bool ok = true;
        uint32_t turn = 0;
        const int u0 = both ? team : 0, du = both ? TEAMS : 1, dt = both ? 1 : TEAMS;
        uint32_t tile = both ? 0 : team;
        for (int nt = blockIdx.y + tile * p.n_ctas; nt < p.n_tiles && ok; nt += dt * p.n_ctas, tile += dt) {
            const uint32_t ys = tile % YS;
            if (warp_sees(&abort_flag) || !warp_wait(yfull0 + 8 * ys, (tile / YS) & 1u, p.wait_ns)) {
                ok = false;
                break;
            }
            const int col = nt * BN + 64 * half;
            const uint32_t box = y_at + ys * Y_BYTES + half * X_BYTES, line = box + row * 128;
            for (int u = u0; u < tl.count; u += du, ++turn) {
                const uint32_t d = team * 2 + (turn & 1);
                if (!warp_wait(dfull0 + 8 * d, (turn >> 1) & 1u, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const bool own = slot == u, any = __any_sync(0xffffffffu, own);
                // half a row's 64 columns at a time (registers), loads of y on their way before its first
                // store: 8192 tokens of 4 adapters mixed, 7168 -> 7168, r = 64, 122 -> 114 us
                const uint32_t taddr = tmem + ((uint32_t)(q4 * 32) << 16) + d * BN + 64 * half;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[32];
                    if (any) {
                        tmem_ld32(taddr + 32 * h, v);
                        tmem_wait_ld();
                    }
                    if (h == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(dempty0 + 8 * d);
                    }
                    if (own && col < p.N) {
                        uint4 q[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) q[c] = lds128(line + (((4 * h + c) ^ (row & 7)) << 4));
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t w[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
                            uint32_t o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                o[i] = pack_bf16x2(bf16lo(w[i]) + __uint_as_float(v[8 * c + 2 * i]),
                                                   bf16hi(w[i]) + __uint_as_float(v[8 * c + 2 * i + 1]));
                            sts128(line + (((4 * h + c) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
                        }
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            fence_async_smem();
            __syncwarp();
            if (both) {  // until the other team's rows are done too; the first team stores them all
                if (lane == 0) mbar_arrive(tdone);
                if (!warp_wait(tdone, tile & 1u, p.wait_ns)) {
                    ok = false;
                    break;
                }
                if (team) continue;
            }
            if (SHARED) {  // rows of its own among those of other blocks
                for (int i = lane >> 3; i < 32; i += 4) {
                    const int at = q4 * 32 + i, c = lane & 7, its = tl.slot[at];
                    if ((its >= 0 || (its == -1 && blockIdx.z == 0)) && m0 + at < p.m && col + 8 * c < p.N)
                        *reinterpret_cast<uint4*>(p.out + (size_t)(m0 + at) * p.ldo + col + 8 * c) =
                            lds128(box + at * 128 + ((c ^ (at & 7)) << 4));
                }
                __syncwarp();
            }
            if (lane == 0) {
                if (!SHARED && col < p.N && m0 + q4 * 32 < p.m) {
                    tma_store_3d(&p.mo, col / 2, m0 + q4 * 32, 0, box + q4 * 4096);
                    tma_store_wait_read();
                }
                mbar_arrive(yempty0 + 8 * ys);
            }
        }
        if (!ok && lane == 0) {
            note_error(p.hdr, DEV_ERR_TIMEOUT, 66);
            abort_flag = 1;
        }
        if (lane == 0) tma_store_wait();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, EXPAND_COLS);
    }
}

int sms() {
    static int n = device_sm_count();
    return n;
}

constexpr int kSmem = 225 * 1024;  // beside the static part (tile lists, barriers)

// Slices of K: as many as fill the device twice over, of at least 4 blocks of 64, and 16 at
// most: every expand block reads them all (1024 tokens, 7168 -> 7168, r = 64, one adapter: 25.7
// us with up to 28, 19.9 with 16, 19.2 with 12; 512 tokens of 64 adapters, 4096 -> 4096, r = 16:
// 53 with 16, 57 with 12).
int split_blocks(int64_t m, int64_t K) {
    const int tiles = (int)std::min<int64_t>((m + BM - 1) / BM, 1 << 20), kblocks = (int)((K + BK - 1) / BK);
    const int splits = std::max(1, std::min({2 * sms() / tiles, kblocks / 4, 16}));
    return ceil_div(kblocks, splits);
}

}  // namespace

// Blocks among which a tile's adapters may be shared, where tiles, slices and outputs leave SMs
// idle: one for each 128 columns that all adapters together have.  Tokens that use one adapter do
// not lose by it (its block works, the others leave), many adapters gain: 256 tokens of 32, 7168 ->
// 2048, r = 64, 67 -> 25.5 us.  With a block for each adapter small ranks lose: 1777 tokens of 6,
// 1016 -> 2728, r = 8, 12.7 -> 13.3.
int shares(int n, int r) {
    return std::max(1, std::min(BM, ceil_div((int)std::min<int64_t>((int64_t)n * r, BM * 128), 128)));
}

// Slices times tokens: tiles * splits is at most two an SM while there are splits.
int64_t lora_part_floats(int64_t m, int64_t r) {
    if (m <= kLoraByToken) return 0;
    return std::max<int64_t>(m, (int64_t)2 * sms() * BM) * r;
}

cudaError_t launch_lora_tiles(LoraArgs& p, cudaStream_t st) {
    const int tiles = ceil_div(p.m, BM);
    p.kblocks = ceil_div(p.K, BK);
    p.split_blocks = split_blocks(p.m, p.K);
    p.splits = ceil_div(p.kblocks, p.split_blocks);
    p.group = std::min(std::min(256 / p.r, p.n), BM);
    const uint64_t bdims[3] = {(uint64_t)p.r / 2, (uint64_t)p.N, (uint64_t)p.n};
    const uint64_t bstrides[2] = {(uint64_t)p.r * 2, (uint64_t)p.N * p.r * 2};
    const uint32_t bbox[3] = {BK / 2, BN, 1};
    if (!ffn_map(&p.mx, p.x, p.m, p.K, p.ldx, BM) || !ffn_map(&p.ma, p.a, (uint64_t)p.n * p.r, p.K, p.K, p.r) ||
        !tmap_encode_words(&p.mb, p.b, 3, bdims, bstrides, bbox) || !ffn_map(&p.my, p.y, p.m, p.N, p.ldy, BM) ||
        !ffn_map(&p.mo, p.out, p.m, p.N, p.ldo, 32))
        return cudaErrorUnknown;
    cudaError_t e = allow_smem<lora_shrink>(SHRINK_SMEM);
    if (e == cudaSuccess) e = allow_smem<lora_expand<false>>(kSmem);
    if (e == cudaSuccess) e = allow_smem<lora_expand<true>>(kSmem);
    if (e != cudaSuccess) return e;
    const int most = shares(p.n, p.r);
    e = launch_pdl(lora_shrink, dim3(tiles, p.splits, std::clamp(2 * sms() / (tiles * p.splits), 1, most)), dim3(SHRINK_THREADS), SHRINK_SMEM, st, p);
    if (e != cudaSuccess) return e;
    const int nb = ceil_div(p.r, BK);
    p.n_tiles = ceil_div(p.N, BN);
    p.n_ctas = std::max(1, std::min(p.n_tiles, sms() / tiles));
    const int room = kSmem - 1024 - 2 * nb * X_BYTES;
    p.stages = std::min(MAX_B, (room - YS * Y_BYTES) / X_BYTES);
    const int z = std::clamp(sms() / (tiles * p.n_ctas), 1, most);
    return launch_pdl(z > 1 ? lora_expand<true> : lora_expand<false>, dim3(tiles, p.n_ctas, z), dim3(EXPAND_THREADS),
                      1024 + 2 * nb * X_BYTES + YS * Y_BYTES + p.stages * X_BYTES, st, p);
}

}  // namespace moe
