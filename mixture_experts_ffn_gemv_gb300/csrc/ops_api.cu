// C-ABI of the operators around the layer and the block: argument checks and
// launches.  Declarations and contracts: include/moe_ffn_ops.h.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "moe_ffn_ops.h"
#include "ops.h"

using namespace moe;

namespace {

constexpr size_t kAlign = 256;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: limit of every bounded mbarrier wait
std::atomic<uint64_t> lora_wait_ns{kWaitNs};
std::atomic<int> lora_stall{0};
constexpr int64_t kMaxRows = INT32_MAX / 64;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// bf16 rows of n elements, ld apart
bool bad_rows(const void* p, int64_t ld, int64_t n) {
    return !p || !aligned(p, 16) || ld < n || ld % 8 || ld > (int64_t)1 << 38;
}
// m rows of n bytes, ld bytes apart
struct Rows {
    uintptr_t at;
    int64_t ld, n;
};
Rows rows16(const void* p, int64_t ld, int64_t n) { return {reinterpret_cast<uintptr_t>(p), 2 * ld, 2 * n}; }
// Whether two matrices of m rows share memory: their spans meet and, where their
// rows are as far apart, so do their columns.
bool share(const Rows& a, const Rows& b, int64_t m) {
    const auto end = [&](const Rows& q) { return (unsigned __int128)q.at + (unsigned __int128)(m - 1) * q.ld + q.n; };
    if (!a.at || !b.at || a.at >= end(b) || b.at >= end(a)) return false;
    if (m == 1 || a.ld != b.ld) return true;
    const int64_t ahead = b.at >= a.at ? (int64_t)(b.at - a.at) % a.ld : (a.ld - (int64_t)(a.at - b.at) % a.ld) % a.ld;
    return ahead < a.n || ahead + b.n > a.ld;
}
// ... where the two may be the same rows
bool share_part(const Rows& a, const Rows& b, int64_t m) {
    return !(a.at == b.at && a.n == b.n && (m == 1 || a.ld == b.ld)) && share(a, b, m);
}
bool bad_words(const void* p) { return !p || !aligned(p, 4); }
int check_norm(int64_t m, int64_t h) {
    if (m < 0 || h <= 0 || h % 8) return MOE_ERR_INVALID_ARG;
    return m > kMaxRows || h > kNormMaxH ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
int check_router(int64_t m, int32_t e, int32_t k, const int32_t* off, int64_t seqs, int scoring) {
    if (m < 0 || e <= 0 || k <= 0 || k > e || seqs <= 0 || (!off && seqs != 1)) return MOE_ERR_INVALID_ARG;
    if (scoring != MOE_SCORING_SOFTMAX && scoring != MOE_SCORING_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (off && !aligned(off, 4)) return MOE_ERR_INVALID_ARG;
    return e > kMaxExperts || k > kMaxTopK || m > kMaxRows || seqs > 1 << 24 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
int status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

__device__ WsHeader captured_errors;  // of workspaces that a graph's pool takes back

__global__ void captured_header(WsHeader* h) {
    pdl_wait();  // the workspace's memory may be in use until then
    pdl_trigger();
    reinterpret_cast<int4*>(h)[threadIdx.x] = make_int4(0, 0, 0, 0);
    __syncthreads();
    if (threadIdx.x == 0) {
        h->errors_at = reinterpret_cast<unsigned long long>(&captured_errors);
        h->errors_at_not = ~h->errors_at;
    }
}

}  // namespace

extern "C" {

int moe_captured_header(void* workspace, void* stream) {
    if (!workspace || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
    return status(launch_pdl(captured_header, dim3(1), dim3(sizeof(WsHeader) / 16), 0, static_cast<cudaStream_t>(stream),
                             static_cast<WsHeader*>(workspace)));
}

int moe_captured_status(void* stream, int32_t* device_code) {
    if (!device_code) return MOE_ERR_INVALID_ARG;
    void* at = nullptr;
    if (cudaGetSymbolAddress(&at, captured_errors) != cudaSuccess) return MOE_ERR_CUDA;
    return moe_device_status(at, stream, device_code);
}

int moe_add_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t m, int64_t h,
                    const float* weight, float eps, void* residual_out, int64_t ldo, void* out, uint8_t* codes,
                    float* scales, void* stream) {
    const int rc = check_norm(m, h);
    if (rc != MOE_OK || m == 0) return rc;
    if (bad_rows(x, ldx, h) || !weight || !aligned(weight, 16) || !(eps >= 0.f) || !std::isfinite(eps))
        return MOE_ERR_INVALID_ARG;
    if (residual ? bad_rows(residual, ldr, h) || bad_rows(residual_out, ldo, h) : residual_out != nullptr)
        return MOE_ERR_INVALID_ARG;
    if ((!out && !codes) || (codes != nullptr) != (scales != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
    const int64_t blocks = (h + 127) / 128;
    const Rows rx = rows16(x, ldx, h), rr = rows16(residual, ldr, h), rn = rows16(residual_out, ldo, h), ro = rows16(out, h, h),
               rc8{reinterpret_cast<uintptr_t>(codes), h, h}, rs{reinterpret_cast<uintptr_t>(scales), 4 * blocks, 4 * blocks};
    if (share_part(rn, rr, m) || share(rn, rx, m) || share_part(ro, rx, m) || share(ro, rr, m) || share(ro, rn, m))
        return MOE_ERR_INVALID_ARG;
    for (const Rows& q : {rx, rr, rn, ro})
        if (share(rc8, q, m) || share(rs, q, m)) return MOE_ERR_INVALID_ARG;
    if (share(rc8, rs, m)) return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.res = static_cast<const uint16_t*>(residual);
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldo = ldo;
    a.w = weight;
    a.eps = eps;
    a.res_out = static_cast<uint16_t*>(residual_out);
    a.out = static_cast<uint16_t*>(out);
    a.codes = codes;
    a.scales = scales;
    a.m = (int)m;
    a.H = (int)h;
    return status(launch_add_rmsnorm(a, static_cast<cudaStream_t>(stream)));
}

int moe_add_rmsnorm_backward_workspace_size(int64_t m, int64_t h, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const int rc = check_norm(m, h);
    if (rc == MOE_OK) *bytes = align_up((size_t)norm_grad_blocks((int)m, (int)h) * h * 4);
    return rc;
}

int moe_add_rmsnorm_backward(const void* dout, int64_t ldd, const void* r, int64_t ldr, int64_t m, int64_t h,
                             const float* weight, float eps, const void* dresidual, int64_t ldq, void* dx,
                             float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    size_t need = 0;
    const int rc = moe_add_rmsnorm_backward_workspace_size(m, h, &need);
    if (rc != MOE_OK || m == 0) return rc;
    if (bad_rows(dout, ldd, h) || bad_rows(r, ldr, h) || !weight || !aligned(weight, 16) || !(eps >= 0.f) ||
        !std::isfinite(eps) || (dresidual && bad_rows(dresidual, ldq, h)) || !dx || !aligned(dx, 16))
        return MOE_ERR_INVALID_ARG;
    const Rows rx = rows16(dx, h, h);
    if (share_part(rx, rows16(dout, ldd, h), m) || share_part(rx, rows16(dresidual, ldq, h), m) || share(rx, rows16(r, ldr, h), m))
        return MOE_ERR_INVALID_ARG;
    if (dweight) {
        if (!aligned(dweight, 4) || !workspace || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
        if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    }
    NormGradArgs a{};
    a.dout = static_cast<const uint16_t*>(dout);
    a.r = static_cast<const uint16_t*>(r);
    a.dres = static_cast<const uint16_t*>(dresidual);
    a.ldd = ldd;
    a.ldr = ldr;
    a.ldq = ldq;
    a.w = weight;
    a.eps = eps;
    a.dx = static_cast<uint16_t*>(dx);
    a.dw = dweight;
    a.part = static_cast<float*>(workspace);
    a.m = (int)m;
    a.H = (int)h;
    return status(launch_add_rmsnorm_backward(a, static_cast<cudaStream_t>(stream)));
}

int moe_balance_loss_workspace_size(int64_t m, int64_t seqs, size_t* bytes) {
    if (m < 0 || seqs <= 0 || !bytes) return MOE_ERR_INVALID_ARG;
    if (m > kMaxRows || seqs > 1 << 24) return MOE_ERR_UNSUPPORTED;
    *bytes = align_up((size_t)seqs * 4) + align_up((size_t)balance_slots(m, seqs) * 8);
    return MOE_OK;
}

int moe_balance_loss(const float* logits, const int32_t* topk_ids, int64_t m, int32_t e, int32_t k,
                     const int32_t* seq_offsets, int64_t seqs, int scoring, float* balance, float* z, int32_t* counts,
                     void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_router(m, e, k, seq_offsets, seqs, scoring);
    if (rc != MOE_OK || m == 0) return rc;
    if (bad_words(logits) || bad_words(topk_ids) || bad_words(balance) || bad_words(z) || bad_words(counts) || !workspace ||
        !aligned(workspace, kAlign))
        return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_balance_loss_workspace_size(m, seqs, &need);
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    RouterArgs a{};
    a.logits = logits;
    a.ids = topk_ids;
    a.off = seq_offsets;
    a.m = (int)m;
    a.E = e;
    a.k = k;
    a.S = (int)seqs;
    a.sigmoid = scoring == MOE_SCORING_SIGMOID;
    a.counts = counts;
    a.balance = balance;
    a.z = z;
    a.ticket = static_cast<int*>(workspace);
    a.part = reinterpret_cast<float2*>(static_cast<char*>(workspace) + align_up((size_t)seqs * 4));
    return status(launch_balance_loss(a, static_cast<cudaStream_t>(stream)));
}

int moe_route_backward(const float* logits, const int32_t* topk_ids, int64_t m, int32_t e, int32_t k, int scoring,
                       int norm_topk_prob, float routed_scaling_factor, const float* dtopk_w,
                       const int32_t* seq_offsets, int64_t seqs, const int32_t* counts, const float* dbalance,
                       const float* dz, float* dlogits, void* stream) {
    const int rc = check_router(m, e, k, seq_offsets, seqs, scoring);
    if (rc != MOE_OK) return rc;
    if (scoring == MOE_SCORING_SIGMOID && ((norm_topk_prob != 0 && norm_topk_prob != 1) || !(routed_scaling_factor > 0.f) ||
                                           !std::isfinite(routed_scaling_factor)))
        return MOE_ERR_INVALID_ARG;
    if (m == 0) return MOE_OK;
    const Rows rl{reinterpret_cast<uintptr_t>(logits), 4 * (int64_t)e, 4 * (int64_t)e}, rd{reinterpret_cast<uintptr_t>(dlogits), rl.ld, rl.n};
    if (bad_words(logits) || bad_words(topk_ids) || bad_words(dlogits) || share(rd, rl, m) || !aligned(dtopk_w, 4) ||
        !aligned(counts, 4) || !aligned(dbalance, 4) || !aligned(dz, 4) || (dbalance && !counts))
        return MOE_ERR_INVALID_ARG;
    RouterArgs a{};
    a.logits = logits;
    a.ids = topk_ids;
    a.off = seq_offsets;
    a.m = (int)m;
    a.E = e;
    a.k = k;
    a.S = (int)seqs;
    a.sigmoid = scoring == MOE_SCORING_SIGMOID;
    a.counts = const_cast<int32_t*>(counts);  // only read
    a.dtopk_w = dtopk_w;
    a.dbalance = dbalance;
    a.dz = dz;
    a.norm = norm_topk_prob;
    a.scale = a.sigmoid ? routed_scaling_factor : 1.f;
    a.dlogits = dlogits;
    return status(launch_route_backward(a, static_cast<cudaStream_t>(stream)));
}

int moe_lora_add_workspace_size(int64_t m, int64_t k, int64_t r, size_t* bytes) {
    if (m < 0 || k <= 0 || k % 8 || r <= 0 || r % 8 || !bytes) return MOE_ERR_INVALID_ARG;
    if (m > kMaxRows || k > 1 << 20 || r > kLoraMaxRank) return MOE_ERR_UNSUPPORTED;
    *bytes = align_up(sizeof(WsHeader)) + align_up((size_t)lora_part_floats(m, r) * 4);
    return MOE_OK;
}

int moe_lora_add(const void* x, int64_t ldx, int64_t m, int64_t k, const void* y, int64_t ldy, int64_t d, const void* a,
                 const void* b, int64_t n, int64_t r, const int32_t* ids, const float* scale, void* out, int64_t ldo,
                 void* workspace, size_t workspace_bytes, void* stream) {
    size_t need = 0;
    const int rc = moe_lora_add_workspace_size(m, k, r, &need);
    if (rc != MOE_OK) return rc;
    if (d <= 0 || d % 8 || n <= 0) return MOE_ERR_INVALID_ARG;
    if (d > 1 << 20 || n > (1 << 30) / r) return MOE_ERR_UNSUPPORTED;
    if (m == 0) return MOE_OK;
    if (bad_rows(x, ldx, k) || bad_rows(y, ldy, d) || bad_rows(out, ldo, d) ||
        share_part(rows16(out, ldo, d), rows16(y, ldy, d), m) || share(rows16(out, ldo, d), rows16(x, ldx, k), m) || !a ||
        !b || !aligned(a, 16) || !aligned(b, 16) || bad_words(ids) || !aligned(scale, 4) || !workspace ||
        !aligned(workspace, kAlign))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    LoraArgs p{};
    p.x = static_cast<const uint16_t*>(x);
    p.y = static_cast<const uint16_t*>(y);
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.out = static_cast<uint16_t*>(out);
    p.scale = scale;
    p.ids = ids;
    p.ldx = ldx;
    p.ldy = ldy;
    p.ldo = ldo;
    p.m = (int)m;
    p.K = (int)k;
    p.N = (int)d;
    p.r = (int)r;
    p.n = (int)n;
    p.hdr = static_cast<WsHeader*>(workspace);
    p.wait_ns = lora_wait_ns.load(std::memory_order_relaxed);
    p.stall = lora_stall.load(std::memory_order_relaxed);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + align_up(sizeof(WsHeader)));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return status(lora_by_token(p.m, p.n, p.r) ? launch_lora_tokens(p, st) : launch_lora_tiles(p, st));
}

int moe_lora_set_wait_limit(uint64_t ns) {
    lora_wait_ns = ns ? ns : kWaitNs;
    return MOE_OK;
}

int moe_lora_stall_test(int kernel) {
    if (kernel < 0 || kernel > 2) return MOE_ERR_INVALID_ARG;
    lora_stall = kernel;
    return MOE_OK;
}

}  // extern "C"
