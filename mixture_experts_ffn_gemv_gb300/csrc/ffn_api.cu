// C-ABI of the dense gated feed-forward block and the MXFP4 operators:
// argument checks, workspace layout and launch sequences.  Declarations and
// contracts: include/moe_ffn_block.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>

#include "common.cuh"
#include "ffn_block.h"
#include "ffn_box.cuh"

using namespace moe;

struct moe_ffn {
    moe_ffn_config cfg;  // first: the sizes below need nothing else of a handle
    int device;
    mutable int last_launches;
    mutable const void* last_ws;  // its header is known to be clean
    uint64_t wait_ns;
    int stall;
    // maps of the weights: along K (128-row boxes), along M or N, MXFP4 codes and scales
    CUtensorMap k1, k3, k2, mn1, mn3, mn2;
    int mn13_order, mn2_order;
    CUtensorMap s1, s3, s2;
};

namespace {

constexpr size_t kAlign = 256;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: limit of every bounded mbarrier wait
constexpr int kMaxDim = 1 << 20;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t scale_bytes(int64_t rows, int64_t n) { return (size_t)((rows + 127) / 128) * ((n + 127) / 128) * 512; }
template <typename T>
inline T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

struct Layout {
    size_t hdr, h, dg, du, xq, xs, hq, hs, total;
};
Layout layout(const moe_ffn* f, int64_t m, bool backward) {
    Layout o{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t p = off;
        off = align_up(off + bytes);
        return p;
    };
    const size_t H = f->cfg.hidden, I = f->cfg.inter;
    o.hdr = take(sizeof(WsHeader));
    if (f->cfg.weights == MOE_WEIGHTS_MXFP4) {
        o.xq = take((size_t)m * H / 2);
        o.xs = take(scale_bytes(m, H));
        o.hq = take((size_t)m * I / 2);
        o.hs = take(scale_bytes(m, I));
    } else {
        if (backward) {
            o.dg = take((size_t)m * I * 2);
            o.du = take((size_t)m * I * 2);
        } else {
            // up to kNarrowParts tokens take 2 kNarrowParts rows; at least as many for more
            // tokens, so that what holds m tokens holds fewer
            o.h = take((size_t)std::max<int64_t>(m, 2 * kNarrowParts) * I * 2);
        }
    }
    o.total = off;
    return o;
}

// The checks every call on a handle makes; *lo is the layout.
int check_call(const moe_ffn* f, int64_t m, bool backward, void* ws, size_t ws_bytes, Layout* lo) {
    if (!f || m < 0) return MOE_ERR_INVALID_ARG;
    if (m > INT32_MAX / 64) return MOE_ERR_UNSUPPORTED;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev != f->device) return MOE_ERR_INVALID_ARG;
    if (m == 0) return MOE_OK;
    *lo = layout(f, m, backward);
    if (!ws || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < lo->total) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

bool bad_rows(const void* p, int64_t ld, int64_t n) { return !p || !aligned(p, 16) || ld < n || ld % 8 || ld > (int64_t)1 << 38; }

FfnProducts products(const moe_ffn* f, void* ws) {
    FfnProducts p{};
    p.act = f->cfg.activation;
    p.hdr = at<WsHeader>(ws, 0);
    p.wait_ns = f->wait_ns;
    p.stall = f->stall;
    return p;
}

// A product of one source, D [M, N] over K.
FfnProduct& add(FfnProducts& p, int M, int N, int K, void* out) {
    FfnProduct& q = p.p[p.count++];
    q.sources = 1;
    q.M = M;
    q.N = N;
    q.kblocks = ceil_div(K, 64);
    q.out = static_cast<uint16_t*>(out);
    return q;
}

// f: the block, or null for a product of its own.
NarrowProduct narrow(const moe_ffn* f, int T, int R, int K, void* ws) {
    NarrowProduct p{};
    p.T = T;
    p.R = R;
    p.K = K;
    p.hdr = at<WsHeader>(ws, 0);
    p.wait_ns = f ? f->wait_ns : kWaitNs;
    p.stall = f ? f->stall : 0;
    return p;
}

// Each product of a bf16 block takes the kernel that suits its size.
int forward_bf16(const moe_ffn* f, const void* x, int64_t ldx, int m, void* out, float* saved, void* h, void* ws,
                 cudaStream_t st) {
    const int H = f->cfg.hidden, I = f->cfg.inter;
    const uint32_t nt = (uint32_t)narrow_tokens(m);
    const bool parts = m <= kNarrowParts && !saved;  // h is not kept: two parts (ffn_narrow.cu)
    float* saved_d = saved ? saved + saved_floats(m, I) : nullptr;
    if (narrow_is_faster(m, I, false)) {
        NarrowProduct g = narrow(f, m, I, H, ws);
        if (!ffn_map(&g.b[0], x, m, H, ldx, nt)) return MOE_ERR_CUDA;
        g.a[0] = f->k1;
        g.a[1] = f->k3;
        g.act = f->cfg.activation;
        g.out = static_cast<uint16_t*>(h);
        g.sa = saved;
        g.sd = saved_d;
        if (launch_ffn_narrow(g, false, parts ? NARROW_GATEUP_PARTS : NARROW_GATEUP, st) != cudaSuccess) return MOE_ERR_CUDA;
    } else {
        FfnProducts p = products(f, ws);
        FfnProduct& gu = add(p, m, I, H, h);
        if (!ffn_map(&gu.a[0], x, m, H, ldx, 128)) return MOE_ERR_CUDA;
        gu.b[0] = f->k1;
        gu.b[1] = f->k3;
        p.a = saved;
        p.d = saved_d;
        if (launch_ffn_products(p, saved ? EPI_GATEUP_SAVE : EPI_GATEUP, st) != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (narrow_is_faster(m, H, false)) {
        NarrowProduct d = narrow(f, m, H, I, ws);
        if (!ffn_map(&d.b[0], h, parts ? 2 * kNarrowParts : m, I, I, nt)) return MOE_ERR_CUDA;
        d.a[0] = f->k2;
        d.early = 1;  // behind the kernel that wrote h
        d.out = static_cast<uint16_t*>(out);
        if (launch_ffn_narrow(d, false, parts ? NARROW_PLAIN_PARTS : NARROW_PLAIN, st) != cudaSuccess) return MOE_ERR_CUDA;
    } else {
        FfnProducts d = products(f, ws);
        FfnProduct& y = add(d, m, H, I, out);
        if (!ffn_map(&y.a[0], h, m, I, I, 128)) return MOE_ERR_CUDA;
        y.b[0] = f->k2;
        if (launch_ffn_products(d, EPI_STORE, st) != cudaSuccess) return MOE_ERR_CUDA;
    }
    f->last_launches = 2;
    return MOE_OK;
}

MxProduct mx_product(const moe_ffn* f, int M, int N, int K, void* ws) {
    MxProduct p{};
    p.M = M;
    p.N = N;
    p.kblocks = ceil_div(K, 256);
    p.hdr = at<WsHeader>(ws, 0);
    p.wait_ns = f ? f->wait_ns : kWaitNs;
    p.stall = f ? f->stall : 0;
    return p;
}

int forward_mxfp4(const moe_ffn* f, const Layout& lo, const void* x, int64_t ldx, int m, void* out, void* ws,
                  cudaStream_t st) {
    const int H = f->cfg.hidden, I = f->cfg.inter;
    uint8_t *xq = at<uint8_t>(ws, lo.xq), *xs = at<uint8_t>(ws, lo.xs), *hq = at<uint8_t>(ws, lo.hq),
            *hs = at<uint8_t>(ws, lo.hs);
    f->last_launches = 3;
    if (narrow_is_faster(m, I, true)) {
        // each kernel after the quantiser streams its weights while the one before drains
        NarrowProduct g = narrow(f, m, I, H, ws), d = narrow(f, m, H, I, ws);
        const uint32_t nt = (uint32_t)narrow_tokens(m);
        const bool fused = m <= kNarrowQuant;  // x is quantised by the gate/up kernel itself
        if (fused) {
            g.x = static_cast<const uint16_t*>(x);
            g.ldx = (size_t)ldx;
        } else if (!mx_code_map(&g.b[0], xq, m, H, nt) || !mx_scale_map(&g.bs, xs, m, H)) {
            return MOE_ERR_CUDA;
        }
        if (!mx_code_map(&d.b[0], hq, m, I, nt) || !mx_scale_map(&d.bs, hs, m, I)) return MOE_ERR_CUDA;
        g.a[0] = f->k1;
        g.a[1] = f->k3;
        g.as[0] = f->s1;
        g.as[1] = f->s3;
        g.act = f->cfg.activation;
        g.codes = hq;
        g.scales = hs;
        g.nkt = ceil_div(I, 128);
        d.a[0] = f->k2;
        d.as[0] = f->s2;
        d.out = static_cast<uint16_t*>(out);
        g.early = !fused;
        d.early = 1;
        f->last_launches = fused ? 2 : 3;
        return (fused || launch_mx_quant(x, false, (size_t)ldx, m, H, xq, xs, st) == cudaSuccess) &&
                       launch_ffn_narrow(g, true, NARROW_GATEUP, st) == cudaSuccess &&
                       launch_ffn_narrow(d, true, NARROW_PLAIN, st) == cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    }
    MxProduct g = mx_product(f, m, I, H, ws), d = mx_product(f, m, H, I, ws);
    if (!mx_code_map(&g.a, xq, m, H, 128) || !mx_scale_map(&g.as, xs, m, H) || !mx_code_map(&d.a, hq, m, I, 128) ||
        !mx_scale_map(&d.as, hs, m, I))
        return MOE_ERR_CUDA;
    g.b[0] = f->k1;
    g.b[1] = f->k3;
    g.bs[0] = f->s1;
    g.bs[1] = f->s3;
    g.act = f->cfg.activation;
    g.codes = hq;
    g.scales = hs;
    g.nkt = ceil_div(I, 128);
    d.b[0] = f->k2;
    d.bs[0] = f->s2;
    d.out = static_cast<uint16_t*>(out);
    return launch_mx_quant(x, false, (size_t)ldx, m, H, xq, xs, st) == cudaSuccess &&
                   launch_mx_product(g, true, st) == cudaSuccess && launch_mx_product(d, false, st) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

// Rows and columns whose pieces of 16 elements the quantisers count in 32 bits.
bool too_large(int64_t rows, int64_t n) {
    return rows > INT32_MAX / 64 || n > INT32_MAX / 64 || rows * ((n + 511) / 512) > (int64_t)1 << 26;
}

int quant(const void* x, bool f32, int64_t ldx, int64_t rows, int64_t n, uint8_t* codes, uint8_t* scales,
          void* stream) {
    if (rows < 0 || n <= 0 || n % 32) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (too_large(rows, n)) return MOE_ERR_UNSUPPORTED;
    if (!x || !aligned(x, 16) || ldx < n || ldx % (f32 ? 4 : 8) || !codes || !scales || !aligned(codes, 16) ||
        !aligned(scales, 16))
        return MOE_ERR_INVALID_ARG;
    return launch_mx_quant(x, f32, (size_t)ldx, (int)rows, (int)n, codes, scales, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

// What moe_mxfp4_gemm and moe_mxfp4_linear check alike.
int check_gemm(int64_t m, int64_t n, int64_t k, const uint8_t* w, const uint8_t* ws, const void* out,
               const void* workspace, size_t bytes, size_t need) {
    if (m > INT32_MAX / 64 || n > kMaxDim || k > kMaxDim) return MOE_ERR_UNSUPPORTED;
    if (m == 0) return MOE_OK;
    if (!workspace || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
    if (bytes < need) return MOE_ERR_WORKSPACE;
    for (const void* p : {(const void*)w, (const void*)ws, out})
        if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// early: the preceding kernel on the stream is the quantiser of A.
int gemm(const uint8_t* a, const uint8_t* as, int m, const uint8_t* b, const uint8_t* bs, int n, int k, void* out,
         void* ws, bool early, cudaStream_t st) {
    if (narrow_is_faster(m, n, true)) {
        NarrowProduct q = narrow(nullptr, m, n, k, ws);
        if (!mx_code_map(&q.a[0], b, n, k, 128) || !mx_scale_map(&q.as[0], bs, n, k) ||
            !mx_code_map(&q.b[0], a, m, k, (uint32_t)narrow_tokens(m)) || !mx_scale_map(&q.bs, as, m, k))
            return MOE_ERR_CUDA;
        q.early = early;
        q.out = static_cast<uint16_t*>(out);
        return launch_ffn_narrow(q, true, NARROW_PLAIN, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    MxProduct g = mx_product(nullptr, m, n, k, ws);
    if (!mx_code_map(&g.a, a, m, k, 128) || !mx_scale_map(&g.as, as, m, k) || !mx_code_map(&g.b[0], b, n, k, 128) ||
        !mx_scale_map(&g.bs[0], bs, n, k))
        return MOE_ERR_CUDA;
    g.out = static_cast<uint16_t*>(out);
    return launch_mx_product(g, false, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

struct LinearLayout {
    size_t codes, scales, total;
};
LinearLayout linear_layout(int64_t m, int64_t k) {
    LinearLayout o;
    o.codes = align_up(sizeof(WsHeader));
    o.scales = align_up(o.codes + (size_t)m * k / 2);
    o.total = align_up(o.scales + scale_bytes(m, k));
    return o;
}

// Whether rows of k bf16 elements, ldx apart, and a dense [m, n] share memory.
bool overlap(const void* x, int64_t ldx, int64_t k, const void* out, int64_t n, int64_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(out);
    return a < b + (size_t)m * n * 2 && b < a + ((size_t)(m - 1) * ldx + k) * 2;
}

int linear(const void* x, bool f32, int64_t ldx, int64_t m, const uint8_t* w, const uint8_t* ws, int64_t n, int64_t k,
           void* out, void* workspace, size_t bytes, void* stream) {
    if (m < 0 || n <= 0 || n % 8 || k <= 0 || k % 32) return MOE_ERR_INVALID_ARG;
    const LinearLayout lo = linear_layout(m, k);
    const int rc = check_gemm(m, n, k, w, ws, out, workspace, bytes, lo.total);
    if (rc != MOE_OK || m == 0) return rc;
    // quantised by the product's kernel itself, whose CTAs read x to the end while
    // others write: only where out is not (part of) x
    if (m <= kNarrowQuant && !f32 && !overlap(x, ldx, k, out, n, m)) {
        if (!x || !aligned(x, 16) || ldx < k || ldx % 8) return MOE_ERR_INVALID_ARG;
        NarrowProduct q = narrow(nullptr, (int)m, (int)n, (int)k, workspace);
        if (!mx_code_map(&q.a[0], w, n, k, 128) || !mx_scale_map(&q.as[0], ws, n, k)) return MOE_ERR_CUDA;
        q.x = static_cast<const uint16_t*>(x);
        q.ldx = (size_t)ldx;
        q.out = static_cast<uint16_t*>(out);
        return launch_ffn_narrow(q, true, NARROW_PLAIN, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    uint8_t *codes = at<uint8_t>(workspace, lo.codes), *scales = at<uint8_t>(workspace, lo.scales);
    const int qc = quant(x, f32, ldx, m, k, codes, scales, stream);
    if (qc != MOE_OK) return qc;
    return gemm(codes, scales, (int)m, w, ws, (int)n, (int)k, out, workspace, true, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int moe_ffn_create(const moe_ffn_config* cfg, const moe_ffn_weights* w, moe_ffn** out) {
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    if (!cfg || !w) return MOE_ERR_INVALID_ARG;
    const moe_ffn_config& c = *cfg;
    if (c.weights != MOE_WEIGHTS_BF16 && c.weights != MOE_WEIGHTS_MXFP4) return MOE_ERR_INVALID_ARG;
    if (c.activation != MOE_ACT_SILU && c.activation != MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
    const bool mx = c.weights == MOE_WEIGHTS_MXFP4;
    const int mult = mx ? 32 : 8;
    if (c.hidden <= 0 || c.inter <= 0) return MOE_ERR_INVALID_ARG;
    if (c.hidden % mult || c.inter % mult || c.hidden > kMaxDim || c.inter > kMaxDim) return MOE_ERR_UNSUPPORTED;
    const void* ptrs[6] = {w->w1, w->w3, w->w2, w->s1, w->s3, w->s2};
    for (int i = 0; i < 6; ++i) {
        if (i >= 3 && !mx) {
            if (ptrs[i]) return MOE_ERR_INVALID_ARG;
        } else if (!ptrs[i] || !aligned(ptrs[i], 16)) {
            return MOE_ERR_INVALID_ARG;
        }
    }
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    moe_ffn* f = new (std::nothrow) moe_ffn();
    if (!f) return MOE_ERR_CUDA;
    f->cfg = c;
    f->device = dev;
    f->wait_ns = kWaitNs;
    const uint64_t H = c.hidden, I = c.inter;
    const bool ok = mx ? mx_code_map(&f->k1, w->w1, I, H, 128) && mx_code_map(&f->k3, w->w3, I, H, 128) &&
                             mx_code_map(&f->k2, w->w2, H, I, 128) && mx_scale_map(&f->s1, w->s1, I, H) &&
                             mx_scale_map(&f->s3, w->s3, I, H) && mx_scale_map(&f->s2, w->s2, H, I)
                       : ffn_map(&f->k1, w->w1, I, H, H, 128) && ffn_map(&f->k3, w->w3, I, H, H, 128) &&
                             ffn_map(&f->k2, w->w2, H, I, I, 128) &&
                             (f->mn13_order = ffn_map_mn(&f->mn1, w->w1, I, H, H)) &&
                             ffn_map_mn(&f->mn3, w->w3, I, H, H) == f->mn13_order &&
                             (f->mn2_order = ffn_map_mn(&f->mn2, w->w2, H, I, I));
    if (!ok) {
        delete f;
        return MOE_ERR_CUDA;
    }
    *out = f;
    return MOE_OK;
}

int moe_ffn_destroy(moe_ffn* f) {
    delete f;
    return MOE_OK;
}

int moe_ffn_set_wait_limit(moe_ffn* f, uint64_t ns) {
    if (!f) return MOE_ERR_INVALID_ARG;
    f->wait_ns = ns ? ns : kWaitNs;
    return MOE_OK;
}

int moe_ffn_stall_test(moe_ffn* f, int enable) {
    if (!f || (enable != 0 && enable != 1)) return MOE_ERR_INVALID_ARG;
    f->stall = enable;
    return MOE_OK;
}

int moe_ffn_workspace_size(const moe_ffn* f, int64_t m, int backward, size_t* bytes) {
    if (!f || m < 0 || !bytes || (backward != 0 && backward != 1)) return MOE_ERR_INVALID_ARG;
    if (m > INT32_MAX / 64) return MOE_ERR_UNSUPPORTED;
    *bytes = layout(f, m, backward != 0).total;
    return MOE_OK;
}

int moe_ffn_saved_size(const moe_ffn* f, int64_t m, size_t* bytes) {
    if (!f || m < 0 || !bytes) return MOE_ERR_INVALID_ARG;
    if (f->cfg.weights != MOE_WEIGHTS_BF16 || m > INT32_MAX / 64) return MOE_ERR_UNSUPPORTED;
    *bytes = saved_floats(m, f->cfg.inter) * 8 + (size_t)m * f->cfg.inter * 2;
    return MOE_OK;
}

int moe_ffn_forward(const moe_ffn* f, const void* x, int64_t ldx, int64_t m, void* out, void* saved, void* workspace,
                    size_t workspace_bytes, void* stream) {
    Layout lo;
    const int rc = check_call(f, m, false, workspace, workspace_bytes, &lo);
    if (rc != MOE_OK || m == 0) return rc;
    if (bad_rows(x, ldx, f->cfg.hidden) || !out || !aligned(out, 16) || (saved && !aligned(saved, 32)))
        return MOE_ERR_INVALID_ARG;
    const bool mx = f->cfg.weights == MOE_WEIGHTS_MXFP4;
    if (mx && (saved || too_large(m, f->cfg.hidden))) return MOE_ERR_UNSUPPORTED;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (clear_header(f->last_ws, workspace, st) != cudaSuccess) return MOE_ERR_CUDA;
    float* sa = static_cast<float*>(saved);
    void* h = saved ? sa + 2 * saved_floats(m, f->cfg.inter) : at<void>(workspace, lo.h);
    return mx ? forward_mxfp4(f, lo, x, ldx, (int)m, out, workspace, st)
              : forward_bf16(f, x, ldx, (int)m, out, sa, h, workspace, st);
}

int moe_ffn_backward(const moe_ffn* f, const void* dout, int64_t ldd, const void* x, int64_t ldx, const void* saved,
                     int64_t m, void* dx, void* dw1, void* dw3, void* dw2, void* workspace, size_t workspace_bytes,
                     void* stream) {
    Layout lo;
    if (f && f->cfg.weights != MOE_WEIGHTS_BF16) return MOE_ERR_UNSUPPORTED;
    const int rc = check_call(f, m, true, workspace, workspace_bytes, &lo);
    if (rc != MOE_OK || m == 0) return rc;
    const int H = f->cfg.hidden, I = f->cfg.inter, n = (int)m;
    const bool dw = dw1 || dw3 || dw2;
    if (bad_rows(dout, ldd, H) || bad_rows(x, ldx, H) || !saved || !aligned(saved, 32) || (dx && !aligned(dx, 16)) ||
        (dw && (!dw1 || !dw3 || !dw2 || !aligned(dw1, 16) || !aligned(dw3, 16) || !aligned(dw2, 16))))
        return MOE_ERR_INVALID_ARG;
    if (!dx && !dw) return MOE_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (clear_header(f->last_ws, workspace, st) != cudaSuccess) return MOE_ERR_CUDA;
    void *dg = at<void>(workspace, lo.dg), *du = at<void>(workspace, lo.du);
    float* sa = static_cast<float*>(const_cast<void*>(saved));  // only read
    float *sd = sa + saved_floats(m, I), *h = sd + saved_floats(m, I);
    const uint32_t nt = (uint32_t)narrow_tokens(n);
    // dh = dout W2 and, in its epilogue, dg and du
    if (narrow_is_faster(n, I, false)) {
        NarrowProduct q = narrow(f, n, I, H, workspace);
        if (!ffn_map(&q.b[0], dout, m, H, ldd, nt)) return MOE_ERR_CUDA;
        q.a[0] = f->mn2;
        q.a_mn = f->mn2_order;
        q.sa = sa;
        q.sd = sd;
        q.out = static_cast<uint16_t*>(dg);
        q.du = static_cast<uint16_t*>(du);
        if (launch_ffn_narrow(q, false, NARROW_DACT, st) != cudaSuccess) return MOE_ERR_CUDA;
    } else {
        FfnProducts p = products(f, workspace);
        FfnProduct& q = add(p, n, I, H, dg);
        if (!ffn_map(&q.a[0], dout, m, H, ldd, 128)) return MOE_ERR_CUDA;
        q.b[0] = f->mn2;
        q.b_mn = f->mn2_order;
        p.a = sa;
        p.d = sd;
        p.out_du = static_cast<uint16_t*>(du);
        if (launch_ffn_products(p, EPI_DACT, st) != cudaSuccess) return MOE_ERR_CUDA;
    }
    f->last_launches = 1;
    // dx, by itself or with the weight gradients in one launch
    FfnProducts r = products(f, workspace);
    if (dx && narrow_is_faster(n, H, false)) {
        NarrowProduct d = narrow(f, n, H, I, workspace);
        if (!ffn_map(&d.b[0], dg, m, I, I, nt) || !ffn_map(&d.b[1], du, m, I, I, nt)) return MOE_ERR_CUDA;
        d.a[0] = f->mn1;
        d.a[1] = f->mn3;
        d.a_mn = f->mn13_order;
        d.early = 1;  // behind the kernel that wrote dg and du
        d.out = static_cast<uint16_t*>(dx);
        if (launch_ffn_narrow(d, false, NARROW_DX, st) != cudaSuccess) return MOE_ERR_CUDA;
        ++f->last_launches;
    }
    const auto add_dx = [&] {
        FfnProduct& d = add(r, n, H, I, dx);
        d.sources = 2;
        d.b[0] = f->mn1;
        d.b[1] = f->mn3;
        d.b_mn = f->mn13_order;
        return ffn_map(&d.a[0], dg, m, I, I, 128) && ffn_map(&d.a[1], du, m, I, I, 128);
    };
    const bool wide_dx = dx && !narrow_is_faster(n, H, false), dx_first = 2 * ceil_div(I, 64) >= ceil_div(n, 64);
    if (wide_dx && dx_first && !add_dx()) return MOE_ERR_CUDA;
    if (dw) {
        // dw1 = dg^T x, dw3 = du^T x, dw2 = dout^T h
        const void* lhs[3] = {dg, du, dout};
        void* out[3] = {dw1, dw3, dw2};
        for (int i = 0; i < 3; ++i) {
            FfnProduct& g = i < 2 ? add(r, I, H, n, out[i]) : add(r, H, I, n, out[i]);
            g.a_mn = i < 2 ? ffn_map_mn(&g.a[0], lhs[i], m, I, I) : ffn_map_mn(&g.a[0], dout, m, H, ldd);
            g.b_mn = i < 2 ? ffn_map_mn(&g.b[0], x, m, H, ldx) : ffn_map_mn(&g.b[0], h, m, I, I);
            if (!g.a_mn || !g.b_mn) return MOE_ERR_CUDA;
        }
    }
    if (wide_dx && !dx_first && !add_dx()) return MOE_ERR_CUDA;
    if (r.count) {
        if (launch_ffn_products(r, EPI_STORE, st) != cudaSuccess) return MOE_ERR_CUDA;
        ++f->last_launches;
    }
    return MOE_OK;
}

int moe_ffn_last_launch_count(const moe_ffn* f) { return f ? f->last_launches : -1; }

int moe_mxfp4_scales_size(int64_t rows, int64_t n, size_t* bytes) {
    if (rows < 0 || n <= 0 || n % 32 || !bytes) return MOE_ERR_INVALID_ARG;
    if (rows > INT32_MAX / 64 || n > INT32_MAX / 64) return MOE_ERR_UNSUPPORTED;
    *bytes = scale_bytes(rows, n);
    return MOE_OK;
}

int moe_mxfp4_quant(const void* x, int64_t ldx, int64_t rows, int64_t n, uint8_t* codes, uint8_t* scales,
                    void* stream) {
    return quant(x, false, ldx, rows, n, codes, scales, stream);
}

int moe_mxfp4_quant_f32(const float* x, int64_t ldx, int64_t rows, int64_t n, uint8_t* codes, uint8_t* scales,
                        void* stream) {
    return quant(x, true, ldx, rows, n, codes, scales, stream);
}

int moe_mxfp4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t n, void* out, void* stream) {
    if (rows < 0 || n <= 0 || n % 32) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (too_large(rows, n)) return MOE_ERR_UNSUPPORTED;
    if (!codes || !scales || !out || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16))
        return MOE_ERR_INVALID_ARG;
    return launch_mx_dequant(codes, scales, (int)rows, (int)n, static_cast<uint16_t*>(out),
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

int moe_mxfp4_gemm_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
    if (m < 0 || n <= 0 || n % 8 || k <= 0 || k % 32 || !bytes) return MOE_ERR_INVALID_ARG;
    *bytes = align_up(sizeof(WsHeader));
    return MOE_OK;
}

int moe_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, const uint8_t* b_codes,
                   const uint8_t* b_scales, int64_t n, int64_t k, void* out, void* workspace, size_t workspace_bytes,
                   void* stream) {
    size_t need = 0;
    int rc = moe_mxfp4_gemm_workspace_size(m, n, k, &need);
    if (rc == MOE_OK) rc = check_gemm(m, n, k, b_codes, b_scales, out, workspace, workspace_bytes, need);
    if (rc != MOE_OK || m == 0) return rc;
    if (!a_codes || !a_scales || !aligned(a_codes, 16) || !aligned(a_scales, 16)) return MOE_ERR_INVALID_ARG;
    return gemm(a_codes, a_scales, (int)m, b_codes, b_scales, (int)n, (int)k, out, workspace, false,
                static_cast<cudaStream_t>(stream));
}

int moe_mxfp4_linear_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
    if (m < 0 || n <= 0 || n % 8 || k <= 0 || k % 32 || !bytes) return MOE_ERR_INVALID_ARG;
    if (m > INT32_MAX / 64 || n > kMaxDim || k > kMaxDim) return MOE_ERR_UNSUPPORTED;
    *bytes = linear_layout(m, k).total;
    return MOE_OK;
}

int moe_mxfp4_linear(const void* x, int64_t ldx, int64_t m, const uint8_t* w_codes, const uint8_t* w_scales, int64_t n,
                     int64_t k, void* out, void* workspace, size_t workspace_bytes, void* stream) {
    return linear(x, false, ldx, m, w_codes, w_scales, n, k, out, workspace, workspace_bytes, stream);
}

int moe_mxfp4_linear_f32(const float* x, int64_t ldx, int64_t m, const uint8_t* w_codes, const uint8_t* w_scales,
                         int64_t n, int64_t k, void* out, void* workspace, size_t workspace_bytes, void* stream) {
    return linear(x, true, ldx, m, w_codes, w_scales, n, k, out, workspace, workspace_bytes, stream);
}

}  // extern "C"
