// ops_internal.h -- parameters passed from the host checks (kda_ops_api.cu) to
// the kernels of include/kda_ops.h, their launchers, and the element-type
// helpers those kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace kda {

struct ConvParams {
    const void* x;
    void* out;                // nullptr: states only
    const void* w;
    const float* bias;
    void* pool;               // [P, W - 1, C] or nullptr
    const int32_t* slot;
    const int32_t* has_state;
    const int32_t* accepted;
    const int32_t* cu;        // nullptr: padded
    int32_t* status;
    int64_t xs[2], os[2];
    int N, T;                 // sequences; tokens a sequence (padded) or in all (packed)
    int64_t total;            // tokens in all
    int C, norm_c, P;
    int silu;
    int tile, cblocks;        // tokens a tile, blocks of channels (set by the launcher)
    float eps;
};
cudaError_t launch_short_conv(const ConvParams& p, int width, bool f16, bool w_f32, int num_sms, cudaStream_t s);

struct RopeParams {
    const void *q, *k, *v;
    void *q_out, *k_out, *k_cache, *v_cache;
    const int64_t* slots;
    const int32_t* positions;
    const float* inv_freq;
    const void *q_w, *k_w;
    int32_t* status;
    int64_t qs[3], ks[3], vs[3], qos[3], kos[3], kcs[3], vcs[3];
    int64_t tokens;           // batch * T
    int T, Hq, Hk, D, rot;
    int64_t cache_rows;       // num_pages * page_size
    int page;
    int norm, interleaved, w_f32;
    int chunks, chunk_passes; // a token's heads are cut into `chunks` runs (set by the launcher)
    float eps, scale;
};
cudaError_t launch_qk_norm_rope(const RopeParams& p, bool f16, int num_sms, cudaStream_t s);

struct TreeParams {
    const void *q, *kc, *vc;
    void* out;
    float* lse;
    const int32_t* table;
    const int32_t* ctx;
    const int32_t* nodes;
    const uint64_t* mask;
    int32_t* status;
    float* part_o;            // partial rows [2 CTAs, slot_rows, D] of items that are cut
    float* part_lse;          // their log-sums, base 2
    int4* parts;              // what they belong to, [2 CTAs]: state (0 nothing, 1 a part, 2 an item's
                              // last), request, key head, block of slot_rows rows
    int64_t qs[3], os[3], ks[3], vs[3], table_stride;
    int R, N, Hq, Hk, G, rows, words;   // rows = N * G, words of a mask row
    int P, page;
    int64_t max_len;          // longest context and nodes of a request (at most what its page row holds)
    uint32_t page_magic, group_magic;   // floor(2^32 / page), floor(2^32 / G) (2^32 - 1 for 1)
    int cluster;              // rows kernel: CTAs that share an item
    int32_t* order;           // the requests, longest first; nullptr: in their order
    int row_blocks, stages;   // set by the launcher
    int k_paged, v_paged;     // mma: the head is part of the map's page coordinate
    int r0, count;            // mma: the requests of a launch (set by the launcher)
    int slots, slot_rows;     // 2 x the CTAs over a line of items, rows of a slot (set by the launcher)
    float scale_log2;         // scale * log2(e)
    uint64_t wait_ns;         // mma: bound of the working waits (set by the entry; a wind-down's are kWaitLimitNs)
    int timeout_probe;        // mma: the softmax warps' first wait runs out (tests)
};
constexpr int kTreeSlice = 256;   // requests a launch of the kernel for many rows takes
// How a call is cut.
struct TreePlan {
    bool mma;            // the kernel for many rows
    bool line;           // rows kernel: CTAs over equal stretches of the line of items
    int row_grid;        // and their number
    int cluster;         // rows kernel: CTAs that share an item
    int grid;            // mma: CTAs
    size_t part_rows;    // partial rows in the workspace (D values and a log-sum each)
    size_t parts;        // int4, for what they belong to
    size_t order;        // int32, for the requests' order
};
TreePlan tree_plan(int R, int Hk, int rows, int D, int64_t max_len, int page, float scale, int num_sms);
cudaError_t launch_tree_attention(const TreeParams& p, const TreePlan& plan, int D, bool f16, cudaStream_t s);
cudaError_t launch_tree_join(const TreeParams& p, int D, bool f16, cudaStream_t s);
// The kernel for many rows; false if the caches' layout has no tensor map.
bool launch_tree_mma(const TreeParams& p, int D, bool f16, int grid, cudaStream_t s, cudaError_t* e);

// n / page for n < 2^32 and magic = floor(2^32 / page): the product is short by at most one.
__device__ __forceinline__ uint32_t page_div(uint32_t n, uint32_t page, uint32_t magic) {
    uint32_t q = __umulhi(n, magic);
    if (n - q * page >= page) ++q;
    return q;
}

// Context and drafted tokens of a request; false (and no tokens) if they do
// not fit the call.
__device__ __forceinline__ bool tree_lengths(const TreeParams& p, int r, int& ctx, int& n) {
    ctx = p.ctx[r];
    n = p.nodes ? p.nodes[r] : p.N;
    const bool ok = ctx >= 0 && n >= 0 && n <= p.N && (int64_t)ctx + n <= p.max_len;
    if (!ok) ctx = n = 0;
    return ok;
}

// Which of the positions tok .. tok + 31 of a request with `ctx` cached tokens and
// positions below `hi` its node sees, a bit each; mask: the node's words, nullptr: a chain.
__device__ __forceinline__ const uint32_t* tree_mask_row(const TreeParams& p, int r, int node) {
    return p.mask ? reinterpret_cast<const uint32_t*>(p.mask + ((int64_t)r * p.N + node) * p.words) : nullptr;
}
__device__ __forceinline__ uint32_t tree_seen(const TreeParams& p, const uint32_t* mask, int node, int ctx, int hi,
                                              int tok) {
    auto node_bits = [&](int w) -> uint32_t {   // drafted nodes 32 w ..
        if (w >= 2 * p.words) return 0u;
        if (mask) return mask[w];
        const int d = node - 32 * w;
        return d >= 31 ? 0xffffffffu : d < 0 ? 0u : (2u << d) - 1u;
    };
    const int rel = tok - ctx, left = hi - tok;
    uint32_t b = 0xffffffffu;
    if (rel >= 0) b = __funnelshift_r(node_bits(rel >> 5), node_bits((rel >> 5) + 1), rel & 31);
    else if (rel > -32) b = (node_bits(0) << -rel) | ((1u << -rel) - 1u);
    return left >= 32 ? b : left <= 0 ? 0u : b & ((1u << left) - 1u);
}

// ---------------------------------------------------------------- element types
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    static __device__ __forceinline__ float one(__nv_bfloat16 x) { return __bfloat162float(x); }
    static constexpr uint32_t kExpMask = 0x7f80u;
};
template <> struct Elem<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    static __device__ __forceinline__ float one(__half x) { return __half2float(x); }
    static constexpr uint32_t kExpMask = 0x7c00u;
};
// Two fp32 values in one 64-bit register pair, for the packed operations.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_parts(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
// 8 elements of 16 bits <-> 4 pairs.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& r, F2 (&f)[4]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = Elem<T>::unpack(w[i]);
        f[i] = f2(v.x, v.y);
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = f2_parts(f[i]);
        w[i] = Elem<T>::pack(v.x, v.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(Elem<T>::pack(f[0], f[1]), Elem<T>::pack(f[2], f[3]), Elem<T>::pack(f[4], f[5]),
                      Elem<T>::pack(f[6], f[7]));
}
// 16-byte asynchronous copies global -> shared.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (Without .ftz the norms take 1 % longer, for sums that an epsilon above 2^-126 keeps away.)
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

}  // namespace kda
