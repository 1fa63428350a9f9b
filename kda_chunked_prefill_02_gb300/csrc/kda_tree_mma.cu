// kda_tree_mma.cu -- kda_tree_attention (include/kda_ops.h) for many query rows
// (a tree of nodes times the query heads of a key head): 128-row tiles on
// tcgen05 tensor cores, S and O in TMEM, K and V pages by TMA.
//
// From about 32 rows on, the products and not the memory bound the warp-level
// kernel of kda_tree.cu; here a tile of 128 rows and 128 keys costs 16
// tcgen05.mma (S = Q K^T, then O += P V).  One CTA an SM, ten warps:
//   warps 0-3, 4-7  two softmax streams: thread = row (TMEM lane), the whole row
//                   of S in registers, so maximum and sum need no exchange; P
//                   goes back over S's columns as 16-bit pairs, the A operand of
//                   the second product;
//   warp 8          the loader: a ring of kBufs tiles, K and V in turn;
//   warp 9          issues the products.
// The streams alternate, so that one's softmax runs under the other's
// products.  With more than 128 rows they are two row tiles over the same keys
// (each K and V tile is read for 256 rows); with fewer they are the even and
// odd key tiles of one row tile, joined at the end.  Long contexts are cut into
// splits as in kda_tree.cu, joined by the same kernel.
//
// The running maximum moves only when a row's scores exceed it by 2^8 (l and O
// stay far inside fp32 and P inside fp16 until then), so that O in TMEM is
// hardly ever rescaled; that is the softmax threads' work, in the time between
// a score tile's arrival (which implies that the product before it is done) and
// their P's.
//
// Keys that a row does not see: only the last tiles hold drafted tokens or
// positions past the end; there every row forms its 128 visibility bits.  In
// those tiles the loader clears V rows past the end and V elements that are not
// finite before the product sees them (0 * NaN is NaN, also for a row whose P is
// zero), and remembers their nodes; the rows that do see such a node take its
// elements at the end.
//
// Every wait is bounded (sm103.cuh); one that runs out sets the abort flag, the
// roles fall through to the end, copies and products in flight are waited for,
// and the status word reports KDA_ERR_TIMEOUT.
#include "kda_internal.h"
#include "ops_internal.h"
#include "sm103.cuh"
#include "tmap.h"

namespace kda {
namespace {

constexpr int kMmaThreads = 320;
constexpr int kKeys = 128;               // keys a tile
constexpr uint32_t kBlock = 128 * 128;   // bytes of 128 rows of 64 elements
constexpr int kMaxBufs = 8;
constexpr uint32_t kTmemS = 0, kTmemO = 256;   // S of stream s at 128 s, O at 256 + 128 s
constexpr float kLazy = 8.f;             // log2 units by which scores may exceed the running maximum

template <int D> struct MmaShape {
    static constexpr uint32_t kTileBytes = (D / 64) * kBlock;
    static constexpr int kBufs = D == 128 ? 5 : 8;
    static constexpr uint32_t kSmem = (2 + kBufs) * kTileBytes + 1024;   // Q of both streams, the ring, alignment
};

template <typename T> struct MmaTypes;
template <> struct MmaTypes<__nv_bfloat16> {
    static __host__ __device__ constexpr uint32_t qk(uint32_t n) { return idesc_bf16_f32(128, n); }
    static __host__ __device__ constexpr uint32_t pv(uint32_t n) { return idesc_bf16_f32_bmn(128, n); }
};
template <> struct MmaTypes<__half> {
    static __host__ __device__ constexpr uint32_t qk(uint32_t n) { return idesc_f16_f32(128, n); }
    static __host__ __device__ constexpr uint32_t pv(uint32_t n) { return idesc_f16_f32_bmn(128, n); }
};

template <typename T, int D>
__global__ void __launch_bounds__(kMmaThreads, 1)
    tree_mma_kernel(const TreeParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    constexpr uint32_t kTileBytes = MmaShape<D>::kTileBytes;
    constexpr int kBufs = MmaShape<D>::kBufs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t kv_full[kMaxBufs], kv_free[kMaxBufs], v_raw, s_full[2], p_ready[2], o_full;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    __shared__ uint32_t s_bad[8];        // drafted nodes with a V element that is not finite
    __shared__ float s_m[128], s_l[128]; // stream 1's row maxima and sums when the streams are joined

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x / p.row_blocks, rb = blockIdx.x - split * p.row_blocks;
    const int kvh = blockIdx.y, r = blockIdx.z, row0 = rb * 256;
    int ctx, n;
    if (!tree_lengths(p, r, ctx, n) && p.status && tid == 0) atomicExch(p.status, 1);
    const int len = ctx + n;
    const int nsplit = max(1, (len + p.chunk - 1) / p.chunk);
    if (split >= nsplit) return;
    const int lo = split * p.chunk, hi = min(lo + p.chunk, len);
    const int ntiles = hi > lo ? (hi - lo + kKeys - 1) / kKeys : 0;
    const bool two = p.rows - row0 > 128;             // two row tiles, or one with its key tiles in turn
    const int units = two ? 2 * ntiles : ntiles;      // unit u: stream u & 1, tile two ? u >> 1 : u
    volatile int* abort = &abort_flag;
    uint8_t* ring = sm + 2 * kTileBytes;
    auto fail = [&]() {
        *abort = 1;
        if (p.status) atomicExch(p.status, 4);
    };

    if (tid == 0) {
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_free[i], 1);
        }
        mbar_init(&v_raw, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_ready[s], 128);
        }
        mbar_init(&o_full, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (tid < 8) s_bad[tid] = 0;
    if (warp == 9) {
        tmem_alloc(&tmem_base_sh, 512);
        tmem_relinquish();
    }
    const int stream = warp >> 2;   // of the softmax warps
    const int row = (two ? row0 + stream * 128 : row0) + (tid & 127);
    if (warp < 8 && (two || stream == 0)) {
        // the query rows as K-major operands in the 128-byte swizzle
        const int i = row / p.G, h = kvh * p.G + (row - i * p.G);
        const T* src = static_cast<const T*>(p.q) + r * p.qs[0] + i * p.qs[1] + h * p.qs[2];
        uint8_t* dst = sm + stream * kTileBytes;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint4 v = row < p.rows ? ldg16(src + c * 8) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(dst + (c >> 3) * kBlock + sw128_off(tid & 127, (c & 7) * 8)) = v;
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tmem_base_sh;

    if (warp == 8) {
        // ---------------------------------------------------------------- loader
        if (lane == 0) {
            tma_prefetch_desc(&kmap);
            tma_prefetch_desc(&vmap);
        }
        const int box = min(p.page, kKeys), per_tile = kKeys / box;
        const int bt = lane / (D / 64), bc = lane % (D / 64);   // this lane's box: tokens bt * box.., columns bc * 64..
        const int shift = 31 - __clz(p.page);
        auto page_of = [&](int tile) -> int {
            const int tok = lo + tile * kKeys + bt * box;
            if (bt >= per_tile || tok >= hi) return -1;
            int id = p.table[r * p.table_stride + (tok >> shift)];
            if (id < 0 || id >= p.P) {
                if (p.status) atomicExch(p.status, 1);
                id = p.P;   // past the map's pages: the copy fills in zeros
            }
            return id;
        };
        int id = ntiles > 0 ? page_of(0) : -1, issued = 0;
        uint32_t raw_uses = 0;
        bool ok = true;
        for (int tile = 0; tile < ntiles && ok; ++tile) {
            const int next = tile + 1 < ntiles ? page_of(tile + 1) : -1;
            const int base = lo + tile * kKeys;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, id >= 0)) * box * 128u;
            for (int v = 0; v < 2 && ok; ++v) {
                const int i = 2 * tile + v, slot = i % kBufs, round = i / kBufs;
                if (round > 0) ok = __all_sync(0xffffffffu, mbar_wait(&kv_free[slot], (round - 1) & 1, abort));
                if (!ok) break;
                uint8_t* dst = ring + slot * kTileBytes;
                const bool special = v == 1 && base + kKeys > ctx;
                uint64_t* bar = special ? &v_raw : &kv_full[slot];
                if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                __syncwarp();
                if (id >= 0)
                    tma_load_4d(dst + bc * kBlock + bt * box * 128, v ? &vmap : &kmap, bc * 64,
                                (base + bt * box) & (p.page - 1), kvh, id, bar);
                issued = i + 1;
                if (special) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&v_raw, raw_uses & 1, abort));
                    ++raw_uses;
                    constexpr uint32_t kExp = Elem<T>::kExpMask;
                    const int first = max(0, ctx - base);
                    for (int e = first * (D / 8) + lane; e < kKeys * (D / 8); e += 32) {
                        const int krow = e / (D / 8), c = e % (D / 8), tok = base + krow;
                        uint4* at = reinterpret_cast<uint4*>(dst + (c >> 3) * kBlock + krow * 128 + (c & 7) * 16);
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (tok < hi) {
                            x = *at;
                            uint32_t w[4] = {x.x, x.y, x.z, x.w};
                            bool bad = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((w[k] & kExp) == kExp) { bad = true; w[k] &= 0xffff0000u; }
                                if (((w[k] >> 16) & kExp) == kExp) { bad = true; w[k] &= 0xffffu; }
                            }
                            if (!bad) continue;
                            atomicOr(&s_bad[(tok - ctx) >> 5], 1u << ((tok - ctx) & 31));
                            x = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        *at = x;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&kv_full[slot]);
                }
            }
            id = next;
        }
        if (!ok) {
            if (lane == 0) fail();
            // copies still on their way into this CTA's memory
            for (int i = max(0, issued - kBufs); i < issued; ++i) mbar_wait(&kv_full[i % kBufs], (i / kBufs) & 1, nullptr);
        }
    } else if (warp == 9) {
        // ---------------------------------------------------------------- products
        if (lane == 0) {
            constexpr uint32_t id_qk = MmaTypes<T>::qk(kKeys), id_pv = MmaTypes<T>::pv(D);
            auto tile_of = [&](int u) { return two ? u >> 1 : u; };
            auto landed = [&](int i) { return mbar_wait(&kv_full[i % kBufs], (i / kBufs) & 1, abort); };
            bool ok = true;
            auto scores = [&](int u) {
                const int s = u & 1, i = 2 * tile_of(u);
                ok = ok && landed(i);
                if (!ok) return;
                tc_fence_after();
                umma_tile(tb + kTmemS + 128 * s, smem_u32(sm + (two ? s : 0) * kTileBytes), kBlock,
                          smem_u32(ring + (i % kBufs) * kTileBytes), kBlock, D, id_qk, false);
                umma_commit(&s_full[s]);
                if (!two || s == 1) umma_commit(&kv_free[i % kBufs]);
            };
            if (units > 0) scores(0);
            if (units > 1) scores(1);
            for (int u = 0; u < units && ok; ++u) {
                const int s = u & 1, i = 2 * tile_of(u) + 1;
                ok = mbar_wait(&p_ready[s], (u >> 1) & 1, abort) && landed(i);
                if (!ok) break;
                tc_fence_after();
                const uint64_t bd = sdesc_mnmajor_sw128(smem_u32(ring + (i % kBufs) * kTileBytes), kBlock, 1024);
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    umma_bf16_ta(tb + kTmemO + 128 * s, tb + kTmemS + 128 * s + 8 * k, bd + k * (2048 >> 4), id_pv,
                                 (u > 1 || k > 0) ? 1u : 0u);
                if (!two || s == 1) umma_commit(&kv_free[i % kBufs]);
                if (u + 2 < units) scores(u + 2);
            }
            if (!ok) fail();
            umma_commit(&o_full);
            if (!ok) mbar_wait(&o_full, 0, nullptr);   // products still in flight
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tb + lane_base + kTmemS + 128 * stream, to = tb + lane_base + kTmemO + 128 * stream;
        const int node = min(row / p.G, p.N - 1);
        const bool live = row - (tid & 31) < p.rows;   // some row of the warp is a row of the call
        const float c = p.scale_log2, lazy = kLazy / c;
        float m = -INFINITY, l = 0.f;
        bool ok = true;

        // 32 drafted nodes' visibility to this row, from node 32 w on
        const uint32_t* mask = p.mask ? reinterpret_cast<const uint32_t*>(p.mask + ((int64_t)r * p.N + node) * p.words)
                                      : nullptr;
        auto node_bits = [&](int w) -> uint32_t {
            if (w >= 2 * p.words) return 0u;
            if (mask) return mask[w];
            const int d = node - 32 * w;
            return d >= 31 ? 0xffffffffu : d < 0 ? 0u : (2u << d) - 1u;
        };
        // visibility of positions tok .. tok + 31
        auto seen = [&](int tok) -> uint32_t {
            const int rel = tok - ctx, left = hi - tok;
            uint32_t b = 0xffffffffu;
            if (rel >= 0) b = __funnelshift_r(node_bits(rel >> 5), node_bits((rel >> 5) + 1), rel & 31);
            else if (rel > -32) b = (node_bits(0) << -rel) | ((1u << -rel) - 1u);
            return left >= 32 ? b : left <= 0 ? 0u : b & ((1u << left) - 1u);
        };

        for (int u = stream; u < units; u += 2) {
            ok = __all_sync(0xffffffffu, mbar_wait(&s_full[stream], (u >> 1) & 1, abort));
            if (!ok) break;
            tc_fence_after();
            if (live) {
                uint32_t raw[8][16];
                float x[128];
#pragma unroll
                for (int k = 0; k < 8; ++k) tmem_ld16_issue(ts + 16 * k, raw[k]);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) tmem_take16(raw[k], &x[16 * k]);
                const int base = lo + (two ? u >> 1 : u) * kKeys;
                if (base + kKeys > ctx) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t b = seen(base + 32 * k);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((b >> e) & 1u)) x[32 * k + e] = -INFINITY;
                    }
                }
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int e = 4; e < 128; ++e) mx[e & 3] = fmaxf(mx[e & 3], x[e]);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (top > m + lazy || m == -INFINITY) {
                    const float alpha = m == -INFINITY ? 1.f : ex2_approx((m - top) * c);
                    m = fmaxf(m, top);
                    l *= alpha;
                    mx[0] = alpha;
                } else {
                    mx[0] = 1.f;
                }
                if (u > 1 && __any_sync(0xffffffffu, mx[0] != 1.f)) {
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        float o[32];
                        uint32_t w[32];
                        tmem_ld32(to + 32 * k, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * mx[0]);
                        tmem_st32(to + 32 * k, w);
                    }
                }
                const float mc = m == -INFINITY ? 0.f : -m * c;
                const F2 c2 = f2(c, c), m2 = f2(mc, mc);
                F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 y = f2_parts(f2_fma(f2(x[32 * k + 2 * e], x[32 * k + 2 * e + 1]), c2, m2));
                        const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
                        sum[e & 1] = f2_add(sum[e & 1], f2(p0, p1));
                        w[e] = Elem<T>::pack(p0, p1);
                    }
                    tmem_st16_issue(ts + 16 * k, w);
                }
                const float2 q = f2_parts(f2_add(sum[0], sum[1]));
                l += q.x + q.y;
                tmem_wait_st();
            }
            tc_fence_before();
            mbar_arrive(&p_ready[stream]);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&o_full, 0, abort)) && ok;
        if (!ok && lane == 0) fail();
        tc_fence_after();

        // the joined rows of an even / odd pair of streams leave through stream 0
        float* so = reinterpret_cast<float*>(ring);   // [D][128]: every tile has been consumed
        float f0 = 1.f, f1 = 0.f;
        if (!two) {
            if (stream == 1) {
                s_m[tid & 127] = m;
                s_l[tid & 127] = l;
                if (units > 1 && ok && live) {
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        float o[32];
                        tmem_ld32(to + 32 * k, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) so[(32 * k + e) * 128 + (tid & 127)] = o[e];
                    }
                }
            }
            named_bar_sync(1, 256);
            if (stream == 0 && units > 1) {
                const float m1 = s_m[tid], mj = fmaxf(m, m1), mu = mj == -INFINITY ? 0.f : mj;
                f0 = ex2_approx((m - mu) * c);
                f1 = ex2_approx((m1 - mu) * c);
                l = l * f0 + s_l[tid] * f1;
                m = mj;
            }
        }
        if (ok && live && units > 0 && (two || stream == 0)) {
            const int i = row / p.G, h = kvh * p.G + (row - i * p.G);
            const bool mine = row < p.rows;
            const bool empty = i >= n || l == 0.f;
            const float inv = empty ? 0.f : 1.f / l;
            const int64_t at = (((int64_t)r * p.Hk + kvh) * p.splits + split) * p.rows + row;
            T* dst = static_cast<T*>(p.out) + r * p.os[0] + i * p.os[1] + h * p.os[2];
            uint32_t any_bad = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) any_bad |= s_bad[w];
            const bool joined = !two && units > 1;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                float o[32];
                tmem_ld32(to + 32 * k, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float y = o[e] * f0;
                    if (joined) y = fmaf(so[(32 * k + e) * 128 + (tid & 127)], f1, y);
                    o[e] = empty ? 0.f : y * inv;
                }
                if (any_bad && !empty) {
                    for (int j = max(0, lo - ctx); j < hi - ctx; ++j) {
                        if (!((s_bad[j >> 5] >> (j & 31)) & 1u) || !(seen(ctx + j) & 1u)) continue;
                        const int tok = ctx + j, id = p.table[r * p.table_stride + tok / p.page];
                        if (id < 0 || id >= p.P) continue;
                        const T* v = static_cast<const T*>(p.vc) + id * p.vs[0] + (tok % p.page) * p.vs[1] +
                                     kvh * p.vs[2] + 32 * k;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = Elem<T>::one(v[e]);
                            if (!isfinite(x)) o[e] += x;
                        }
                    }
                }
                if (!mine) continue;
                if (nsplit == 1) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(dst + 32 * k + e) =
                            make_uint4(Elem<T>::pack(o[e], o[e + 1]), Elem<T>::pack(o[e + 2], o[e + 3]),
                                       Elem<T>::pack(o[e + 4], o[e + 5]), Elem<T>::pack(o[e + 6], o[e + 7]));
                } else {
                    float4* po = reinterpret_cast<float4*>(p.part_o + at * D + 32 * k);
#pragma unroll
                    for (int e = 0; e < 8; ++e) po[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            const float lse = empty ? -INFINITY : m * c + log2f(l);
            if (mine && nsplit > 1) p.part_lse[at] = lse;
            else if (mine && p.lse) p.lse[((int64_t)r * p.N + i) * p.Hq + h] = lse * 0.6931471805599453f;
        } else if (ok && units == 0 && row < p.rows && (two || stream == 0)) {
            // nothing to see at all
            const int i = row / p.G, h = kvh * p.G + (row - i * p.G);
            T* dst = static_cast<T*>(p.out) + r * p.os[0] + i * p.os[1] + h * p.os[2];
#pragma unroll
            for (int e = 0; e < D; e += 8) *reinterpret_cast<uint4*>(dst + e) = make_uint4(0, 0, 0, 0);
            if (p.lse) p.lse[((int64_t)r * p.N + i) * p.Hq + h] = -INFINITY;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
}

template <typename T, int D>
cudaError_t launch_mma_t(const TreeParams& q, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
    TreeParams p = q;
    p.row_blocks = (p.rows + 255) / 256;
    static std::atomic<uint64_t> smem_set;
    cudaError_t e = set_smem_limit_once((const void*)tree_mma_kernel<T, D>, (int)MmaShape<D>::kSmem, smem_set);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(p.splits * p.row_blocks), (unsigned)p.Hk, (unsigned)p.R);
    tree_mma_kernel<T, D><<<grid, kMmaThreads, MmaShape<D>::kSmem, s>>>(p, kmap, vmap);
    return cudaGetLastError();
}

// Tensor map of a cache as [channel, row of a page, head, page]; a box is the
// rows of a page that a tile takes, 64 channels wide.
bool cache_map(CUtensorMap* map, const void* base, const int64_t (&st)[3], const TreeParams& p, int D, bool f16) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.page, (uint64_t)p.Hk, (uint64_t)p.P};
    const uint64_t strides[3] = {(uint64_t)st[1] * 2, (uint64_t)st[2] * 2, (uint64_t)st[0] * 2};
    const uint32_t box[4] = {64, (uint32_t)(p.page < kKeys ? p.page : kKeys), 1, 1};
    return make_tensor_map(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
                           strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

bool launch_tree_mma(const TreeParams& p, int D, bool f16, cudaStream_t s, cudaError_t* e) {
    CUtensorMap kmap, vmap;
    if (!cache_map(&kmap, p.kc, p.ks, p, D, f16) || !cache_map(&vmap, p.vc, p.vs, p, D, f16)) return false;
    if (f16) *e = D == 64 ? launch_mma_t<__half, 64>(p, kmap, vmap, s) : launch_mma_t<__half, 128>(p, kmap, vmap, s);
    else *e = D == 64 ? launch_mma_t<__nv_bfloat16, 64>(p, kmap, vmap, s)
                      : launch_mma_t<__nv_bfloat16, 128>(p, kmap, vmap, s);
    return true;
}

}  // namespace kda
