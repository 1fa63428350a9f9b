// kda_tree.cu -- attention of drafted tokens over a paged cache
// (kda_tree_attention in include/kda_ops.h): the kernel for few query rows and
// the kernel that joins the splits of a long context.
//
// The rows of one (request, key head) are its nodes times the G query heads
// that share the key head, so that a key is read once for all of them.  One
// pass over the keys with the running maximum m and sum l of the softmax:
//
//     m' = max(m, max_p s_p),  o' = o 2^(m - m') + sum_p 2^(s_p - m') v_p,  l' likewise,
//
// s in units of log2 (scale * log2 e is folded into one multiplier).  With at
// most 32 rows a key costs 4 D rows flops for its 4 D bytes, so the kernel is
// bound by HBM bandwidth and what matters is bytes in flight: 64-token tiles of
// K and V come in by 16-byte asynchronous copies, three tiles deep, two CTAs an
// SM.  Rows go through warp-level m16n8k16 products (16 rows a product; the
// 128-row tcgen05 products would be mostly padding here).  The four warps
// split a tile's tokens, not its rows: every key is read from shared memory by
// one warp only, the probabilities stay in registers (the product's
// accumulator layout is the next product's operand layout), and the warps meet
// once, at the end, to join their (m, l, o).
//
// Where there are too few (request, head) pairs to fill the GPU, a context is the
// work of a cluster of up to 8 CTAs, an equal stretch of its tiles each (of the
// length that the device sees), which join their rows through distributed shared
// memory: no second launch and no workspace.  Longer contexts are first cut into
// splits of `chunk` tokens, one cluster each; the splits leave normalised rows and
// their log-sum in the workspace, joined in a fixed order by tree_join_kernel.
//
// Where one CTA an item is more than the GPU runs at once, the requests go longest
// first (tree_order_kernel ranks them, as the chunk table ranks prefill's
// sequences), so that the last CTAs are short ones.
//
// Keys that a row does not see are taken out of the scores by a select, and
// rows of V past the end are zero-filled in shared memory.  V of a drafted
// token is seen by some rows only, and 0 * NaN is NaN: a tile that holds
// drafted tokens whose V is not finite takes a scalar product that leaves out
// what a row does not see.
#include "kda_internal.h"
#include "ops_internal.h"

namespace kda {
namespace {

constexpr int kTreeThreads = 128;
constexpr int kTile = 64;      // tokens a tile, 16 a warp
constexpr int kStages = 3;
constexpr int kOrderMax = 1024;   // requests that are ranked

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory of the cluster's CTA `rank` at this CTA's address `addr`.
__device__ __forceinline__ uint32_t remote_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 remote_ld4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 remote_ld2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool take) {
    const int n = take ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte piece c of row r in a tile of rows of D elements.
template <int D>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    return (uint32_t)r * (D * 2) + (uint32_t)((c ^ (r & 7)) << 4);
}

template <typename T, int D, int MT, bool kCluster>
__global__ void __launch_bounds__(kTreeThreads) tree_rows_kernel(const TreeParams p) {
    constexpr int kRows = 16 * MT;
    constexpr uint32_t kKV = kTile * D * 2, kStage = 2 * kKV;
    extern __shared__ __align__(128) uint8_t smt[];
    uint8_t* sq = smt + kStages * kStage;
    int* spage = reinterpret_cast<int*>(sq + kRows * D * 2);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const int cluster = kCluster ? p.cluster : 1, rank = kCluster ? blockIdx.x % cluster : 0, bx = blockIdx.x / cluster;
    const int split = bx / p.row_blocks, rb = bx - split * p.row_blocks;
    if (p.order) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int kvh = blockIdx.y, r = p.order ? p.order[blockIdx.z] : blockIdx.z, row0 = rb * kRows;
    int ctx, n;
    if (!tree_lengths(p, r, ctx, n) && p.status && tid == 0) atomicExch(p.status, 1);
    const int len = ctx + n;
    const int nsplit = max(1, (len + p.chunk - 1) / p.chunk);
    if (split >= nsplit) return;   // the whole cluster
    // this CTA's tiles of the split
    const int lo0 = split * p.chunk, hi0 = min(lo0 + p.chunk, len), tiles0 = max(0, hi0 - lo0 + kTile - 1) / kTile;
    const int lo = lo0 + tiles0 * rank / cluster * kTile, hi = min(lo0 + tiles0 * (rank + 1) / cluster * kTile, hi0);

    // this split's pages
    const int pg0 = lo / p.page;
    const int npages = hi > lo ? (hi - 1) / p.page - pg0 + 1 : 0;
    for (int e = tid; e < npages; e += kTreeThreads) {
        int id = p.table[r * p.table_stride + pg0 + e];
        if (id < 0 || id >= p.P) {
            id = -1;
            if (p.status) atomicExch(p.status, 1);
        }
        spage[e] = id;
    }
    __syncthreads();

    const uint32_t s0 = smem_addr(smt);
    const T* kbase = static_cast<const T*>(p.kc) + kvh * p.ks[2];
    const T* vbase = static_cast<const T*>(p.vc) + kvh * p.vs[2];
    const uint32_t pos0 = (uint32_t)(lo - pg0 * p.page);
    constexpr int kPieces = D / 8, kRowsPass = kTreeThreads / kPieces;
    auto load = [&](int tile) {
        if (lo + tile * kTile < hi) {
            const uint32_t dst = s0 + (tile % kStages) * kStage;
            const int c = tid % kPieces;
#pragma unroll
            for (int j = 0; j < kTile / kRowsPass; ++j) {
                const int row = tid / kPieces + j * kRowsPass;
                const int tok = tile * kTile + row;
                const uint32_t at = pos0 + tok, pg = page_div(at, p.page, p.page_magic);
                const bool in = lo + tok < hi;
                const int id = in ? spage[pg] : -1;
                const int64_t rem = at - pg * p.page, page = id < 0 ? 0 : id;
                const uint32_t off = tile_off<D>(row, c);
                cp_async16_or_zero(dst + off, kbase + page * p.ks[0] + (id < 0 ? 0 : rem) * p.ks[1] + c * 8, id >= 0);
                cp_async16_or_zero(dst + kKV + off, vbase + page * p.vs[0] + (id < 0 ? 0 : rem) * p.vs[1] + c * 8,
                                   id >= 0);
            }
        }
        cp_async_commit();
    };
    const int ntiles = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load(i);

    // query rows
    for (int e = tid; e < kRows * kPieces; e += kTreeThreads) {
        const int row = e / kPieces, c = e - row * kPieces, q = row0 + row;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (q < p.rows) {
            const int i = q / p.G, h = kvh * p.G + (q - i * p.G);
            v = ldg16(static_cast<const T*>(p.q) + r * p.qs[0] + i * p.qs[1] + h * p.qs[2] + c * 8);
        }
        *reinterpret_cast<uint4*>(sq + tile_off<D>(row, c)) = v;
    }

    float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int a = 0; a < MT; ++a) {
#pragma unroll
        for (int b = 0; b < D / 8; ++b)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[a][b][c] = 0.f;
        m[a][0] = m[a][1] = -INFINITY;
        l[a][0] = l[a][1] = 0.f;
    }
    // does row `row` of this block see position tok (< hi)?
    auto sees = [&](int row, int tok) -> bool {
        if (tok < ctx) return true;
        const int i = min((row0 + row) / p.G, p.N - 1), j = tok - ctx;
        if (!p.mask) return j <= i;
        return (p.mask[((int64_t)r * p.N + i) * p.words + (j >> 6)] >> (j & 63)) & 1;
    };

    for (int tile = 0; tile < ntiles; ++tile) {
        cp_async_wait<kStages - 2>();
        __syncthreads();   // the tile has landed for every thread; the tile before it is consumed
        load(tile + kStages - 1);
        const int tok0 = lo + tile * kTile + warp * 16;
        if (tok0 >= hi) continue;
        const uint32_t sk = s0 + (tile % kStages) * kStage, sv = sk + kKV;

        float s[MT][2][4];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[a][b][c] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t kb[4];
            ldmatrix4(kb, sk + tile_off<D>(warp * 16 + (lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)));
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                uint32_t qa[4];
                ldmatrix4(qa, smem_addr(sq) + tile_off<D>(a * 16 + (lane & 15), ks * 2 + (lane >> 4)));
                mma16816<T>(s[a][0], qa, kb[0], kb[1]);
                mma16816<T>(s[a][1], qa, kb[2], kb[3]);
            }
        }
        const bool ragged = tok0 + 16 > hi || tok0 + 16 > ctx;
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[a][b][c] *= p.scale_log2;
                    if (ragged) {
                        const int tok = tok0 + b * 8 + tq * 2 + (c & 1);
                        if (tok >= hi || !sees(a * 16 + g + (c >> 1) * 8, tok)) s[a][b][c] = -INFINITY;
                    }
                }
        bool moved = false;
        float alpha[MT][2];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float mx = fmaxf(fmaxf(s[a][0][2 * h], s[a][0][2 * h + 1]), fmaxf(s[a][1][2 * h], s[a][1][2 * h + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[a][h], mx), mu = mn == -INFINITY ? 0.f : mn;
                moved |= mn != m[a][h];
                alpha[a][h] = ex2_approx(m[a][h] - mu);
                m[a][h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float& x = s[a][b][2 * h + c];
                        x = ex2_approx(x - mu);
                        sum += x;
                    }
                l[a][h] = fmaf(l[a][h], alpha[a][h], sum);
            }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int b = 0; b < D / 8; ++b)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[a][b][c] *= alpha[a][c >> 1];
        }
        bool plain = true;
        if (tok0 + 16 > ctx) {
            // drafted tokens: is all of their V finite?
            bool bad = false;
            constexpr uint32_t kExp = Elem<T>::kExpMask;
            for (int e = lane; e < 16 * kPieces; e += 32) {
                const uint4 v = *reinterpret_cast<const uint4*>(smt + (sv - s0) + (uint32_t)warp * 16 * (D * 2) + e * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    bad |= (w[k] & kExp) == kExp || ((w[k] >> 16) & kExp) == kExp;
            }
            plain = !__any_sync(0xffffffffu, bad);
        }
        if (plain) {
            uint32_t pa[MT][4];
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                pa[a][0] = Elem<T>::pack(s[a][0][0], s[a][0][1]);
                pa[a][1] = Elem<T>::pack(s[a][0][2], s[a][0][3]);
                pa[a][2] = Elem<T>::pack(s[a][1][0], s[a][1][1]);
                pa[a][3] = Elem<T>::pack(s[a][1][2], s[a][1][3]);
            }
#pragma unroll
            for (int b = 0; b < D / 16; ++b) {
                uint32_t vb[4];
                ldmatrix4_trans(vb, sv + tile_off<D>(warp * 16 + (lane & 15), b * 2 + (lane >> 4)));
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    mma16816<T>(o[a][2 * b], pa[a], vb[0], vb[1]);
                    mma16816<T>(o[a][2 * b + 1], pa[a], vb[2], vb[3]);
                }
            }
        } else {
#pragma unroll 1
            for (int t = 0; t < 16 && tok0 + t < hi; ++t) {
                const int src = (lane & ~3) | ((t & 7) >> 1);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const float lo0 = (t & 1) ? s[a][0][1] : s[a][0][0], hi0 = (t & 1) ? s[a][0][3] : s[a][0][2];
                    const float lo1 = (t & 1) ? s[a][1][1] : s[a][1][0], hi1 = (t & 1) ? s[a][1][3] : s[a][1][2];
                    const float p0 = __shfl_sync(0xffffffffu, t < 8 ? lo0 : lo1, src);
                    const float p1 = __shfl_sync(0xffffffffu, t < 8 ? hi0 : hi1, src);
                    const bool see0 = sees(a * 16 + g, tok0 + t), see1 = sees(a * 16 + g + 8, tok0 + t);
#pragma unroll
                    for (int b = 0; b < D / 8; ++b) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(
                            smt + (sv - s0) + tile_off<D>(warp * 16 + t, b) + tq * 4);
                        const float2 v = Elem<T>::unpack(w);
                        if (see0) {
                            o[a][b][0] = fmaf(p0, v.x, o[a][b][0]);
                            o[a][b][1] = fmaf(p0, v.y, o[a][b][1]);
                        }
                        if (see1) {
                            o[a][b][2] = fmaf(p1, v.x, o[a][b][2]);
                            o[a][b][3] = fmaf(p1, v.y, o[a][b][3]);
                        }
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();   // every tile is consumed: its memory takes the warps' (m, l, o)

    float* so = reinterpret_cast<float*>(smt);                  // [4][kRows][D]
    float* sml = so + 4 * kRows * D;                            // [4][kRows][2]
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float sum = l[a][h];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const int row = a * 16 + g + 8 * h;
            if (tq == 0) {
                sml[(warp * kRows + row) * 2] = m[a][h];
                sml[(warp * kRows + row) * 2 + 1] = sum;
            }
#pragma unroll
            for (int b = 0; b < D / 8; ++b)
                *reinterpret_cast<float2*>(so + (warp * kRows + row) * D + b * 8 + tq * 2) =
                    make_float2(o[a][b][2 * h], o[a][b][2 * h + 1]);
        }
    __syncthreads();
    // the four warps' rows joined: the running maximum (0 if there is none), the sum, and
    // 8 values of the row
    auto joined = [&](int row, int c, float& mu, float& sum, float (&y)[8]) {
        float mw[4], mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            mw[w] = sml[(w * kRows + row) * 2];
            mx = fmaxf(mx, mw[w]);
        }
        mu = mx == -INFINITY ? 0.f : mx;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = ex2_approx(mw[w] - mu);
            sum = fmaf(sml[(w * kRows + row) * 2 + 1], f, sum);
            const float* src = so + (w * kRows + row) * D + c * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = fmaf(src[k], f, y[k]);
        }
    };
    float* const sx = sml + 4 * kRows * 2;      // cluster: this CTA's rows [kRows][D], then (maximum, sum) [kRows]
    if (kCluster) {
        for (int e = tid; e < kRows * kPieces; e += kTreeThreads) {
            const int row = e / kPieces, c = e - row * kPieces;
            float mu, sum, y[8];
            joined(row, c, mu, sum, y);
            float4* dst = reinterpret_cast<float4*>(sx + row * D + c * 8);
            dst[0] = make_float4(y[0], y[1], y[2], y[3]);
            dst[1] = make_float4(y[4], y[5], y[6], y[7]);
            if (c == 0) *reinterpret_cast<float2*>(sx + kRows * D + 2 * row) = make_float2(sum == 0.f ? -INFINITY : mu, sum);
        }
        cluster_sync();
    }
    const uint32_t sx_at = smem_addr(sx);
    for (int e = rank * kTreeThreads + tid; e < kRows * kPieces; e += cluster * kTreeThreads) {
        const int row = e / kPieces, c = e - row * kPieces, q = row0 + row;
        if (q >= p.rows) break;
        float mu, sum, y[8];
        if (!kCluster) {
            joined(row, c, mu, sum, y);
        } else {
            float mx = -INFINITY;
            for (int w = 0; w < cluster; ++w) mx = fmaxf(mx, remote_ld2(remote_addr(sx_at + (kRows * D + 2 * row) * 4, w)).x);
            mu = mx == -INFINITY ? 0.f : mx;
            sum = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = 0.f;
            for (int w = 0; w < cluster; ++w) {
                const float2 ml = remote_ld2(remote_addr(sx_at + (kRows * D + 2 * row) * 4, w));
                const uint32_t src = remote_addr(sx_at + (row * D + c * 8) * 4, w);
                const float4 a = remote_ld4(src), b = remote_ld4(src + 16);
                const float f = ex2_approx(ml.x - mu);
                sum = fmaf(ml.y, f, sum);
                y[0] = fmaf(a.x, f, y[0]); y[1] = fmaf(a.y, f, y[1]); y[2] = fmaf(a.z, f, y[2]); y[3] = fmaf(a.w, f, y[3]);
                y[4] = fmaf(b.x, f, y[4]); y[5] = fmaf(b.y, f, y[5]); y[6] = fmaf(b.z, f, y[6]); y[7] = fmaf(b.w, f, y[7]);
            }
        }
        const int i = q / p.G;
        const bool empty = i >= n || sum == 0.f;
        const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = empty ? 0.f : y[k] * inv;
        const float lse = empty ? -INFINITY : mu + log2f(sum);
        if (nsplit == 1) {
            const int h = kvh * p.G + (q - i * p.G);
            *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + r * p.os[0] + i * p.os[1] + h * p.os[2] + c * 8) =
                pack8<T>(y);
            if (p.lse && c == 0) p.lse[((int64_t)r * p.N + i) * p.Hq + h] = lse * 0.6931471805599453f;
        } else {
            const int64_t at = (((int64_t)r * p.Hk + kvh) * p.splits + split) * p.rows + q;
            float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + c * 8);
            dst[0] = make_float4(y[0], y[1], y[2], y[3]);
            dst[1] = make_float4(y[4], y[5], y[6], y[7]);
            if (c == 0) p.part_lse[at] = lse;
        }
    }
    if (kCluster) cluster_sync();   // the others have read this CTA's rows
}

// order[k]: the request of rank k by descending length (ties by index).
__global__ void __launch_bounds__(1024) tree_order_kernel(const TreeParams p) {
    __shared__ int len[kOrderMax];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // they wait for this grid's end themselves
    const int r = threadIdx.x;
    int ctx = 0, n = 0;
    if (r < p.R) tree_lengths(p, r, ctx, n);
    const int mine = ctx + n;
    len[r] = mine;
    __syncthreads();
    if (r >= p.R) return;
    int rank = 0;
    for (int i = 0; i < p.R; ++i) rank += len[i] > mine || (len[i] == mine && i < r);
    p.order[rank] = r;
}

// Joins the splits of a row: out = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M).
// One warp a row, in a fixed order of the splits.
template <typename T, int D>
__global__ void __launch_bounds__(128) tree_join_kernel(const TreeParams p) {
    constexpr int kVec = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, q = blockIdx.x * 4 + (threadIdx.x >> 5), kvh = blockIdx.y, r = blockIdx.z;
    int ctx, n;
    tree_lengths(p, r, ctx, n);
    const int nsplit = (ctx + n + p.chunk - 1) / p.chunk;
    if (nsplit <= 1 || q >= p.rows) return;
    const int64_t at = (((int64_t)r * p.Hk + kvh) * p.splits) * p.rows + q;
    const float* lses = p.part_lse + at;
    float mx = -INFINITY;
    for (int s = lane; s < nsplit; s += 32) mx = fmaxf(mx, lses[(int64_t)s * p.rows]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mu = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, y[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) y[i] = 0.f;
#pragma unroll 4
    for (int s = 0; s < nsplit; ++s) {
        const float f = ex2_approx(lses[(int64_t)s * p.rows] - mu);
        const float* src = p.part_o + (at + (int64_t)s * p.rows) * D + lane * kVec;
        sum += f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[i] = fmaf(src[i], f, y[i]);
    }
    const int i = q / p.G, h = kvh * p.G + (q - i * p.G);
    const bool empty = sum == 0.f;
    const float inv = empty ? 0.f : 1.f / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + r * p.os[0] + i * p.os[1] + h * p.os[2] +
                                                lane * kVec);
#pragma unroll
    for (int k = 0; k < kVec; k += 2) dst[k / 2] = Elem<T>::pack(y[k] * inv, y[k + 1] * inv);
    if (p.lse && lane == 0)
        p.lse[((int64_t)r * p.N + i) * p.Hq + h] = empty ? -INFINITY : (mu + log2f(sum)) * 0.6931471805599453f;
}

int rows_per_block(int rows, int D) { return rows <= 16 || D > 128 ? 16 : 32; }

template <typename T, int D, int MT, bool kCluster>
cudaError_t launch_rows_c(const TreeParams& p, cudaStream_t s) {
    const size_t pages = (size_t)p.chunk / p.page + 2;
    const size_t smem = (size_t)kStages * 2 * kTile * D * 2 + 16 * MT * D * 2 + pages * sizeof(int);
    static std::atomic<uint64_t> smem_set;
    // the largest page list (see tree_plan)
    const int limit = kStages * 2 * kTile * D * 2 + 16 * MT * D * 2 + 1026 * (int)sizeof(int);
    const auto kernel = tree_rows_kernel<T, D, MT, kCluster>;
    cudaError_t e = set_smem_limit_once((const void*)kernel, limit, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    if (kCluster) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)p.cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    } else {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // right after tree_order_kernel
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = dim3((unsigned)(p.splits * p.row_blocks * p.cluster), (unsigned)p.Hk, (unsigned)p.R);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster || p.order ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <typename T, int D, int MT>
cudaError_t launch_rows_t(const TreeParams& q, cudaStream_t s) {
    TreeParams p = q;
    p.row_blocks = (p.rows + 16 * MT - 1) / (16 * MT);
    if (p.order) {
        tree_order_kernel<<<1, kOrderMax, 0, s>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return p.cluster > 1 ? launch_rows_c<T, D, MT, true>(p, s) : launch_rows_c<T, D, MT, false>(p, s);
}

template <typename T>
cudaError_t launch_rows(const TreeParams& p, int D, cudaStream_t s) {
    const bool one = rows_per_block(p.rows, D) == 16;
    if (D == 64) return one ? launch_rows_t<T, 64, 1>(p, s) : launch_rows_t<T, 64, 2>(p, s);
    if (D == 128) return one ? launch_rows_t<T, 128, 1>(p, s) : launch_rows_t<T, 128, 2>(p, s);
    return launch_rows_t<T, 256, 1>(p, s);
}

template <typename T>
cudaError_t launch_join(const TreeParams& p, int D, cudaStream_t s) {
    const dim3 grid((unsigned)((p.rows + 3) / 4), (unsigned)p.Hk, (unsigned)p.R);
    const auto kernel = D == 64 ? tree_join_kernel<T, 64> : D == 128 ? tree_join_kernel<T, 128> : tree_join_kernel<T, 256>;
    return launch_maybe_pdl(kernel, grid, dim3(128), 0, s, true, p);
}

}  // namespace

TreePlan tree_plan(int R, int Hk, int rows, int D, int64_t max_len, int page, float scale, int num_sms) {
    TreePlan t;
    // The 128-row products where there are more rows than one product of the
    // warp-level kernel takes and enough work to outlast their longer way in (about
    // 10 us): 38 requests x 4 key heads x 32 rows over 1024 tokens 21 us against 48,
    // 8 x 2 x 512 rows over 300 28 against 37; but 16 x 8 x 32 over 500 24 against 22
    // and 1 x 8 x 32 over 1000 21 against 17.  Pages have to be whole 8-row groups of a
    // tile (and the line of work, in key tiles, stays inside 32 bits).
    const int64_t blocks = (rows + 31) / 32;
    t.mma = rows > 16 && (int64_t)R * Hk * blocks * max_len > 65536 && D <= 128 && page >= 8 &&
            (page & (page - 1)) == 0 && scale > 0.f && max_len / 128 + 1 < (1 << 22);
    // The rows kernel's cut (also for a cache without a tensor map): as many CTAs as run
    // at once (two an SM), so that no context's end is alone on the GPU, at least 128
    // tokens each.  Up to 8 are a cluster, which joins its rows itself (one request, 2
    // key heads, 1000 tokens: 8.5 us against 9.7 with a second launch, and no workspace);
    // more are splits, of at most 1024 pages (one request, 8 key heads, 131072 tokens: 95
    // us against 104 in clusters).  One request, 8 key heads, 64000 tokens: 56 us with as
    // many splits, 78 with twice as many, 112 with four times.
    const int block = rows_per_block(rows, D);
    const int64_t items = (int64_t)R * Hk * ((rows + block - 1) / block);
    const int64_t most = (max_len + 127) / 128;
    int64_t parts = 2LL * num_sms / items;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    t.cluster = parts >= 16 ? 1 : parts >= 8 ? 8 : parts >= 4 ? 4 : parts >= 2 ? 2 : 1;
    int64_t splits = parts / t.cluster;
    int64_t chunk = (max_len + splits - 1) / splits;
    if (chunk > 1024LL * page) chunk = 1024LL * page;
    chunk = (chunk + kTile - 1) / kTile * kTile;
    if (chunk < kTile) chunk = kTile;
    splits = (max_len + chunk - 1) / chunk;
    t.chunk = (int)chunk;
    t.splits = (int)(splits > 0 ? splits : 1);
    // Ranked where the items outnumber the CTAs that run at once: 256 requests x 8 key heads
    // of 0.2 to 1 times 4096 tokens 406 us against 437.
    t.order = !t.mma && t.splits == 1 && t.cluster == 1 && R > 1 && R <= kOrderMax && items > 2LL * num_sms ? R : 0;
    t.grid = num_sms;
    t.parts = t.mma ? (size_t)2 * t.grid : 0;
    t.part_rows = t.splits > 1 ? (size_t)R * Hk * rows * t.splits : 0;
    if (t.mma && t.part_rows < (size_t)2 * t.grid * 256) t.part_rows = (size_t)2 * t.grid * 256;
    return t;
}

cudaError_t launch_tree_attention(const TreeParams& p, const TreePlan& plan, int D, bool f16, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (plan.mma && launch_tree_mma(p, D, f16, plan.grid, s, &e)) return e;
    e = f16 ? launch_rows<__half>(p, D, s) : launch_rows<__nv_bfloat16>(p, D, s);
    if (e != cudaSuccess || p.splits == 1) return e;
    return f16 ? launch_join<__half>(p, D, s) : launch_join<__nv_bfloat16>(p, D, s);
}

}  // namespace kda
