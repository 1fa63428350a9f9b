// kda_chunk.cu -- attention of chunks of new tokens over a paged cache
// (kda_chunk_attention in include/kda_ops.h): the kernel for few rows and for caches
// that have no tensor map, and the choice between the kernels.
//
// The rows of one (request, key head) are its new tokens times the G query heads that
// share the key head.  One pass over the keys with the running maximum m and sum l of
// the softmax:
//
//     m' = max(m, max_p s_p),  o' = o 2^(m - m') + sum_p 2^(s_p - m') v_p,  l' likewise,
//
// s in units of log2.  A CTA takes a block of 16 or 32 rows and the keys that its last
// token sees, in 64-token tiles by 16-byte asynchronous copies, three tiles deep; the
// four warps split a tile's tokens and join their rows at the end, as in kda_tree.cu.
// Where the blocks are few, a cluster of up to 8 CTAs shares one, an equal stretch of
// its tiles each, and joins the rows through distributed shared memory.
//
// Which request a block belongs to is found on the device, by a search in cu_seqlens: a
// call's grid has floor(tokens * G / rows) + requests blocks, as many as ragged requests can
// need.
//
// Few rows are bound by a chain of latencies (lengths, page table, K and V, products, join): one
// token over 1000 keys, 8 / 2 heads 7.6 us, 16 tokens 10.4.
//
// Keys behind a row's own are taken out of the scores by a select; V rows past the
// request's end are zero-filled, and a tile in which some row does not see a key whose V
// is not finite takes a scalar product that leaves out what a row does not see
// (0 * NaN is NaN).
#include <math.h>

#include "kda_internal.h"
#include "ops_internal.h"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace kda {
namespace {

constexpr int kChunkThreads = 128;
constexpr int kTile = 64;      // tokens a tile, 16 a warp
constexpr int kStages = 3;
constexpr int kWindow = 256;   // pages listed at a time (a tile has at most kTile)
template <typename T> constexpr bool elem_is_f16() { return std::is_same<T, __half>::value; }
// The probabilities meet V in its type.  fp16 ends at 2^-24, and a long context may have its
// weight in keys far below the largest, so there they are 2^15 times as large (the sum of the
// softmax too; only the log-sum takes the factor back).
template <typename T> constexpr float kWeightShift = elem_is_f16<T>() ? 15.f : 0.f;

template <typename T, int D, int MT, bool kCluster>
__global__ void __launch_bounds__(kChunkThreads) chunk_rows_kernel(const ChunkParams p) {
    constexpr int kRows = 16 * MT;
    constexpr uint32_t kKV = kTile * D * 2, kStage = 2 * kKV;
    extern __shared__ __align__(128) uint8_t smt[];
    __shared__ int spage[kWindow];
    __shared__ int s_request, s_block;
    uint8_t* sq = smt + p.stages * kStage;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const int cluster = kCluster ? p.cluster : 1, rank = kCluster ? blockIdx.x % cluster : 0;
    const int kvh = blockIdx.y;
    const int64_t at = blockIdx.x / cluster;
    if (p.cu) {
        // Request r has the blocks from floor(cu[r] G / kRows) + r up to the next one's: never fewer
        // than it needs.  A warp looks at 32 requests at a time, evenly spread over those left.
        if (warp == 0) {
            const auto begin = [&](int i) { return (int64_t)p.cu[i] * p.G / kRows + i; };
            int lo = 0, hi = p.R;   // begin(lo) <= at < begin(hi)
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32, i = lo + step * lane;
                const uint32_t before = __ballot_sync(0xffffffffu, i < hi && begin(i) <= at) | 1u;
                const int last = 31 - __clz(before);
                hi = min(hi, lo + step * (last + 1));
                lo += step * last;
            }
            if (lane == 0) {
                s_request = lo;
                s_block = (int)max((int64_t)0, min(at - begin(lo), (int64_t)INT32_MAX / kRows));
            }
        }
        // every request's lengths are looked at by one thread (there are R blocks at least)
        const int64_t mine = at * kChunkThreads + tid;
        if (kvh == 0 && rank == 0 && p.status && mine < p.R) {
            int first, n, len;
            if (!chunk_request(p, (int)mine, first, n, len)) atomicMax(p.status, 1);
        }
        __syncthreads();
    } else {
        const int64_t each = ((int64_t)p.T * p.G + kRows - 1) / kRows;
        s_request = (int)(at / each);   // (all threads write the same)
        s_block = (int)(at - at / each * each);
        __syncthreads();
    }
    const int r = s_request, row0 = s_block * kRows;
    int first, n, len;
    if (!chunk_request(p, r, first, n, len) && !p.cu && p.status && tid == 0) atomicMax(p.status, 1);
    if (row0 >= n * p.G) return;   // no such block (all CTAs of a cluster)
    const int rows = n * p.G, ctx = len - n;   // without keys (len 0) no row sees any
    const int token0 = (int)page_div((uint32_t)row0, p.G, p.group_magic);
    const int token1 = min((int)page_div((uint32_t)(row0 + kRows - 1), p.G, p.group_magic), n - 1);
    const int end = len == 0 ? 0 : ctx + token1 + 1;   // keys of the block's last token
    const int tiles = (end + kTile - 1) / kTile;
    const int t0 = tiles * rank / cluster, t1 = tiles * (rank + 1) / cluster;
    const int lo = t0 * kTile, hi = min(t1 * kTile, end);
    const T* qbase = static_cast<const T*>(p.q) + (p.cu ? first * p.qs[1] : r * p.qs[0]);
    T* obase = static_cast<T*>(p.out) + (p.cu ? first * p.os[1] : r * p.os[0]);

    // the pages of this part, kWindow at a time
    int page0 = 0;
    auto list_pages = [&](int tok) {
        page0 = (int)page_div((uint32_t)tok, p.page, p.page_magic);
        const int count = hi > tok ? min(kWindow, (int)page_div((uint32_t)(hi - 1), p.page, p.page_magic) - page0 + 1) : 0;
        for (int e = tid; e < count; e += kChunkThreads) {
            int id = p.table[r * p.table_stride + page0 + e];
            if (id < 0 || id >= p.P) {
                id = -1;
                if (p.status) atomicMax(p.status, 1);
            }
            spage[e] = id;
        }
        __syncthreads();
    };
    list_pages(lo);

    const uint32_t s0 = smem_addr(smt);
    const T* kbase = static_cast<const T*>(p.kc) + kvh * p.ks[2];
    const T* vbase = static_cast<const T*>(p.vc) + kvh * p.vs[2];
    constexpr int kPieces = D / 8, kRowsPass = kChunkThreads / kPieces;
    auto load = [&](int tile) {
        if (lo + tile * kTile < hi) {
            const uint32_t dst = s0 + (tile % kStages) * kStage;
            const int c = tid % kPieces;
#pragma unroll
            for (int j = 0; j < kTile / kRowsPass; ++j) {
                const int row = tid / kPieces + j * kRowsPass;
                const uint32_t tok = (uint32_t)(lo + tile * kTile + row), pg = page_div(tok, p.page, p.page_magic);
                const int id = (int)tok < hi ? spage[(int)pg - page0] : -1;
                const int64_t rem = id < 0 ? 0 : tok - pg * p.page, page = id < 0 ? 0 : id;
                const uint32_t off = tile_off<D>(row, c);
                cp_async16_or_zero(dst + off, kbase + page * p.ks[0] + rem * p.ks[1] + c * 8, id >= 0);
                cp_async16_or_zero(dst + kKV + off, vbase + page * p.vs[0] + rem * p.vs[1] + c * 8, id >= 0);
            }
        }
        cp_async_commit();
    };
    const int ntiles = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load(i);

    // query rows
    for (int e = tid; e < kRows * kPieces; e += kChunkThreads) {
        const int row = e / kPieces, c = e - row * kPieces, q = row0 + row;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (q < rows) {
            const int i = (int)page_div((uint32_t)q, p.G, p.group_magic), h = kvh * p.G + (q - i * p.G);
            v = ldg16(qbase + i * p.qs[1] + h * p.qs[2] + c * 8);
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
    // how many of the positions from tok on row `row` of this block sees
    auto sees = [&](int row, int tok) -> int {
        const int i = (int)page_div((uint32_t)(row0 + row), p.G, p.group_magic);
        return min(ctx + i + 1, hi) - tok;
    };

    for (int tile = 0; tile < ntiles; ++tile) {
        cp_async_wait<kStages - 2>();
        __syncthreads();   // the tile has landed for every thread; the tile before it is consumed
        const int next = lo + (tile + kStages - 1) * kTile;
        if (next < hi && (int)page_div((uint32_t)min(next + kTile, hi) - 1, p.page, p.page_magic) - page0 >= kWindow)
            list_pages(next);
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
        // some row of the block does not see some of these keys
        const bool ragged = tok0 + 16 > min(hi, ctx + token0 + 1);
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[a][b][c] *= p.scale_log2;
        if (ragged) {
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int count = sees(a * 16 + g + 8 * h, tok0 + tq * 2);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (b * 8 + c >= count) s[a][b][2 * h + c] = -INFINITY;
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
                const float mn = fmaxf(m[a][h], mx), at0 = mn == -INFINITY ? 0.f : mn, mu = at0 - kWeightShift<T>;
                moved |= mn != m[a][h];
                alpha[a][h] = ex2_approx(m[a][h] - at0);
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
        if (ragged) {
            // is all of their V finite?
            bool bad = false;
            constexpr uint32_t kExp = Elem<T>::kExpMask;
#pragma unroll 8
            for (int e = lane; e < 16 * kPieces; e += 32) {
                const uint4 v = *reinterpret_cast<const uint4*>(smt + (sv - s0) + (uint32_t)warp * 16 * (D * 2) + e * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) bad |= (w[k] & kExp) == kExp || ((w[k] >> 16) & kExp) == kExp;
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
                    const bool see0 = sees(a * 16 + g, tok0 + t) > 0, see1 = sees(a * 16 + g + 8, tok0 + t) > 0;
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

    float* so = reinterpret_cast<float*>(smt);                  // [4][kRows][D], a row's 8-value pieces c at c ^ (row % 8)
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
                *reinterpret_cast<float2*>(so + (warp * kRows + row) * D + ((b ^ (row & 7)) * 8) + tq * 2) =
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
            const float* src = so + (w * kRows + row) * D + ((c ^ (row & 7)) * 8);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = fmaf(src[k], f, y[k]);
        }
    };
    float* const sx = sml + 4 * kRows * 2;      // cluster: this CTA's rows [kRows][D], then (maximum, sum) [kRows]
    if (kCluster) {
        for (int e = tid; e < kRows * kPieces; e += kChunkThreads) {
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
    for (int e = rank * kChunkThreads + tid; e < kRows * kPieces; e += cluster * kChunkThreads) {
        const int row = e / kPieces, c = e - row * kPieces, q = row0 + row;
        if (q >= rows) break;
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
        const int i = (int)page_div((uint32_t)q, p.G, p.group_magic), h = kvh * p.G + (q - i * p.G);
        const bool empty = sum == 0.f;
        const float inv = 1.f / sum;   // (every score -inf: 0 / 0)
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = len == 0 ? 0.f : y[k] * inv;
        *reinterpret_cast<uint4*>(obase + i * p.os[1] + h * p.os[2] + c * 8) = pack8<T>(y);
        if (p.lse && c == 0)
            p.lse[((p.cu ? (int64_t)first : (int64_t)r * p.T) + i) * p.Hq + h] =
                empty ? -INFINITY : (mu + log2f(sum) - kWeightShift<T>) * 0.6931471805599453f;
    }
    if (kCluster) cluster_sync();   // the others have read this CTA's rows
}

// Joins the parts of an item that kda_chunk_mma.cu has cut: out = sum_c 2^(lse_c - M) o_c /
// sum_c 2^(lse_c - M) over the stretches c that hold one, in their order: slot 1 of a
// stretch, then slot 0 of those behind it up to the item's last part.  A row is the work
// of one warp that takes part after part, or of the block's 8 warps, of every 8th part each
// (the order of the sums is fixed all the same).  A block takes rows blockIdx.y (times 8, with
// a warp a row), and so on: with a block for every 8 rows of a pair the kernel took 6 us where
// nothing was cut.
template <typename T, int D, int W>
__global__ void __launch_bounds__(256) chunk_join_kernel(const ChunkParams p) {
    constexpr int kVec = D / 32;
    __shared__ float sy[W > 1 ? 8 : 1][W > 1 ? D : 1], ssum[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // this block's stretches, one of each wave (kMaxWaves at most), are looked at together
    const int ctas = p.ctas, mine = (int)blockIdx.x + lane * (int)gridDim.x;
    const int4 items = mine < ctas ? p.parts[2 * mine + 1] : make_int4(0, 0, 0, 0);
    for (uint32_t cut = __ballot_sync(0xffffffffu, items.x != 0); cut; cut &= cut - 1) {
        const int wave = __ffs(cut) - 1, cta = (int)blockIdx.x + wave * (int)gridDim.x;
        // its item: request, key head, pair of row tiles
        const int4 item = make_int4(1, __shfl_sync(0xffffffffu, items.y, wave), __shfl_sync(0xffffffffu, items.z, wave),
                                    __shfl_sync(0xffffffffu, items.w, wave));
        int first, n, len;
        chunk_request(p, item.y, first, n, len);
        int count = 1;   // parts, from their states, 32 at a time
        for (int c = cta + 1;; c += 32) {
            const int state = c + lane < ctas ? p.parts[2 * (c + lane)].x : 0;
            const uint32_t stop = __ballot_sync(0xffffffffu, state != 1);
            const int k = stop ? __ffs(stop) - 1 : 32;
            count += k;
            if (stop) {
                if (__shfl_sync(0xffffffffu, state, k) == 2) ++count;
                break;
            }
        }
        for (int in = (int)blockIdx.y * (8 / W) + warp / W; in < 256; in += (int)gridDim.y * (8 / W)) {
            const int row = in & 127, in_token = (int)page_div((uint32_t)row, p.G, p.group_magic);
            const int token = (2 * item.w + (in >> 7)) * p.tile_tokens + in_token;
            if (in_token >= p.tile_tokens || token >= n) continue;   // all of a row's warps
            const auto part = [&](int k) { return (int64_t)(k ? 2 * (cta + k) : 2 * cta + 1) * 256 + in; };
            float mx = -INFINITY, sum = 0.f, y[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) y[i] = 0.f;
            for (int k = lane; k < count; k += 32) mx = fmaxf(mx, p.part_lse[part(k)]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mu = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
            for (int k = W > 1 ? warp : 0; k < count; k += W) {
                const float f = ex2_approx(p.part_lse[part(k)] - mu);
                const float* src = p.part_o + part(k) * D + lane * kVec;
                sum += f;
#pragma unroll
                for (int i = 0; i < kVec; ++i) y[i] = fmaf(src[i], f, y[i]);
            }
            if (W > 1) {
                __syncthreads();   // the row before has been read
                if (lane == 0) ssum[warp] = sum;
#pragma unroll
                for (int i = 0; i < kVec; ++i) sy[warp][lane * kVec + i] = y[i];
                __syncthreads();
                if (warp > 0) continue;
                sum = 0.f;
#pragma unroll
                for (int i = 0; i < kVec; ++i) y[i] = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    sum += ssum[w];
#pragma unroll
                    for (int i = 0; i < kVec; ++i) y[i] += sy[w][lane * kVec + i];
                }
            }
            const int h = item.z * p.G + (row - in_token * p.G);
            const bool empty = sum == 0.f;
            const float inv = 1.f / sum;   // (every score -inf: 0 / 0; a request without keys is not cut)
            uint32_t* dst = reinterpret_cast<uint32_t*>(
                static_cast<T*>(p.out) + (p.cu ? (int64_t)(first + token) * p.os[1] : item.y * p.os[0] + token * p.os[1]) +
                h * p.os[2] + lane * kVec);
#pragma unroll
            for (int k = 0; k < kVec; k += 2) dst[k / 2] = Elem<T>::pack(y[k] * inv, y[k + 1] * inv);
            if (p.lse && lane == 0)
                p.lse[((p.cu ? (int64_t)first : (int64_t)item.y * p.T) + token) * p.Hq + h] =
                    empty ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
        }
    }
}

// Pairs of row tiles of all requests, at most.
int64_t row_pairs(int R, int T, bool packed, int G) {
    const int tt = 128 / G, pt = 2 * tt;
    return packed ? (int64_t)T / pt + R : (int64_t)R * ((T + pt - 1) / pt);
}

// Waves that chunk_mma_kernel may walk, at most: its own conditions (there on the lengths
// themselves), with what they can come to for requests that fit the call.  Pairs beside a
// request's first are together `more` at most, so the row tiles of a head walk no more than
// keys + len * more keys, which has to be above 4 * keys (some request's five pairs or more);
// a wave has kWaveBytes of K and V, and 64 key tiles a stretch.  What a call may need of the
// workspace follows it: 60 single tokens and four pieces of 512 over 4096 (32 / 8 heads of 128)
// 40 MB, where room for eight waves is 321.
int most_waves(int R, int T, bool packed, int Hk, int G, int D, int64_t max_len, int stretches) {
    const int pt = 2 * (128 / G), beside = (T - 1) / pt;
    if (beside < 4) return 1;
    const double more = packed ? (double)beside : (double)R * beside;
    const double len = (double)max_len, requests = packed && T < R ? T : R;
    const double keys = requests * len < len * more / 3 ? requests * len : len * more / 3;
    const double by_keys = ceil(keys * Hk * 4 * D / kWaveBytes);
    const double by_line = floor(Hk * (keys + len * more + kItemKeys * (more + requests)) / (64.0 * 128 * stretches));
    const double waves = by_keys < by_line ? by_keys : by_line;
    return waves < 1 ? 1 : waves > kMaxWaves ? kMaxWaves : (int)waves;
}

template <typename T, int W>
cudaError_t launch_join_w(const ChunkParams& p, int D, cudaStream_t s) {
    const dim3 grid((unsigned)(p.ctas / p.waves), 16);
    const auto kernel = D == 64 ? chunk_join_kernel<T, 64, W>
                                : D == 128 ? chunk_join_kernel<T, 128, W> : chunk_join_kernel<T, 256, W>;
    return launch_maybe_pdl(kernel, grid, dim3(256), 0, s, true, p);
}
template <typename T>
cudaError_t launch_join(const ChunkParams& p, int D, cudaStream_t s) {
    if (p.ctas <= 1) return cudaSuccess;   // one CTA cuts nothing
    // Eight warps a row where the rows are few and are cut into many parts.
    const bool wide = (int64_t)p.T * p.G <= 64 && p.ctas >= 8 * row_pairs(p.R, p.T, p.cu != nullptr, p.G) * p.Hk;
    return wide ? launch_join_w<T, 8>(p, D, s) : launch_join_w<T, 1>(p, D, s);
}

int rows_per_block(int64_t rows, int D) { return rows <= 16 || D > 128 ? 16 : 32; }
// Blocks of rows of all requests: exactly (padded), or at most (packed).
int64_t row_blocks(int R, int T, bool packed, int G, int block) {
    const int64_t rows = (int64_t)T * G;
    return packed ? rows / block + R : (int64_t)R * ((rows + block - 1) / block);
}

template <typename T, int D, int MT, bool kCluster>
cudaError_t launch_rows_t(const ChunkParams& q, cudaStream_t s) {
    ChunkParams p = q;
    // no more tiles in flight than a CTA has, so that more CTAs of short contexts share an SM
    const int64_t tiles = ((p.max_len + kTile - 1) / kTile + p.cluster - 1) / p.cluster;
    p.stages = tiles < 1 ? 1 : tiles < kStages ? (int)tiles : kStages;
    const auto bytes = [](int stages) -> size_t {
        const size_t load = (size_t)stages * 2 * kTile * D * 2 + 16 * MT * D * 2;
        const size_t join = (size_t)16 * MT * (kCluster ? 5 * D + 10 : 4 * D + 8) * sizeof(float);
        return load > join ? load : join;
    };
    const auto kernel = chunk_rows_kernel<T, D, MT, kCluster>;
    static std::atomic<uint64_t> smem_set;
    cudaError_t e = set_smem_limit_once((const void*)kernel, (int)bytes(kStages), smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(row_blocks(p.R, p.T, p.cu != nullptr, p.G, 16 * MT) * p.cluster), (unsigned)p.Hk);
    cfg.blockDim = dim3(kChunkThreads);
    cfg.dynamicSmemBytes = bytes(p.stages);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <typename T, int D, int MT>
cudaError_t launch_rows_m(const ChunkParams& p, cudaStream_t s) {
    return p.cluster > 1 ? launch_rows_t<T, D, MT, true>(p, s) : launch_rows_t<T, D, MT, false>(p, s);
}
template <typename T>
cudaError_t launch_rows(const ChunkParams& p, int D, cudaStream_t s) {
    const bool one = rows_per_block((int64_t)p.T * p.G, D) == 16;
    if (D == 64) return one ? launch_rows_m<T, 64, 1>(p, s) : launch_rows_m<T, 64, 2>(p, s);
    if (D == 128) return one ? launch_rows_m<T, 128, 1>(p, s) : launch_rows_m<T, 128, 2>(p, s);
    return launch_rows_m<T, 256, 1>(p, s);
}

}  // namespace

ChunkPlan chunk_plan(int R, int T, bool packed, int Hk, int G, int D, int64_t max_len, int page, float scale, bool in_place,
                     int num_sms) {
    ChunkPlan t;
    // Pages have to be whole 8-row groups of a tile, a row tile whole tokens, the scale's
    // reciprocal finite.  With head size 256 the two CTAs of an item both read all of its
    // queries and each writes a half of its results, in no order: not where the results
    // replace the queries.
    t.mma = page % 8 == 0 && G <= 128 && scale > 1e-30f && num_sms > 1 && !(in_place && D == 256);
    t.grid = num_sms;
    t.stretches = t.mma ? D == 256 ? t.grid / 2 : t.grid : 0;
    t.waves = 1;
    // The rows kernel (also for layouts without a tensor map): clusters where the blocks are
    // fewer than the CTAs that run at once (what the tiles in flight leave room for, or for D
    // 64 the registers), at least 128 tokens a CTA.
    const int at_once = num_sms * (D == 64 ? 4 : D == 128 ? 2 : 1);
    const int64_t blocks = row_blocks(R, T, packed, G, rows_per_block((int64_t)T * G, D)) * Hk;
    const int64_t tiles = (max_len + kTile - 1) / kTile;
    int64_t parts = blocks > 0 ? at_once / blocks : 1;
    if (parts > (tiles + 1) / 2) parts = (tiles + 1) / 2;
    t.cluster = parts >= 8 ? 8 : parts >= 4 ? 4 : parts >= 2 ? 2 : 1;
    if (t.mma) {
        // The kernel for few rows where its estimated time (us) is the shorter one by a margin, since
        // ragged contexts are the other's strength: a 64-key tile a CTA and wave against the
        // tensor-core kernel's 17 us of set-up and join and its stretch of the line of work, in
        // 128-key tiles.  Head size 128: 1 request, 2 key heads, 1 token over 250 keys 6.9 us
        // against 13.8, over 4000 13.4 and 17.3, over 16000 35.7 and 20.8; 256 tokens, 8 key heads
        // over 250 19 and 25, over 1000 37 and 29; 16 requests x 1 token, 8 key heads over up to
        // 1000 18 and 23, over 4000 53 and 41.
        const double waves = (double)((blocks * t.cluster + at_once - 1) / at_once);
        const double rows_us = 4.0 + waves * ((tiles + t.cluster - 1) / t.cluster) * (D == 64 ? 0.9 : D == 128 ? 1.15 : 2.2);
        const double keys = (double)row_pairs(R, T, packed, G) * Hk * (0.8 * max_len + 256.0) / t.stretches;
        const double mma_us = 17.0 + keys / 128 * (D == 64 ? 1.15 : D == 128 ? 1.4 : 2.1);
        t.mma = mma_us < 1.25 * rows_us;
        if (!t.mma) t.stretches = 0;
        else t.waves = most_waves(R, T, packed, Hk, G, D, max_len, t.stretches);
        t.stretches *= t.waves;
    }
    return t;
}

cudaError_t launch_chunk_attention(const ChunkParams& p, const ChunkPlan& plan, int D, bool f16, cudaStream_t s) {
    ChunkParams q = p;
    q.cluster = plan.cluster;
    q.ctas = plan.stretches;
    q.waves = plan.waves;
    q.tile_tokens = 128 / q.G;
    cudaError_t e = cudaSuccess;
    if (plan.mma && launch_chunk_mma(q, D, f16, plan.grid, s, &e)) {
        if (e != cudaSuccess) return e;
        return f16 ? launch_join<__half>(q, D, s) : launch_join<__nv_bfloat16>(q, D, s);
    }
    return f16 ? launch_rows<__half>(q, D, s) : launch_rows<__nv_bfloat16>(q, D, s);
}

}  // namespace kda
