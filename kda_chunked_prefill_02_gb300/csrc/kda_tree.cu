// kda_tree.cu -- attention of drafted tokens over a paged cache
// (kda_tree_attention in include/kda_ops.h): the kernel for few query rows, the
// kernel that joins the parts of long contexts, and the choice between the kernels.
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
// How a call is cut.  Where the (request, key head, block of rows) items are more
// than the CTAs that run at once, a CTA takes an item, the requests longest first
// (tree_order_kernel ranks them, as the chunk table ranks prefill's sequences), so
// that the last CTAs are short ones.  Where they are fewer and short, an item is the
// work of a cluster of up to 8 CTAs, an equal stretch of its tiles each, which join
// their rows through distributed shared memory: no second launch and no workspace.
// Where they are fewer and long, the tiles of all items make one line, of which every
// CTA takes an equal stretch, so that ragged contexts leave no SM idle; the parts of
// an item that is cut leave normalised rows and their log-sum in the workspace, joined
// in the CTAs' order by tree_join_kernel (also kda_tree_mma.cu's).
//
// Measured (bf16, D 128): 256 requests x 8 key heads x 16 rows over 0.2 to 1 times
// 4096 tokens 387 us, 6.7 TB/s; one request, 8 key heads, 4 rows, 131072 tokens 87 us,
// 6.2 TB/s; one request, 2 key heads, 1000 tokens 6.8 us.
//
// Keys that a row does not see are taken out of the scores by a select, and
// rows of V past the end are zero-filled in shared memory.  V of a drafted
// token is seen by some rows only, and 0 * NaN is NaN: a tile that holds
// drafted tokens whose V is not finite takes a scalar product that leaves out
// what a row does not see.
#include "kda_internal.h"
#include "ops_internal.h"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace kda {
namespace {

constexpr int kTreeThreads = 128;
constexpr int kTile = 64;      // tokens a tile, 16 a warp
constexpr int kStages = 3;
constexpr int kOrderMax = 1024;   // requests that are ranked
constexpr int kLineMax = 512;    // requests on a line
// Tiles' worth of the line that an item's way in and out takes (20 requests x 2 key heads of
// up to 4000 tokens: 17.8 us with 0, 16.7 with 1, 16.2 with 2, 16.4 with 4).
constexpr int kItem = 2;
constexpr int kWindow = 256;      // pages listed at a time (a tile has at most kTile)
// How the rows kernel is cut: a CTA, a cluster an item, or CTAs over equal stretches of the line of items.
constexpr int kByItem = 0, kByCluster = 1, kByLine = 2;
constexpr int kJoinParts = 4, kJoinRows = 64;   // see launch_join
template <typename T> constexpr bool elem_is_f16() { return std::is_same<T, __half>::value; }
// The probabilities meet V in its type.  fp16 ends at 2^-24, and a long context may have its
// weight in keys far below the largest, so there they are 2^15 times as large (the sum of the
// softmax too; only the log-sum takes the factor back).
template <typename T> constexpr float kWeightShift = elem_is_f16<T>() ? 15.f : 0.f;

template <typename T, int D, int MT, int kMode>
__global__ void __launch_bounds__(kTreeThreads) tree_rows_kernel(const TreeParams p) {
    constexpr bool kCluster = kMode == kByCluster, kLine = kMode == kByLine;
    constexpr int kRows = 16 * MT;
    constexpr uint32_t kKV = kTile * D * 2, kStage = 2 * kKV;
    extern __shared__ __align__(128) uint8_t smt[];
    __shared__ int spage[kWindow];
    __shared__ int32_t s_start[kLine ? kLineMax + 1 : 1];   // where every request begins on the line, in tiles
    uint8_t* sq = smt + p.stages * kStage;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const int cluster = kCluster ? p.cluster : 1, rank = kCluster ? blockIdx.x % cluster : 0;
    // the item: request, key head, block of rows; its tiles and this CTA's part t0 .. t1 of them
    int r = kLine ? 0 : blockIdx.z, kvh = blockIdx.y, row0 = (int)(blockIdx.x / cluster) * kRows, tiles = 0, t0 = 0, t1 = 0;
    // line: head and block, where the item begins, this CTA's stretch; an item takes kItem
    // tiles' worth of the line for its way in and out, then its tiles
    int hb = 0, item = 0, at = 0, end = 0;
    const auto start = [&](int i) { return s_start[i] + i * kItem; };   // of request i, a head's and block's part
    if (kLine) {
        if (warp == 0) {
            int sum = 0;
            for (int r0 = 0; r0 < p.R; r0 += 32) {
                int ctx, len, t = 0;
                if (r0 + lane < p.R) {
                    tree_lengths(p, r0 + lane, ctx, len);
                    t = max(1, (ctx + len + kTile - 1) / kTile);   // rows that see nothing are written too
                }
                int upto = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                if (r0 + lane < p.R) s_start[r0 + lane] = sum + upto - t;
                sum += __shfl_sync(0xffffffffu, upto, 31);
            }
            if (lane == 0) s_start[p.R] = sum;
        }
        __syncthreads();
        const int per = p.Hk * p.row_blocks, total = start(p.R) * per;
        const int ctas = max(1, min((int)gridDim.x, s_start[p.R] * per / 2));   // at least two tiles each
        if (tid < 2) p.parts[2 * blockIdx.x + tid] = make_int4(0, 0, 0, 0);
        if ((int)blockIdx.x >= ctas) return;
        const int each = total / ctas, rest = total - each * ctas, b = blockIdx.x;
        at = each * b + min(b, rest);
        end = at + each + (b < rest ? 1 : 0);
        int hi = p.R;
        while (hi - r > 1) {
            const int mid = (r + hi) >> 1;
            if (start(mid) * per <= at) r = mid; else hi = mid;
        }
        tiles = s_start[r + 1] - s_start[r];
        const int off = at - start(r) * per;
        hb = off / (tiles + kItem);
        item = at - (off - hb * (tiles + kItem));
        __syncthreads();   // parts are cleared before a thread writes one
    } else if (p.order) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        r = p.order[r];
    }

    for (;;) {   // once, or an item of the line after the other
        if (kLine && item + kItem >= end) break;   // none of its tiles
        int ctx, n;
        if (!tree_lengths(p, r, ctx, n) && p.status && tid == 0) atomicMax(p.status, 1);
        const int len = ctx + n;
        if (kLine) {
            kvh = hb / p.row_blocks;
            row0 = (hb - kvh * p.row_blocks) * kRows;
            t0 = max(0, at - item - kItem);
            t1 = min(tiles, end - item - kItem);
        } else {
            tiles = (len + kTile - 1) / kTile;
            t0 = tiles * rank / cluster;
            t1 = tiles * (rank + 1) / cluster;
        }
        const int lo = t0 * kTile, hi = min(t1 * kTile, len);

        // the pages of this part, kWindow at a time
        int page0 = 0;
        auto list_pages = [&](int tok) {
            page0 = (int)page_div((uint32_t)tok, p.page, p.page_magic);
            const int count = hi > tok ? min(kWindow, (int)page_div((uint32_t)(hi - 1), p.page, p.page_magic) - page0 + 1) : 0;
            for (int e = tid; e < count; e += kTreeThreads) {
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
        constexpr int kPieces = D / 8, kRowsPass = kTreeThreads / kPieces;
        auto load = [&](int tile) {
            if (lo + tile * kTile < hi) {
                const uint32_t dst = s0 + (tile % kStages) * kStage;
                const int c = tid % kPieces;
#pragma unroll
                for (int j = 0; j < kTile / kRowsPass; ++j) {
                    const int row = tid / kPieces + j * kRowsPass;
                    const uint32_t tok = (uint32_t)(lo + tile * kTile + row), pg = page_div(tok, p.page, p.page_magic);
                    const bool in = (int)tok < hi;
                    const int id = in ? spage[(int)pg - page0] : -1;
                    const int64_t rem = tok - pg * p.page, page = id < 0 ? 0 : id;
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
                const int i = (int)page_div((uint32_t)q, p.G, p.group_magic), h = kvh * p.G + (q - i * p.G);
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
        // visibility of positions tok .. tok + 31 to row `row` of this block
        auto seen = [&](int row, int tok) -> uint32_t {
            const int i = min((int)page_div((uint32_t)(row0 + row), p.G, p.group_magic), p.N - 1);
            return tree_seen(p, tree_mask_row(p, r, i), i, ctx, hi, tok);
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
            const bool ragged = tok0 + 16 > hi || tok0 + 16 > ctx;
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
                        const uint32_t bits = seen(a * 16 + g + 8 * h, tok0) >> (tq * 2);
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (!((bits >> (b * 8 + c)) & 1u)) s[a][b][2 * h + c] = -INFINITY;
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
            if (tok0 + 16 > ctx) {
                // drafted tokens: is all of their V finite?
                bool bad = false;
                constexpr uint32_t kExp = Elem<T>::kExpMask;
#pragma unroll 8
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
                        const bool see0 = seen(a * 16 + g, tok0) >> t & 1u, see1 = seen(a * 16 + g + 8, tok0) >> t & 1u;
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
        const bool whole = t0 == 0 && t1 == tiles;
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
            const int i = (int)page_div((uint32_t)q, p.G, p.group_magic);
            const bool empty = i >= n || sum == 0.f;
            const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = empty ? 0.f : y[k] * inv;
            const float lse = empty ? -INFINITY : mu + log2f(sum) - kWeightShift<T>;
            if (!kLine || whole) {
                const int h = kvh * p.G + (q - i * p.G);
                *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + r * p.os[0] + i * p.os[1] + h * p.os[2] + c * 8) =
                    pack8<T>(y);
                if (p.lse && c == 0) p.lse[((int64_t)r * p.N + i) * p.Hq + h] = lse * 0.6931471805599453f;
            } else {
                const int64_t part = (int64_t)(2 * blockIdx.x + (t0 > 0 ? 0 : 1)) * kRows + row;
                float4* dst = reinterpret_cast<float4*>(p.part_o + part * D + c * 8);
                dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                if (c == 0) p.part_lse[part] = lse;
            }
        }
        if (kCluster) cluster_sync();   // the others have read this CTA's rows
        if (!kLine) break;
        if (!whole && tid == 0)
            p.parts[2 * blockIdx.x + (t0 > 0 ? 0 : 1)] = make_int4(t1 == tiles ? 2 : 1, r, kvh, row0 / kRows);
        item += kItem + tiles;
        if (item >= end) break;
        if (++hb == p.Hk * p.row_blocks) {
            hb = 0;
            ++r;
            tiles = s_start[r + 1] - s_start[r];
        }
        __syncthreads();   // the rows have been read: their memory takes the next tiles
    }
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

// Joins the parts of a cut item: out = sum_c 2^(lse_c - M) o_c / sum_c 2^(lse_c - M)
// over the CTAs c that hold one, in their order: slot 1 of CTA blockIdx.x, then
// slot 0 of those behind it up to the item's last part.  A row is the work of one
// warp that takes part after part, or of W > 1 warps, of every W-th part each (the
// order of the sums is fixed all the same).
template <typename T, int D, int W>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p) {
    constexpr int kVec = D / 32;
    __shared__ float sy[W > 1 ? 8 : 1][W > 1 ? D : 1], ssum[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in = blockIdx.y * (8 / W) + warp / W;
    const int cta = blockIdx.x, ctas = p.slots / 2;
    const int4 item = p.parts[2 * cta + 1];   // state, request, key head, block of rows
    const int row = item.w * p.slot_rows + in;
    if (item.x == 0 || in >= p.slot_rows || row >= p.rows) return;   // all of a row's warps
    const auto part = [&](int k) { return (int64_t)(k ? 2 * (cta + k) : 2 * cta + 1) * p.slot_rows + in; };
    float mx = -INFINITY, sum = 0.f, y[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) y[i] = 0.f;
    if (W == 1) {
        for (int k = 0, state = item.x;;) {
            const float lse = p.part_lse[part(k)];
            const float* src = p.part_o + part(k) * D + lane * kVec;
            float o[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) o[i] = src[i];
            const float mn = fmaxf(mx, lse), mu = mn == -INFINITY ? 0.f : mn;
            const float fo = ex2_approx(mx - mu), fn = ex2_approx(lse - mu);
            sum = sum * fo + fn;
#pragma unroll
            for (int i = 0; i < kVec; ++i) y[i] = y[i] * fo + o[i] * fn;
            mx = mn;
            if (state == 2 || cta + ++k >= ctas) break;
            state = p.parts[2 * (cta + k)].x;
            if (state == 0) break;
        }
    } else {
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
        for (int k = lane; k < count; k += 32) mx = fmaxf(mx, p.part_lse[part(k)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mu = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
        for (int k = warp % W; k < count; k += W) {
            const float f = ex2_approx(p.part_lse[part(k)] - mu);
            const float* src = p.part_o + part(k) * D + lane * kVec;
            sum += f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) y[i] = fmaf(src[i], f, y[i]);
        }
        if (lane == 0) ssum[warp] = sum;
#pragma unroll
        for (int i = 0; i < kVec; ++i) sy[warp][lane * kVec + i] = y[i];
        named_bar_sync(1 + warp / W, 32 * W);
        if (warp % W > 0) return;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[i] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            sum += ssum[warp + w];
#pragma unroll
            for (int i = 0; i < kVec; ++i) y[i] += sy[warp + w][lane * kVec + i];
        }
    }
    const int r = item.y, i = (int)page_div((uint32_t)row, p.G, p.group_magic), h = item.z * p.G + (row - i * p.G);
    const bool empty = sum == 0.f;
    const float inv = empty ? 0.f : 1.f / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + r * p.os[0] + i * p.os[1] + h * p.os[2] +
                                                lane * kVec);
#pragma unroll
    for (int k = 0; k < kVec; k += 2) dst[k / 2] = Elem<T>::pack(y[k] * inv, y[k + 1] * inv);
    if (p.lse && lane == 0)
        p.lse[((int64_t)r * p.N + i) * p.Hq + h] = empty ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
}

int rows_per_block(int rows, int D) { return rows <= 16 || D > 128 ? 16 : 32; }

template <typename T, int D, int MT, int kMode>
cudaError_t launch_rows_mode(const TreeParams& q, const TreePlan& plan, cudaStream_t s) {
    TreeParams p = q;
    // no more tiles in flight than a CTA has, so that more CTAs of short contexts share an SM
    const int64_t tiles = ((p.max_len + kTile - 1) / kTile + p.cluster - 1) / p.cluster;
    p.stages = tiles < 1 ? 1 : tiles < kStages ? (int)tiles : kStages;
    // the tiles in flight and the queries; then the warps' rows, and a cluster's
    const auto bytes = [](int stages) -> size_t {
        const size_t load = (size_t)stages * 2 * kTile * D * 2 + 16 * MT * D * 2;
        const size_t join = (size_t)16 * MT * (kMode == kByCluster ? 5 * D + 10 : 4 * D + 8) * sizeof(float);
        return load > join ? load : join;
    };
    const auto kernel = tree_rows_kernel<T, D, MT, kMode>;
    static std::atomic<uint64_t> smem_set;
    cudaError_t e = set_smem_limit_once((const void*)kernel, (int)bytes(kStages), smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    if (kMode == kByCluster) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)p.cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    } else {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // right after tree_order_kernel
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = kMode == kByLine ? dim3((unsigned)plan.row_grid)
                                   : dim3((unsigned)(p.row_blocks * p.cluster), (unsigned)p.Hk, (unsigned)p.R);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = bytes(p.stages);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = kMode == kByCluster || p.order ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <typename T, int D, int MT>
cudaError_t launch_rows_t(const TreeParams& q, const TreePlan& plan, cudaStream_t s) {
    TreeParams p = q;
    p.row_blocks = (p.rows + 16 * MT - 1) / (16 * MT);
    if (plan.line) {
        p.slots = 2 * plan.row_grid;
        p.slot_rows = 16 * MT;
        const cudaError_t e = launch_rows_mode<T, D, MT, kByLine>(p, plan, s);
        return e == cudaSuccess ? launch_tree_join(p, D, elem_is_f16<T>(), s) : e;
    }
    if (p.cluster > 1) return launch_rows_mode<T, D, MT, kByCluster>(p, plan, s);
    if (p.order) {
        tree_order_kernel<<<1, kOrderMax, 0, s>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return launch_rows_mode<T, D, MT, kByItem>(p, plan, s);
}

template <typename T>
cudaError_t launch_rows(const TreeParams& p, const TreePlan& plan, int D, cudaStream_t s) {
    const bool one = rows_per_block(p.rows, D) == 16;
    if (D == 64) return one ? launch_rows_t<T, 64, 1>(p, plan, s) : launch_rows_t<T, 64, 2>(p, plan, s);
    if (D == 128) return one ? launch_rows_t<T, 128, 1>(p, plan, s) : launch_rows_t<T, 128, 2>(p, plan, s);
    return launch_rows_t<T, 256, 1>(p, plan, s);
}

template <typename T, int W>
cudaError_t launch_join_w(const TreeParams& p, int D, cudaStream_t s) {
    const int rows = p.rows < p.slot_rows ? p.rows : p.slot_rows;
    const dim3 grid((unsigned)(p.slots / 2 - 1), (unsigned)((rows * W + 7) / 8));
    const auto kernel = D == 64 ? tree_join_kernel<T, 64, W>
                                : D == 128 ? tree_join_kernel<T, 128, W> : tree_join_kernel<T, 256, W>;
    return launch_maybe_pdl(kernel, grid, dim3(256), 0, s, true, p);
}
template <typename T>
cudaError_t launch_join(const TreeParams& p, int D, cudaStream_t s) {
    if (p.slots <= 2) return cudaSuccess;   // one CTA cuts nothing
    const int64_t items = (int64_t)p.R * p.Hk * ((p.rows + p.slot_rows - 1) / p.slot_rows);
    // Warps a row, by the parts that an item is about cut into.  One request, 2 key heads of
    // 16000 tokens (125 parts): 17 us with 8 warps, 44 with one; 16 rows a request, 8 key
    // heads, 131072 tokens (19 parts): 87 and 94; but 192 items of 488 rows (1.6 parts): 136
    // with one, 180 with 8.  Many rows make as many blocks, most of which find no cut item:
    // 8 items x 248 rows over 16000 tokens 44 us with 8 warps, 36 with 2.
    if (p.slots / 2 < kJoinParts * items) return launch_join_w<T, 1>(p, D, s);
    return p.rows <= kJoinRows ? launch_join_w<T, 8>(p, D, s) : launch_join_w<T, 2>(p, D, s);
}

}  // namespace

TreePlan tree_plan(int R, int Hk, int rows, int D, int64_t max_len, int page, float scale, int num_sms) {
    TreePlan t;
    // The 128-row products where there are more rows than one product of the warp-level
    // kernel takes and enough work to outlast their longer way in and out (some 15 us).
    // In one block of 32 rows the rows kernel reads a key once too, and what decides is the
    // context (20 rows, 8 items over up to 1000 tokens 17 us against 11, over 4000 17 against
    // 19; 304 items 37 against 33 and 77 against 84); in more it reads a key once a block (80
    // items x 64 rows over up to 1000 tokens 21 us against 24, over 120 20 against 12; 16 x 64
    // over 2000 21 against 17; 304 x 248 over 120 34 against 79, 16 x 248 over 500 26 against
    // 18; head size 256, blocks of 16: 152 x 64 over 4000 125 against 275, 306 x 40 over 10 47
    // against 25, 304 x 512 over 4000 653 against 4421).  Pages have to be whole 8-row groups
    // of a tile, the scale's reciprocal finite (and the line of work, in key tiles, stays inside
    // 32 bits).
    const int block = rows_per_block(rows, D);
    const int64_t row_blocks = (rows + block - 1) / block, items = (int64_t)R * Hk * row_blocks;
    const int64_t work = items * (max_len + 64);
    t.mma = rows > 16 && page % 8 == 0 && num_sms > 1 && scale > 1e-30f && max_len / 128 + 1 < (1 << 22) &&
            (row_blocks == 1 ? max_len >= 2560 : work >= 98304 && (row_blocks > 2 || max_len >= 512));
    // The rows kernel's cut (also for a cache without a tensor map); at_once is what the
    // tiles in flight leave room for, or for D 64 the registers.
    const int at_once = num_sms * (D == 64 ? 4 : D == 128 ? 2 : 1);
    const int64_t tiles = (max_len + kTile - 1) / kTile;
    // Fewer items than CTAs at once: clusters of up to 8, at least 128 tokens a CTA (one
    // request, 2 key heads, 1000 tokens: 8.5 us, 10.2 as a line), until a CTA's tiles outweigh
    // the line's second launch: 8 rows, 48 items of up to 1000 tokens 11.0 us and 12.1 as a
    // line, 1500 13.3 and 12.5, 4000 25 and 18, 160 items of up to 4000 81 and 43, 80 of head
    // size 256 107 and 50; head size 64, 72 items of up to 4000 14.5 and 15.6, 8000 22.6 and
    // 22.0.  Where a CTA an item fills the GPU nearly as well, the line pays late (304 items
    // of up to 4000 tokens 82 us and 69).
    int64_t parts = items > 0 ? at_once / items : 1;
    if (parts > (tiles + 1) / 2) parts = (tiles + 1) / 2;
    t.cluster = parts >= 8 ? 8 : parts >= 4 ? 4 : parts >= 2 ? 2 : 1;
    t.line = R <= kLineMax && items <= at_once && items * tiles < (1 << 30) &&
             tiles > t.cluster * (items * 8 > at_once * 7 ? 24 : D == 64 ? 12 : 5);
    if (t.line) t.cluster = 1;
    t.row_grid = t.line ? at_once : 0;
    // Ranked where the items outnumber the CTAs that run at once: 100 requests x 8 key heads
    // of 0.2 to 1 times 1000 tokens 53 us against 59, but 22 against 25 the other way with
    // 202 requests of up to 41 (and 34 both ways with 150 of up to 250).
    t.order = !t.mma && !t.line && t.cluster == 1 && R > 1 && R <= kOrderMax && items > at_once && tiles > 4 ? R : 0;
    t.grid = num_sms;
    const int stretches = t.mma ? D == 256 ? t.grid / 2 : t.grid : 0;   // with head size 256 two CTAs share one
    t.parts = (size_t)2 * (stretches > t.row_grid ? stretches : t.row_grid);
    t.part_rows = (size_t)2 * t.row_grid * block;
    if (t.part_rows < (size_t)2 * stretches * 256) t.part_rows = (size_t)2 * stretches * 256;
    return t;
}

cudaError_t launch_tree_join(const TreeParams& p, int D, bool f16, cudaStream_t s) {
    return f16 ? launch_join<__half>(p, D, s) : launch_join<__nv_bfloat16>(p, D, s);
}

cudaError_t launch_tree_attention(const TreeParams& p, const TreePlan& plan, int D, bool f16, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    // With head size 256 the two CTAs of an item both read all of its queries and each
    // writes a half of its results, in no order: not where the results replace the queries.
    const bool in_place = p.out == p.q;
    if (plan.mma && !(in_place && D == 256) && launch_tree_mma(p, D, f16, plan.grid, s, &e)) return e;
    return f16 ? launch_rows<__half>(p, plan, D, s) : launch_rows<__nv_bfloat16>(p, plan, D, s);
}

}  // namespace kda
