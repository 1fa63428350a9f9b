// kda_pool.cu -- copies between the entries of pools (kda_pool_copy in
// include/kda_ops.h: cache pages, KDA states, convolution states of requests that are
// forked) and the rows of a verified tree's accepted nodes moved together behind their
// context in the caches of all layers (kda_cache_commit).
//
// Both move bytes: each is read and written once, and what counts is that many 16-byte
// loads are on their way before the first store.  All pools of a call (48 a launch) go in
// one grid, since a layer's share alone would not fill the GPU.  Measured (GPU time): 16
// states in 12 pools (805 MB read and written) 117 us, 6.9 TB/s; 24 pages in 32 caches 18.8 us
// (5.6); the accepted rows of 256 requests in 32 caches 28 us for 108 MB, two waves of CTAs of some
// 60 KB, bound by the chain of path, page table and rows and the barriers between their reads and
// writes, one request 3 us.
#include "kda_internal.h"
#include "ops_internal.h"

namespace kda {
namespace {

constexpr int kPoolThreads = 256;
constexpr int kBatch = 8;                             // pieces a thread has on their way
constexpr int kSlicePieces = kPoolThreads * kBatch;   // pieces a CTA of the copy takes

// Byte offset of piece e of an entry (its rows and columns in order).
__device__ __forceinline__ int64_t piece_at(const PoolDesc& d, uint32_t e) {
    const uint32_t run = page_div(e, (uint32_t)d.pieces, d.piece_magic), piece = e - run * (uint32_t)d.pieces;
    const uint32_t row = page_div(run, (uint32_t)d.cols, d.col_magic), col = run - row * (uint32_t)d.cols;
    return row * d.st[1] + col * d.st[2] + (int64_t)piece * 16;
}

__global__ void __launch_bounds__(kPoolThreads) pool_copy_kernel(const __grid_constant__ PoolCopyParams p) {
    const PoolDesc& d = p.pool[blockIdx.z];
    const int i = blockIdx.y;
    const int src = p.src[i], dst = p.dst[i], given = p.rows ? p.rows[i] : d.rows;
    if (src < 0 || dst < 0 || src == dst) return;
    if (src >= d.entries || dst >= d.entries || given < 0 || given > d.rows) {
        if (p.status && threadIdx.x == 0 && blockIdx.x == 0) atomicMax(p.status, 1);
        return;
    }
    const uint32_t total = (uint32_t)given * (uint32_t)d.cols * (uint32_t)d.pieces;
    const char* from = d.data + src * d.st[0];
    char* to = d.data + dst * d.st[0];
    for (uint32_t base = blockIdx.x * (uint32_t)kSlicePieces + threadIdx.x; base < total; base += gridDim.x * (uint32_t)kSlicePieces) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t e = base + k * kPoolThreads;
            if (e < total) v[k] = *reinterpret_cast<const uint4*>(from + piece_at(d, e));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t e = base + k * kPoolThreads;
            if (e < total) *reinterpret_cast<uint4*>(to + piece_at(d, e)) = v[k];
        }
    }
}

constexpr int kPathMax = 256;
// As kBatch.  With 8 the case below takes 47 us instead of 30 where six CTAs share an SM
// (registers spill), and 29, hardly less, where four do.
constexpr int kCommitBatch = 4;

// A CTA takes a request's path in `group` caches (or a split of the rows' pieces).  The path
// ascends, so path[j] >= j: in the order of j no row is written before it has been read, and a
// batch of pieces in that order can be read as a whole before it is written.  The pieces of
// all of the CTA's caches, which have rows of the same size then, are one sequence: finding the
// rows' places is a chain of four loads, which a CTA a cache paid each time (256 requests, 32
// caches, rows of 2 KB, calls one after the other: 30 us, 37 with a CTA a cache).
__global__ void __launch_bounds__(kPoolThreads, 6) cache_commit_kernel(const __grid_constant__ CacheCommitParams p) {
    __shared__ int2 s_from[kPathMax], s_to[kPathMax];   // page (< 0: none) and row of a moved node and of its new place
    __shared__ int s_first;
    __shared__ uint32_t s_magic[2];   // of the two divisions of a piece's number
    const int k0 = blockIdx.z * p.group, caches = min(p.group, p.pools - k0);
    const PoolDesc& d0 = p.pool[k0];
    const int r = blockIdx.y, tid = threadIdx.x;
    const int ctx = p.ctx[r], n = p.accepted[r];
    const int32_t* path = p.path + (int64_t)r * p.max_path;
    const bool report = p.status && blockIdx.x == 0;
    if (ctx < 0 || n < 0 || n > p.max_path) {
        if (report && tid == 0) atomicMax(p.status, 1);
        return;
    }
    if (tid == 0) s_first = n;
    __syncthreads();
    bool ok = true;
    if (tid < n) {   // n <= kPathMax = kPoolThreads
        const int node = path[tid];
        ok = (tid == 0 ? node >= 0 : node > path[tid - 1]) && (int64_t)ctx + node < p.room;
        if (ok && node != tid) {
            const auto place = [&](int at) {
                const int pg = (int)page_div((uint32_t)at, p.page, p.page_magic);
                return make_int2(p.table[r * p.table_stride + pg], at - pg * p.page);
            };
            s_from[tid] = place(ctx + node);
            s_to[tid] = place(ctx + tid);
            atomicMin(&s_first, tid);
        }
    }
    if (!__syncthreads_and(ok)) {
        if (report && tid == 0) atomicMax(p.status, 1);
        return;
    }
    // path[j] = j up to s_first, and never again behind it
    const int first = s_first;
    if (first == n) return;   // nothing moves
    const uint32_t row_pieces = (uint32_t)(d0.cols * d0.pieces);
    const uint32_t c0 = (uint32_t)((uint64_t)row_pieces * blockIdx.x / gridDim.x),
                   width = (uint32_t)((uint64_t)row_pieces * (blockIdx.x + 1) / gridDim.x) - c0;
    const uint32_t each = (uint32_t)(n - first) * width, total = each * (uint32_t)caches;
    if (tid < 2) {
        const uint32_t d = tid ? width : each;
        s_magic[tid] = d == 1 ? 0xffffffffu : (uint32_t)((1ull << 32) / d);
    }
    __syncthreads();
    const uint32_t each_magic = s_magic[0], width_magic = s_magic[1];
    for (uint32_t base = tid; base - tid < total; base += kCommitBatch * kPoolThreads) {
        uint4 v[kCommitBatch];
        char* to[kCommitBatch];
#pragma unroll
        for (int k = 0; k < kCommitBatch; ++k) {
            const uint32_t e = base + k * kPoolThreads;
            to[k] = nullptr;
            if (e < total) {
                const uint32_t cache = page_div(e, each, each_magic), in = e - cache * each;
                const uint32_t j = page_div(in, width, width_magic), c = c0 + (in - j * width);
                const PoolDesc& d = p.pool[k0 + cache];
                const int2 a = s_from[first + j], b = s_to[first + j];
                const uint32_t col = page_div(c, (uint32_t)d0.pieces, d0.piece_magic), piece = c - col * (uint32_t)d0.pieces;
                const int64_t in_row = col * d.st[2] + (int64_t)piece * 16;
                if (a.x >= 0 && a.x < d.entries && b.x >= 0 && b.x < d.entries) {
                    v[k] = *reinterpret_cast<const uint4*>(d.data + a.x * d.st[0] + a.y * d.st[1] + in_row);
                    to[k] = d.data + b.x * d.st[0] + b.y * d.st[1] + in_row;
                } else if (p.status) {
                    atomicMax(p.status, 1);
                }
            }
        }
        __syncthreads();   // the batch is read
#pragma unroll
        for (int k = 0; k < kCommitBatch; ++k)
            if (to[k]) *reinterpret_cast<uint4*>(to[k]) = v[k];
    }
}

}  // namespace

cudaError_t launch_pool_copy(const PoolCopyParams& q, cudaStream_t s) {
    int64_t most = 1;
    for (int k = 0; k < q.pools; ++k) {
        const int64_t n = (int64_t)q.pool[k].rows * q.pool[k].cols * q.pool[k].pieces;
        most = n > most ? n : most;
    }
    const int64_t slices = (most + kSlicePieces - 1) / kSlicePieces;
    const dim3 grid((unsigned)(slices < 65535 ? slices : 65535), (unsigned)q.count, (unsigned)q.pools);
    pool_copy_kernel<<<grid, kPoolThreads, 0, s>>>(q);
    return cudaGetLastError();
}

cudaError_t launch_cache_commit(const CacheCommitParams& q, int num_sms, cudaStream_t s) {
    CacheCommitParams p = q;
    const auto row = [&](int k) { return p.pool[k].cols * p.pool[k].pieces; };
    int least = row(0);
    bool same = true;   // rows of one size in every cache (a layout of their own each)
    for (int k = 1; k < p.pools; ++k) {
        same = same && p.pool[k].cols == p.pool[0].cols && p.pool[k].pieces == p.pool[0].pieces;
        least = row(k) < least ? row(k) : least;
    }
    // Some 12 CTAs an SM, two waves: so many caches a CTA, or where the (request, cache) pairs are fewer than
    // two CTAs an SM the rows are cut, at least 8 pieces (128 bytes) a CTA.
    const int64_t pairs = (int64_t)p.R * p.pools;
    p.group = same ? (int)((pairs + 12 * num_sms - 1) / (12 * num_sms)) : 1;
    if (p.group > p.pools) p.group = p.pools;
    // a CTA's pieces are counted in 32 bits
    while (p.group > 1 && (int64_t)p.max_path * row(0) * p.group > (1 << 30)) p.group /= 2;
    int64_t splits = 2 * num_sms / pairs;
    if (splits > least / 8) splits = least / 8;
    if (splits < 1) splits = 1;
    const dim3 grid((unsigned)splits, (unsigned)p.R, (unsigned)((p.pools + p.group - 1) / p.group));
    cache_commit_kernel<<<grid, kPoolThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
