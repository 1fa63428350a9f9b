// kda_tree_mma.cu -- kda_tree_attention (include/kda_ops.h) for many query rows
// (a tree of nodes times the query heads of a key head): 128-row tiles on
// tcgen05 tensor cores, S and O in TMEM, K and V pages by TMA.
//
// From about 16 rows on, the products and not the memory bound the warp-level
// kernel of kda_tree.cu; here a tile of 128 rows and 128 keys costs 16
// tcgen05.mma (S = Q K^T, then O += P V).  Persistent CTAs, one an SM:
//   warps 0-3, 4-7  two softmax streams: thread = row (TMEM lane), the whole row
//                   of S in registers, so maximum and sum need no exchange; P
//                   goes back over S's columns as 16-bit pairs, the A operand of
//                   the second product;
//   warp 8          the loader: a ring of K and V tiles in turn;
//   warp 9          issues the products;
//   warp 10         deals out the work, item by item;
//   warp 11         cleans the V tiles that need it.
// The streams alternate, so that one's softmax runs under the other's
// products.  With more than 128 rows they are two row tiles over the same keys
// (each K and V tile is read for 256 rows); with fewer they are the even and
// odd key tiles of one row tile, joined at the end.
//
// The work of a call is one line of key tiles, ordered by request, key head and
// pair of row tiles, and every CTA takes an equal stretch of it (a tile for two
// row tiles counts 5, for one 4, as measured: 1.92 and 1.52 us; an item's way in and
// out as much as several tiles: 24 requests of 4 key heads and 488 rows over up to
// 9000 tokens 136 us without, 124 with), so that ragged contexts leave no SM idle.  A stretch cuts at most two items; the parts of a
// cut item leave normalised rows and their log-sum in the workspace (slot 0 of
// a CTA: a later part of an item, slot 1: the first), joined in the CTAs' order
// by tree_join_kernel (kda_tree.cu).  The loader and the issuer run from
// one item into the next without a halt; only the rows' way out and the next
// queries' way in are between two items.
//
// Head size 256: S of two row tiles and a whole O (256 columns each) do not fit TMEM,
// so two neighbouring CTAs take the same stretch, both with all of S and each with
// one half of V's columns.  That is 3 products where 2 are due, but the keys are read
// for 256 rows at a time (a whole O would leave room for 128) and come out of L2 the
// second time.
//
// Measured: 19 requests x 4 key heads x 512 rows of 128 over 16384 tokens 216 us, 1.51
// PFLOP/s; 38 x 4 x 256 over 8192 122 us, 1.34 PFLOP/s and 5.2 TB/s; head size 256, 152 x 2
// x 512 rows over 0.2 to 1 times 16000 2.24 ms, 1.14 PFLOP/s (15.8 ms in the kernel for
// few rows).
//
// The running maximum moves only when a row's scores exceed it by a factor of
// 2^8 (2^4 in fp16; l and O stay far inside fp32 and P inside its type until
// then), so that O in TMEM is hardly ever rescaled (a published refinement of the softmax in one pass); that is the softmax threads' work, in the time between
// a score tile's arrival (which implies that the product before it is done) and
// their P's.
//
// Keys that a row does not see: only the last tiles hold drafted tokens or
// positions past the end; there every row forms its 128 visibility bits.  In
// those tiles a warp of its own clears V rows past the end and V elements that are not
// finite before the product sees them (0 * NaN is NaN, also for a row whose P is
// zero), and remembers their nodes; the rows that do see such a node take its
// elements at the end.
//
// The third warpgroup gives most of its registers to the softmax warps (56 of
// 168 kept, 224 taken: 4 x 56 + 8 x 224 = 12 x 168), whose threads hold a row of
// 128 scores.
//
// Every wait is bounded; one that runs out sets the abort flag, the roles fall
// through to the end, and the status word reports KDA_ERR_TIMEOUT.  Whatever the
// others do, the loader and the issuer end by waiting for their last copies and
// products (with the full kWaitLimitNs), so that none is in flight when the CTA's
// memory goes to the next.
#include "attn_mma.cuh"
#include "kda_internal.h"
#include "ops_internal.h"
#include "sm103.cuh"

namespace kda {
namespace {

constexpr int kMmaThreads = 384;   // three warpgroups: two softmax streams, loader and issuer
constexpr int kMaxBufs = 8;
constexpr uint32_t kTmemS = 0, kTmemO = 256;   // S of stream s at 128 s, O at 256 + 128 s
// Floats of the rows' way out: a patch a warp, 32 columns of stream 1, its maxima and sums.
constexpr int kPatch = 32 * 36, kWayOut = 8 * kPatch + 34 * 128;
constexpr int kCostTwo = 5, kCostOne = 4;  // cost of a key tile for two row tiles, for one

template <int D> struct MmaShape {
    static constexpr int kV = D == 256 ? 128 : D;   // value columns a CTA
    static constexpr int kHalves = D / kV;          // CTAs that share a stretch, each with its columns
    static constexpr int kPer = kHalves + 1;        // ring slots a key tile: K by kV channels, V
    // Cost of an item's way in and out (some 9 us) beside a key tile's kCostTwo.  With 0, 12,
    // 16, 24, 32: head size 128, 24 requests x 4 key heads x 488 rows over up to 9000 tokens
    // 136, 128, 126, 124, 125 us; 256, 20 x 2 x 248 over up to 6555 100, 93, 94, 97, 98; 64,
    // 20 x 16 x 64 over up to 9286 134, 127, 127, 130, 135.
    static constexpr int kCostItem = D == 256 ? 12 : D == 128 ? 24 : 16;
    static constexpr uint32_t kSlotBytes = (kV / 64) * kBlock, kQBytes = (D / 64) * kBlock;
    // K and V tiles as the copies leave them: groups of 8 keys, in a group 64 channels
    // after the other, 8 rows of 128 bytes each.
    static constexpr uint32_t kGroupBytes = (kV / 64) * 1024;
    // The queries, where the rows also pass on their way out, and the ring of K and V.  With
    // head size 256 one row tile's queries leave room for more of the ring.
    static __host__ __device__ constexpr uint32_t front(int rows) {
        return D == 64 ? 56 * 1024 : D == 256 && rows <= 128 ? kQBytes : 2 * kQBytes;
    }
    static __host__ __device__ constexpr int bufs(int rows) { return D == 64 ? 8 : D == 256 && rows > 128 ? 3 : 5; }
    static constexpr uint32_t smem(int rows) { return front(rows) + bufs(rows) * kSlotBytes + 1024; }   // and alignment
};

static_assert(kWayOut * 4 <= MmaShape<64>::front(1) && kWayOut * 4 <= MmaShape<128>::front(1) &&
                  kWayOut * 4 <= MmaShape<256>::front(1),
              "the way out fits the front");

// One CTA's part of an item (request, key head, pair of row tiles).
struct Item {
    int r, h, rb;      // request, key head, row tiles 2 rb and 2 rb + 1
    int t0, t1;        // key tiles (t1 < 0: no more items)
    int ctx, n;        // the request's context and nodes
    bool two, whole;   // two row tiles; all of the item's key tiles
};
constexpr int kItems = 4;   // items dealt out ahead
// What a wait may take beside its bound, a key tile of the longest context: the cleaner waits
// for an item's last tiles from its first on, and the other roles and the dealer for what the
// kItems items before are done with.  A tile takes some 2 us.
constexpr uint64_t kTileWaitNs = 20000 * (kItems + 1);

template <typename T, int D>
__global__ void __launch_bounds__(kMmaThreads, 1)
    tree_mma_kernel(const TreeParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using Shape = MmaShape<D>;
    constexpr uint32_t kSlotBytes = Shape::kSlotBytes, kQBytes = Shape::kQBytes, kGroupBytes = Shape::kGroupBytes;
    constexpr int kV = Shape::kV, kHalves = Shape::kHalves, kPer = Shape::kPer;
    const int bufs = Shape::bufs(p.rows);
    const int cta = (int)blockIdx.x / kHalves, half = (int)blockIdx.x % kHalves;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t kv_full[kMaxBufs], kv_free[kMaxBufs], kv_raw[kMaxBufs], q_ready, s_full[2], p_half[2], p_ready[2], o_full, o_free;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    // Drafted nodes with a V element that is not finite, for eight items in turn
    // (the ring holds at most four items' tiles ahead of the rows' way out).
    __shared__ uint32_t s_bad[8][8];
    __shared__ int32_t s_start[kTreeSlice + 1];   // where every request begins on the line, in key tiles
    __shared__ Item s_item[kItems];
    __shared__ uint64_t item_full[kItems], item_free[kItems], never;   // never: the probe's, nothing arrives on it

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    volatile int* abort = &abort_flag;
    const uint64_t limit = p.wait_ns;
    uint8_t* ring = sm + Shape::front(p.rows);
    auto fail = [&]() {
        *abort = 1;
        if (p.status) atomicExch(p.status, 4);
    };

    if (tid == 0) {
        for (int i = 0; i < bufs; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_free[i], 1);
            mbar_init(&kv_raw[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_free[i], 4);   // loader, issuer, cleaner, softmax
        }
        mbar_init(&q_ready, 8);   // one arrival a warp
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_half[s], 4);
            mbar_init(&p_ready[s], 4);
        }
        mbar_init(&o_full, 1);
        mbar_init(&o_free, 8);
        mbar_init(&never, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (tid < 64) s_bad[tid >> 3][tid & 7] = 0;
    if (warp == 9) {
        tmem_alloc(&tmem_base_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tmem_base_sh;
    // The k-th item of this CTA; false after the last (or on an abort).
    auto take = [&](int k, Item& x, bool& ok) -> bool {
        ok = ok && wait_for(&item_full[k % kItems], (k / kItems) & 1, abort, limit);
        if (!ok) return false;
        x = s_item[k % kItems];
        return x.t1 >= 0;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 8) {
            // ------------------------------------------------------------ loader
            if (lane == 0) {
                tma_prefetch_desc(&kmap);
                tma_prefetch_desc(&vmap);
            }
            const int box = box_of(p.page), per_tile = kKeys / box;   // this lane's box: tokens lane * box ..
            int issued = 0, item = 0;   // tiles asked for, items begun
            uint32_t raw = 0, raw_phases = ~0u;   // slots whose last copy was a raw one, those copies' phases
            bool ok = true;
            Item x;
            for (; __all_sync(0xffffffffu, take(item, x, ok)) && ok; ++item) {
                if (lane == 0) mbar_arrive(&item_free[item % kItems]);
                const int ctx = x.ctx, hi = ctx + x.n;
                const int32_t* table = p.table + x.r * p.table_stride;
                // this lane's page of a tile, -1: none (asked for a tile ahead, looked at
                // later), and its first row there
                int row_ahead = 0;
                auto page_of = [&](int tile) -> int64_t {
                    const int tok = tile * kKeys + lane * box;
                    const int at = (int)page_div((uint32_t)tok, p.page, p.page_magic);
                    row_ahead = tok - at * p.page;
                    return tile < x.t1 && lane < per_tile && tok < hi ? (int64_t)(uint32_t)table[at] : -1;
                };
                int64_t ahead = page_of(x.t0);
                for (int tile = x.t0; tile < x.t1 && ok; ++tile) {
                    const int id = ahead < 0 ? -1 : (int)min(ahead, (int64_t)p.P);
                    if (ahead >= p.P && p.status) atomicMax(p.status, 1);   // reads zeros: past the map's pages
                    const int row = row_ahead;
                    ahead = page_of(tile + 1);
                    const int base = tile * kKeys;
                    const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, id >= 0)) * box * kV * 2u;
                    for (int part = 0; part < kPer; ++part) {   // K by kV channels, then V
                        const bool v = part == kHalves;
                        const int slot = issued % bufs, round = issued / bufs;
                        if (round > 0) ok = __all_sync(0xffffffffu, wait_for(&kv_free[slot], (round - 1) & 1, abort, limit));
                        if (!ok) break;
                        uint8_t* dst = ring + slot * kSlotBytes;
                        const bool special = v && base + kKeys > ctx;
                        uint64_t* bar = special ? &kv_raw[slot] : &kv_full[slot];   // raw: to warp 11 first
                        raw = special ? raw | 1u << slot : raw & ~(1u << slot);
                        if (special) raw_phases ^= 1u << slot;
                        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                        __syncwarp();
                        if (id >= 0)
                            tma_load_5d(dst + lane * box * kV * 2, v ? &vmap : &kmap, 0, 0,
                                        ((v ? p.v_paged : p.k_paged) ? 0 : x.h * (D / 64)) +
                                            (v ? half : part) * (kV / 64),
                                        row / 8,
                                        (v ? p.v_paged : p.k_paged) ? id * p.Hk + x.h : id, bar);
                        ++issued;
                    }
                }
            }
            if (!__all_sync(0xffffffffu, ok) && lane == 0) fail();
            // the last copies into this CTA's memory
            for (int i = max(0, issued - bufs); i < issued; ++i)
                if (!((raw >> (i % bufs)) & 1)) wait_for(&kv_full[i % bufs], (i / bufs) & 1, nullptr, kWaitLimitNs);
                else wait_for(&kv_raw[i % bufs], (raw_phases >> (i % bufs)) & 1, nullptr, kWaitLimitNs);
        } else if (warp == 9) {
            // ------------------------------------------------------------ products
            // The whole warp walks the loop and one elected lane issues, with every
            // operand a warp-uniform value (taken from lane 0 where it comes from
            // memory): the products' operands live in uniform registers, and a lone
            // thread that has to bring them there issues a product in about 105 cycles,
            // whatever its size.
            constexpr uint32_t id_qk = MmaTypes<T>::qk(kKeys), id_pv = MmaTypes<T>::pv(kV);
            const uint32_t tbu = __shfl_sync(0xffffffffu, tb, 0);
            const uint32_t q_at = __shfl_sync(0xffffffffu, smem_u32(sm), 0),
                           ring_at = q_at + Shape::front(p.rows);
            bool ok = true;
            int item = 0;
            int base = 0;                      // ring tiles before this item
            int done0 = 0, done1 = 0;          // P tiles taken, by stream
            auto landed = [&](int i) { return wait_for(&kv_full[i % bufs], (i / bufs) & 1, abort, limit); };
            Item x;
            for (; __all_sync(0xffffffffu, take(item, x, ok)); ++item) {
                if (lane == 0) mbar_arrive(&item_free[item % kItems]);
                const bool two = __shfl_sync(0xffffffffu, (int)x.two, 0) != 0;
                const int tiles = __shfl_sync(0xffffffffu, x.t1 - x.t0, 0);
                const int units = (two ? 2 : 1) * tiles;   // unit u: stream u & 1, tile two ? u >> 1 : u
                auto keys_landed = [&](int i) {
                    bool all = true;
#pragma unroll
                    for (int part = 0; part < kHalves; ++part) all = all && landed(i + part);
                    return all;
                };
                auto scores = [&](int u) {
                    const int s = u & 1, i = base + kPer * (two ? u >> 1 : u);
                    if (!two) ok = __all_sync(0xffffffffu, ok && keys_landed(i));
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t ad = sdesc_kmajor_sw128(q_at + (two ? s : 0) * kQBytes);
#pragma unroll
                    for (int part = 0; part < kHalves; ++part) {   // kV channels of K
                        const int slot = (i + part) % bufs;
                        const uint64_t bd = sdesc_keys(ring_at + slot * kSlotBytes, kGroupBytes);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < kV / 16; ++k)
                                umma_bf16(tbu + kTmemS + 128 * s,
                                          ad + ((part * kV / 16 + k) >> 2) * (kBlock >> 4) + (k & 3) * 2,
                                          bd + (k >> 2) * (1024 >> 4) + (k & 3) * 2, id_qk, part + k > 0 ? 1u : 0u);
                            if (part == kHalves - 1) umma_commit(&s_full[s]);
                            if (!two || s == 1) umma_commit(&kv_free[slot]);
                        }
                    }
                    __syncwarp();
                };
                ok = __all_sync(0xffffffffu, ok && wait_for(&q_ready, item & 1, abort, limit));
                if (two) ok = __all_sync(0xffffffffu, ok && keys_landed(base));
                scores(0);
                if (units > 1) scores(1);
                for (int u = 0; u < units && ok; ++u) {
                    const int s = u & 1, i = base + kPer * (two ? u >> 1 : u) + kHalves;
                    // O still holds the item before until its rows are out
                    if (u == 0 && item > 0) ok = wait_for(&o_free, (item - 1) & 1, abort, limit);
                    // This tile's V, and with two row tiles the next K before P is there (the
                    // second stream's tiles are the first's); with one row tile memory is the
                    // bound, and waiting for a K would hold up the V before it.
                    if (!two || s == 0) ok = ok && landed(i) && (!two || u + 2 >= units || keys_landed(i + 1));
                    const uint32_t phase = (s ? done1 : done0) & 1;
                    if (s) ++done1; else ++done0;
                    const uint64_t bd = sdesc_mnmajor_sw128(ring_at + (i % bufs) * kSlotBytes, 1024, kGroupBytes);
                    // the two halves of P as they come
                    auto product = [&](int k0, uint64_t* ready) {
                        ok = __all_sync(0xffffffffu, ok && wait_for(ready, phase, abort, limit));
                        if (!ok) return;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < kKeys / 32; ++k)
                                umma_bf16_ta(tbu + kTmemO + 128 * s, tbu + kTmemS + 128 * s + 8 * (k0 + k),
                                             bd + (k0 + k) * (kGroupBytes >> 3), id_pv, (u > 1 || k0 + k > 0) ? 1u : 0u);
                            if (k0 && (!two || s == 1)) umma_commit(&kv_free[i % bufs]);
                        }
                        __syncwarp();
                    };
                    product(0, &p_half[s]);
                    product(kKeys / 32, &p_ready[s]);
                    if (!ok) break;
                    if (u + 2 < units) scores(u + 2);
                }
                if (elect_one()) umma_commit(&o_full);
                __syncwarp();
                base += kPer * tiles;
            }
            if (!ok && lane == 0) fail();
            if (item > 0) wait_for(&o_full, (item - 1) & 1, nullptr, kWaitLimitNs);   // the last products
            __syncwarp();
        } else if (warp == 10) {
            // ------------------------------------------------------------ work
            // where every request begins on the line: at least one tile each, so that
            // rows that see nothing are written too
            int64_t at = 0;
            for (int r0 = 0; r0 < p.count; r0 += 32) {
                const int r = r0 + lane;
                int ctx, n, t = 0;
                if (r < p.count) {
                    if (!tree_lengths(p, p.r0 + r, ctx, n) && p.status) atomicMax(p.status, 1);
                    t = max(1, (ctx + n + kKeys - 1) / kKeys);
                }
                int sum = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                if (r < p.count) s_start[r] = (int)at + sum - t;
                at += __shfl_sync(0xffffffffu, sum, 31);
            }
            if (lane == 0) s_start[p.count] = (int)at;
            __syncwarp();
            if (lane == 0) {
                const int pairs = (p.rows + 255) / 256;
                const bool odd = (p.rows - 1) % 256 < 128;   // the last pair has one row tile
                const int head_cost = pairs * kCostTwo - (odd ? kCostTwo - kCostOne : 0);   // of a key tile
                const int pairs_cost = pairs * Shape::kCostItem;
                // where request r begins on the line
                const auto start = [&](int r) { return ((int64_t)s_start[r] * head_cost + (int64_t)r * pairs_cost) * p.Hk; };
                const int64_t total = start(p.count);
                // at least a key tile a CTA
                const int64_t most = quotient(at * head_cost * p.Hk, kCostTwo);
                const int room = (int)gridDim.x / kHalves, ctas = most < 1 ? 1 : most < room ? (int)most : room;
                int4 slots[2] = {make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
                int k = 0;
                bool ok = true;
                auto deal = [&](const Item& x) {
                    if (k >= kItems) ok = wait_for(&item_free[k % kItems], (k / kItems - 1) & 1, abort, limit);
                    if (!ok) return;
                    s_item[k % kItems] = x;
                    mbar_arrive(&item_full[k % kItems]);
                    ++k;
                };
                Item x{};
                if (cta < ctas) {
                    const int64_t begin = quotient(total * cta, ctas), end = quotient(total * (cta + 1), ctas);
                    // the item that holds the stretch's begin
                    int lo = 0, hi = p.count;
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) >> 1;
                        if (start(mid) <= begin) lo = mid; else hi = mid;
                    }
                    int r = lo, tiles = s_start[r + 1] - s_start[r];
                    int64_t item = start(r), off = begin - item;
                    const int64_t per_head = (int64_t)tiles * head_cost + pairs_cost;
                    const int64_t per_pair = (int64_t)tiles * kCostTwo + Shape::kCostItem;
                    x.h = (int)quotient(off, per_head);
                    off -= x.h * per_head;
                    x.rb = min((int)quotient(off, per_pair), pairs - 1);
                    off -= x.rb * per_pair;
                    item = begin - off;
                    tree_lengths(p, p.r0 + r, x.ctx, x.n);
                    while (item < end && ok) {
                        x.two = !(odd && x.rb == pairs - 1);
                        const int cost = x.two ? kCostTwo : kCostOne;
                        const int64_t first = item + Shape::kCostItem, next = first + (int64_t)tiles * cost;
                        x.r = p.r0 + r;
                        x.t0 = first < begin ? (int)quotient(begin - first + cost - 1, cost) : 0;
                        x.t1 = next <= end ? tiles : first < end ? (int)quotient(end - first + cost - 1, cost) : 0;
                        x.whole = x.t0 == 0 && x.t1 == tiles;
                        if (x.t1 > x.t0) {
                            if (!x.whole) slots[x.t0 > 0 ? 0 : 1] = make_int4(x.t1 == tiles ? 2 : 1, x.r, x.h, x.rb);
                            deal(x);
                        }
                        item = next;
                        if (++x.rb == pairs) {
                            x.rb = 0;
                            if (++x.h == p.Hk) {
                                x.h = 0;
                                if (++r == p.count) break;
                                tiles = s_start[r + 1] - s_start[r];
                                tree_lengths(p, p.r0 + r, x.ctx, x.n);
                            }
                        }
                    }
                }
                x.t1 = -1;
                deal(x);
                // what the two slots hold: 0 nothing, 1 a part of item (r, h, rb), 2 its last
                if (half == 0) {
                    p.parts[2 * cta] = slots[0];
                    p.parts[2 * cta + 1] = slots[1];
                }
                if (!ok) fail();
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ cleaning
            // V tiles with drafted tokens or positions past the end, between their copy
            // and the products, so that the loader can go on.
            int base_kv = 0, item = 0;      // ring tiles before this item, items begun
            uint32_t phases = 0;            // of the slots' raw barriers
            bool ok = true;
            Item x;
            for (; __all_sync(0xffffffffu, take(item, x, ok)) && ok; ++item) {
                if (lane == 0) mbar_arrive(&item_free[item % kItems]);
                const int ctx = x.ctx, hi = ctx + x.n;
                for (int tile = max(x.t0, ctx / kKeys); tile < x.t1 && ok; ++tile) {
                    const int i = base_kv + kPer * (tile - x.t0) + kHalves, slot = i % bufs, base = tile * kKeys;
                    uint8_t* const dst = ring + slot * kSlotBytes;
                    ok = __all_sync(0xffffffffu, wait_for(&kv_raw[slot], (phases >> slot) & 1, abort, limit));
                    if (!ok) break;
                    phases ^= 1u << slot;
                    constexpr uint32_t kExp = Elem<T>::kExpMask;
                    constexpr int kPieces = kV / 8;
                    auto piece = [&](int e) -> uint4* {   // 16-byte piece e of the tile, rows in order
                        const int c = e % kPieces, krow = e / kPieces;
                        return reinterpret_cast<uint4*>(dst + (krow >> 3) * kGroupBytes + (c >> 3) * 1024 +
                                                        (krow & 7) * 128 + (c & 7) * 16);
                    };
                    const int drafted = max(0, ctx - base), past = max(0, min(hi - base, kKeys));
                    for (int e = past * kPieces + lane; e < kKeys * kPieces; e += 32) *piece(e) = make_uint4(0, 0, 0, 0);
#pragma unroll 4
                    for (int e = drafted * kPieces + lane; e < past * kPieces; e += 32) {
                        const uint4 y = *piece(e);
                        uint32_t w[4] = {y.x, y.y, y.z, y.w};
                        bool bad = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((w[k] & kExp) == kExp) { bad = true; w[k] &= 0xffff0000u; }
                            if (((w[k] >> 16) & kExp) == kExp) { bad = true; w[k] &= 0xffffu; }
                        }
                        if (bad) {
                            const int j = base + e / kPieces - ctx;
                            atomicOr(&s_bad[item & 7][j >> 5], 1u << (j & 31));
                            *piece(e) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&kv_full[slot]);
                }
                base_kv += kPer * (x.t1 - x.t0);
            }
            if (!__all_sync(0xffffffffu, ok) && lane == 0) fail();
        }
    } else {
        // ---------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int stream = warp >> 2, row_in = tid & 127;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tb + lane_base + kTmemS + 128 * stream, to = tb + lane_base + kTmemO + 128 * stream;
        const float c = p.scale_log2, lazy = kLazy<T> / c;   // in units of the scores
        bool ok = true;
        int item = 0, seen_s = 0;   // items begun, score tiles taken
        for (;; ++item) {
            ok = __all_sync(0xffffffffu, wait_for(&item_full[item % kItems], (item / kItems) & 1, abort, limit));
            if (!ok && lane == 0) fail();
            const Item& x = s_item[item % kItems];
            if (named_bar_or(1, 256, !ok || x.t1 < 0)) break;   // all stop if one has given up
            const bool two = x.two;
            const int row0 = x.rb * 256, r = x.r, kvh = x.h;
            {
                // the query rows as K-major operands in the 128-byte swizzle, D / 8 lanes a
                // row; all of them are on their way at once
                constexpr int kPieces = D / 8, kRowsPass = 256 / kPieces, kPasses = 256 / kRowsPass;
                const int piece = tid % kPieces, in0 = tid / kPieces;
                // node and head of the thread's rows, kRowsPass rows on each time
                const int di = (int)page_div(kRowsPass, p.G, p.group_magic), dg = kRowsPass - di * p.G;
                const int64_t step = di * p.qs[1] + dg * p.qs[2], wrap = p.qs[1] - p.G * p.qs[2];
                const int i0 = (int)page_div((uint32_t)(row0 + in0), p.G, p.group_magic);
                int left = p.rows - row0 - in0, g = row0 + in0 - i0 * p.G;
                const T* src = static_cast<const T*>(p.q) + r * p.qs[0] + i0 * p.qs[1] + (kvh * p.G + g) * p.qs[2] +
                               piece * 8;
                uint8_t* const dst = sm + (piece >> 3) * kBlock;
#pragma unroll
                for (int k = 0; k < kPasses; ++k) {
                    const int in = k * kRowsPass + in0;   // row of the pair of tiles
                    if (k < kPasses / 2 || two) {
                        uint8_t* at = dst + (k * kRowsPass >> 7) * kQBytes + sw128_off(in & 127, (piece & 7) * 8);
                        if (left > 0) cp_async16(at, src);
                        else *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
                    }
                    left -= kRowsPass;
                    g += dg;
                    src += step;
                    if (g >= p.G) {
                        g -= p.G;
                        src += wrap;
                    }
                }
                cp_async_commit();
            }
            const int ctx = x.ctx, hi = ctx + x.n;
            const int row = row0 + (two ? stream * 128 : 0) + row_in;
            const int node = min((int)page_div((uint32_t)row, p.G, p.group_magic), p.N - 1);
            const bool live = row - lane < p.rows;   // some row of the warp is a row of the call
            cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready);

            // visibility of positions tok .. tok + 31 to this row
            const uint32_t* mask = tree_mask_row(p, r, node);
            auto seen = [&](int tok) -> uint32_t { return tree_seen(p, mask, node, ctx, hi, tok); };

            const int tile0 = x.t0, ctx_in = x.ctx;
            float m = -INFINITY, l = 0.f;
            const int units = (two ? 2 : 1) * (x.t1 - x.t0);
            if (p.timeout_probe && item == 0) ok = __all_sync(0xffffffffu, wait_for(&never, 0, abort, limit));
            for (int u = stream; u < units && ok; u += 2) {
                ok = __all_sync(0xffffffffu, wait_for(&s_full[stream], seen_s & 1, abort, limit));
                if (!ok) break;
                ++seen_s;
                tc_fence_after();
                if (live) {
                    uint32_t raw[8][16];
                    float v[128];
#pragma unroll
                    for (int k = 0; k < 8; ++k) tmem_ld16_issue(ts + 16 * k, raw[k]);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k) tmem_take16(raw[k], &v[16 * k]);
                    const int base = (tile0 + (two ? u >> 1 : u)) * kKeys;
                    if (base + kKeys > ctx_in) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t b = seen(base + 32 * k);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((b >> e) & 1u)) v[32 * k + e] = -INFINITY;
                        }
                    }
                    float mx[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e] = v[e];
#pragma unroll
                    for (int e = 8; e < 128; ++e) mx[e & 7] = fmaxf(mx[e & 7], v[e]);
                    const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                            fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                    float alpha = 1.f;
                    if (top > m + lazy || m == -INFINITY) {
                        const float mn = fmaxf(m, kShift<T> == 0.f ? top : fmaf(lazy, -kShift<T> / kLazy<T>, top));
                        if (m != -INFINITY) alpha = ex2_approx((m - mn) * c);
                        m = mn;
                        l *= alpha;
                    }
                    if (u > 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                        for (int k = 0; k < kV / 32; ++k) {
                            float o[32];
                            uint32_t w[32];
                            tmem_ld32(to + 32 * k, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * alpha);
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
                            const float2 y = f2_parts(f2_fma(f2(v[32 * k + 2 * e], v[32 * k + 2 * e + 1]), c2, m2));
                            const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
                            sum[e & 1] = f2_add(sum[e & 1], f2(p0, p1));
                            w[e] = Elem<T>::pack(p0, p1);
                        }
                        tmem_st16_issue(ts + 16 * k, w);
                        if (k == 1) {   // half of P: its product may start
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&p_half[stream]);
                        }
                    }
                    const float2 q = f2_parts(f2_add(sum[0], sum[1]));
                    l += q.x + q.y;
                    tmem_wait_st();
                } else if (lane == 0) {
                    mbar_arrive(&p_half[stream]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[stream]);
            }
            ok = __all_sync(0xffffffffu, wait_for(&o_full, item & 1, abort, limit)) && ok;
            if (!ok && lane == 0) fail();
            tc_fence_after();

            // The rows' way out.  The products are done, so the queries' memory is free:
            // a patch a warp (32 rows at a pitch of 36 floats) through which the stores
            // to memory become whole sectors, and behind the patches 32 columns of
            // stream 1's rows on their way to stream 0 when the two are joined.
            float* const patch = reinterpret_cast<float*>(sm) + warp * kPatch;
            float* const other = reinterpret_cast<float*>(sm) + 8 * kPatch;   // [32][128], then m and l
            float f0 = 1.f, f1 = 0.f;
            const bool joined = !two && units > 1;
            if (joined) {
                if (stream == 1) {
                    other[32 * 128 + row_in] = m;
                    other[33 * 128 + row_in] = l;
                }
                named_bar_sync(1, 256);
                if (stream == 0) {
                    const float m1 = other[32 * 128 + row_in], mj = fmaxf(m, m1), mu = mj == -INFINITY ? 0.f : mj;
                    f0 = ex2_approx((m - mu) * c);
                    f1 = ex2_approx((m1 - mu) * c);
                    l = l * f0 + other[33 * 128 + row_in] * f1;
                    m = mj;
                }
            }
            const bool empty = node >= x.n || l == 0.f, whole = x.whole;
            const float inv = empty ? 0.f : 1.f / l;
            f0 *= inv;
            f1 *= inv;
            const int64_t part = ((int64_t)(2 * cta + (x.t0 > 0 ? 0 : 1)) * 256 + (row - row0));
            const bool out = ok && live && (two || stream == 0);
            uint32_t any_bad = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) any_bad |= s_bad[item & 7][w];
            // Where this lane stores: whole rows 4 lanes a row (8 elements each), partial ones
            // 8 lanes a row (4 floats each).
            T* dst[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int q = row - lane + 8 * g + (lane >> 2), qi = (int)page_div((uint32_t)q, p.G, p.group_magic);
                dst[g] = q < p.rows ? static_cast<T*>(p.out) + r * p.os[0] + qi * p.os[1] +
                                          (kvh * p.G + q - qi * p.G) * p.os[2] + half * kV + (lane & 3) * 8
                                    : nullptr;
            }
            float* const pdst = p.part_o + (part - lane + (lane >> 3)) * D + half * kV + (lane & 7) * 4;
            // rolled: the code runs once an item, and fetching it costs more than running it
#pragma unroll 1
            for (int k = 0; k < kV / 32; ++k) {
                float o[32];
                if (live && ok && (out || joined)) tmem_ld32(to + 32 * k, o);
                if (joined) {
                    if (stream == 1) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) other[e * 128 + row_in] = o[e];
                    }
                    named_bar_sync(1, 256);
                }
                if (out) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = empty ? 0.f : o[e] * f0;
                    if (joined && !empty) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = fmaf(other[e * 128 + row_in], f1, o[e]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(patch + lane * 36 + 4 * e) =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    if (any_bad && !empty) {
                        for (int j = max(0, x.t0 * kKeys - ctx); j < min(hi, x.t1 * kKeys) - ctx; ++j) {
                            if (!((s_bad[item & 7][j >> 5] >> (j & 31)) & 1u) || !(seen(ctx + j) & 1u)) continue;
                            const int tok = ctx + j, id = p.table[r * p.table_stride + tok / p.page];
                            if (id < 0 || id >= p.P) continue;
                            const T* src = static_cast<const T*>(p.vc) + id * p.vs[0] + (tok % p.page) * p.vs[1] +
                                           kvh * p.vs[2] + half * kV + 32 * k;
#pragma unroll 1
                            for (int e = 0; e < 32; ++e) {
                                const float y = Elem<T>::one(src[e]);
                                if (!isfinite(y)) patch[lane * 36 + e] += y;
                            }
                        }
                    }
                    __syncwarp();
                    if (whole) {
                        const float* src = patch + (lane >> 2) * 36 + (lane & 3) * 8;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const float4 y0 = *reinterpret_cast<const float4*>(src + 8 * g * 36),
                                         y1 = *reinterpret_cast<const float4*>(src + 8 * g * 36 + 4);
                            if (dst[g])
                                *reinterpret_cast<uint4*>(dst[g] + 32 * k) =
                                    make_uint4(Elem<T>::pack(y0.x, y0.y), Elem<T>::pack(y0.z, y0.w),
                                               Elem<T>::pack(y1.x, y1.y), Elem<T>::pack(y1.z, y1.w));
                        }
                    } else {
                        const float* src = patch + (lane >> 3) * 36 + (lane & 7) * 4;
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            if (row - lane + 4 * g + (lane >> 3) < p.rows)
                                *reinterpret_cast<float4*>(pdst + 4 * g * D + 32 * k) =
                                    *reinterpret_cast<const float4*>(src + 4 * g * 36);
                    }
                }
                if (joined) named_bar_sync(1, 256);   // stream 1's columns are taken
            }
            if (out && row < p.rows && half == 0) {
                const float lse = empty ? -INFINITY : m * c + log2f(l);
                if (!whole) p.part_lse[part] = lse;
                else if (p.lse)
                    p.lse[((int64_t)r * p.N + node) * p.Hq + kvh * p.G + (row - node * p.G)] = lse * 0.6931471805599453f;
            }
            tc_fence_before();
            named_bar_sync(1, 256);   // every warp's patch and s_bad have been read
            if (tid < 8) s_bad[item & 7][tid] = 0;
            if (tid == 0) mbar_arrive(&item_free[item % kItems]);
            if (lane == 0) mbar_arrive(&o_free);
        }
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
}

template <typename T, int D>
cudaError_t launch_mma_t(const TreeParams& q, const CUtensorMap& kmap, const CUtensorMap& vmap, int grid, cudaStream_t s) {
    using Shape = MmaShape<D>;
    static std::atomic<uint64_t> smem_set;
    constexpr uint32_t most = Shape::smem(1) > Shape::smem(256) ? Shape::smem(1) : Shape::smem(256);
    cudaError_t e = set_smem_limit_once((const void*)tree_mma_kernel<T, D>, (int)most, smem_set);
    grid -= grid % Shape::kHalves;
    for (int r0 = 0; r0 < q.R && e == cudaSuccess; r0 += kTreeSlice) {
        TreeParams p = q;
        p.r0 = r0;
        p.slots = 2 * (grid / Shape::kHalves);
        p.slot_rows = 256;
        p.count = q.R - r0 < kTreeSlice ? q.R - r0 : kTreeSlice;
        tree_mma_kernel<T, D><<<grid, kMmaThreads, Shape::smem(p.rows), s>>>(p, kmap, vmap);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = launch_tree_join(p, D, std::is_same<T, __half>::value, s);
    }
    return e;
}

template <typename T>
cudaError_t launch_mma(const TreeParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int D, int grid,
                       cudaStream_t s) {
    return D == 64 ? launch_mma_t<T, 64>(p, kmap, vmap, grid, s)
                   : D == 128 ? launch_mma_t<T, 128>(p, kmap, vmap, grid, s) : launch_mma_t<T, 256>(p, kmap, vmap, grid, s);
}

}  // namespace

bool launch_tree_mma(const TreeParams& q, int D, bool f16, int grid, cudaStream_t s, cudaError_t* e) {
    CUtensorMap kmap, vmap;
    TreeParams p = q;
    p.wait_ns += (uint64_t)((p.max_len + kKeys - 1) / kKeys) * kTileWaitNs;
    if (!cache_map(&kmap, p.kc, p.ks, p.Hk, p.P, p.page, D, f16, &p.k_paged) || !cache_map(&vmap, p.vc, p.vs, p.Hk, p.P, p.page, D, f16, &p.v_paged))
        return false;
    if (f16) *e = launch_mma<__half>(p, kmap, vmap, D, grid, s);
    else *e = launch_mma<__nv_bfloat16>(p, kmap, vmap, D, grid, s);
    return true;
}

}  // namespace kda
