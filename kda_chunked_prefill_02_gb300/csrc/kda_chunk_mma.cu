// kda_chunk_mma.cu -- kda_chunk_attention (include/kda_ops.h) on tcgen05 tensor cores:
// tiles of 128 query rows (the new tokens times the query heads of a key head) and 128
// keys, S and O in TMEM, queries and the pages of K and V by TMA.
//
// A tile of rows and keys costs 16 tcgen05.mma (S = Q K^T, then O += P V).  Persistent
// CTAs, one an SM:
//   warps 0-3, 4-7  two softmax streams: thread = row (TMEM lane), the whole row of S in
//                   registers, so maximum and sum need no exchange; P goes back over S's
//                   columns as 16-bit pairs, the A operand of the second product;
//   warps 8-11      the rows' way out: O from TMEM, divided by the sum, to memory;
//   warp 12         deals out the work, item by item, and loads it: query tiles and a ring
//                   of K and V tiles;
//   warps 13, 14    issue the products, a stream each (one warp for both was what bound the
//                   kernel: some 2300 cycles a unit of waits, commits and 16 products that
//                   take 1024);
//   warp 15         cleans the V tiles that need it.
// An item is a pair of row tiles over the same keys, one a stream, each K and V tile read
// for 256 rows; or a last single row tile, whose even and odd key tiles go to the two
// streams and whose two halves are joined on the way out.  The streams run without a break
// from item to item: while an item's last rows are on their way out, the next
// one's first scores are formed and its softmax runs (its queries come into a buffer of
// their own); what is left of an item's change is some 4 us.
//
// A row tile holds whole tokens (128 / G of them, G query heads a key head), so that its
// queries are one box of the query tensor a block of 64 channels.
//
// The work of a call is one line, ordered by request, key head and pair of row tiles, an
// item's length on it the keys that its last token sees and a constant for its way in and
// out; every CTA takes an equal stretch, so that ragged batches and the causal triangle
// leave no SM idle.  Where row tiles share more keys than L2 keeps, the CTAs walk the line in
// waves, all on one part of it and then on the next (2048 tokens over 126976: 2970 us without,
// 2610 with four waves, 2570 with eight).  A stretch cuts at most two items; the parts of a
// cut item leave normalised rows and their log-sum in the workspace (slot 0 of a CTA: a later
// part of an item, slot 1: the first), joined in the CTAs' order by chunk_join_kernel
// (kda_chunk.cu).
//
// Head size 256: S of two row tiles and a whole O do not fit TMEM, so two neighbouring
// CTAs take the same stretch, both with all of S and each with one half of V's columns.
//
// The running maximum moves only when a row's scores exceed it by a factor of 2^8 (2^4 in
// fp16), so that O in TMEM is hardly ever rescaled; that is the softmax threads' work, in
// the time between a score tile's arrival (which implies that the product before it is
// done) and their P's.
//
// Keys behind a row's own: only an item's last tiles hold any; there every row compares
// its 128 positions.  In those tiles a warp of its own clears V rows that no row of the
// item sees and V elements that are not finite before the product sees them (0 * NaN is
// NaN, also for a row whose P is zero), and remembers their positions; the rows that do
// see such a position take its elements on their way out.
//
// Measured (us of GPU time, 32 / 8 heads of 128, bf16; rates of the products that rows see):
// a prompt of 8192 tokens 341 (1.61 PFLOP/s, the tensor pipe 75 % busy), of 32768 5000 (1.75),
// 2048 tokens over 126976 2600 (1.65), 32 prompts of 512 118 (0.58), 64 single tokens over 4096
// 175 (6.1 TB/s of K and V).  What bounds it: with many tiles an item the products and the
// exponentials together (head size 64: neither, 8192 tokens 279 with the tensor pipe 44 % and the
// exponentials' 45 % busy, but a stream's chain of one score tile after the other), with few an
// item's change, most of which is fetching the roles' code (77 KB) into the instruction cache.
//
// Registers: 512 threads start with 128 each; the softmax warps take 168, the way out
// keeps 80, the last four warps 96 (2 x 168 + 80 + 96 = 4 x 128).
//
// Every wait is bounded; one that runs out sets the abort flag, the roles fall through to
// the end, and the status word reports KDA_ERR_TIMEOUT.  Whatever the others do, the loader
// and the issuer end by waiting for their last copies and products (with the full
// kWaitLimitNs), so that none is in flight when the CTA's memory goes to the next.
#include "attn_mma.cuh"
#include "kda_internal.h"
#include "ops_internal.h"
#include "sm103.cuh"

namespace kda {
namespace {

constexpr int kThreads = 512;
constexpr uint32_t kTmemS = 0, kTmemO = 256;   // S of stream s at 128 s, O at 256 + 128 s
constexpr int kMaxSlots = 8, kMaxQ = 3;
constexpr int kItems = 4;         // items dealt out ahead
constexpr int kBadWords = 12;     // positions of an item's last tiles (three at most), a bit each
// What a wait may take beside its bound, a key tile of the longest context (see kda_tree_mma.cu).
constexpr uint64_t kTileWaitNs = 20000 * (kItems + 1);

// One CTA's part of an item.
struct Item {
    int r, h, token0, tokens;   // request, key head, the pair's first token and its tokens
    int t0, t1;                 // key tiles (t1 < 0: no more items)
    int ctx, first;             // the request's context, and its first row of q (packed: in all)
    int end;                    // keys that the last token sees (0: a request that does not fit the call)
    int part;                   // where its partial rows go (not whole)
    uint8_t two, whole;         // two row tiles; all of the key tiles
};

// A CTA's memory behind the queries and the ring.
struct Misc {
    uint64_t kv_full[kMaxSlots], kv_free[kMaxSlots], kv_raw[kMaxSlots];
    uint64_t q_full[kItems][2], q_free[kMaxQ];   // full: an item's row tiles
    uint64_t s_full[2], p_full[2][2], o_full[2], o_free[2], ml_full[2], ml_free[2];
    uint64_t item_full[kItems], item_free[kItems], drained[2], never;   // never: the probe's, nothing arrives on it
    float2 ml[2][128];          // the rows' maximum and sum, a stream each
    alignas(16) uint32_t bad[kItems][kBadWords];   // positions with a V element that is not finite
    Item item[kItems];
    uint32_t tmem;
    int abort;
};

template <int D> struct Shape {
    static constexpr int kV = D == 256 ? 128 : D;   // value columns a CTA
    static constexpr int kHalves = D / kV;          // CTAs that share a stretch, each with its columns
    static constexpr int kPer = kHalves + 1;        // ring slots a key tile: K by kV channels, V
    static constexpr uint32_t kSlotBytes = (kV / 64) * kBlock, kQBytes = (D / 64) * kBlock;
    static constexpr uint32_t kGroupBytes = (kV / 64) * 1024;   // 8 keys, 64 channels after the other
    // query tiles: three where memory allows it, so that an item's first comes in while the
    // two of the item before are still needed
    static constexpr int kQ = D == 256 ? 2 : 3;
    static constexpr int kSlots = D == 64 ? 8 : D == 128 ? 4 : 3;
    static constexpr uint32_t kMiscAt = kQ * kQBytes + kSlots * kSlotBytes;
    static constexpr uint32_t kBytes = kMiscAt + sizeof(Misc);
};
static_assert(Shape<128>::kBytes <= 232448 && Shape<256>::kBytes <= 232448, "a CTA's shared memory");

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Whether N pieces of 8 elements are finite: the sum of their products with 0 is 0 or NaN.
template <typename T, int N>
__device__ __forceinline__ bool all_finite(const uint4 (&y)[N]) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    uint32_t sum = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t w[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t zero = 0;
            const T2 r = __hfma2(*reinterpret_cast<const T2*>(&w[i]), *reinterpret_cast<const T2*>(&zero),
                                 *reinterpret_cast<const T2*>(&sum));
            sum = *reinterpret_cast<const uint32_t*>(&r);
        }
    }
    return (sum & 0x7fff7fffu) == 0;
}

// The waits are loops of few instructions: the roles' code does not fit the instruction cache
// together, and an item's change takes as long as fetching it (unrolled by the compiler, the
// same waits cost 32 prompts of 512 tokens 133 us instead of 119).
//
// The rows' way out waits by the clock, up to 20 us a try: its polls take issue slots from the
// softmax (head size 64: 8192 tokens 302 us without that, 286 with it).
__device__ __forceinline__ bool wait_out(uint64_t* bar, uint32_t parity, const volatile int* abort, uint64_t limit_ns) {
    uint64_t t0 = 0;
#pragma unroll 1
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
            : "memory");
        if (done) return true;
        if (*abort) return false;
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        else if (t - t0 > limit_ns) return false;
    }
}
// The other roles' wait has no clock.  What holds a role up holds up the rows' way out too,
// whose waits run out and set the abort flag; the number of tries ends this one in any case.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, const volatile int* abort) {
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort || i >> 31) return false;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_mma_kernel(const ChunkParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<D>;
    constexpr uint32_t kSlotBytes = S::kSlotBytes, kQBytes = S::kQBytes, kGroupBytes = S::kGroupBytes;
    constexpr int kV = S::kV, kHalves = S::kHalves, kPer = S::kPer, kSlots = S::kSlots, kQ = S::kQ;
    const int cta = (int)blockIdx.x / kHalves, half = (int)blockIdx.x % kHalves;
    extern __shared__ __align__(1024) uint8_t sm[];   // at the window's begin: there is no static shared memory
    uint8_t* const ring = sm + kQ * kQBytes;
    Misc& m = *reinterpret_cast<Misc*>(sm + S::kMiscAt);

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    volatile int* abort = &m.abort;
    const uint64_t limit = p.wait_ns;
    const int tt = p.tile_tokens, G = p.G;      // tokens a row tile, query heads a key head
    auto fail = [&]() {
        *abort = 1;
        if (p.status) atomicExch(p.status, 4);
    };
    if (smem_u32(sm) & 1023u) {   // the swizzled tiles' alignment (never seen: all threads leave)
        if (p.status && tid == 0) atomicExch(p.status, 4);
        if (half == 0 && tid < 2 * p.waves)   // no parts for the join
            p.parts[2 * (cta + (tid >> 1) * ((int)gridDim.x / kHalves)) + (tid & 1)] = make_int4(0, 0, 0, 0);
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&m.kv_full[i], 1);
            mbar_init(&m.kv_free[i], 2);    // both streams' products
            mbar_init(&m.kv_raw[i], 1);
        }
        for (int i = 0; i < kMaxQ; ++i) mbar_init(&m.q_free[i], 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.s_full[s], 1);
            mbar_init(&m.p_full[s][0], 4);     // the halves of P: one arrival a warp
            mbar_init(&m.p_full[s][1], 4);
            mbar_init(&m.o_full[s], 1);
            mbar_init(&m.o_free[s], 4);
            mbar_init(&m.ml_full[s], 4);
            mbar_init(&m.ml_free[s], 4);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&m.item_full[i], 1);
            mbar_init(&m.q_full[i][0], 1);
            mbar_init(&m.q_full[i][1], 1);
            mbar_init(&m.item_free[i], 15);   // 8 softmax warps, 4 of the way out, 2 issuers, the cleaner
        }
        for (int s = 0; s < 2; ++s) mbar_init(&m.drained[s], 1);
        mbar_init(&m.never, 1);
        m.abort = 0;
        fence_mbar_init();
    }
    if (warp == 13) {
        tmem_alloc(&m.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // chunk_join_kernel waits for this grid's end itself
    const uint32_t tb = m.tmem;
    // The k-th item of this CTA; false after the last (or on an abort).
    auto take = [&](int k, Item& x, bool& ok) -> bool {
        ok = ok && wait_on(&m.item_full[k % kItems], (k / kItems) & 1, abort);
        if (!ok) return false;
        x = m.item[k % kItems];
        return x.t1 >= 0;
    };
    auto release = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.item_free[k % kItems]);
    };
    // Keys that the last row of stream s sees, and how many of the item's key tiles are its
    // units (one at least, so that rows without keys are written too).
    auto stream_end = [&](const Item& x, int s) -> int { return x.two && s == 0 ? min(x.end, x.ctx + x.token0 + tt) : x.end; };
    auto stream_units = [&](const Item& x, int s) -> int {
        if (!x.two) return (x.t1 - x.t0 + 1 - s) / 2;   // every other tile
        return max(1, min(x.t1, (stream_end(x, s) + kKeys - 1) / kKeys) - x.t0);
    };
    // Keys from which on some row of an item does not see V: the tiles that are cleaned.
    auto clean_from = [&](const Item& x) -> int { return min(x.end, x.ctx + x.token0 + 1) / kKeys; };

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == 12) {
            // ------------------------------------------------------------ work and loader
            if (lane == 0) {
                tma_prefetch_desc(&qmap);
                tma_prefetch_desc(&kmap);
                tma_prefetch_desc(&vmap);
            }
            // A request's length on the line: over its pairs of row tiles, the keys of each one's
            // last token (a last single row tile four fifths of them: 60 single tokens over 4096 and
            // four pieces 225 us, 252 with all of them) and kItemKeys, times the key heads.
            const int pt = 2 * tt;          // tokens a pair
            // where pair `rb` begins on a head's part of the line
            auto pair_at = [&](int ctx, int rb) -> int64_t {
                return (int64_t)rb * (uint32_t)(kItemKeys + ctx + tt * (rb + 1));   // (32 bits: contexts and tokens have 30)
            };
            // four fifths of a single row tile's keys
            auto single = [](int keys) -> int { return keys - (int)(((uint32_t)keys + 4u) / 5u) + 1; };
            const int room = (int)gridDim.x / kHalves;
            const int box = box_of(p.page), per_tile = kKeys / box;   // this lane's box: tokens lane * box ..
            int item = 0, issued = 0, queries = 0;   // items dealt, K and V tiles and query tiles asked for
            uint32_t raw = 0, raw_phases = ~0u;      // slots whose last copy was a raw one, those copies' phases
            int q_asked = 0, q_phase = 0;            // q_full barriers with a copy, those copies' phases
            bool ok = true;
            Item x{};
            // The item to the other warps.
            auto deal = [&]() {
                const int at = item % kItems;
                if (item >= kItems) ok = __all_sync(0xffffffffu, wait_on(&m.item_free[at], (item / kItems - 1) & 1, abort));
                if (!ok) return;
                if (lane == 0) {
                    m.item[at] = x;
                    mbar_arrive(&m.item_full[at]);
                }
                __syncwarp();
                ++item;
            };
            // Its queries and its tiles.
            auto load = [&]() {
                if (!ok) return;
                const int32_t* table = p.table + x.r * p.table_stride;
                const int special = clean_from(x);
                // this lane's page of a tile, -1: none (asked for a tile ahead, looked at
                // later), and its first row there
                int row_ahead = 0;
                auto page_of = [&](int tile) -> int64_t {
                    const int tok = tile * kKeys + lane * box;
                    const int at = (int)page_div((uint32_t)tok, p.page, p.page_magic);
                    row_ahead = tok - at * p.page;
                    return tile < x.t1 && lane < per_tile && tok < x.end ? (int64_t)(uint32_t)table[at] : -1;
                };
                // row tile a of the item: a box of whole tokens a block of 64 channels (rows past
                // the request's end, or the call's, are some other rows or zeros, and not stored)
                auto load_queries = [&](int a) {
                    const int b = queries % kQ, round = queries / kQ;
                    if (round > 0) ok = __all_sync(0xffffffffu, ok && wait_on(&m.q_free[b], (round - 1) & 1, abort));
                    if (!ok) return;
                    const int at = (item - 1) % kItems, bit = 1 << (2 * at + a);   // the item is dealt already
                    uint64_t* bar = &m.q_full[at][a];
                    q_asked |= bit;
                    q_phase = ((item - 1) / kItems) & 1 ? q_phase | bit : q_phase & ~bit;
                    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(G * tt) * 128u * (D / 64));
                    __syncwarp();
                    if (lane < D / 64)
                        tma_load_5d(sm + b * kQBytes + lane * kBlock, &qmap, 0, x.h * G, (p.cu ? x.first : 0) + x.token0 + a * tt, lane,
                                    p.cu ? 0 : x.r, bar);
                    ++queries;
                };
                int64_t ahead = page_of(x.t0);
                if (!x.two) {   // no second row tile: its phase all the same (a copy four items before is over)
                    q_asked &= ~(2 << (2 * ((item - 1) % kItems)));
                    if (lane == 0) mbar_arrive(&m.q_full[(item - 1) % kItems][1]);
                }
#pragma unroll 1
                for (int tile = x.t0; tile < x.t1 && ok; ++tile) {
                    const int id = ahead < 0 ? -1 : (int)min(ahead, (int64_t)p.P);
                    if (ahead >= p.P && p.status) atomicMax(p.status, 1);   // reads zeros: past the map's pages
                    const int row = row_ahead;
                    ahead = page_of(tile + 1);
                    const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, id >= 0)) * box * kV * 2u;
#pragma unroll 1
                    for (int part = 0; part < kPer; ++part) {   // K by kV channels, then V
                        const bool v = part == kHalves;
                        if (tile == x.t0 && (part == 0 || (v && x.two))) load_queries(v);   // a row tile's queries before each
                        const int slot = issued % kSlots, round = issued / kSlots;
                        if (round > 0) ok = __all_sync(0xffffffffu, ok && wait_on(&m.kv_free[slot], (round - 1) & 1, abort));
                        if (!ok) break;
                        uint8_t* dst = ring + slot * kSlotBytes;
                        const bool to_clean = v && tile >= special;
                        uint64_t* bar = to_clean ? &m.kv_raw[slot] : &m.kv_full[slot];   // raw: to warp 15 first
                        raw = to_clean ? raw | 1u << slot : raw & ~(1u << slot);
                        if (to_clean) raw_phases ^= 1u << slot;
                        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                        __syncwarp();
                        if (id >= 0)
                            tma_load_5d(dst + lane * box * kV * 2, v ? &vmap : &kmap, 0, 0,
                                        ((v ? p.v_paged : p.k_paged) ? 0 : x.h * (D / 64)) + (v ? half : part) * (kV / 64),
                                        row / 8, (v ? p.v_paged : p.k_paged) ? id * p.Hk + x.h : id, bar);
                        ++issued;
                    }
                }
            };
            // Of a request (its lengths at q): true if they fit the call; its first token, new tokens,
            // context, pairs of row tiles and length on a key head's line.
            auto request = [&](int r, const ChunkLengths& q, int& first, int& n, int& ctx, int& pairs, int64_t& head) -> bool {
                int len;
                const bool fits = chunk_request(p, r, q, first, n, len);
                ctx = fits ? len - n : 0;
                pairs = 0;
                head = 0;
                if (n > 0) {
                    pairs = (n - 1) / pt + 1;
                    const int all = ctx + n;
                    head = pair_at(ctx, pairs - 1) + kItemKeys + (n - (pairs - 1) * pt <= tt ? single(all) : all);
                }
                return fits;
            };
            // The line's length.  Until the first tile is loaded the ring keeps the length of every 32
            // requests, so that this CTA begins with its own.  Lengths are asked for four rounds ahead.
            int64_t* const groups = reinterpret_cast<int64_t*>(ring);
            int64_t total = 0, each = 0, rest = 0, tokens = 0, keys = 0, walked = 0;   // walked: the keys of all row tiles
            const auto lengths = [&](int r) { return chunk_lengths(p, min(r, p.R - 1)); };
            ChunkLengths q0 = lengths(lane), q1 = lengths(lane + 32), q2 = lengths(lane + 64), q3 = lengths(lane + 96);
#pragma unroll 1
            for (int r0 = 0; r0 < p.R; r0 += 32) {
                const ChunkLengths q = q0;
                q0 = q1;
                q1 = q2;
                q2 = q3;
                q3 = lengths(r0 + 128 + lane);
                int first, n = 0, ctx, pairs;
                int64_t head = 0;
                if (r0 + lane < p.R) {
                    const bool fits = request(r0 + lane, q, first, n, ctx, pairs, head);
                    if (!fits && p.status && blockIdx.x == 0) atomicMax(p.status, 1);
                    if (n > 0) {
                        tokens += n;
                        keys += ctx + n;
                        walked += head - (int64_t)pairs * kItemKeys;
                    }
                }
                head *= p.Hk;
#pragma unroll 1
                for (int o = 16; o > 0; o >>= 1) head += __shfl_xor_sync(0xffffffffu, head, o);
                total += head;
                if (lane == 0) groups[r0 / 32] = head;
            }
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) {
                keys += __shfl_xor_sync(0xffffffffu, keys, o);
                walked += __shfl_xor_sync(0xffffffffu, walked, o);
                tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
            }
            __syncwarp();
            if (p.cu && tokens > p.T) total = 0;   // a cu_seqlens that goes back again and again: any amount of work
            // Equal stretches, of at least two key tiles.  Where the row tiles of a key head share
            // keys that do not stay in L2 (kWaveBytes of K and V), the line is walked in waves: all
            // CTAs on one part of it, then on the next, of at least 64 key tiles a CTA.
            const int64_t most = total / (2 * kKeys);
            const int ctas = most < 1 ? 1 : most < room ? (int)most : room;
            int waves = 1;
#pragma unroll 1
            while (waves < p.waves && walked > 4 * keys && keys * p.Hk * (4 * D) > waves * kWaveBytes &&
                   total >= (waves + 1) * ctas * (int64_t)(64 * kKeys))
                ++waves;
            rest = total;   // a division in few instructions: it runs once
#pragma unroll 1
            for (int bit = 46; bit >= 0; --bit)
                if (rest >> bit >= ctas * waves) {
                    rest -= (int64_t)(ctas * waves) << bit;
                    each += (int64_t)1 << bit;
                }
            if (half == 0 && lane < 2)   // the stretches that are not there
                for (int k = ctas * waves + cta; k < room * p.waves; k += room) p.parts[2 * k + lane] = make_int4(0, 0, 0, 0);
            // This CTA's stretches of the line, the requests 32 at a time.
            const int mine = cta < ctas ? waves : 0;
#pragma unroll 1
            for (int wave = 0; wave < mine; ++wave) {
                int4 slots[2] = {make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
                const int stretch = wave * ctas + cta;
                const int64_t begin = each * stretch + min((int64_t)stretch, rest);
                const int64_t end = begin + each + (stretch < rest ? 1 : 0);
                int64_t before = 0;         // length of the requests before r0
                int r0 = 0;
                if (wave == 0) {
#pragma unroll 1
                    for (; r0 + 32 < p.R && before + groups[r0 / 32] <= begin; r0 += 32) before += groups[r0 / 32];
                    fence_proxy_async_smem();   // the ring is the copies' from here on
                    __syncwarp();
                }
#pragma unroll 1
                for (; r0 < p.R && ok; r0 += 32) {
                    int first = 0, n = 0, ctx = 0, pairs = 0;
                    bool fits = true;
                    int64_t head = 0;
                    if (r0 + lane < p.R) fits = request(r0 + lane, lengths(r0 + lane), first, n, ctx, pairs, head);
                    int64_t upto = head * p.Hk;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += y;
                    }
                    const int64_t here = before;
                    before += __shfl_sync(0xffffffffu, upto, 31);
                    if (here >= end) break;
                    // the requests of these that meet the stretch
                    uint32_t meet = __ballot_sync(0xffffffffu, n > 0 && here + upto > begin && here + upto - head * p.Hk < end);
#pragma unroll 1
                    while (meet && ok) {
                        const int who = __ffs(meet) - 1;
                        meet &= meet - 1;
                        const int q_n = __shfl_sync(0xffffffffu, n, who), q_ctx = __shfl_sync(0xffffffffu, ctx, who),
                                  q_pairs = __shfl_sync(0xffffffffu, pairs, who);
                        const bool q_fits = __shfl_sync(0xffffffffu, (int)fits, who) != 0;
                        const int64_t q_head = __shfl_sync(0xffffffffu, head, who);
                        int64_t place = __shfl_sync(0xffffffffu, here + upto - head * p.Hk, who);   // of the item on the line
                        x.r = r0 + who;
                        x.first = __shfl_sync(0xffffffffu, first, who);
                        x.ctx = q_ctx;
                        x.h = 0;
                        int rb = 0;
                        if (place < begin) {   // the head, and the pair, that hold the stretch's begin
                            int hi = p.Hk;
#pragma unroll 1
                            while (hi - x.h > 1) {
                                const int mid = (x.h + hi) >> 1;
                                if (place + mid * q_head <= begin) x.h = mid; else hi = mid;
                            }
                            place += x.h * q_head;
                            hi = q_pairs;
#pragma unroll 1
                            while (hi - rb > 1) {
                                const int mid = (rb + hi) >> 1;
                                if (place + pair_at(q_ctx, mid) <= begin) rb = mid; else hi = mid;
                            }
                            place += pair_at(q_ctx, rb);
                        }
#pragma unroll 1
                        while (ok && place < end) {
                            x.token0 = rb * pt;
                            x.tokens = min(q_n - x.token0, pt);
                            x.two = x.tokens > tt;
                            const int keys_all = q_ctx + x.token0 + x.tokens;
                            x.end = q_fits ? keys_all : 0;
                            const int tiles = max(1, (x.end + kKeys - 1) / kKeys);
                            // key tiles before a place on the line: one in 128 (102.4) of the keys' part
                            const int64_t next = place + kItemKeys + (x.two ? keys_all : single(keys_all));
                            auto tiles_before = [&](int64_t to) -> int {
                                const int64_t in = max((int64_t)0, to - place - kItemKeys);
                                return (int)min((int64_t)tiles, x.two ? (in + 127) >> 7 : (5 * in + 511) >> 9);
                            };
                            x.t0 = next <= begin ? tiles : tiles_before(begin);   // (an item before the stretch)
                            x.t1 = next <= end ? tiles : tiles_before(end);
                            place = next;
                            x.whole = x.t0 == 0 && x.t1 == tiles;
                            if (x.t1 > x.t0) {
                                x.part = 2 * stretch + (x.t0 > 0 ? 0 : 1);
                                if (!x.whole) slots[x.t0 > 0 ? 0 : 1] = make_int4(x.t1 == tiles ? 2 : 1, x.r, x.h, rb);
                                deal();
                                load();
                            }
                            if (++rb == q_pairs) {
                                rb = 0;
                                if (++x.h == p.Hk) break;
                            }
                        }
                    }
                }
                // what the two slots hold: 0 nothing, 1 a part of item (r, h, rb), 2 its last
                if (half == 0 && lane == 0) {
                    p.parts[2 * stretch] = slots[0];
                    p.parts[2 * stretch + 1] = slots[1];
                }
            }
            x.t1 = -1;
            if (ok) deal();
            if (!__all_sync(0xffffffffu, ok) && lane == 0) fail();
            // the last copies into this CTA's memory
#pragma unroll 1
            for (int i = 0; i < 2 * kItems; ++i)
                if ((q_asked >> i) & 1) wait_for(&m.q_full[i >> 1][i & 1], (q_phase >> i) & 1, nullptr, kWaitLimitNs);
#pragma unroll 1
            for (int i = max(0, issued - kSlots); i < issued; ++i)
                if (!((raw >> (i % kSlots)) & 1)) wait_for(&m.kv_full[i % kSlots], (i / kSlots) & 1, nullptr, kWaitLimitNs);
                else wait_for(&m.kv_raw[i % kSlots], (raw_phases >> (i % kSlots)) & 1, nullptr, kWaitLimitNs);
        } else if (warp < 15) {
            // ------------------------------------------------------------ products
            // A warp a stream: a tile's second product, as soon as its P is there, and the next
            // tile's scores behind it, also those of the next item.  The whole warp walks the
            // loop and one elected lane issues, with every operand a warp-uniform value (see
            // kda_tree_mma.cu).
            constexpr uint32_t id_qk = MmaTypes<T>::qk(kKeys), id_pv = MmaTypes<T>::pv(kV);
            const int s = warp - 13;
            const uint32_t tbu = __shfl_sync(0xffffffffu, tb, 0);
            const uint32_t tsu = tbu + kTmemS + 128 * s, tou = tbu + kTmemO + 128 * s;
            const uint32_t q_at = __shfl_sync(0xffffffffu, smem_u32(sm), 0), ring_at = q_at + kQ * kQBytes;
            bool ok = true, two = false;
            int item = 0, base = 0, queries = 0;   // ring and query tiles before the item
            int tiles = 0, step = 1, j = 0;        // the item's key tiles; this stream's are j, j + step ..
            int units = 0, left = 0;               // how many of them are still to come; keys from the item's first tile on
            uint32_t p_phase = 0, outs = 0;        // items whose O this stream has formed
            auto landed = [&](int i) { return wait_on(&m.kv_full[i % kSlots], (i / kSlots) & 1, abort); };
            auto keys_landed = [&](int t) {
                bool all = true;
#pragma unroll
                for (int part = 0; part < kHalves; ++part) all = all && landed(base + kPer * t + part);
                return all;
            };
            // A tile of the other stream's (one row tile): seen and given back all the same, so that
            // neither stream is ever a phase ahead of, or behind, a place of the ring.
            auto pass = [&](int t) {
                ok = ok && keys_landed(t) && landed(base + kPer * t + kHalves);
                ok = __all_sync(0xffffffffu, ok);
                if (ok && lane <= kHalves) mbar_arrive(&m.kv_free[(base + kPer * t + lane) % kSlots]);
                __syncwarp();
            };
            // The next item with tiles for this stream, and the tile before its first there;
            // false after the last.
            auto enter = [&]() -> bool {
                for (;; ++item) {
                    ok = __all_sync(0xffffffffu, ok && wait_on(&m.item_full[item % kItems], (item / kItems) & 1, abort));
                    if (!ok) return false;
                    const Item& x = m.item[item % kItems];
                    const int t1 = __shfl_sync(0xffffffffu, x.t1, 0);
                    if (t1 < 0) return false;
                    tiles = t1 - __shfl_sync(0xffffffffu, x.t0, 0);
                    two = __shfl_sync(0xffffffffu, (int)x.two, 0) != 0;
                    units = __shfl_sync(0xffffffffu, stream_units(x, s), 0);
                    left = __shfl_sync(0xffffffffu, stream_end(x, s) - x.t0 * kKeys, 0);
                    release(item);
                    j = two ? 0 : s;
                    step = two ? 1 : 2;
                    if (j > 0) pass(0);
                    if (!ok) return false;
                    if (units > 0) return true;
                    base += kPer * tiles;
                    queries += 1;
                }
            };
            // Keys of tile t that the stream's rows see, in steps of 16 (one at least): products
            // behind them are left out.
            auto steps_of = [&](int t) { return max(1, min(kKeys / 16, (left - t * kKeys + 15) >> 4)); };
            auto scores = [&](int j, int units) {   // one elected lane
                const int b = (queries + (two ? s : 0)) % kQ;
                    const uint32_t id = id_qk - ((uint32_t)(kKeys - 16 * steps_of(j)) >> 3 << 17);   // N keys
                    const uint64_t ad = sdesc_kmajor_sw128(q_at + b * kQBytes);
#pragma unroll
                    for (int part = 0; part < kHalves; ++part) {   // kV channels of K
                        const uint64_t bd = sdesc_keys(ring_at + (base + kPer * j + part) % kSlots * kSlotBytes, kGroupBytes);
#pragma unroll
                        for (int k = 0; k < kV / 16; ++k)
                            umma_bf16(tsu, ad + ((part * kV / 16 + k) >> 2) * (kBlock >> 4) + (k & 3) * 2,
                                      bd + (k >> 2) * (1024 >> 4) + (k & 3) * 2, id, part + k > 0 ? 1u : 0u);
                    }
                    umma_commit(&m.s_full[s]);
                    if (!two) {
#pragma unroll 1
                        for (int part = 0; part < kHalves; ++part) umma_commit(&m.kv_free[(base + kPer * j + part) % kSlots]);
                        if (units == 1) {   // two arrivals free a row tile's queries: a stream's each, or one's both
                            umma_commit(&m.q_free[b]);
                            if (tiles == 1) umma_commit(&m.q_free[b]);
                        }
                    }
            };
            // One place in the code for an item's change and for what both ends of the line share:
            // what an item's change costs is fetching it.
            bool fresh = true, begun = false, pending = false;
#pragma unroll 1
            while (ok) {
                bool waited = false;   // for the next scores' keys
                if (pending) {
                    // the second product of tile j
                    const int slot = (base + kPer * j + kHalves) % kSlots, steps = steps_of(j);
                    const bool last = units == 1;
                    // O still holds the rows of the item before until they are out
                    if (!begun && outs > 0) ok = wait_on(&m.o_free[s], (outs - 1) & 1, abort);
                    ok = ok && landed(base + kPer * j + kHalves);
                    // with two row tiles the next scores' keys before P is there; with one, memory is the
                    // bound, and waiting for a K would hold up the V before it
                    if (two && !last) {
                        ok = ok && keys_landed(j + step);
                        waited = true;
                    }
                    const uint64_t bd = sdesc_mnmajor_sw128(ring_at + slot * kSlotBytes, 1024, kGroupBytes);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // the two halves of P as they come
                        ok = __all_sync(0xffffffffu, ok && wait_on(&m.p_full[s][h], p_phase, abort));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < kKeys / 32; ++k)
                                if (4 * h + k < steps)
                                    umma_bf16_ta(tou, tsu + 32 * h + 8 * k, bd + (4 * h + k) * (kGroupBytes >> 3), id_pv,
                                                 begun || h + k > 0 ? 1u : 0u);
                            if (h && waited) scores(j + step, units - 1);
                            if (h && (!two || last)) umma_commit(&m.kv_free[slot]);
                            if (h && last) umma_commit(&m.o_full[s]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    p_phase ^= 1;
                    begun = true;
                    // tiles of the other stream, or that this stream's rows do not see
                    if (!two || last) {
#pragma unroll 1
                        for (int t = j + 1; t < (two ? tiles : min(tiles, j + 2)) && ok; ++t) pass(t);
                        if (!ok) break;
                    }
                    --units;
                    j += step;
                    if (last) {
                        ++outs;
                        begun = false;
                        base += kPer * tiles;
                        queries += two ? 2 : 1;
                        ++item;
                        fresh = true;
                    }
                }
                if (fresh && !enter()) break;
                fresh = false;
                // Scores of tile j: as many keys as its rows see.  With two row tiles the softmax warps
                // give K, V and the queries back, once they have seen the scores: a commit takes the
                // issuer and the tensor pipe some 100 cycles.
                if (!waited) {
                    if (!begun) ok = ok && wait_on(&m.q_full[item % kItems][two ? s : 0], (item / kItems) & 1, abort);
                    ok = __all_sync(0xffffffffu, ok && keys_landed(j));
                    if (!ok) break;
                    tc_fence_after();
                }
                if (!waited) {
                    if (elect_one()) scores(j, units);
                    __syncwarp();
                }
                pending = true;
            }
            if (!ok && lane == 0) fail();
            if (elect_one()) umma_commit(&m.drained[s]);
            __syncwarp();
            wait_for(&m.drained[s], 0, nullptr, kWaitLimitNs);   // the last products
            __syncwarp();
        } else {
            // ------------------------------------------------------------ cleaning
            // V tiles with positions that some row of the item does not see, between their copy
            // and the products, so that the loader can go on.
            int base_kv = 0, item = 0;      // ring tiles before this item, items begun
            uint32_t phases = 0;            // of the slots' raw barriers
            bool ok = true;
            Item x;
            for (; __all_sync(0xffffffffu, take(item, x, ok)) && ok; ++item) {
                const int special = clean_from(x);
                if (lane < kBadWords) m.bad[item % kItems][lane] = 0;   // the way out of four items before has read them
                __syncwarp();
                for (int tile = max(x.t0, special); tile < x.t1 && ok; ++tile) {
                    const int i = base_kv + kPer * (tile - x.t0) + kHalves, slot = i % kSlots, base = tile * kKeys;
                    uint8_t* const dst = ring + slot * kSlotBytes;
                    ok = __all_sync(0xffffffffu, wait_on(&m.kv_raw[slot], (phases >> slot) & 1, abort));
                    if (!ok) break;
                    phases ^= 1u << slot;
                    constexpr uint32_t kExp = Elem<T>::kExpMask;
                    constexpr int kPieces = kV / 8;
                    auto piece = [&](int e) -> uint4* {   // 16-byte piece e of the tile, rows in order
                        const int c = e % kPieces, krow = e / kPieces;
                        return reinterpret_cast<uint4*>(dst + (krow >> 3) * kGroupBytes + (c >> 3) * 1024 +
                                                        (krow & 7) * 128 + (c & 7) * 16);
                    };
                    // rows behind what any row sees (in the last step of 16 keys alone: the products
                    // leave the others out), and those that every row sees
                    const int past = max(0, min(x.end - base, kKeys)), seen = max(0, min(x.ctx + x.token0 + 1, x.end) - base);
                    const int upto = max(16, (past + 15) & ~15);
#pragma unroll 1
                    for (int e = past * kPieces + lane; e < upto * kPieces; e += 32) *piece(e) = make_uint4(0, 0, 0, 0);
                    // is anything between not finite?  0 times such a value is NaN, and so is a sum with it
                    bool bad = false;
                    int e = seen * kPieces + lane;
#pragma unroll 1
                    for (; e < past * kPieces; e += 8 * 32) {
                        uint4 y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = e + 32 * k < past * kPieces ? *piece(e + 32 * k) : make_uint4(0, 0, 0, 0);
                        bad |= !all_finite<T, 8>(y);
                    }
                    if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
                        for (e = seen * kPieces + lane; e < past * kPieces; e += 32) {
                            const uint4 y = *piece(e);
                            uint32_t w[4] = {y.x, y.y, y.z, y.w};
                            bad = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((w[k] & kExp) == kExp) { bad = true; w[k] &= 0xffff0000u; }
                                if (((w[k] >> 16) & kExp) == kExp) { bad = true; w[k] &= 0xffffu; }
                            }
                            if (bad) {
                                const int j = base + e / kPieces - special * kKeys;
                                atomicOr(&m.bad[item % kItems][j >> 5], 1u << (j & 31));
                                *piece(e) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m.kv_full[slot]);
                }
                base_kv += kPer * (x.t1 - x.t0);
                release(item);
            }
            if (!__all_sync(0xffffffffu, ok) && lane == 0) fail();
        }
    } else if (warp >= 8) {
        // ---------------------------------------------------------------- the rows' way out
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const int row = tid & 127;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const int in_token = (int)page_div((uint32_t)row, G, p.group_magic), in_head = row - in_token * G;
        const float c = p.scale_log2;
        uint32_t outs = 0;            // items of each stream, odd or even
        bool ok = true;
        Item x;
        for (int item = 0;; ++item) {
            ok = ok && wait_out(&m.item_full[item % kItems], (item / kItems) & 1, abort, limit);
            if (!__all_sync(0xffffffffu, take(item, x, ok)) || !ok) break;
            const bool joined = !x.two && x.t1 - x.t0 > 1;
            const int special = clean_from(x);
            const bool cleaned = x.t1 > special;   // (otherwise the flags are not this item's)
            // one row tile: one pass over both streams; two: a pass each
            for (int a = 0; a < (x.two ? 2 : 1) && ok; ++a) {
                const int s = a, s2 = a ^ 1;
#pragma unroll 1
                for (int w = 0; w < (joined ? 4 : 2); ++w) {   // the rows' statistics and O, of s and then of s2
                    const int t = w < 2 ? s : s2;
                    ok = ok && wait_out(w & 1 ? &m.o_full[t] : &m.ml_full[t], (outs >> t) & 1, abort, limit);
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                outs ^= joined ? 3 : 1 << s;
                float2 ml = m.ml[s][row];
                float f0 = 1.f, f1 = 0.f;
                if (joined) {
                    const float2 o = m.ml[s2][row];
                    const float mj = fmaxf(ml.x, o.x), mu = mj == -INFINITY ? 0.f : mj;
                    f0 = ex2_approx((ml.x - mu) * c);
                    f1 = ex2_approx((o.x - mu) * c);
                    ml = make_float2(mj, ml.y * f0 + o.y * f1);
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&m.ml_free[s]);
                    if (joined) mbar_arrive(&m.ml_free[s2]);
                }
                const int token = x.token0 + a * tt + in_token;   // of the request
                const bool live = in_token < tt && token < x.token0 + x.tokens;
                const bool empty = ml.y == 0.f, whole = x.whole;
                // no weight: zeros for a part without keys or a request that does not fit the call; a whole
                // row whose scores are all -inf is 0 / 0
                const float inv = empty && (!whole || x.end == 0) ? 0.f : 1.f / ml.y;
                f0 *= inv;
                f1 *= inv;
                const int64_t part = (int64_t)x.part * 256 + a * 128 + row;
                T* const dst = static_cast<T*>(p.out) + (p.cu ? (int64_t)(x.first + token) * p.os[1]
                                                              : x.r * p.os[0] + token * p.os[1]) +
                               (x.h * G + in_head) * p.os[2] + half * kV;
                float* const pdst = p.part_o + part * D + half * kV;
                uint32_t any_bad = 0;
                if (cleaned) {
#pragma unroll
                    for (int w = 0; w < kBadWords; w += 4) {
                        const uint4 y = *reinterpret_cast<const uint4*>(&m.bad[item % kItems][w]);
                        any_bad |= y.x | y.y | y.z | y.w;
                    }
                }
                const uint32_t to = tb + lane_base + kTmemO + 128 * s, to2 = tb + lane_base + kTmemO + 128 * s2;
#pragma unroll 1
                for (int k = 0; k < kV / 16; ++k) {
                    uint32_t r0[16], r1[16];
                    float o[16];
                    tmem_ld16_issue(to + 16 * k, r0);
                    if (joined) tmem_ld16_issue(to2 + 16 * k, r1);
                    tmem_wait_ld();
                    tmem_take16(r0, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= f0;   // (0 where no key is seen: then O is 0 too)
                    if (joined) {
                        float y[16];
                        tmem_take16(r1, y);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = fmaf(y[e], f1, o[e]);
                    }
                    if (k == kV / 16 - 1) {   // O is read: the next item's may come
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&m.o_free[s]);
                            if (joined) mbar_arrive(&m.o_free[s2]);
                        }
                    }
                    if (!live) continue;
                    uint32_t w[8];
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = Elem<T>::pack(o[2 * e], o[2 * e + 1]);
                        store32(dst + 16 * k, w, p.wide_out);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[8 * i + e]);
                            store32(pdst + 16 * k + 8 * i, w, true);
                        }
                    }
                }
                if (any_bad && live && !empty) {   // elements of V that are not finite, to the rows that see them
                    const int to_key = min(x.ctx + token + 1, min(x.end, x.t1 * kKeys));
#pragma unroll 1
                    for (int pos = max(special, x.t0) * kKeys; pos < to_key; ++pos) {
                        const int j = pos - special * kKeys;
                        if (!((m.bad[item % kItems][j >> 5] >> (j & 31)) & 1u)) continue;
                        const int pg = (int)page_div((uint32_t)pos, p.page, p.page_magic), id = p.table[x.r * p.table_stride + pg];
                        if (id < 0 || id >= p.P) continue;
                        const T* src = static_cast<const T*>(p.vc) + id * p.vs[0] + (pos - pg * p.page) * p.vs[1] + x.h * p.vs[2] + half * kV;
#pragma unroll 1
                        for (int e = 0; e < kV; ++e) {
                            const float y = Elem<T>::one(src[e]);
                            if (isfinite(y)) continue;
                            if (whole) dst[e] = static_cast<T>(Elem<T>::one(dst[e]) + y);
                            else pdst[e] += y;
                        }
                    }
                }
                if (live && half == 0 && (!whole || p.lse)) {
                    const float lse = empty ? -INFINITY : ml.x * c + lg2_approx(ml.y);
                    if (!whole) p.part_lse[part] = lse;
                    else
                        p.lse[((p.cu ? (int64_t)x.first : (int64_t)x.r * p.T) + token) * p.Hq + x.h * G + in_head] =
                            lse * 0.6931471805599453f;
                }
            }
            if (ok) release(item);
        }
        if (!__all_sync(0xffffffffu, ok) && lane == 0) fail();
    } else {
        // ---------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int stream = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tb + lane_base + kTmemS + 128 * stream, to = tb + lane_base + kTmemO + 128 * stream;
        const float c = p.scale_log2, lazy = kLazy<T> / c;   // in units of the scores
        const int in_token = (int)page_div((uint32_t)row, G, p.group_magic);
        bool ok = true;
        uint32_t seen_s = 0, items_s = 0;   // score tiles taken, items with work for this stream
        int ring = 0, queries = 0;          // ring and query tiles before the item
        for (int item = 0;; ++item) {
            Item x;
            if (!__all_sync(0xffffffffu, take(item, x, ok)) || !ok) break;
            release(item);
            const bool two = x.two;
            const int units = stream_units(x, stream), step = two ? 1 : 2;
            const int ring_base = ring, b = (queries + stream) % kQ;   // (of two row tiles)
            ring += kPer * (x.t1 - x.t0);
            queries += two ? 2 : 1;
            if (units == 0) continue;
            // keys that this row sees, and the warp's first
            const int token = x.ctx + x.token0 + (two && stream ? tt : 0) + in_token;
            const int sees = min(token + 1, x.end), least = __shfl_sync(0xffffffffu, sees, 0);
            const int tile0 = x.t0 + (two ? 0 : stream);
            float mx = -INFINITY, l = 0.f;
            if (p.timeout_probe && item == 0) ok = __all_sync(0xffffffffu, wait_on(&m.never, 0, abort));
            for (int u = 0; u < units && ok; ++u) {
                ok = __all_sync(0xffffffffu, wait_on(&m.s_full[stream], seen_s & 1, abort));
                if (!ok) break;
                ++seen_s;
                tc_fence_after();
                if (two && (warp & 3) == 0 && lane == 0) {
                    // these scores are formed, and the stream's second product before them: this K and
                    // that V are free, and with the last scores the row tile's queries
                    const int at = ring_base + kPer * u;
#pragma unroll
                    for (int part = 0; part < kHalves; ++part) mbar_arrive(&m.kv_free[(at + part) % kSlots]);
                    if (u > 0) mbar_arrive(&m.kv_free[(at - 1) % kSlots]);
                    if (u == units - 1) {
                        mbar_arrive(&m.q_free[b]);   // for both streams
                        mbar_arrive(&m.q_free[b]);
                    }
                }
                uint32_t raw[8][16];
                float v[128];
#pragma unroll
                for (int k = 0; k < 8; ++k) tmem_ld16_issue(ts + 16 * k, raw[k]);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) tmem_take16(raw[k], &v[16 * k]);
                const int base = (tile0 + u * step) * kKeys;
                if (base + kKeys > least) {
                    const int n = sees - base, n_all = least - base;   // what this row sees, and all of the warp's
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        if (32 * g + 32 <= n_all) continue;
                        const uint32_t hidden = n >= 32 * g + 32 ? 0u : n <= 32 * g ? ~0u : ~0u << (n - 32 * g);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if ((hidden >> e) & 1u) v[32 * g + e] = -INFINITY;
                    }
                }
                float t8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t8[e] = max3(v[e], v[8 + e], v[16 + e]);
#pragma unroll
                for (int e = 24; e < 120; e += 16)
#pragma unroll
                    for (int i = 0; i < 8; ++i) t8[i] = max3(t8[i], v[e + i], v[e + 8 + i]);
                const float top = fmaxf(max3(max3(t8[0], t8[1], v[120]), max3(t8[2], t8[3], v[121]), max3(t8[4], t8[5], v[122])),
                                        max3(max3(t8[6], t8[7], v[123]), max3(v[124], v[125], v[126]), v[127]));
                float alpha = 1.f;
                if (top > mx + lazy || mx == -INFINITY) {
                    const float mn = fmaxf(mx, kShift<T> == 0.f ? top : fmaf(lazy, -kShift<T> / kLazy<T>, top));
                    if (mx != -INFINITY) alpha = ex2_approx((mx - mn) * c);
                    mx = mn;
                    l *= alpha;
                }
                if (u > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                    for (int k = 0; k < kV / 16; ++k) {
                        float o[16];
                        uint32_t w[16];
                        tmem_ld16(to + 16 * k, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
                        tmem_st16(to + 16 * k, w);
                    }
                }
                const float mc = mx == -INFINITY ? 0.f : -mx * c;
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
                        if (lane == 0) mbar_arrive(&m.p_full[stream][0]);
                    }
                }
                const float2 q = f2_parts(f2_add(sum[0], sum[1]));
                l += q.x + q.y;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.p_full[stream][1]);
            }
            // the rows' maximum and sum, once those of the stream's item before have been taken
            if (items_s > 0) ok = ok && wait_on(&m.ml_free[stream], (items_s - 1) & 1, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++items_s;
            m.ml[stream][row] = make_float2(mx, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.ml_full[stream]);
        }
        if (!ok && lane == 0) fail();
    }
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
}

template <typename T, int D>
cudaError_t launch_t(const ChunkParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, int grid,
                     cudaStream_t s) {
    static std::atomic<uint64_t> smem_set;
    cudaError_t e = set_smem_limit_once((const void*)chunk_mma_kernel<T, D>, (int)Shape<D>::kBytes, smem_set);
    if (e != cudaSuccess) return e;
    chunk_mma_kernel<T, D><<<grid - grid % Shape<D>::kHalves, kThreads, Shape<D>::kBytes, s>>>(p, qmap, kmap, vmap);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_d(const ChunkParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, int D,
                     int grid, cudaStream_t s) {
    return D == 64 ? launch_t<T, 64>(p, qmap, kmap, vmap, grid, s)
                   : D == 128 ? launch_t<T, 128>(p, qmap, kmap, vmap, grid, s) : launch_t<T, 256>(p, qmap, kmap, vmap, grid, s);
}

// Tensor map of the queries as [64 channels, heads, tokens, blocks of 64 channels, requests],
// a box the query heads of a key head of a row tile's tokens.
bool query_map(CUtensorMap* map, const ChunkParams& p, int D, bool f16) {
    const uint64_t dims[5] = {64, (uint64_t)p.Hq, (uint64_t)p.T, (uint64_t)D / 64, p.cu ? 1u : (uint64_t)p.R};
    const uint64_t strides[4] = {(uint64_t)p.qs[2] * 2, (uint64_t)p.qs[1] * 2, 128, (uint64_t)(p.cu ? p.qs[1] : p.qs[0]) * 2};
    const uint32_t box[5] = {64, (uint32_t)p.G, (uint32_t)p.tile_tokens, 1, 1};
    return make_tensor_map(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, p.q, dims, strides,
                           box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

bool launch_chunk_mma(const ChunkParams& q, int D, bool f16, int grid, cudaStream_t s, cudaError_t* e) {
    CUtensorMap qmap, kmap, vmap;
    ChunkParams p = q;
    p.tile_tokens = 128 / p.G;
    p.wait_ns += (uint64_t)((p.max_len + kKeys - 1) / kKeys) * kTileWaitNs;
    p.wide_out = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0 && p.os[0] % 16 == 0 && p.os[1] % 16 == 0 && p.os[2] % 16 == 0;
    if (!query_map(&qmap, p, D, f16) || !cache_map(&kmap, p.kc, p.ks, p.Hk, p.P, p.page, D, f16, &p.k_paged) ||
        !cache_map(&vmap, p.vc, p.vs, p.Hk, p.P, p.page, D, f16, &p.v_paged))
        return false;
    if (f16) *e = launch_d<__half>(p, qmap, kmap, vmap, D, grid, s);
    else *e = launch_d<__nv_bfloat16>(p, qmap, kmap, vmap, D, grid, s);
    return true;
}

}  // namespace kda
