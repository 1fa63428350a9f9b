// attn_mma.cuh -- what the attention kernels on tcgen05 tensor cores (kda_tree_mma.cu,
// kda_chunk_mma.cu) share: tiles, operand descriptors, bounded waits, and the tensor map
// of a paged cache.
#pragma once

#include "ops_internal.h"
#include "sm103.cuh"
#include "tmap.h"

namespace kda {

constexpr int kKeys = 128;               // keys a tile
constexpr uint32_t kBlock = 128 * 128;   // Q: bytes of 128 rows of 64 elements
// P enters its product in the element type.  bf16: scores may exceed the running maximum by 8
// log2 units.  fp16 ends at 2^-24, and a long context may have its weight in keys far below the
// largest, so there the maximum is held 11 units lower than the scores and they may exceed it
// by 15: P uses fp16's range up to 2^15 (l carries the same factor, the log-sum m c + log2 l
// none).  A maximum that moves at 4 units instead of 8 is not slower to measure.
template <typename T> constexpr float kLazy = std::is_same<T, __half>::value ? 15.f : 8.f;
template <typename T> constexpr float kShift = std::is_same<T, __half>::value ? 11.f : 0.f;

// mbar_wait (sm103.cuh) with the clock and the abort flag looked at every 64th time
// only: between a phase's end and this thread's next step there is then nothing but
// the try_wait itself, where a look at the global timer takes longer than the wait.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const volatile int* abort, uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (i % 64) continue;
        if (abort && *abort) return false;
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        else if (t - t0 > limit_ns) return false;
    }
}

template <typename T> struct MmaTypes;
template <> struct MmaTypes<__nv_bfloat16> {
    static __host__ __device__ constexpr uint32_t qk(uint32_t n) { return idesc_bf16_f32(128, n); }
    static __host__ __device__ constexpr uint32_t pv(uint32_t n) { return idesc_bf16_f32_bmn(128, n); }
};
template <> struct MmaTypes<__half> {
    static __host__ __device__ constexpr uint32_t qk(uint32_t n) { return idesc_f16_f32(128, n); }
    static __host__ __device__ constexpr uint32_t pv(uint32_t n) { return idesc_f16_f32_bmn(128, n); }
};

// Rows a copy brings: the largest power of two that divides the page, a tile's at most,
// so that no copy goes past a tile's or a page's end.
__host__ __device__ constexpr int box_of(int page) { return page % kKeys == 0 ? kKeys : page & -page; }

// K-major operand in the 128-byte swizzle with its 8-row groups `group` bytes apart.
__device__ __forceinline__ uint64_t sdesc_keys(uint32_t saddr, uint32_t group) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(group >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
        : "memory");
}

// a / b of numbers that hardly ever need 64 bits: the division that does takes some
// 500 cycles of the way to a CTA's first item.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0;
}

// Tensor map of a cache as [64 channels, 8 rows, blocks of 64 channels, groups of 8
// rows, pages], a box the rows of a page that a tile takes with all their channels
// of one head: one copy a page (a copy costs about 120 cycles, whatever its size,
// which with pages of 16 is what bounds copies of 64 channels).  The head is part
// of the block dimension where a row's heads follow one another, of the page
// dimension (*paged) where a page's heads do.  False for any other layout.
inline bool cache_map(CUtensorMap* map, const void* base, const int64_t (&st)[3], int Hk, int pages, int page, int D, bool f16,
                      int* paged) {
    const bool rows = Hk == 1 || st[2] == D;
    if (!rows && st[0] != st[2] * Hk) return false;
    *paged = !rows;
    const uint64_t dims[5] = {64, 8, (uint64_t)(rows ? Hk : 1) * (D / 64), (uint64_t)page / 8,
                              (uint64_t)pages * (rows ? 1 : Hk)};
    const uint64_t strides[4] = {(uint64_t)st[1] * 2, 128, (uint64_t)st[1] * 16, (uint64_t)(rows ? st[0] : st[2]) * 2};
    const uint32_t box[5] = {64, 8, (uint32_t)(D == 256 ? 128 : D) / 64, (uint32_t)box_of(page) / 8, 1};
    if (dims[4] > INT32_MAX) return false;
    return make_tensor_map(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dims,
                           strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace kda
