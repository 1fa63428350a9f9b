// kda_rope.cu -- RMS norm of every query and key head and the rotation by the
// token's position in one pass, the keys and values put into their rows of a
// paged cache on the way (kda_qk_norm_rope in include/kda_ops.h).
//
// With r = 1 / sqrt(mean(x^2) + eps), the channel c of a rotated pair and its
// partner c', the two steps fold into
//
//     out_c = r (A_c x_c + B_c x_c'),   A_c = s w_c cos t,  B_c = -+ s w_c' sin t,
//
// and A and B depend on the token and the channel only, not on the head.  So a
// warp takes one token and a run of its heads, forms A and B once in registers
// (8 channels a lane) and then spends a square, two FMAs and a product on every
// element; each element is read once and written once, and the kernel is bound
// by HBM bandwidth (4 bytes an element).  A head's channels are kLanes adjacent
// lanes (8, 16 or 32 for head sizes up to 64, 128 and 256); the sum of squares
// is a shuffle reduction over them, and the partner of a half-split pair lies in
// another lane's piece, since rot_dim / 2 is a multiple of a lane's 8 channels.
//
// All of a warp's pieces are asked for at once by 16-byte asynchronous copies
// into shared memory (up to kMaxPasses of 512 bytes), and A and B are formed
// while they fly; with the loads in registers, four at a time, the same sums
// took 171 us for 32768 tokens of 32 + 8 heads of 128.
//
// The angle.  t = position * f reaches 1e5 and more in a long context, where a
// rounded fp32 product is off by 1e-2.  The product is kept in two fp32 parts
// (hi = round(p f), lo = fma(p, f, -hi), exact while p is) and hi is reduced by
// the nearest multiple of 2 pi with 2 pi in two parts, each step one FMA whose
// result is small; positions or products of 2^24 and beyond are reduced in
// double.
#include "kda_internal.h"
#include "ops_internal.h"

namespace kda {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kMaxPasses = 23;   // 512 bytes each, and as many zeros: 48 KB for a CTA's four warps

// position * f modulo 2 pi, in about [-5, 5], within 1e-6.
__device__ __forceinline__ float reduced_angle(int pos, float f) {
    constexpr float kTwoPi = 6.283185307179586f;   // rounded; the rest follows
    constexpr float kTwoPiRest = (float)(6.283185307179586476925 - (double)6.283185307179586f);
    const float p = (float)pos, hi = p * f, lo = fmaf(p, f, -hi);
    if (pos > -(1 << 24) && pos < (1 << 24) && fabsf(hi) < 16777216.f) {
        // k below 2^22: k * kTwoPi is exact inside the FMA and the difference is
        // below 5, so it is off by 2^-22 at most; so is the last sum
        const float k = rintf(hi * 0.15915494309189535f);
        return fmaf(-k, kTwoPiRest, fmaf(-k, kTwoPi, hi)) + lo;
    }
    const double a = (double)pos * (double)f;
    return (float)(a - 6.283185307179586476925 * rint(a * 0.15915494309189533577));
}

template <typename T, int kLanes>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
    constexpr int kGroup = 32 / kLanes;   // heads a warp takes at a time
    const int lane = threadIdx.x & 31, sub = lane / kLanes, c0 = (lane % kLanes) * 8;
    const int64_t item = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t token = item / p.chunks;
    if (token >= p.tokens) return;
    const int chunk = (int)(item - token * p.chunks);
    const int64_t b = token / p.T, t = token - b * p.T;
    const bool act = c0 < p.D;
    const int cc = act ? c0 : 0;

    const int qp = (p.Hq + kGroup - 1) / kGroup, kp = (p.Hk + kGroup - 1) / kGroup;
    const int first = chunk * p.chunk_passes;   // passes: q heads, k heads, v heads
    const int end = min(first + p.chunk_passes, qp + kp + (p.v_cache ? kp : 0));

    // where the token's cache row is
    int64_t kc_off = -1, vc_off = -1;
    if (p.slots && end > qp) {
        const int64_t slot = p.slots[token];
        if (slot >= p.cache_rows) {
            if (p.status && lane == 0) atomicExch(p.status, 1);
        } else if (slot >= 0) {
            const int64_t page = slot / p.page, row = slot - page * p.page;
            kc_off = page * p.kcs[0] + row * p.kcs[1];
            vc_off = page * p.vcs[0] + row * p.vcs[1];
        }
    }

    // every piece of this run of heads, on its way to shared memory
    extern __shared__ __align__(16) uint4 pieces[];
    uint4* const mine = pieces + (threadIdx.x >> 5) * (p.chunk_passes + 1) * 32;   // [pass][lane], then 32 zeros
    const bool values = vc_off >= 0 && p.v_cache;
    auto fetch = [&](int i0, int i1, int base, const T* src, int64_t hs, int heads) {
        uint4* dst = mine + (i0 - first) * 32 + lane;
        int h = (i0 - base) * kGroup + sub;
        src += h * hs + cc;
        for (int i = i0; i < i1; ++i) {
            if (act && h < heads) cp_async16(dst, src);
            else *dst = make_uint4(0, 0, 0, 0);
            dst += 32;
            h += kGroup;
            src += kGroup * hs;
        }
    };
    if (first < qp)
        fetch(first, min(end, qp), 0, static_cast<const T*>(p.q) + b * p.qs[0] + t * p.qs[1], p.qs[2], p.Hq);
    if (end > qp && first < qp + kp)
        fetch(max(first, qp), min(end, qp + kp), qp, static_cast<const T*>(p.k) + b * p.ks[0] + t * p.ks[1], p.ks[2],
              p.Hk);
    if (end > qp + kp && values)
        fetch(max(first, qp + kp), end, qp + kp, static_cast<const T*>(p.v) + b * p.vs[0] + t * p.vs[1], p.vs[2], p.Hk);
    cp_async_commit();
    mine[p.chunk_passes * 32 + lane] = make_uint4(0, 0, 0, 0);

    const bool rotates = c0 < p.rot;
    const int half = p.rot >> 1;
    const bool low = c0 < half;
    // first of the partner channels (half-split; interleaved pairs lie within the piece)
    const int pc0 = (p.interleaved || !rotates) ? cc : low ? cc + half : cc - half;
    // Where a pass's partner piece is: for channels that do not rotate the zeros,
    // so that they take no part of another channel, not even 0 * inf.
    const int mate = rotates ? lane + (pc0 - cc) / 8 : p.chunk_passes * 32 + lane;
    const int mate_step = rotates ? 32 : 0;
    float cs[8], sn[8];
    if (first < qp + kp) {
        const int pos = rotates ? p.positions[token] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = 1.f;
            sn[i] = 0.f;
            if (rotates && !(p.interleaved && (i & 1))) {
                const int pair = p.interleaved ? (c0 + i) >> 1 : (low ? c0 + i : c0 + i - half);
                const float a = reduced_angle(pos, __ldg(p.inv_freq + pair));
                cs[i] = p.scale * __cosf(a);
                sn[i] = p.scale * __sinf(a);
            }
        }
        if (rotates && p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                cs[i + 1] = cs[i];
                sn[i + 1] = sn[i];
            }
        }
    }
    auto weights = [&](const void* w, int c, float (&f)[8]) {
        if (!w) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 1.f;
        } else if (p.w_f32) {
            const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
            const float4 a = __ldg(src), e = __ldg(src + 1);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = e.x; f[5] = e.y; f[6] = e.z; f[7] = e.w;
        } else {
            F2 x[4];
            unpack8<T>(ldg16(static_cast<const T*>(w) + c), x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = f2_parts(x[i]);
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    };
    bool landed = false;
    const float inv_d = 1.f / (float)p.D;

    // passes [i0, i1), whose first is head 0 of a tensor at pass `base`, normed and rotated
    auto rotate = [&](int i0, int i1, int base, int heads, const void* w, T* dst, int64_t dhs, T* dst2, int64_t dhs2) {
        F2 A[4], B[4];
        {
            float own[8], other[8];
            weights(w, cc, own);
            weights(w, pc0, other);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                A[k] = f2(own[2 * k] * cs[2 * k], own[2 * k + 1] * cs[2 * k + 1]);
                B[k] = p.interleaved
                           ? f2(-other[2 * k + 1] * sn[2 * k], other[2 * k] * sn[2 * k + 1])
                           : f2(other[2 * k] * (low ? -sn[2 * k] : sn[2 * k]),
                                other[2 * k + 1] * (low ? -sn[2 * k + 1] : sn[2 * k + 1]));
            }
        }
        if (!landed) {
            cp_async_wait<0>();
            __syncwarp();   // partners are read from other lanes' pieces
            landed = true;
        }
        const uint4* src = mine + (i0 - first) * 32 + lane;
        const uint4* msrc = mine + (i0 - first) * mate_step + mate;
        int h = (i0 - base) * kGroup + sub;
        if (dst) dst += h * dhs + cc;
        if (dst2) dst2 += h * dhs2 + cc;
#pragma unroll 2
        for (int i = i0; i < i1; ++i) {
            F2 x[4], y[4];
            unpack8<T>(*src, x);
            uint4 m = *msrc;
            src += 32;
            msrc += mate_step;
            float r = 1.f;
            if (p.norm) {
                F2 s2 = f2_mul(x[0], x[0]);
#pragma unroll
                for (int k = 1; k < 4; ++k) s2 = f2_fma(x[k], x[k], s2);
                const float2 s = f2_parts(s2);
                float ss = s.x + s.y;
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                r = rsqrt_approx(fmaf(ss, inv_d, p.eps));
            }
            if (p.interleaved) {   // the partner is the other half of a 32-bit word
                m.x = __byte_perm(m.x, 0, 0x1032);
                m.y = __byte_perm(m.y, 0, 0x1032);
                m.z = __byte_perm(m.z, 0, 0x1032);
                m.w = __byte_perm(m.w, 0, 0x1032);
            }
            unpack8<T>(m, y);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = f2_mul(f2(r, r), f2_fma(A[k], x[k], f2_mul(B[k], y[k])));
            if (act && h < heads) {
                const uint4 o = pack8<T>(y);
                if (dst) *reinterpret_cast<uint4*>(dst) = o;
                if (dst2) *reinterpret_cast<uint4*>(dst2) = o;
            }
            h += kGroup;
            dst += kGroup * dhs;
            dst2 += kGroup * dhs2;
        }
    };
    if (first < qp)
        rotate(first, min(end, qp), 0, p.Hq, p.q_w, static_cast<T*>(p.q_out) + b * p.qos[0] + t * p.qos[1], p.qos[2],
               nullptr, 0);
    if (end > qp && first < qp + kp) {
        T* out = p.k_out ? static_cast<T*>(p.k_out) + b * p.kos[0] + t * p.kos[1] : nullptr;
        T* cache = kc_off >= 0 ? static_cast<T*>(p.k_cache) + kc_off : nullptr;
        rotate(max(first, qp), min(end, qp + kp), qp, p.Hk, p.k_w, out, out ? p.kos[2] : 0, cache,
               cache ? p.kcs[2] : 0);
    }
    cp_async_wait<0>();
    if (end > qp + kp && values) {
        int i = max(first, qp + kp), h = (i - qp - kp) * kGroup + sub;
        T* dst = static_cast<T*>(p.v_cache) + vc_off + h * p.vcs[2] + cc;
        for (; i < end; ++i) {
            if (act && h < p.Hk) *reinterpret_cast<uint4*>(dst) = mine[(i - first) * 32 + lane];
            h += kGroup;
            dst += kGroup * p.vcs[2];
        }
    }
}

template <typename T>
cudaError_t launch_rope_t(RopeParams& p, int num_sms, cudaStream_t s) {
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32, group = 32 / lanes;
    const int qp = (p.Hq + group - 1) / group, kp = (p.Hk + group - 1) / group;
    const int passes = qp + kp + (p.v_cache ? kp : 0);
    // A warp takes all of a token's heads (A and B are formed once), as far as
    // its shared memory goes, unless that leaves fewer than 16 warps an SM: then
    // the heads are cut further, down to two passes.
    int chunks = (passes + kMaxPasses - 1) / kMaxPasses;
    while (p.tokens * chunks < 16LL * num_sms && chunks * 2 < passes) chunks <<= 1;
    p.chunk_passes = (passes + chunks - 1) / chunks;
    p.chunks = (passes + p.chunk_passes - 1) / p.chunk_passes;
    const size_t smem = (size_t)(kRopeThreads / 32) * (p.chunk_passes + 1) * 512;
    const int64_t items = p.tokens * p.chunks, per = kRopeThreads / 32;
    const int64_t grid = (items + per - 1) / per;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (lanes == 8) qk_norm_rope_kernel<T, 8><<<(unsigned)grid, kRopeThreads, smem, s>>>(p);
    else if (lanes == 16) qk_norm_rope_kernel<T, 16><<<(unsigned)grid, kRopeThreads, smem, s>>>(p);
    else qk_norm_rope_kernel<T, 32><<<(unsigned)grid, kRopeThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& q, bool f16, int num_sms, cudaStream_t s) {
    RopeParams p = q;
    return f16 ? launch_rope_t<__half>(p, num_sms, s) : launch_rope_t<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace kda
