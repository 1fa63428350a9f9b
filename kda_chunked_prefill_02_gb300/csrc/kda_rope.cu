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
// is a shuffle reduction over them and the partner of a half-split pair one
// shuffle of the packed input, since rot_dim / 2 is a multiple of a lane's 8
// channels.
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
constexpr int kRopeUnroll = 4;

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
    const int first = chunk * p.chunk_passes, end = first + p.chunk_passes;   // passes: q heads, k heads, v heads

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

    const bool rotates = c0 < p.rot;
    const int half = p.rot >> 1;
    const bool low = c0 < half;
    // lane that holds the partner channels (itself unless a half-split pair)
    const int mate = (!p.interleaved && rotates) ? lane + (low ? half / 8 : -half / 8) : lane;
    float cs[8], sn[8];
    if (first < qp + kp) {
        const int pos = rotates ? p.positions[token] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = 1.f;
            sn[i] = 0.f;
            if (rotates) {
                const int pair = p.interleaved ? (c0 + i) >> 1 : (low ? c0 + i : c0 + i - half);
                const float a = reduced_angle(pos, p.inv_freq[pair]);
                cs[i] = p.scale * __cosf(a);
                sn[i] = p.scale * __sinf(a);
            }
        }
    }
    auto weight = [&](const void* w, int c) -> float {
        if (!w) return 1.f;
        return p.w_f32 ? static_cast<const float*>(w)[c] : Elem<T>::one(static_cast<const T*>(w)[c]);
    };

    // heads [h0, h1) of one tensor, normed and rotated
    auto rotate = [&](const T* src, int64_t hs, const void* w, T* dst, int64_t dhs, T* dst2, int64_t dhs2, int h0,
                      int h1) {
        float A[8], B[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pc = !rotates ? cc + i : p.interleaved ? (cc + i) ^ 1 : low ? cc + i + half : cc + i - half;
            const bool minus = p.interleaved ? (i & 1) == 0 : low;
            A[i] = act ? weight(w, cc + i) * cs[i] : 0.f;
            B[i] = act ? weight(w, pc) * (minus ? -sn[i] : sn[i]) : 0.f;
        }
        for (int h = h0; h < h1; h += kGroup * kRopeUnroll) {
            uint4 raw[kRopeUnroll];
#pragma unroll
            for (int u = 0; u < kRopeUnroll; ++u) {
                const int hh = h + u * kGroup + sub;
                raw[u] = (act && hh < h1) ? *reinterpret_cast<const uint4*>(src + hh * hs + cc) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kRopeUnroll; ++u) {
                const int hh = h + u * kGroup + sub;
                if (h + u * kGroup >= h1) break;
                float x[8], y[8];
                unpack8<T>(raw[u], x);
                float r = 1.f;
                if (p.norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    r = rsqrt_approx(ss / (float)p.D + p.eps);
                }
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
                } else {
                    uint4 m;
                    m.x = __shfl_sync(0xffffffffu, raw[u].x, mate);
                    m.y = __shfl_sync(0xffffffffu, raw[u].y, mate);
                    m.z = __shfl_sync(0xffffffffu, raw[u].z, mate);
                    m.w = __shfl_sync(0xffffffffu, raw[u].w, mate);
                    unpack8<T>(m, y);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // channels that do not rotate take no part of another, not even 0 * inf
                    const float rest = rotates ? B[i] * y[i] : 0.f;
                    y[i] = r * fmaf(A[i], x[i], rest);
                }
                const uint4 o = pack8<T>(y);
                if (act && hh < h1) {
                    if (dst) *reinterpret_cast<uint4*>(dst + hh * dhs + cc) = o;
                    if (dst2) *reinterpret_cast<uint4*>(dst2 + hh * dhs2 + cc) = o;
                }
            }
        }
    };
    if (first < qp) {
        rotate(static_cast<const T*>(p.q) + b * p.qs[0] + t * p.qs[1], p.qs[2], p.q_w,
               static_cast<T*>(p.q_out) + b * p.qos[0] + t * p.qos[1], p.qos[2], nullptr, 0, first * kGroup,
               min(end * kGroup, p.Hq));
    }
    if (end > qp && first < qp + kp) {
        T* out = p.k_out ? static_cast<T*>(p.k_out) + b * p.kos[0] + t * p.kos[1] : nullptr;
        T* cache = kc_off >= 0 ? static_cast<T*>(p.k_cache) + kc_off : nullptr;
        rotate(static_cast<const T*>(p.k) + b * p.ks[0] + t * p.ks[1], p.ks[2], p.k_w, out, p.kos[2], cache, p.kcs[2],
               max(first - qp, 0) * kGroup, min((end - qp) * kGroup, p.Hk));
    }
    if (end > qp + kp && vc_off >= 0 && p.v_cache) {
        const T* src = static_cast<const T*>(p.v) + b * p.vs[0] + t * p.vs[1];
        T* dst = static_cast<T*>(p.v_cache) + vc_off;
        const int h1 = min((end - qp - kp) * kGroup, p.Hk);
        for (int h = max(first - qp - kp, 0) * kGroup + sub; h < h1; h += kGroup)
            if (act) *reinterpret_cast<uint4*>(dst + h * p.vcs[2] + cc) = ldg16(src + h * p.vs[2] + cc);
    }
}

template <typename T>
cudaError_t launch_rope_t(RopeParams& p, int num_sms, cudaStream_t s) {
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32, group = 32 / lanes;
    const int qp = (p.Hq + group - 1) / group, kp = (p.Hk + group - 1) / group;
    const int passes = qp + kp + (p.v_cache ? kp : 0);
    // A warp takes all of a token's heads (A and B are formed once) unless that
    // leaves fewer than 16 warps an SM: then the heads are cut further, down to
    // one unrolled run.
    int chunks = 1;
    while (p.tokens * chunks < 16LL * num_sms && chunks * kRopeUnroll < passes) chunks <<= 1;
    p.chunk_passes = (passes + chunks - 1) / chunks;
    p.chunks = (passes + p.chunk_passes - 1) / p.chunk_passes;
    const int64_t items = p.tokens * p.chunks, per = kRopeThreads / 32;
    const int64_t grid = (items + per - 1) / per;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (lanes == 8) qk_norm_rope_kernel<T, 8><<<(unsigned)grid, kRopeThreads, 0, s>>>(p);
    else if (lanes == 16) qk_norm_rope_kernel<T, 16><<<(unsigned)grid, kRopeThreads, 0, s>>>(p);
    else qk_norm_rope_kernel<T, 32><<<(unsigned)grid, kRopeThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& q, bool f16, int num_sms, cudaStream_t s) {
    RopeParams p = q;
    return f16 ? launch_rope_t<__half>(p, num_sms, s) : launch_rope_t<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace kda
