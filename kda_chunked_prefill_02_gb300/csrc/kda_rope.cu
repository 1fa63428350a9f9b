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
// All of a warp's pieces are asked for at once by 16-byte asynchronous copies into
// shared memory (up to kMaxPasses of 512 bytes), and A and B are formed while they
// fly: every angle by one lane, the cosines and sines through shared memory (formed
// by every lane that turns by them they take 0.5 us of a small call's 3.8; 41 us
// against 37 with 18318 tokens of 12 + 3 heads of 96, 36.5 against 35.3 with 8191
// tokens of 16 + 2 heads of 256).  The arithmetic is near the issue limit (a pass of
// 32 pieces has some 90 cycles of a scheduler at the memory's rate), and it takes 20
// warps an SM to keep up: two passes go together, whose sums of squares share one
// reduction and one root.  Measured: 32768 tokens of 32 + 8 heads of 128, fp16, 104
// us (6.4 TB/s; 171 with the loads in registers, 118 with a reduction a pass, 103
// with four passes together, but then the wide heads take 38 us against 36; 153 with
// persistent warps and two buffers, which leave 8 warps an SM).
//
// The angle.  t = position * f reaches 1e5 and more in a long context, where a
// rounded fp32 product is off by 1e-2.  The product is kept in two fp32 parts
// (hi = round(p f), lo = fma(p, f, -hi), exact while p is) and hi is reduced by
// the nearest multiple of 2 pi with 2 pi in two parts, each step one FMA whose
// result is small; positions or products of 2^24 and beyond are reduced in
// the same way in double.
#include "kda_internal.h"
#include "ops_internal.h"

namespace kda {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kMaxPasses = 20;   // of an item
// Rows of 512 bytes a warp has: its passes, the token's cosines and sines (which are also
// read, and not used, past an odd number of passes, two at a time), and zeros.
__host__ __device__ constexpr int turn_rows(int rot) { return rot > 128 ? 2 : 1; }
__host__ __device__ constexpr int warp_rows(int passes, int rot) { return passes + turn_rows(rot) + 1; }
static_assert(kRopeThreads / 32 * warp_rows(kMaxPasses, 256) * 512 <= 48 * 1024, "fits without an opt-in");

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
    // the same in double: the product has up to 55 bits, and its rounding and that of 2 pi count
    // from frequencies of some 16 on
    constexpr double kTwoPiD = 6.283185307179586, kTwoPiDRest = 2.4492935982947064e-16;
    const double d = (double)pos, a = d * (double)f, rest = fma(d, (double)f, -a), k = rint(a * 0.15915494309189533577);
    return (float)(fma(-k, kTwoPiDRest, fma(-k, kTwoPiD, a)) + rest);
}

// 1 / sqrt(a[k] / D + eps) of two sums over groups of kLanes lanes, each to all of
// its group: a halving step leaves every lane a half of one of the sums.
template <int kLanes>
__device__ __forceinline__ void inverse_norms(float (&a)[2], float inv_d, float eps, int lane) {
    constexpr int kHalf = kLanes / 2;
    const bool h = lane & kHalf;
    float s = (h ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, h ? a[0] : a[1], kHalf);
#pragma unroll
    for (int o = kLanes / 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float r = rsqrt_approx(fmaf(s, inv_d, eps)), o = __shfl_xor_sync(0xffffffffu, r, kHalf);
    a[0] = h ? o : r;
    a[1] = h ? r : o;
}

template <typename T, int kLanes>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
    constexpr int kGroup = 32 / kLanes;   // heads a pass
    const int lane = threadIdx.x & 31, sub = lane / kLanes, c0 = (lane % kLanes) * 8;
    const int64_t items = p.tokens * p.chunks;
    const int64_t item = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (item >= items) return;
    const bool act = c0 < p.D;
    const int cc = act ? c0 : 0;
    const int P = p.chunk_passes;
    extern __shared__ __align__(16) uint4 pieces[];
    uint4* const mine = pieces + (threadIdx.x >> 5) * warp_rows(P, p.rot) * 32;
    float2* const turn = reinterpret_cast<float2*>(mine + P * 32);
    uint4* const zeros = mine + (P + turn_rows(p.rot)) * 32;
    zeros[lane] = make_uint4(0, 0, 0, 0);

    // passes of a token: its query heads, its key heads, its value heads
    const int qp = (p.Hq + kGroup - 1) / kGroup, kp = (p.Hk + kGroup - 1) / kGroup;
    const int all = qp + kp + (p.v_cache ? kp : 0);
    const bool rotates = c0 < p.rot;
    const int half = p.rot >> 1;
    const bool low = c0 < half;
    // first of the partner channels (half-split; interleaved pairs lie within the piece)
    const int pc0 = (p.interleaved || !rotates) ? cc : low ? cc + half : cc - half;
    const float inv_d = 1.f / (float)p.D;

    struct Place {
        int64_t b, t, slot;
        int first, end, pos;   // passes [first, end); position
    };
    auto place = [&](int64_t it) {
        Place x;
        const uint32_t token = (uint32_t)(p.chunks == 1 ? it : it / p.chunks), b = token / (uint32_t)p.T;   // below 2^31
        x.b = b;
        x.t = token - b * (uint32_t)p.T;
        x.first = (int)(it - (int64_t)token * p.chunks) * P;
        x.end = min(x.first + P, all);
        x.pos = p.rot ? __ldg(p.positions + token) : 0;
        x.slot = p.slots ? __ldg(reinterpret_cast<const long long*>(p.slots) + token) : -1;
        return x;
    };
    // an item's pieces on their way into a buffer
    auto fetch = [&](const Place& x, uint4* buf) {
        auto run = [&](int i0, int i1, int base, const T* src, int64_t hs, int heads) {
            uint4* dst = buf + (i0 - x.first) * 32 + lane;
            int h = (i0 - base) * kGroup + sub;
            src += h * hs + cc;
#pragma unroll 4
            for (int i = i0; i < i1; ++i) {
                if (act && h < heads) cp_async16(dst, src);
                else *dst = make_uint4(0, 0, 0, 0);
                dst += 32;
                h += kGroup;
                src += kGroup * hs;
            }
        };
        if (x.first < qp)
            run(x.first, min(x.end, qp), 0, static_cast<const T*>(p.q) + x.b * p.qs[0] + x.t * p.qs[1], p.qs[2], p.Hq);
        if (x.end > qp && x.first < qp + kp)
            run(max(x.first, qp), min(x.end, qp + kp), qp, static_cast<const T*>(p.k) + x.b * p.ks[0] + x.t * p.ks[1],
                p.ks[2], p.Hk);
        if (x.end > qp + kp)
            run(max(x.first, qp + kp), x.end, qp + kp, static_cast<const T*>(p.v) + x.b * p.vs[0] + x.t * p.vs[1],
                p.vs[2], p.Hk);
    };
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

    const Place cur = place(item);
    uint4* const buf = mine;
    fetch(cur, buf);
    cp_async_commit();
    {
        // where the token's cache row is
        int64_t kc_off = -1, vc_off = -1;
        if (cur.slot >= p.cache_rows) {
            if (p.slots && cur.end > qp && p.status && lane == 0) atomicMax(p.status, 1);
        } else if (cur.slot >= 0) {
            const int64_t page = cur.slot / p.page, row = cur.slot - page * p.page;
            kc_off = page * p.kcs[0] + row * p.kcs[1];
            vc_off = page * p.vcs[0] + row * p.vcs[1];
        }
        // every angle once, to all lanes that turn by it
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = 1.f;
            sn[i] = 0.f;
        }
        if (cur.first < qp + kp) {
            for (int j = lane; j < half; j += 32) {
                const float a = reduced_angle(cur.pos, __ldg(p.inv_freq + j));
                turn[j] = make_float2(p.scale * __cosf(a), p.scale * __sinf(a));
            }
            __syncwarp();
            if (rotates) {
                const float4* src = reinterpret_cast<const float4*>(turn + (p.interleaved ? c0 / 2 : low ? c0 : c0 - half));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (p.interleaved) {
                        const float2 y = reinterpret_cast<const float2*>(src)[i];
                        cs[2 * i] = cs[2 * i + 1] = y.x;
                        sn[2 * i] = sn[2 * i + 1] = y.y;
                    } else {
                        const float4 y = src[i];
                        cs[2 * i] = y.x;
                        sn[2 * i] = y.y;
                        cs[2 * i + 1] = y.z;
                        sn[2 * i + 1] = y.w;
                    }
                }
            }
        }
        bool landed = false;

        // passes [i0, i1), whose first is head 0 of a tensor at pass `base`, normed and rotated
        auto rotate = [&](int i0, int i1, int base, int heads, const void* w, T* dst, int64_t dhs, T* dst2,
                          int64_t dhs2) {
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
            const uint4* src = buf + (i0 - cur.first) * 32 + lane;
            // Where a pass's partner piece is: for channels that do not rotate the zeros, so
            // that they take no part of another channel, not even 0 * inf.
            const uint4* msrc = rotates ? src + (pc0 - cc) / 8 : zeros + lane;
            const int mstep = rotates ? 32 : 0;
            int h = (i0 - base) * kGroup + sub;
            if (dst) dst += h * dhs + cc;
            if (dst2) dst2 += h * dhs2 + cc;
#pragma unroll 1
            for (int i = i0; i < i1; i += 2) {
                F2 x[2][4];
                float r[2] = {1.f, 1.f};
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    unpack8<T>(src[u * 32], x[u]);
                    if (p.norm) {
                        F2 s2 = f2_mul(x[u][0], x[u][0]);
#pragma unroll
                        for (int k = 1; k < 4; ++k) s2 = f2_fma(x[u][k], x[u][k], s2);
                        const float2 s = f2_parts(s2);
                        r[u] = s.x + s.y;
                    }
                }
                if (p.norm) inverse_norms<kLanes>(r, inv_d, p.eps, lane);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 m = msrc[u * mstep];
                    if (p.interleaved) {   // the partner is the other half of a 32-bit word
                        m.x = __byte_perm(m.x, 0, 0x1032);
                        m.y = __byte_perm(m.y, 0, 0x1032);
                        m.z = __byte_perm(m.z, 0, 0x1032);
                        m.w = __byte_perm(m.w, 0, 0x1032);
                    }
                    F2 y[4];
                    unpack8<T>(m, y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[k] = f2_mul(f2(r[u], r[u]), f2_fma(A[k], x[u][k], f2_mul(B[k], y[k])));
                    if (act && i + u < i1 && h + u * kGroup < heads) {
                        const uint4 o = pack8<T>(y);
                        if (dst) *reinterpret_cast<uint4*>(dst + u * kGroup * dhs) = o;
                        if (dst2) *reinterpret_cast<uint4*>(dst2 + u * kGroup * dhs2) = o;
                    }
                }
                src += 2 * 32;
                msrc += 2 * mstep;
                h += 2 * kGroup;
                dst += 2 * kGroup * dhs;
                dst2 += 2 * kGroup * dhs2;
            }
        };
        if (cur.first < qp)
            rotate(cur.first, min(cur.end, qp), 0, p.Hq, p.q_w,
                   static_cast<T*>(p.q_out) + cur.b * p.qos[0] + cur.t * p.qos[1], p.qos[2], nullptr, 0);
        if (cur.end > qp && cur.first < qp + kp) {
            T* out = p.k_out ? static_cast<T*>(p.k_out) + cur.b * p.kos[0] + cur.t * p.kos[1] : nullptr;
            T* cache = kc_off >= 0 ? static_cast<T*>(p.k_cache) + kc_off : nullptr;
            rotate(max(cur.first, qp), min(cur.end, qp + kp), qp, p.Hk, p.k_w, out, out ? p.kos[2] : 0, cache,
                   cache ? p.kcs[2] : 0);
        }
        if (!landed) cp_async_wait<0>();
        if (cur.end > qp + kp && vc_off >= 0) {
            int i = max(cur.first, qp + kp), h = (i - qp - kp) * kGroup + sub;
            T* dst = static_cast<T*>(p.v_cache) + vc_off + h * p.vcs[2] + cc;
            for (; i < cur.end; ++i) {
                if (act && h < p.Hk) *reinterpret_cast<uint4*>(dst) = buf[(i - cur.first) * 32 + lane];
                h += kGroup;
                dst += kGroup * p.vcs[2];
            }
        }
    }
    cp_async_wait<0>();
}

template <typename T>
cudaError_t launch_rope_t(RopeParams& p, int num_sms, cudaStream_t s) {
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32, group = 32 / lanes;
    const int qp = (p.Hq + group - 1) / group, kp = (p.Hk + group - 1) / group;
    const int passes = qp + kp + (p.v_cache ? kp : 0);
    // A warp takes all of a token's heads (A and B are formed once), as far as
    // its shared memory goes, unless that leaves fewer than 8 warps an SM: then
    // the heads are cut further, down to two passes (1024 drafts of 32 + 2 x 8 heads: 7.3
    // us; 10.6 where 16 warps an SM are asked for, 16.4 with 64).
    int chunks = (passes + kMaxPasses - 1) / kMaxPasses;
    while (p.tokens * chunks < 8LL * num_sms && chunks * 2 < passes) chunks <<= 1;
    p.chunk_passes = (passes + chunks - 1) / chunks;
    p.chunks = (passes + p.chunk_passes - 1) / p.chunk_passes;
    const size_t smem = (size_t)(kRopeThreads / 32) * warp_rows(p.chunk_passes, p.rot) * 512;
    const int64_t blocks = (p.tokens * p.chunks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    const auto kernel = lanes == 8 ? qk_norm_rope_kernel<T, 8> : lanes == 16 ? qk_norm_rope_kernel<T, 16>
                                                                             : qk_norm_rope_kernel<T, 32>;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    kernel<<<(unsigned)blocks, kRopeThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& q, bool f16, int num_sms, cudaStream_t s) {
    RopeParams p = q;
    return f16 ? launch_rope_t<__half>(p, num_sms, s) : launch_rope_t<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace kda
