// kda_conv.cu -- the short causal convolution in front of a KDA layer, with
// SiLU, the per-head L2 norm of the q and k channels and the conv-state pool
// (kda_short_conv in include/kda_ops.h; the conv caches that the TensorRT-LLM
// page "Kimi K3 work for Rubin (SM107)", Description, keeps beside the KDA
// states).
//
// y_t[c] = act(bias[c] + sum_j w[c][j] x_{t-W+1+j}[c]): every input is used W
// times and every output written once, so the kernel streams x once and is
// bound by HBM bandwidth (4 bytes an element).  Thread = 8 channels (16 bytes a
// token), walking down a tile of tokens with the last W - 1 inputs in fp32
// registers.  The tokens ahead come by 16-byte asynchronous copies into a ring
// of kRing rows in shared memory, of which every thread reads only what it
// copied itself: the loads in flight cost no registers (so five CTAs fit an SM)
// and need no barrier.  Arithmetic is in packed fp32 pairs, without which the
// issue slots, not the memory, set the time.  A head's 128 channels are 16
// adjacent lanes, so its L2 norm is four shuffles.
//
// Tiles cut the flat token range, whatever sequences they meet, so that ragged
// batches need no host knowledge of cu_seqlens and leave no empty CTA.  The
// tile that holds a sequence's first token owns it: it alone reads the old
// conv state, writes the new one, and computes the first W - 1 tokens (which
// see the old state) even where they reach past the tile's end.  No other tile
// touches the pool entry, so the update in place needs no ordering between
// CTAs.
#include "kda_internal.h"
#include "ops_internal.h"

namespace kda {
namespace {

constexpr int kConvThreads = 128;
constexpr int kConvVec = 8;
constexpr int kStep = 4;            // tokens a copy group
constexpr int kRing = 4 * kStep;    // tokens in flight
constexpr int kTokenSeqs = 4;       // sequences a CTA of the single-token kernel takes

// z sigmoid(z) of 8 values.  Two values share one reciprocal (1/(ab) times b
// and a), which takes the special-function work from 2 to 1.5 operations a
// value; the exponent is clamped at 2^62 so that the product stays finite.
__device__ __forceinline__ void silu8(F2 (&z)[4]) {
    constexpr float kLog2e = 1.4426950408889634f;
    const F2 m = f2(-kLog2e, -kLog2e), one = f2(1.f, 1.f);
    F2 a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = f2_parts(f2_mul(z[i], m));
        a[i] = f2_add(f2(ex2_approx(fminf(u.x, 62.f)), ex2_approx(fminf(u.y, 62.f))), one);
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 ab = f2_parts(f2_mul(a[i], a[i + 1]));
        const F2 r = f2(rcp_approx(ab.x), rcp_approx(ab.y));
        z[i] = f2_mul(z[i], f2_mul(r, a[i + 1]));
        z[i + 1] = f2_mul(z[i + 1], f2_mul(r, a[i]));
    }
}

// A thread's channels: its weights by tap, bias, and the step from inputs to outputs.
template <typename T, int W, bool kWF32>
struct Channels {
    F2 w[W][4], bias[4];
    bool warp_norm, lane_norm;

    __device__ __forceinline__ Channels(const ConvParams& p, int c0, int cc) {
        warp_norm = c0 - (int)(threadIdx.x & 31) * kConvVec < p.norm_c;
        lane_norm = c0 < p.norm_c;
        float f[8 * W];
        if (kWF32) {
            const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + (int64_t)cc * W);
#pragma unroll
            for (int i = 0; i < 2 * W; ++i) {
                const float4 v = __ldg(src + i);
                f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
            }
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.w) + (int64_t)cc * W);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint4 v = __ldg(src + i);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x = Elem<T>::unpack(u[k]);
                    f[8 * i + 2 * k] = x.x;
                    f[8 * i + 2 * k + 1] = x.y;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = f2(f[2 * i * W + j], f[(2 * i + 1) * W + j]);
            bias[i] = f2(0.f, 0.f);
        }
        if (p.bias) {
            const float4 b0 = __ldg(reinterpret_cast<const float4*>(p.bias + cc)),
                         b1 = __ldg(reinterpret_cast<const float4*>(p.bias + cc + 4));
            bias[0] = f2(b0.x, b0.y); bias[1] = f2(b0.z, b0.w);
            bias[2] = f2(b1.x, b1.y); bias[3] = f2(b1.z, b1.w);
        }
    }
    // One output row from the window (oldest first) and the current input.
    __device__ __forceinline__ uint4 row(const ConvParams& p, const F2 (&win)[W - 1][4], const F2 (&x)[4]) const {
        F2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = f2_fma(w[W - 1][i], x[i], bias[i]);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) y[i] = f2_fma(w[j][i], win[j][i], y[i]);
        }
        if (p.silu) silu8(y);
        if (warp_norm) {
            F2 s2 = f2_mul(y[0], y[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) s2 = f2_fma(y[i], y[i], s2);
            const float2 s = f2_parts(s2);
            float ss = s.x + s.y;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = lane_norm ? rsqrt_approx(ss + p.eps) : 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = f2_mul(y[i], f2(r, r));
        }
        return pack8<T>(y);
    }
};

template <typename T, int W, bool kWF32>
__global__ void __launch_bounds__(kConvThreads, 5) short_conv_kernel(const ConvParams p) {
    __shared__ uint4 ring[kRing][kConvThreads];
    const int tid = threadIdx.x, c0 = (blockIdx.y * kConvThreads + tid) * kConvVec;
    if (c0 - (tid & 31) * kConvVec >= p.C) return;  // the whole warp is past the channels
    const bool act = c0 < p.C;
    const int cc = act ? c0 : 0;
    const Channels<T, W, kWF32> ch(p, c0, cc);

    const int total = (int)p.total;
    const int t0 = (int)blockIdx.x * p.tile, t1 = min(t0 + p.tile, total);
    const bool last = t1 == total;
    auto start = [&](int n) -> int { return p.cu ? p.cu[n] : n * p.T; };
    auto report = [&]() {
        if (p.status && tid == 0) atomicExch(p.status, 1);
    };
    if (p.cu && blockIdx.x == 0 && (p.cu[0] != 0 || p.cu[p.N] != total)) report();

    // first sequence that starts at or after t0, or the one that runs into it
    int n;
    if (p.cu) {
        int lo = 0, hi = p.N;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid] >= t0) hi = mid; else lo = mid + 1;
        }
        n = lo;
        if (n > 0 && (n == p.N || p.cu[n] > t0)) --n;
    } else {
        n = p.T > 0 ? t0 / p.T : 0;
    }

    for (; n < p.N; ++n) {
        const int s = start(n);
        if (s >= t1 && !(last && s == total)) break;
        const int e = start(n + 1), len = e - s;
        const int a = p.accepted ? p.accepted[n] : len;
        const int slot = p.slot ? p.slot[n] : n;
        if (s < 0 || len < 0 || e > total || a < 0 || a > len ||
            (p.pool && (slot < 0 || slot >= p.P))) {
            report();
            continue;
        }
        const T* xb = static_cast<const T*>(p.x) + (p.cu ? (int64_t)s * p.xs[1] : (int64_t)n * p.xs[0]) + cc;
        const bool owner = s >= t0;
        // tokens of this sequence that the tile computes
        const int tb = owner ? 0 : max(t0 - s, W - 1);
        const int te = p.out ? (owner ? min(len, max(t1 - s, W - 1)) : min(len, t1 - s)) : 0;
        const int64_t step = p.xs[1];
        const T* xf = xb + tb * step;                 // next token to ask for
        int left = te - tb;                           // tokens not yet asked for
        auto fetch = [&](uint4* rows) {               // kStep tokens into their rows of the ring
            if (left >= kStep) {
#pragma unroll
                for (int u = 0; u < kStep; ++u) {
                    cp_async16(rows + u * kConvThreads, xf);
                    xf += step;
                }
            } else {
#pragma unroll
                for (int u = 0; u < kStep - 1; ++u) {
                    if (u < left) cp_async16(rows + u * kConvThreads, xf);
                    xf += step;
                }
            }
            left -= kStep;
            cp_async_commit();
        };
        uint4* const mine = &ring[0][tid];
        constexpr int kGroup = kStep * kConvThreads;  // pieces of a copy group
#pragma unroll
        for (int g = 0; g < kRing / kStep - 1; ++g) fetch(mine + g * kGroup);
        F2 win[W - 1][4];
        if (owner) {
            uint4 old[W - 1];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) old[i] = make_uint4(0, 0, 0, 0);
            if (p.pool) {
                uint4* pool = reinterpret_cast<uint4*>(static_cast<T*>(p.pool) + (int64_t)slot * (W - 1) * p.C + cc);
                const int64_t row = p.C / kConvVec;
                if (!p.has_state || p.has_state[n] != 0) {
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) old[i] = pool[i * row];
                }
                // inputs a .. a + W - 2 of [old state, tokens]
#pragma unroll
                for (int i = 0; i < W - 1; ++i) {
                    uint4 r;
                    if (a + i >= W - 1) {
                        r = ldg16(xb + (int64_t)(a + i - (W - 1)) * p.xs[1]);
                    } else {
                        r = old[i];
#pragma unroll
                        for (int k = i + 1; k < W - 1; ++k)
                            if (a + i == k) r = old[k];
                    }
                    if (act) pool[i * row] = r;
                }
            }
#pragma unroll
            for (int i = 0; i < W - 1; ++i) unpack8<T>(old[i], win[i]);
        } else if (tb < te) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) unpack8<T>(ldg16(xb + (int64_t)(tb - (W - 1) + i) * p.xs[1]), win[i]);
        }
        T* o = static_cast<T*>(p.out) + (p.cu ? (int64_t)s * p.os[1] : (int64_t)n * p.os[0]) + tb * p.os[1] + cc;
        auto token = [&](const uint4* piece) {
            F2 x[4];
            unpack8<T>(*piece, x);
            const uint4 y = ch.row(p, win, x);
            if (act) *reinterpret_cast<uint4*>(o) = y;
            o += p.os[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
                win[W - 2][i] = x[i];
            }
        };
        int g = 0;
        int t = tb;
        for (; t + kStep <= te; t += kStep) {
            cp_async_wait<kRing / kStep - 2>();
            // the group that comes in goes to the rows that the last round emptied
            fetch(mine + ((g + kRing / kStep - 1) % (kRing / kStep)) * kGroup);
            const uint4* rows = mine + g * kGroup;
            g = (g + 1) % (kRing / kStep);
#pragma unroll
            for (int u = 0; u < kStep; ++u) token(rows + u * kConvThreads);
        }
        if (t < te) {
            cp_async_wait<0>();
            const uint4* rows = mine + g * kGroup;
            for (int u = 0; t + u < te; ++u) token(rows + u * kConvThreads);
        }
        cp_async_wait<0>();   // groups past the end hold nothing, but the next sequence counts anew
    }
}

// One token a sequence (decoding): the token, the old state and the new one
// are 2 W rows, all independent, so a thread has the loads of kTokenSeqs
// sequences in flight at once and its weights serve them all.
template <typename T, int W, bool kWF32>
__global__ void __launch_bounds__(kConvThreads) short_conv_token_kernel(const ConvParams p) {
    const int tid = threadIdx.x, c0 = (blockIdx.y * kConvThreads + tid) * kConvVec;
    if (c0 - (tid & 31) * kConvVec >= p.C) return;
    const bool act = c0 < p.C;
    const int cc = act ? c0 : 0;
    const int64_t row = p.C / kConvVec;
    uint4 raw[kTokenSeqs][W];
    uint4* pool[kTokenSeqs];
    int a[kTokenSeqs];
    bool ok[kTokenSeqs];
#pragma unroll
    for (int u = 0; u < kTokenSeqs; ++u) {
        const int n = blockIdx.x * kTokenSeqs + u;
        ok[u] = n < p.N;
        pool[u] = nullptr;
        a[u] = 1;
        if (!ok[u]) continue;
        const int slot = p.slot ? p.slot[n] : n;
        if (p.accepted) a[u] = p.accepted[n];
        if (a[u] < 0 || a[u] > 1 || (p.pool && (slot < 0 || slot >= p.P))) {
            if (p.status && tid == 0) atomicExch(p.status, 1);
            ok[u] = false;
            continue;
        }
        const bool keep = p.pool && (!p.has_state || p.has_state[n] != 0);
        if (p.pool) pool[u] = reinterpret_cast<uint4*>(static_cast<T*>(p.pool) + (int64_t)slot * (W - 1) * p.C + cc);
        raw[u][W - 1] = ldg16(static_cast<const T*>(p.x) + (int64_t)n * p.xs[0] + cc);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) raw[u][i] = keep ? pool[u][i * row] : make_uint4(0, 0, 0, 0);
    }
    const Channels<T, W, kWF32> ch(p, c0, cc);
#pragma unroll
    for (int u = 0; u < kTokenSeqs; ++u) {
        if (!ok[u]) continue;
        if (pool[u] && act) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) pool[u][i * row] = a[u] ? raw[u][i + 1] : raw[u][i];
        }
        if (!p.out) continue;
        F2 win[W - 1][4], x[4];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) unpack8<T>(raw[u][i], win[i]);
        unpack8<T>(raw[u][W - 1], x);
        const uint4 y = ch.row(p, win, x);
        const int64_t n = blockIdx.x * kTokenSeqs + u;
        if (act) *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + n * p.os[0] + cc) = y;
    }
}

template <typename T, int W, bool kWF32>
cudaError_t launch_conv_t(ConvParams& p, int num_sms, cudaStream_t s) {
    const unsigned cblocks = (unsigned)((p.C + kConvThreads * kConvVec - 1) / (kConvThreads * kConvVec));
    if (!p.cu && p.T == 1) {
        const dim3 grid((unsigned)((p.N + kTokenSeqs - 1) / kTokenSeqs), cblocks);
        short_conv_token_kernel<T, W, kWF32><<<grid, kConvThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    // The longest tile (at most 64 tokens) that still gives every SM eight CTAs.
    int tile = 64;
    while (tile > 1 && (p.total + tile - 1) / tile * cblocks < 8LL * num_sms) tile >>= 1;
    p.tile = tile;
    const int64_t tiles = p.total > 0 ? (p.total + tile - 1) / tile : 1;
    short_conv_kernel<T, W, kWF32><<<dim3((unsigned)tiles, cblocks), kConvThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int W>
cudaError_t launch_conv_w(ConvParams& p, bool w_f32, int num_sms, cudaStream_t s) {
    return w_f32 ? launch_conv_t<T, W, true>(p, num_sms, s) : launch_conv_t<T, W, false>(p, num_sms, s);
}
template <typename T>
cudaError_t launch_conv(ConvParams& p, int width, bool w_f32, int num_sms, cudaStream_t s) {
    switch (width) {
        case 2: return launch_conv_w<T, 2>(p, w_f32, num_sms, s);
        case 3: return launch_conv_w<T, 3>(p, w_f32, num_sms, s);
        default: return launch_conv_w<T, 4>(p, w_f32, num_sms, s);
    }
}

}  // namespace

cudaError_t launch_short_conv(const ConvParams& q, int width, bool f16, bool w_f32, int num_sms, cudaStream_t s) {
    ConvParams p = q;
    return f16 ? launch_conv<__half>(p, width, w_f32, num_sms, s)
               : launch_conv<__nv_bfloat16>(p, width, w_f32, num_sms, s);
}

}  // namespace kda
