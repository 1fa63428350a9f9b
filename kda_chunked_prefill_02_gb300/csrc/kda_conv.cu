// kda_conv.cu -- the short causal convolution in front of a KDA layer, with
// SiLU, the per-head L2 norm of the q and k channels and the conv-state pool
// (kda_short_conv in include/kda_ops.h; the conv caches that the TensorRT-LLM
// page "Kimi K3 work for Rubin (SM107)", Description, keeps beside the KDA
// states).
//
// y_t[c] = act(bias[c] + sum_j w[c][j] x_{t-W+1+j}[c]): every input is used W
// times and every output written once, so the kernel streams x once and is
// bound by HBM bandwidth (4 bytes an element).  Thread = 4 channels (8 bytes a
// token), walking down a tile of tokens with the last W - 1 inputs in fp32
// registers.  The tokens ahead come by 8-byte asynchronous copies into a ring
// of kRing rows in shared memory, of which every thread reads only what it
// copied itself: the loads in flight cost no registers and need no barrier.  A
// token is a chain of some 400 cycles (taps, exponential, reciprocal, the sum
// over the head), which other warps hide, and the issue slots leave some 85 cycles
// a warp and token at the memory's rate: so few channels a thread (many warps),
// packed fp32 pairs, and four tokens at a time, whose norms share one reduction
// and one root.  Measured, 32768 tokens of 12288 channels, bf16: 247 us, 6.5 TB/s
// (372 us with 8 channels a thread, plain fp32 and loads in registers; 292 us
// with everything but the four tokens' shared reduction and the folded log2 e).
// Drafts (256 sequences of 4 tokens of 12288 channels, accepted = 0): 22.1 us, their
// bytes 13.0; the commit alone 14.1.  A tile walks its seven or so short sequences
// one after the other.
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
constexpr int kConvVec = 4;         // channels a thread
constexpr int kPairs = kConvVec / 2;
using Piece = uint2;                // their elements
constexpr int kStep = 4;            // tokens a copy group
constexpr int kRing = 4 * kStep;    // tokens in flight
constexpr int kTokenSeqs = 2;       // sequences a CTA of the single-token kernel takes (256 of them: 9.7 us; 10.6 with 1, 11.7 with 4)

template <typename T>
__device__ __forceinline__ void unpack(const Piece& r, F2 (&f)[kPairs]) {
    const float2 a = Elem<T>::unpack(r.x), b = Elem<T>::unpack(r.y);
    f[0] = f2(a.x, a.y);
    f[1] = f2(b.x, b.y);
}
template <typename T>
__device__ __forceinline__ Piece pack(const F2 (&f)[kPairs]) {
    const float2 a = f2_parts(f[0]), b = f2_parts(f[1]);
    return make_uint2(Elem<T>::pack(a.x, a.y), Elem<T>::pack(b.x, b.y));
}
__device__ __forceinline__ Piece load(const void* p) { return __ldg(static_cast<const Piece*>(p)); }
__device__ __forceinline__ void copy_async(Piece* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;

// z sigmoid(z) of 4 values from u = z log2 e (the weights carry the factor):
// u / (log2 e + log2 e 2^-u); far below zero the denominator is infinite and the
// quotient 0.
__device__ __forceinline__ void silu(F2 (&u)[kPairs]) {
    const F2 l = f2(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const float2 v = f2_parts(u[i]);
        const float2 a = f2_parts(f2_fma(f2(ex2_approx(-v.x), ex2_approx(-v.y)), l, l));
        u[i] = f2_mul(u[i], f2(rcp_approx(a.x), rcp_approx(a.y)));
    }
}

// The sums of a[0..3] over the warp's 32 lanes, each to every lane as
// 1 / sqrt(sum + eps): two halving steps leave lane l with a quarter of the sum of
// value (l >> 3), so that one reduction and one root serve all four.
__device__ __forceinline__ void inverse_norms(float (&a)[4], float eps, int lane) {
    const bool h = lane & 16, q = lane & 8;
    const float b0 = (h ? a[2] : a[0]) + __shfl_xor_sync(0xffffffffu, h ? a[0] : a[2], 16);
    const float b1 = (h ? a[3] : a[1]) + __shfl_xor_sync(0xffffffffu, h ? a[1] : a[3], 16);
    float s = (q ? b1 : b0) + __shfl_xor_sync(0xffffffffu, q ? b0 : b1, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float r = rsqrt_approx(s + eps);
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = __shfl_sync(0xffffffffu, r, 8 * k);
}

// A thread's channels: its weights by tap, bias, and the step from inputs to outputs.
template <typename T, int W, bool kWF32>
struct Channels {
    F2 w[W][kPairs], bias[kPairs];
    bool warp_norm;   // a warp is a head

    __device__ __forceinline__ Channels(const ConvParams& p, int c0, int cc) {
        warp_norm = c0 < p.norm_c;
        const float factor = p.silu ? kLog2e : 1.f;   // see silu
        float f[kConvVec * W];
        if (kWF32) {
            const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + (int64_t)cc * W);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float4 v = __ldg(src + i);
                f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
            }
        } else {
            const uint2* src = reinterpret_cast<const uint2*>(static_cast<const T*>(p.w) + (int64_t)cc * W);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint2 v = __ldg(src + i);
                const float2 x = Elem<T>::unpack(v.x), y = Elem<T>::unpack(v.y);
                f[4 * i] = x.x; f[4 * i + 1] = x.y; f[4 * i + 2] = y.x; f[4 * i + 3] = y.y;
            }
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = f2(f[2 * i * W + j] * factor, f[(2 * i + 1) * W + j] * factor);
            bias[i] = f2(0.f, 0.f);
        }
        if (p.bias) {
            const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + cc));
            bias[0] = f2(b.x * factor, b.y * factor);
            bias[1] = f2(b.z * factor, b.w * factor);
        }
    }
    // The activation of one token from the window (oldest first) and the current input.
    __device__ __forceinline__ void taps(const ConvParams& p, const F2 (&win)[W - 1][kPairs], const F2 (&x)[kPairs],
                                         F2 (&y)[kPairs]) const {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            y[i] = f2_fma(w[W - 1][i], x[i], bias[i]);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) y[i] = f2_fma(w[j][i], win[j][i], y[i]);
        }
        if (p.silu) silu(y);
    }
    static __device__ __forceinline__ float squares(const F2 (&y)[kPairs]) {
        const float2 s = f2_parts(f2_fma(y[1], y[1], f2_mul(y[0], y[0])));
        return s.x + s.y;
    }
    static __device__ __forceinline__ void scale(F2 (&y)[kPairs], float r) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) y[i] = f2_mul(y[i], f2(r, r));
    }
    // One output row.
    __device__ __forceinline__ Piece row(const ConvParams& p, const F2 (&win)[W - 1][kPairs], const F2 (&x)[kPairs]) const {
        F2 y[kPairs];
        taps(p, win, x, y);
        if (warp_norm) {
            float ss = squares(y);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            scale(y, rsqrt_approx(ss + p.eps));
        }
        return pack<T>(y);
    }
};

template <typename T, int W>
__device__ __forceinline__ void shift(F2 (&win)[W - 1][kPairs], const F2 (&x)[kPairs]) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
#pragma unroll
        for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
        win[W - 2][i] = x[i];
    }
}

template <typename T, int W, bool kWF32>
__global__ void __launch_bounds__(kConvThreads) short_conv_kernel(const ConvParams p) {
    __shared__ Piece ring[kRing][kConvThreads];
    const int cb = blockIdx.x % p.cblocks, tile = blockIdx.x / p.cblocks;
    const int tid = threadIdx.x, c0 = (cb * kConvThreads + tid) * kConvVec;
    const int total = (int)p.total;
    if (p.cu && cb == 0 && p.status) {
        // Every pair of cu is looked at once: the tiles below search cu as a sorted
        // array, and need not meet the places where it is not.
        const int64_t step = (int64_t)(gridDim.x / p.cblocks) * kConvThreads;
        for (int64_t n = (int64_t)tile * kConvThreads + tid; n < p.N; n += step) {
            const int s = p.cu[n], e = p.cu[n + 1];
            if (s < 0 || e < s || e > total || (n == 0 && s != 0) || (n == p.N - 1 && e != total))
                atomicExch(p.status, 1);
        }
    }
    if (c0 - (tid & 31) * kConvVec >= p.C) return;  // the whole warp is past the channels
    const bool act = c0 < p.C;
    const int cc = act ? c0 : 0;
    const Channels<T, W, kWF32> ch(p, c0, cc);

    const int t0 = tile * p.tile, t1 = (int)min((unsigned)t0 + p.tile, (unsigned)total);   // total may be 2^31 - 1
    const bool last = t1 == total;
    auto start = [&](int n) -> int { return p.cu ? p.cu[n] : n * p.T; };
    auto report = [&]() {
        if (p.status && tid == 0) atomicExch(p.status, 1);
    };

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
        auto fetch = [&](Piece* rows) {               // kStep tokens into their rows of the ring
            if (left >= kStep) {
#pragma unroll
                for (int u = 0; u < kStep; ++u) {
                    copy_async(rows + u * kConvThreads, xf);
                    xf += step;
                }
            } else {
#pragma unroll
                for (int u = 0; u < kStep - 1; ++u) {
                    if (u < left) copy_async(rows + u * kConvThreads, xf);
                    xf += step;
                }
            }
            left -= kStep;
            cp_async_commit();
        };
        Piece* const mine = &ring[0][tid];
        constexpr int kGroup = kStep * kConvThreads;  // pieces of a copy group
#pragma unroll
        for (int g = 0; g < kRing / kStep - 1; ++g) fetch(mine + g * kGroup);
        F2 win[W - 1][kPairs];
        if (owner) {
            Piece old[W - 1];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) old[i] = make_uint2(0, 0);
            if (p.pool) {
                Piece* pool = reinterpret_cast<Piece*>(static_cast<T*>(p.pool) + (int64_t)slot * (W - 1) * p.C + cc);
                const int64_t row = p.C / kConvVec;
                if (!p.has_state || p.has_state[n] != 0) {
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) old[i] = pool[i * row];
                }
                // inputs a .. a + W - 2 of [old state, tokens]
#pragma unroll
                for (int i = 0; i < W - 1; ++i) {
                    Piece r;
                    if (a + i >= W - 1) {
                        r = load(xb + (int64_t)(a + i - (W - 1)) * p.xs[1]);
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
            for (int i = 0; i < W - 1; ++i) unpack<T>(old[i], win[i]);
        } else if (tb < te) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) unpack<T>(load(xb + (int64_t)(tb - (W - 1) + i) * p.xs[1]), win[i]);
        }
        T* o = static_cast<T*>(p.out) + (p.cu ? (int64_t)s * p.os[1] : (int64_t)n * p.os[0]) + tb * p.os[1] + cc;
        const int64_t ostep = p.os[1];
        int g = 0;
        int t = tb;
        for (const int last_step = te - kStep; t <= last_step; t += kStep) {   // te may be 2^31 - 1
            cp_async_wait<kRing / kStep - 2>();
            // the group that comes in goes to the rows that the last round emptied
            fetch(mine + ((g + kRing / kStep - 1) % (kRing / kStep)) * kGroup);
            const Piece* rows = mine + g * kGroup;
            g = (g + 1) % (kRing / kStep);
            F2 y[kStep][kPairs];
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                F2 x[kPairs];
                unpack<T>(rows[u * kConvThreads], x);
                ch.taps(p, win, x, y[u]);
                shift<T, W>(win, x);
            }
            if (ch.warp_norm) {
                float ss[kStep];
#pragma unroll
                for (int u = 0; u < kStep; ++u) ss[u] = ch.squares(y[u]);
                inverse_norms(ss, p.eps, tid & 31);
#pragma unroll
                for (int u = 0; u < kStep; ++u) ch.scale(y[u], ss[u]);
            }
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                if (act) *reinterpret_cast<Piece*>(o) = pack<T>(y[u]);
                o += ostep;
            }
        }
        if (t < te) {
            cp_async_wait<0>();
            const Piece* rows = mine + g * kGroup;
            for (; t < te; ++t, rows += kConvThreads, o += ostep) {
                F2 x[kPairs];
                unpack<T>(*rows, x);
                const Piece y = ch.row(p, win, x);
                if (act) *reinterpret_cast<Piece*>(o) = y;
                shift<T, W>(win, x);
            }
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
    Piece raw[kTokenSeqs][W];
    Piece* pool[kTokenSeqs];
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
        if (p.pool) pool[u] = reinterpret_cast<Piece*>(static_cast<T*>(p.pool) + (int64_t)slot * (W - 1) * p.C + cc);
        raw[u][W - 1] = load(static_cast<const T*>(p.x) + (int64_t)n * p.xs[0] + cc);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) raw[u][i] = keep ? pool[u][i * row] : make_uint2(0, 0);
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
        F2 win[W - 1][kPairs], x[kPairs];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) unpack<T>(raw[u][i], win[i]);
        unpack<T>(raw[u][W - 1], x);
        const Piece y = ch.row(p, win, x);
        const int64_t n = blockIdx.x * kTokenSeqs + u;
        if (act) *reinterpret_cast<Piece*>(static_cast<T*>(p.out) + n * p.os[0] + cc) = y;
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
    // Tiles of about 64 tokens (the W - 1 inputs before a tile are read twice), cut so
    // that the CTAs fill a whole number of the GPU's waves, where there is work for one.
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, short_conv_kernel<T, W, kWF32>, kConvThreads, 0);
    if (e != cudaSuccess) return e;
    const int64_t wave = (int64_t)num_sms * per_sm / cblocks;   // tiles a wave
    int64_t tile = 1;
    if (wave > 0) {
        const int64_t waves = (p.total + 64 * wave - 1) / (64 * wave);
        tile = waves > 0 ? (p.total + waves * wave - 1) / (waves * wave) : 1;
    } else if (p.total > 0) {
        tile = p.total < 64 ? p.total : 64;
    }
    p.tile = (int)tile;
    const int64_t tiles = p.total > 0 ? (p.total + tile - 1) / tile : 1;
    p.cblocks = (int)cblocks;
    short_conv_kernel<T, W, kWF32><<<(unsigned)(tiles * cblocks), kConvThreads, 0, s>>>(p);
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
