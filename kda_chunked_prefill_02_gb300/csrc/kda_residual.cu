// kda_residual.cu -- a block's output added to the residual stream, with its own norm,
// a gate and a scale, and the norm in front of the next block (kda_residual_norm in
// include/kda_ops.h).
//
//     u = y [/ rms(y) * post_weight] [* gate],   x' = x + alpha u,   h = x' / rms(x') * weight
//
// Every element is read and written once and takes part in two sums over its row, so the
// kernel is bound by HBM bandwidth: 2 bytes an element for each of y, x, the gate, x' and
// h (4 for x and x' in fp32).  A row is a CTA's (or, up to 512 elements, a warp's): all of
// its pieces are asked for before the first is used, 2 of 8 elements a thread, so that few
// registers hold a row and 2048 threads an SM keep some 100 KB on their way; sums, x'
// and both norms stay in fp32, and x' and h are rounded once, h from the unrounded x'.
// Measured (GPU time): 32768 tokens of 4096 with both norms and a gate 207 us (6.5 TB/s), 8191
// of 1288 in fp16 over an fp32 stream 23.7 us (6.2), one token of 2048 2.4 us (a launch and one
// chain of loads).  Rows of fewer than 256 channels leave lanes of their warp idle: the sum and the
// norm of 2^27 elements move 7.1 TB/s in rows of 512, 6.0 in rows of 256, 3.6 of 128, 1.9 of 64.
#include "kda_internal.h"
#include "ops_internal.h"

namespace kda {
namespace {

constexpr int kWarpRows = 4;      // rows a CTA where a row is one warp's

// 8 elements as pairs of fp32.
template <typename S> struct Raw { uint4 v; };
template <> struct Raw<float> { uint4 v, w; };
template <typename S>
__device__ __forceinline__ Raw<S> load_raw(const S* p) {
    Raw<S> r;
    r.v = ldg16(p);
    if constexpr (std::is_same<S, float>::value) r.w = ldg16(p + 4);
    return r;
}
template <typename S>
__device__ __forceinline__ void unpack_raw(const Raw<S>& r, F2 (&f)[4]) {
    if constexpr (std::is_same<S, float>::value) {
        f[0] = f2(__uint_as_float(r.v.x), __uint_as_float(r.v.y));
        f[1] = f2(__uint_as_float(r.v.z), __uint_as_float(r.v.w));
        f[2] = f2(__uint_as_float(r.w.x), __uint_as_float(r.w.y));
        f[3] = f2(__uint_as_float(r.w.z), __uint_as_float(r.w.w));
    } else {
        unpack8<S>(r.v, f);
    }
}
template <typename S>
__device__ __forceinline__ void store8(S* p, const F2 (&f)[4]) {
    if constexpr (std::is_same<S, float>::value) {
        float2 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = f2_parts(f[i]);
        reinterpret_cast<float4*>(p)[0] = make_float4(a[0].x, a[0].y, a[1].x, a[1].y);
        reinterpret_cast<float4*>(p)[1] = make_float4(a[2].x, a[2].y, a[3].x, a[3].y);
    } else {
        *reinterpret_cast<uint4*>(p) = pack8<S>(f);
    }
}
// 8 weights (ones where there are none).
template <typename T>
__device__ __forceinline__ void weights8(const void* w, bool f32, int at, F2 (&f)[4]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f2(1.f, 1.f);
    } else if (f32) {
        unpack_raw<float>(load_raw(static_cast<const float*>(w) + at), f);
    } else {
        unpack_raw<T>(load_raw(static_cast<const T*>(w) + at), f);
    }
}

// Sum over the threads of a row: a warp's, or (kBlock) the CTA's, by way of sh[32].
template <bool kBlock>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (kBlock) {
        const int warps = (int)blockDim.x / 32, lane = threadIdx.x & 31;
        if (lane == 0) sh[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? sh[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}
__device__ __forceinline__ float squares(const F2 (&f)[4]) {
    const float2 a = f2_parts(f2_add(f2_fma(f[0], f[0], f2_mul(f[1], f[1])), f2_fma(f[2], f[2], f2_mul(f[3], f[3]))));
    return a.x + a.y;
}

// T: type of y, gate and h; X: of the residual stream; N: pieces a thread.
template <typename T, typename X, int N, bool kBlock>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const ResidualParams p) {
    __shared__ float sh[2][32];
    const int lane = kBlock ? (int)threadIdx.x : (int)threadIdx.x & 31, step = kBlock ? (int)blockDim.x : 32;
    const int64_t row = kBlock ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5);
    if (row >= p.tokens) return;   // a whole warp's (a CTA's) row
    const int pieces = p.E / 8;
    const T* y = static_cast<const T*>(p.y);
    const T* gate = static_cast<const T*>(p.gate);
    Raw<X> rx[N];
    Raw<T> ry[N], rg[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = lane + i * step;
        if (c < pieces) {
            if (y) ry[i] = load_raw(y + row * p.ys + 8 * c);
            rx[i] = load_raw(static_cast<const X*>(p.x) + row * p.xs + 8 * c);
            if (gate) rg[i] = load_raw(gate + row * p.gs + 8 * c);
        }
    }
    const float inv_e = 1.f / (float)p.E;
    float post = 1.f;
    if (p.post) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + i * step < pieces) {
                F2 f[4];
                unpack_raw(ry[i], f);
                sum += squares(f);
            }
        post = rsqrt_approx(fmaf(row_sum<kBlock>(sum, sh[0]), inv_e, p.eps));
    }
    F2 x[N][4];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = lane + i * step;
        if (c >= pieces) continue;
        unpack_raw(rx[i], x[i]);
        if (y) {
            F2 u[4];
            unpack_raw(ry[i], u);
            if (p.post) {
                F2 w[4];
                weights8<T>(p.post_w, p.w_f32, 8 * c, w);
                const F2 r = f2(post, post);
#pragma unroll
                for (int k = 0; k < 4; ++k) u[k] = f2_mul(f2_mul(u[k], r), w[k]);
            }
            if (gate) {
                F2 g[4];
                unpack_raw(rg[i], g);
                if (p.sigmoid) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 z = f2_parts(g[k]);
                        g[k] = f2(rcp_approx(1.f + ex2_approx(z.x * -1.4426950408889634f)),
                                  rcp_approx(1.f + ex2_approx(z.y * -1.4426950408889634f)));
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) u[k] = f2_mul(u[k], g[k]);
            }
            const F2 a = f2(p.alpha, p.alpha);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][k] = f2_fma(u[k], a, x[i][k]);
            if (p.x_out) store8(static_cast<X*>(p.x_out) + row * p.xos + 8 * c, x[i]);
        }
        sum += squares(x[i]);
    }
    if (!p.out) return;
    const float r = rsqrt_approx(fmaf(row_sum<kBlock>(sum, sh[1]), inv_e, p.eps));
    const F2 r2 = f2(r, r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = lane + i * step;
        if (c >= pieces) continue;
        F2 w[4];
        weights8<T>(p.w, p.w_f32, 8 * c, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i][k] = f2_mul(f2_mul(x[i][k], r2), w[k]);
        store8(static_cast<T*>(p.out) + row * p.os + 8 * c, x[i]);
    }
}

template <typename T, typename X>
cudaError_t launch_t(const ResidualParams& p, cudaStream_t s) {
    const int pieces = p.E / 8;
    if (pieces <= 64) {
        const unsigned grid = (unsigned)((p.tokens + kWarpRows - 1) / kWarpRows);
        residual_norm_kernel<T, X, 2, false><<<grid, 32 * kWarpRows, 0, s>>>(p);
    } else {
        residual_norm_kernel<T, X, 2, true><<<(unsigned)p.tokens, (unsigned)((pieces + 63) / 64 * 32), 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualParams& p, bool f16, bool x_f32, cudaStream_t s) {
    if (f16) return x_f32 ? launch_t<__half, float>(p, s) : launch_t<__half, __half>(p, s);
    return x_f32 ? launch_t<__nv_bfloat16, float>(p, s) : launch_t<__nv_bfloat16, __nv_bfloat16>(p, s);
}

}  // namespace kda
