// fno_act8.cu -- activation checkpoints in 8 bits: pack, unpack, and GELU's
// backward from a checkpoint.
//
// A checkpoint halves (16-bit) or quarters (float32) what a training step
// keeps between forward and backward; all three calls read and write each
// element once and are bound by memory bandwidth.
#include "fno_ops_internal.h"

using namespace fno;
using namespace fno::ops;

namespace {

constexpr int kThreads = 256;

// Both pack kernels are bound by bytes.  Rows whose length is a multiple of a
// 16-byte load: 128 / kVec lanes hold a
// group, each one load of it, so a warp packs 1 (float32) or 2 groups a step,
// and takes four steps' loads before the first is used.
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_act8_pack(const T *__restrict__ x, int8_t *__restrict__ codes, float *__restrict__ scales,
            int64_t cols, int64_t groups_per_row, int64_t groups) {
    constexpr int V = kVec<T>, L = kGroup / V, N = 32 / L, U = 4;
    const int lane = threadIdx.x & 31, sub = lane / L, off = (lane % L) * V;
    const uint32_t mask = L == 32 ? 0xffffffffu : 0xffffu << (16 * sub);
    const int64_t first = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * (N * U);
    Pack<T, V> d[U];
    int64_t at[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t g = first + k * N + sub, row = g / groups_per_row;
        const int64_t c = (g - row * groups_per_row) * kGroup + off;
        at[k] = g < groups && c < cols ? row * cols + c : -1;
        if (at[k] >= 0) d[k] = *reinterpret_cast<const Pack<T, V> *>(x + at[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        float v[V];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = at[k] >= 0 ? Storage<T>::load(&d[k].v[i]) : 0.0f;
            m = max(m, abs_bits(v[i]));
        }
        m = __reduce_max_sync(mask, m);
        const Group8 s = group8(m);
        Pack<int8_t, V> q;
#pragma unroll
        for (int i = 0; i < V; ++i) q.v[i] = (int8_t)code8(v[i], s.inv);
        if (at[k] >= 0) {
            *reinterpret_cast<Pack<int8_t, V> *>(codes + at[k]) = q;
            if (off == 0) scales[first + k * N + sub] = s.scale;
        }
    }
}

// Rows of any length: consecutive groups are consecutive in memory, so a CTA
// brings 32 groups in by aligned 16-byte loads of the range that they cover,
// packs them from shared memory, and writes the codes back by aligned 16-byte
// stores (single bytes at the two ends).
constexpr int kStage = 32;    // groups

template <typename T>
__global__ void __launch_bounds__(kThreads)
k_act8_pack_any(const T *__restrict__ x, int8_t *__restrict__ codes, float *__restrict__ scales,
                int64_t cols, int64_t groups_per_row, int64_t groups, int64_t n) {
    constexpr int V = kVec<T>;
    __shared__ alignas(16) T sx[kStage * kGroup + V];
    __shared__ alignas(16) int8_t sq[kStage * kGroup + 16];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t g0 = (int64_t)blockIdx.x * kStage, g1 = min(groups, g0 + kStage);
    const auto start = [&](int64_t g) {
        const int64_t row = g / groups_per_row;
        return row * cols + (g - row * groups_per_row) * kGroup;
    };
    const int64_t e0 = start(g0), e1 = start(g1);      // elements (start(groups) = n)
    const int64_t a0 = e0 / V * V;
    for (int64_t e = a0 + (int64_t)threadIdx.x * V; e < e1; e += (int64_t)kThreads * V) {
        if (e + V <= n) {
            *reinterpret_cast<Pack<T, V> *>(sx + (e - a0)) =
                *reinterpret_cast<const Pack<T, V> *>(x + e);
        } else {
            for (int i = 0; i < V && e + i < n; ++i) sx[e - a0 + i] = x[e + i];
        }
    }
    __syncthreads();
    const int64_t c0 = e0 / 16 * 16;                   // the codes' 16-byte window
#pragma unroll
    for (int k = 0; k < kStage / 8; ++k) {
        const int64_t g = g0 + w + 8 * k;
        if (g >= g1) break;
        const int64_t b = start(g);
        const int len = (int)(start(g + 1) - b);
        const T *src = sx + (b - a0);
        float v[4];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = lane + 32 * j < len ? Storage<T>::load(src + lane + 32 * j) : 0.0f;
            m = max(m, abs_bits(v[j]));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        const Group8 s = group8(m);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (lane + 32 * j < len) sq[b - c0 + lane + 32 * j] = (int8_t)code8(v[j], s.inv);
        if (lane == 0) scales[g] = s.scale;
    }
    __syncthreads();
    for (int64_t e = c0 + (int64_t)threadIdx.x * 16; e < e1; e += (int64_t)kThreads * 16) {
        if (e >= e0 && e + 16 <= e1) {
            *reinterpret_cast<uint4 *>(codes + e) = *reinterpret_cast<uint4 *>(sq + (e - c0));
        } else {
            for (int i = 0; i < 16; ++i)
                if (e + i >= e0 && e + i < e1) codes[e + i] = sq[e - c0 + i];
        }
    }
}

// Derivative of GELU: Phi(v) + v phi(v), the normal distribution and density.
// 1 - erf is Abramowitz & Stegun 7.1.26, poly(t) e^{-x^2} with x = |v| / sqrt 2
// (absolute error 1.5e-7, as in fno_gelu.cuh), whose exponential is also the
// density's: one exponential and one reciprocal an element, where erfcf and
// expf would make the arithmetic cost more than the bytes.  Two elements at a
// time: 15 instructions an element.
__device__ __forceinline__ float2 gelu_slope2(float2 v) {
    constexpr float p = 0.3275911f * 0.70710678118654752f;
    constexpr float a1 = 0.254829592f, a2 = -0.284496736f, a3 = 1.421413741f,
                    a4 = -1.453152027f, a5 = 1.061405429f;
    const float2 d = fma2(f2(p), make_float2(fabsf(v.x), fabsf(v.y)), f2(1.0f));
    const float2 t = make_float2(__fdividef(1.0f, d.x), __fdividef(1.0f, d.y));
    const float2 w = mul2(mul2(v, v), f2(-0.5f));
    const float2 e = make_float2(__expf(w.x), __expf(w.y));
    float2 q = fma2(t, f2(a5), f2(a4));
    q = fma2(t, q, f2(a3));
    q = fma2(t, q, f2(a2));
    q = fma2(t, q, f2(a1));
    // Phi(-|v|) = q t e / 2, and Phi(v) = 1/2 + sign(v) (1/2 - Phi(-|v|))
    const float2 r = fma2(mul2(mul2(q, t), e), f2(-0.5f), f2(0.5f));
    const float2 phi = add2(make_float2(copysignf(r.x, v.x), copysignf(r.y, v.y)), f2(0.5f));
    return fma2(mul2(v, f2(0.3989422804014327f)), e, phi);
}
// of a pair's values and gradients, or the values themselves
template <bool GELU>
__device__ __forceinline__ float2 result2(float2 v, float2 dy) {
    return GELU ? mul2(dy, gelu_slope2(v)) : v;
}

// the scale of the element after column c
template <typename I>
__device__ __forceinline__ float step_scale(const float *scales, I cols, I &c, I &at, float s) {
    ++c;
    if (c == cols) {
        c = 0;
        return scales[++at];           // a row's first group follows the last row's last
    }
    return c % kGroup == 0 ? scales[++at] : s;
}

// out = value, or dy * GELU'(value).  The tensors are walked as flat arrays by
// 16-byte vectors of the storage type whatever the row length; a vector that
// crosses a group's or a row's end looks its scales up one by one.  I: 32 bits
// where the element count allows (the division by the row length is the
// largest part of the index arithmetic).  GELU of 2048 x 65536: float32 at the copy
// rate (6.7 TB/s), fp16 141 us (4.8 TB/s; 640 us element by element with erfcf).
template <typename T, bool GELU, typename I>
__global__ void __launch_bounds__(kThreads)
k_act8_read(const int8_t *__restrict__ codes, const float *__restrict__ scales, const T *dy,
            T *out, I cols, I groups_per_row, I n) {
    constexpr int V = kVec<T>, U = 2;
    const I block = (I)blockIdx.x * (kThreads * V * U);
    Pack<int8_t, V> q[U];
    Pack<T, V> d[U];
    I first[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        first[k] = block + (I)(k * kThreads + threadIdx.x) * V;
        if (first[k] < n && n - first[k] >= V) {
            q[k] = *reinterpret_cast<const Pack<int8_t, V> *>(codes + first[k]);
            if (GELU) d[k] = *reinterpret_cast<const Pack<T, V> *>(dy + first[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (first[k] >= n) continue;
        const I row = first[k] / cols, col = first[k] - row * cols;
        const bool one = cols - col >= V && col % kGroup <= kGroup - V;
        I at = row * groups_per_row + col / kGroup;
        if (n - first[k] >= V) {
            float f[V];
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                uint32_t u;
                memcpy(&u, &q[k].v[i], 4);
                code_values4(u, f + i);
            }
            float s = scales[at], t = s;
            I c = col;
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                if (!one) {                    // scales element by element
                    if (i > 0) s = step_scale(scales, cols, c, at, s);
                    t = step_scale(scales, cols, c, at, s);
                }
                const float2 v = mul2(make_float2(f[i], f[i + 1]), make_float2(s, t));
                const float2 dv = GELU ? make_float2(Storage<T>::load(&d[k].v[i]),
                                                     Storage<T>::load(&d[k].v[i + 1]))
                                       : v;
                const float2 r = result2<GELU>(v, dv);
                Storage<T>::store(&d[k].v[i], r.x);
                Storage<T>::store(&d[k].v[i + 1], r.y);
                s = t;
            }
            *reinterpret_cast<Pack<T, V> *>(out + first[k]) = d[k];
        } else {
            float s = scales[at];
            I c = col;
            for (int i = 0; (I)i < n - first[k]; ++i) {
                if (i > 0) s = step_scale(scales, cols, c, at, s);
                const float v = (float)codes[first[k] + i] * s;
                const float dv = GELU ? Storage<T>::load(dy + first[k] + i) : v;
                Storage<T>::store(out + first[k] + i, result2<GELU>(f2(v), f2(dv)).x);
            }
        }
    }
}

fno_status_t check_shape(int64_t rows, int64_t cols, fno_dtype_t dtype) {
    if (rows < 1 || cols < 1 || !valid_dtype(dtype)) return FNO_ERR_INVALID_ARG;
    // (the second: a grid of 32 groups a block)
    if ((double)rows * (double)cols > kMaxElems ||
        (double)rows * (double)ceil_div(cols, kGroup) > 32.0 * 2147483647.0)
        return FNO_ERR_UNSUPPORTED;
    return FNO_OK;
}

template <bool GELU>
fno_status_t read_call(int64_t rows, int64_t cols, fno_dtype_t dtype, const int8_t *codes,
                       const float *scales, const void *dy, void *out, fno_stream_t stream) {
    fno_status_t st = check_shape(rows, cols, dtype);
    if (st != FNO_OK) return st;
    if (!codes || !scales || !out || (GELU && !dy)) return FNO_ERR_INVALID_ARG;
    const int64_t n = rows * cols, gpr = ceil_div(cols, kGroup);
    const size_t xb = (size_t)n * elem_bytes(dtype);
    st = check_operands({{codes, (size_t)n, false}, {scales, (size_t)(rows * gpr) * 4, false},
                         {dy, xb, false}, {out, xb, true, dy}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    with_storage(dtype, [&](auto t) {
        using T = decltype(t);
        const unsigned blocks = (unsigned)ceil_div(n, (int64_t)kThreads * kVec<T> * 2);
        const auto launch = [&](auto i) {
            using I = decltype(i);
            k_act8_read<T, GELU, I><<<blocks, kThreads, 0,
                                      reinterpret_cast<cudaStream_t>(stream)>>>(
                codes, scales, static_cast<const T *>(dy), static_cast<T *>(out), (I)cols, (I)gpr,
                (I)n);
        };
        // a block's first element may lie a block beyond n
        if (n < (int64_t)1 << 31) launch(uint32_t());
        else launch(uint64_t());
    });
    return launched();
}

}  // namespace

extern "C" {

fno_status_t fno_act8_pack(int64_t rows, int64_t cols, fno_dtype_t dtype, const void *x,
                           int8_t *codes, float *scales, fno_stream_t stream) {
    fno_status_t st = check_shape(rows, cols, dtype);
    if (st != FNO_OK) return st;
    if (!x || !codes || !scales) return FNO_ERR_INVALID_ARG;
    const int64_t n = rows * cols, gpr = ceil_div(cols, kGroup);
    st = check_operands({{x, (size_t)n * elem_bytes(dtype), false}, {codes, (size_t)n, true},
                         {scales, (size_t)(rows * gpr) * 4, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    with_storage(dtype, [&](auto t) {
        using T = decltype(t);
        cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
        const int64_t groups = rows * gpr;
        if (cols % kVec<T> == 0) {
            const int64_t per = (kThreads / 32) * 4 * (kVec<T> * 32 / kGroup);
            k_act8_pack<T><<<(unsigned)ceil_div(groups, per), kThreads, 0, cs>>>(
                static_cast<const T *>(x), codes, scales, cols, gpr, groups);
        } else {
            k_act8_pack_any<T><<<(unsigned)ceil_div(groups, kStage), kThreads, 0, cs>>>(
                static_cast<const T *>(x), codes, scales, cols, gpr, groups, n);
        }
    });
    return launched();
}

fno_status_t fno_act8_unpack(int64_t rows, int64_t cols, fno_dtype_t dtype, const int8_t *codes,
                             const float *scales, void *x, fno_stream_t stream) {
    return read_call<false>(rows, cols, dtype, codes, scales, nullptr, x, stream);
}

fno_status_t fno_act8_gelu_backward(int64_t rows, int64_t cols, fno_dtype_t dtype,
                                    const int8_t *codes, const float *scales, const void *dy,
                                    void *dx, fno_stream_t stream) {
    return read_call<true>(rows, cols, dtype, codes, scales, dy, dx, stream);
}

}  // extern "C"
