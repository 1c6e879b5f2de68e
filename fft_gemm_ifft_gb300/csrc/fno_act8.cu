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

// One warp per group of 128 elements, lane l on elements l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_act8_pack(const T *__restrict__ x, int8_t *__restrict__ codes, float *__restrict__ scales,
            int64_t cols, int64_t groups_per_row, int64_t groups) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t g = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); g < groups;
         g += step) {
        const int64_t row = g / groups_per_row, c0 = (g - row * groups_per_row) * kGroup;
        const int64_t base = row * cols + c0;
        const int n = (int)min((int64_t)kGroup, cols - c0);
        float v[4];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = lane + 32 * j;
            v[j] = e < n ? Storage<T>::load(x + base + e) : 0.0f;
            m = max(m, abs_bits(v[j]));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        const Group8 s = group8(m);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = lane + 32 * j;
            if (e < n) codes[base + e] = (int8_t)code8(v[j], s.inv);
        }
        if (lane == 0) scales[g] = s.scale;
    }
}

// Derivative of GELU: Phi(v) + v phi(v), the normal distribution and density.
__device__ __forceinline__ float gelu_slope(float v) {
    const float phi = 0.3989422804014327f * expf(-0.5f * v * v);
    return fmaf(v, phi, 0.5f * erfcf(-0.70710678118654752f * v));
}


// out = value, or dy * GELU'(value), element by element
template <typename T, bool GELU>
__global__ void __launch_bounds__(kThreads)
k_act8_read(const int8_t *__restrict__ codes, const float *__restrict__ scales, const T *dy,
            T *out, int64_t cols, int64_t groups_per_row, int64_t n) {
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
        const int64_t row = i / cols, c = i - row * cols;
        const float v = (float)codes[i] * scales[row * groups_per_row + c / kGroup];
        Storage<T>::store(out + i, GELU ? Storage<T>::load(dy + i) * gelu_slope(v) : v);
    }
}

fno_status_t check_shape(int64_t rows, int64_t cols, fno_dtype_t dtype) {
    if (rows < 1 || cols < 1 || !valid_dtype(dtype)) return FNO_ERR_INVALID_ARG;
    if ((double)rows * (double)cols > kMaxElems) return FNO_ERR_UNSUPPORTED;
    return FNO_OK;
}

int blocks_for(int64_t items, int64_t per_block) {
    const int64_t b = ceil_div(items, per_block);
    return (int)(b < 152 * 8 ? b : 152 * 8);
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
        k_act8_read<T, GELU><<<blocks_for(n, kThreads), kThreads, 0,
                               reinterpret_cast<cudaStream_t>(stream)>>>(
            codes, scales, static_cast<const T *>(dy), static_cast<T *>(out), cols, gpr, n);
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
        k_act8_pack<T><<<blocks_for(rows * gpr, kThreads / 32), kThreads, 0,
                         reinterpret_cast<cudaStream_t>(stream)>>>(
            static_cast<const T *>(x), codes, scales, cols, gpr, rows * gpr);
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
