// fno_causal_conv.h -- what the causal convolution's translation units share.
#pragma once

#include "fno_ops_internal.h"

struct fno_causal_conv_s {
    int64_t batch, length;
    int channels, width;
    fno_act_t act;
    fno_dtype_t dtype;
    uint32_t flags;
    int sms;
    int run;                   // tokens of a thread forward
    int bwd_run;               // and backward
    int parts;                 // of the weights' gradients
    size_t workspace;
};

namespace fno {
namespace conv {

using namespace ops;

constexpr int kThreads = 256;
// Blocks of the gradients' kernel on an SM: 3 (80 registers) up to 4 taps of 16-bit types and 3
// of float32, else 2, as more is spilled than the warps hide (4 taps, 4 x 4096 tokens of 2048
// channels, float32: 110 us, by 3 blocks 126; 4 x 8192 in bfloat16: 173 by 3, 208 by 2).
constexpr int grad_blocks(int width, int elem_bytes) {
    return width <= (elem_bytes == 4 ? 3 : 4) ? 3 : 2;
}

struct Args {
    const void *x, *s0, *dy, *dsT;
    const float *w, *bias;
    const int32_t *lengths;
    void *y, *sT, *dx, *ds0;
    float *part;               // per part: dw (width, channels), then dbias
    int64_t rows;              // runs of all sequences
    int length, channels, run, across, chunks;
    bool silu;
};

// v / (1 + e^-v) and its slope (fast quotient and exponential, 1e-6 for |v| up to 10)
__device__ __forceinline__ float silu(float v) {
    return v * rcp_fast(1.0f + exp2_fast(-kLog2e * v));
}
__device__ __forceinline__ float silu_slope(float v) {
    const float s = rcp_fast(1.0f + exp2_fast(-kLog2e * v));
    return s * fmaf(v, 1.0f - s, 1.0f);
}

// Input s of a sequence (s < 0: of its initial state).
template <typename T, bool WIDE, int W>
__device__ __forceinline__ float2 input(const Args &p, int64_t b, int s, int c, int left) {
    if (s >= 0)
        return to_float2(load_pair(
            static_cast<const T *>(p.x) + (b * p.length + s) * p.channels + c, WIDE, left));
    if (!p.s0) return f2(0.0f);
    return to_float2(load_pair(
        static_cast<const T *>(p.s0) + (b * (W - 1) + s + W - 1) * p.channels + c, WIDE, left));
}
__device__ __forceinline__ int tokens(const Args &p, int64_t b) {
    return p.lengths ? max(0, min(p.lengths[b], p.length)) : p.length;
}
// The weights (channels, W) of two channels, tap by tap.
template <int W>
__device__ __forceinline__ void load_weights(const Args &p, int c, int left, float2 (&w)[W],
                                             float2 &bias) {
    const float *from = p.w + (int64_t)c * W;
#pragma unroll
    for (int j = 0; j < W; ++j)
        w[j] = make_float2(left > 0 ? from[j] : 0.0f, left > 1 ? from[W + j] : 0.0f);
    bias = f2(0.0f);
    if (p.bias) bias = make_float2(left > 0 ? p.bias[c] : 0.0f, left > 1 ? p.bias[c + 1] : 0.0f);
}
// A pair as it was loaded.
template <typename T>
__device__ __forceinline__ void store_raw(T *p, const Pair<T> &v, bool wide, int left) {
    const T *e = reinterpret_cast<const T *>(&v);
    if (wide) *reinterpret_cast<Pair<T> *>(p) = v;
    else {
        p[0] = e[0];
        if (left > 1) p[1] = e[1];
    }
}
template <int W>
__device__ __forceinline__ float2 taps(const float2 (&w)[W], const float2 (&win)[W], float2 s) {
#pragma unroll
    for (int j = 0; j < W; ++j)
        s = make_float2(fmaf(w[j].x, win[j].x, s.x), fmaf(w[j].y, win[j].y, s.y));
    return s;
}

// A block: `across` threads over a chunk of the channels, the rest over runs.  Neighbouring
// blocks have neighbouring chunks, so that whole rows are read at about the same time (forward,
// 5 x 4099 tokens of 1001 channels in fp16, ragged: 34 us; 42 with neighbouring runs).
__device__ __forceinline__ int chunk(const Args &p) {
    return (int)(blockIdx.x % (unsigned)p.chunks);
}
__device__ __forceinline__ unsigned block(const Args &p) { return blockIdx.x / (unsigned)p.chunks; }
// Which run of which sequence:
struct Run {
    int64_t b;
    int t0, t1;
    __device__ Run(const Args &p, int64_t row) {
        const int runs = (p.length + p.run - 1) / p.run;
        b = row <= 0xffffffffll ? (int64_t)((uint32_t)row / (uint32_t)runs) : row / runs;
        t0 = (int)(row - b * runs) * p.run;
        t1 = min(t0 + p.run, p.length);
    }
};

// Calls f with the width as a constant.
template <class F>
fno_status_t with_width(int width, F &&f) {
    switch (width) {
        case 2: return f(std::integral_constant<int, 2>());
        case 3: return f(std::integral_constant<int, 3>());
        case 4: return f(std::integral_constant<int, 4>());
        case 5: return f(std::integral_constant<int, 5>());
        case 6: return f(std::integral_constant<int, 6>());
        case 7: return f(std::integral_constant<int, 7>());
        default: return f(std::integral_constant<int, 8>());
    }
}
// The gradients' passes (fno_causal_conv_bwd.cu).
fno_status_t gradients(const fno_causal_conv_s &p, const Args &a, float *dw, float *db,
                       cudaStream_t s);

}  // namespace conv
}  // namespace fno
