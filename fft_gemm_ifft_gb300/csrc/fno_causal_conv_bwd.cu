// fno_causal_conv_bwd.cu -- the causal convolution's gradients.
#include "fno_causal_conv.h"

using namespace fno;
using namespace fno::conv;

namespace {

// Gradients.  Token t's pre-activation gets g_t = dy_t act'(pre_t), worked out from the
// inputs again; then dx_s = sum_j w_j g_{s + W - 1 - j}, for which a run goes on W - 1
// tokens, and dw_j = sum_t g_t x_{t - W + 1 + j}.  A block takes every `parts`-th group of
// runs and leaves one sum of its dw and dbias.  Neighbouring blocks have neighbouring channels
// (4 x 8192 tokens of 2048 channels in bfloat16: 175 us; 198 with neighbouring runs), but runs
// where rows are odd and read by elements (5 x 4099 tokens of 1001 channels in fp16, ragged:
// 51 us, the kernel 45; 56 with neighbouring channels.  Without ragged ends it is the other way
// round: 75 and 73 us; 4 x 8192 of 2047 in bfloat16: 235 and 202; 8 x 2048 of 4095 in float32:
// 237 and 212).
//
// Far from its bytes (59 us for these 2048 channels): x and dy of 4 tokens in registers are 24 KB
// an SM on their way, of 2 tokens above 4 taps 8 KB (8 taps in fp16: 323 us).
template <typename T, bool WIDE, int W>
__global__ void __launch_bounds__(kThreads, grad_blocks(W, sizeof(T)))
k_conv_grad(const Args p) {
    __shared__ float2 sums[kThreads];
    constexpr int U = W <= 4 ? 4 : 2;          // tokens whose loads are on their way
    const int lane = threadIdx.x % p.across, down = kThreads / p.across;
    const int rank = threadIdx.x / p.across;
    const int c = ((int)(WIDE ? blockIdx.x : blockIdx.y) * p.across + lane) * 2;
    const int left = p.channels - c;
    float2 w[W], bias, dw[W], db = f2(0.0f);
    load_weights<W>(p, c, left, w, bias);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j] = f2(0.0f);
    for (int64_t row = (int64_t)(WIDE ? blockIdx.y : blockIdx.x) * down + rank;
         left > 0 && row < p.rows;
         row += (int64_t)(WIDE ? gridDim.y : gridDim.x) * down) {
        const Run r(p, row);
        const int n = tokens(p, r.b), t0 = r.t0, t1 = r.t1;
        // win: inputs t - W + 1 .. t; acc: the gradients of these inputs so far
        float2 win[W], acc[W];
        const int64_t at = (r.b * p.length + t0) * p.channels + c;
        const int end = min(t1 + W - 1, n);                // tokens that reach the run's inputs
        // gradients that come from the final state: input n - W + 1 + j has state j
        const auto from_state = [&](int s) {
            const int j = s - n + W - 1;
            if (!p.dsT || s >= n || j < 0) return f2(0.0f);
            return to_float2(load_pair(static_cast<const T *>(p.dsT) +
                                           (r.b * (W - 1) + j) * p.channels + c, WIDE, left));
        };
        T *const dx = static_cast<T *>(p.dx) + at;
        const auto finish = [&](int s, float2 v) {             // input s is complete
            if (s >= t0 && s < t1)
                store_pair(dx + (int64_t)(s - t0) * p.channels, v, WIDE, left);
            else if (s < 0 && t0 == 0 && p.ds0)
                store_pair(static_cast<T *>(p.ds0) + (r.b * (W - 1) + s + W - 1) * p.channels + c,
                           v, WIDE, left);
        };
        const T *x = static_cast<const T *>(p.x) + at, *dy = static_cast<const T *>(p.dy) + at;
        Pair<T> xn[U], gn[U];
        const auto fetch = [&](int t) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                xn[k] = load_pair(x, WIDE, t + k < end ? left : 0);
                gn[k] = load_pair(dy, WIDE, t + k < end ? left : 0);
                x += p.channels;
                dy += p.channels;
            }
        };
        if (t0 < n || t0 == 0) {
            if (t0 < end) fetch(t0);
#pragma unroll
            for (int j = 1; j < W; ++j) {
                win[j] = input<T, WIDE, W>(p, r.b, t0 - W + j, c, left);
                acc[j] = from_state(t0 - W + j);
            }
        }
        for (int t = t0; t < end; t += U) {
            Pair<T> xin[U], gin[U];
#pragma unroll
            for (int k = 0; k < U; ++k) xin[k] = xn[k], gin[k] = gn[k];
            if (t + U < end) fetch(t + U);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (t + k >= end) break;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1], acc[j] = acc[j + 1];
                win[W - 1] = to_float2(xin[k]);
                acc[W - 1] = from_state(t + k);
                float2 g = to_float2(gin[k]);
                if (p.silu) {
                    const float2 s = taps<W>(w, win, bias);
                    g = make_float2(g.x * silu_slope(s.x), g.y * silu_slope(s.y));
                }
#pragma unroll
                for (int j = 0; j < W; ++j)
                    acc[j] = make_float2(fmaf(w[j].x, g.x, acc[j].x), fmaf(w[j].y, g.y, acc[j].y));
                if (t + k < t1) {
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        dw[j] = make_float2(fmaf(g.x, win[j].x, dw[j].x),
                                            fmaf(g.y, win[j].y, dw[j].y));
                    db = add2(db, g);
                }
                finish(t + k - W + 1, acc[0]);
            }
        }
        // what the last tokens leave: inputs end - W + 1 .. end - 1 (those in front of the
        // first token where the sequence has none)
        if (t0 < n || t0 == 0) {
            const int e = max(end, t0);
#pragma unroll
            for (int j = 1; j < W; ++j) finish(e - W + j, acc[j]);
        }
        for (int s = max(t0, n); s < t1; ++s)
            store_pair(dx + (int64_t)(s - t0) * p.channels, f2(0.0f), WIDE, left);
    }
    float *out = p.part + (int64_t)(WIDE ? blockIdx.y : blockIdx.x) * (W + 1) * p.channels;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
        sums[threadIdx.x] = j < W ? dw[j < W ? j : 0] : db;
        __syncthreads();
        if (rank == 0) {
            float2 v = sums[lane];
            for (int k = 1; k < down; ++k) v = add2(v, sums[k * p.across + lane]);
            if (left > 0) out[(int64_t)j * p.channels + c] = v.x;
            if (left > 1) out[(int64_t)j * p.channels + c + 1] = v.y;
        }
    }
}

// dw (channels, width) and dbias: the sums of the parts.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows)
k_conv_sum(const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ db,
           int channels, int width, int parts) {
    __shared__ float s[kSumRows][33];
    const int64_t n = (int64_t)channels * (width + 1);
    const int64_t i = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float v = 0.0f;
    if (i < n) {
#pragma unroll 8
        for (int k = threadIdx.y; k < parts; k += kSumRows) v += part[k * n + i];
    }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y || i >= n) return;
    for (int k = 1; k < kSumRows; ++k) v += s[k][threadIdx.x];
    const int64_t j = i / channels, c = i - j * channels;
    if (j < width) dw[c * width + j] = v;
    else if (db) db[c] = v;
}

}  // namespace

namespace fno {
namespace conv {

fno_status_t gradients(const fno_causal_conv_s &p, const Args &a, float *dw, float *db,
                       cudaStream_t s) {
    const dim3 grid = p.channels % 2 ? dim3((unsigned)p.parts, (unsigned)a.chunks)
                                     : dim3((unsigned)a.chunks, (unsigned)p.parts);
    return with_storage(p.dtype, [&](auto t) {
        using T = decltype(t);
        return with_width(p.width, [&](auto width) {
            constexpr int W = decltype(width)::value;
            if (p.channels % 2) k_conv_grad<T, false, W><<<grid, kThreads, 0, s>>>(a);
            else k_conv_grad<T, true, W><<<grid, kThreads, 0, s>>>(a);
            const int64_t outs = (int64_t)p.channels * (W + 1);
            k_conv_sum<<<(unsigned)ceil_div(outs, 32), dim3(32, kSumRows), 0, s>>>(
                a.part, dw, db, p.channels, W, p.parts);
            return launched();
        });
    });
}

}  // namespace conv
}  // namespace fno
