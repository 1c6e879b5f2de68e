// fno_causal_conv.cu -- short causal convolutions of every channel along time, with their
// activation: whole sequences, gradients, single tokens.
//
// 2 width multiply-adds an element: bound by bytes.  A thread takes two channels (one, where
// their number is odd) of a run of tokens with the last inputs in registers, so that an input
// is loaded once and the width - 1 in front of a run once more.  Two channels and no more:
// the weights, the window and eight tokens' loads then take few enough registers for the
// warps that keep enough loads on their way.
#include "fno_ops_internal.h"

using namespace fno;
using namespace fno::ops;

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

namespace {

constexpr int kThreads = 256;

struct Args {
    const void *x, *s0, *dy, *dsT;
    const float *w, *bias;
    const int32_t *lengths;
    void *y, *sT, *dx, *ds0;
    float *part;               // per part: dw (width, channels), then dbias
    int64_t rows;              // runs of all sequences
    int length, channels, run, across;
    bool silu;
};

// v / (1 + e^-v) and its slope (fast quotient and exponential, 1e-6 for |v| up to 10)
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }
__device__ __forceinline__ float silu_slope(float v) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-v));
    return s * fmaf(v, 1.0f - s, 1.0f);
}

template <typename T, int V>
__device__ __forceinline__ void load(const T *p, float *v) {
    const Pack<T, V> a = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = Storage<T>::load(&a.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float *v) {
    Pack<T, V> a;
#pragma unroll
    for (int i = 0; i < V; ++i) Storage<T>::store(&a.v[i], v[i]);
    *reinterpret_cast<Pack<T, V> *>(p) = a;
}

// Input s of a sequence (s < 0: of its initial state).
template <typename T, int V, int W>
__device__ __forceinline__ void input(const Args &p, int64_t b, int s, int c, float *v) {
    if (s >= 0) {
        load<T, V>(static_cast<const T *>(p.x) + (b * p.length + s) * p.channels + c, v);
    } else if (p.s0) {
        load<T, V>(static_cast<const T *>(p.s0) + (b * (W - 1) + s + W - 1) * p.channels + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
    }
}
__device__ __forceinline__ int tokens(const Args &p, int64_t b) {
    return p.lengths ? max(0, min(p.lengths[b], p.length)) : p.length;
}
// The weights (channels, W) of V channels, tap by tap.
template <int V, int W>
__device__ __forceinline__ void load_weights(const Args &p, int c, float (&w)[W][V],
                                             float (&bias)[V]) {
    float flat[V * W];
    const float *from = p.w + (int64_t)c * W;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        const Pack<float, V> a = *reinterpret_cast<const Pack<float, V> *>(from + k * V);
#pragma unroll
        for (int i = 0; i < V; ++i) flat[k * V + i] = a.v[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = flat[i * W + j];
        bias[i] = p.bias ? p.bias[c + i] : 0.0f;
    }
}
// A block: `across` threads over channels (all blockIdx.y make), the rest over runs.  Which
// run of which sequence:
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

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
k_conv(const Args p) {
    constexpr int U = 8;                       // tokens whose loads are in flight
    const int lane = threadIdx.x % p.across, rank = threadIdx.x / p.across;
    const int c = (blockIdx.y * p.across + lane) * V;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / p.across) + rank;
    if (row >= p.rows || c >= p.channels) return;
    const Run r(p, row);
    const int n = tokens(p, r.b), end = min(r.t1, n);
    float w[W][V], bias[V], win[W - 1][V];     // win: the inputs in front, oldest first
    load_weights<V, W>(p, c, w, bias);
    const int64_t at = (r.b * p.length + r.t0) * p.channels + c;
    T *y = static_cast<T *>(p.y) + at;
    const T *x = static_cast<const T *>(p.x) + at;
    if (r.t0 < end) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input<T, V, W>(p, r.b, r.t0 - (W - 1) + j, c, win[j]);
    }
    for (int t = r.t0; t < end; t += U) {
        Pack<T, V> in[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (t + k < end)
                in[k] = *reinterpret_cast<const Pack<T, V> *>(x + (int64_t)k * p.channels);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (t + k >= end) break;
            float v[V], o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = Storage<T>::load(&in[k].v[i]);
                float s = bias[i];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][i], win[j][i], s);
                s = fmaf(w[W - 1][i], v[i], s);
                o[i] = p.silu ? silu(s) : s;
#pragma unroll
                for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
                win[W - 2][i] = v[i];
            }
            store<T, V>(y, o);
            y += p.channels;
        }
        x += (int64_t)U * p.channels;
    }
    const float zero[V] = {};
    y = static_cast<T *>(p.y) + at;
    for (int t = max(r.t0, end); t < r.t1; ++t)
        store<T, V>(y + (int64_t)(t - r.t0) * p.channels, zero);
    if (p.sT && r.t0 == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float v[V];
            input<T, V, W>(p, r.b, n - (W - 1) + j, c, v);
            store<T, V>(static_cast<T *>(p.sT) + (r.b * (W - 1) + j) * p.channels + c, v);
        }
    }
}

// Gradients.  Token t's pre-activation gets g_t = dy_t act'(pre_t), worked out from the
// inputs again; then dx_s = sum_j w_j g_{s + W - 1 - j}, for which a run goes on W - 1
// tokens, and dw_j = sum_t g_t x_{t - W + 1 + j}.  A block takes every gridDim.x-th group of
// runs and leaves one sum of its dw and dbias.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
k_conv_grad(const Args p) {
    __shared__ float sums[kThreads * V];
    constexpr int U = 4;
    const int lane = threadIdx.x % p.across, down = kThreads / p.across;
    const int rank = threadIdx.x / p.across, c = (blockIdx.y * p.across + lane) * V;
    const bool there = c < p.channels;
    float w[W][V], bias[V], dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = dw[j][i] = 0.0f;
        bias[i] = db[i] = 0.0f;
    }
    if (there) load_weights<V, W>(p, c, w, bias);
    for (int64_t row = (int64_t)blockIdx.x * down + rank; there && row < p.rows;
         row += (int64_t)gridDim.x * down) {
        const Run r(p, row);
        const int n = tokens(p, r.b), t0 = r.t0, t1 = r.t1;
        // win: inputs t - W + 1 .. t; acc: the gradients of these inputs so far
        float win[W][V], acc[W][V];
        const int64_t at = (r.b * p.length + t0) * p.channels + c;
        const int end = min(t1 + W - 1, n);                // tokens that reach the run's inputs
        // gradients that come from the final state: input n - W + 1 + j has state j
        const auto from_state = [&](int s, float *v) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.0f;
            const int j = s - n + W - 1;
            if (p.dsT && s < n && j >= 0)
                load<T, V>(static_cast<const T *>(p.dsT) + (r.b * (W - 1) + j) * p.channels + c, v);
        };
        const auto finish = [&](int s, const float *v) {       // input s is complete
            if (s >= t0 && s < t1) {
                store<T, V>(static_cast<T *>(p.dx) + at + (int64_t)(s - t0) * p.channels, v);
            } else if (s < 0 && t0 == 0 && p.ds0) {
                store<T, V>(static_cast<T *>(p.ds0) + (r.b * (W - 1) + s + W - 1) * p.channels + c,
                            v);
            }
        };
        if (t0 < n || t0 == 0) {
#pragma unroll
            for (int j = 1; j < W; ++j) {
                input<T, V, W>(p, r.b, t0 - W + j, c, win[j]);
                from_state(t0 - W + j, acc[j]);
            }
        }
        const T *x = static_cast<const T *>(p.x) + at, *dy = static_cast<const T *>(p.dy) + at;
        for (int t = t0; t < end; t += U) {
            Pack<T, V> xin[U], gin[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (t + k < end) {
                    xin[k] = *reinterpret_cast<const Pack<T, V> *>(x + (int64_t)k * p.channels);
                    gin[k] = *reinterpret_cast<const Pack<T, V> *>(dy + (int64_t)k * p.channels);
                }
            x += (int64_t)U * p.channels;
            dy += (int64_t)U * p.channels;
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (t + k >= end) break;
                float last[V];
                from_state(t + k, last);
                const float mine = t + k < t1 ? 1.0f : 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        win[j][i] = win[j + 1][i];
                        acc[j][i] = acc[j + 1][i];
                    }
                    win[W - 1][i] = Storage<T>::load(&xin[k].v[i]);
                    acc[W - 1][i] = last[i];
                    float g = Storage<T>::load(&gin[k].v[i]);
                    if (p.silu) {
                        float s = bias[i];
#pragma unroll
                        for (int j = 0; j < W; ++j) s = fmaf(w[j][i], win[j][i], s);
                        g *= silu_slope(s);
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[j][i] = fmaf(w[j][i], g, acc[j][i]);
                    if (mine != 0.0f) {
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][i] = fmaf(g, win[j][i], dw[j][i]);
                        db[i] += g;
                    }
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
        const float zero[V] = {};
        for (int s = max(t0, n); s < t1; ++s)
            store<T, V>(static_cast<T *>(p.dx) + at + (int64_t)(s - t0) * p.channels, zero);
    }
    float *out = p.part + (int64_t)blockIdx.x * (W + 1) * p.channels;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i)
            sums[(rank * V + i) * p.across + lane] = j < W ? dw[j < W ? j : 0][i] : db[i];
        __syncthreads();
        for (int i = threadIdx.x; i < p.across * V; i += kThreads) {
            float v = 0.0f;
            for (int k = 0; k < down; ++k) v += sums[k * V * p.across + i];
            const int64_t ch = (int64_t)(blockIdx.y * p.across + i % p.across) * V + i / p.across;
            if (ch < p.channels) out[(int64_t)j * p.channels + ch] = v;
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

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
k_conv_step(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
            const int32_t *__restrict__ slots, int64_t num_slots, const T *state, T *new_state,
            T *__restrict__ y, int64_t batch, int channels, bool act) {
    const int cols = channels / V;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x, b = id / cols;
    if (b >= batch) return;
    const int c = (int)(id - b * cols) * V;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    if (slot >= 0 && slot < num_slots) {
        Pack<T, V> in[W];
        const int64_t at = slot * (W - 1) * channels + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            in[j] = *reinterpret_cast<const Pack<T, V> *>(state + at + (int64_t)j * channels);
        in[W - 1] = *reinterpret_cast<const Pack<T, V> *>(x + b * channels + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s = bias ? bias[c + i] : 0.0f;
#pragma unroll
            for (int j = 0; j < W; ++j)
                s = fmaf(w[(int64_t)(c + i) * W + j], Storage<T>::load(&in[j].v[i]), s);
            o[i] = act ? silu(s) : s;
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            *reinterpret_cast<Pack<T, V> *>(new_state + at + (int64_t)j * channels) = in[j + 1];
    }
    store<T, V>(y + b * channels + c, o);
}

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
struct Sizes {
    size_t row, w, c, s, len;    // bytes of x, w, bias, a state, lengths
};
Sizes sizes(const fno_causal_conv_s &p, int64_t length) {
    const size_t e = elem_bytes(p.dtype), n = (size_t)p.batch;
    return {n * length * p.channels * e, (size_t)p.channels * p.width * 4,
            (size_t)p.channels * 4, n * (p.width - 1) * p.channels * e, n * 4};
}

// Channels of a thread, and threads of a block over the channels.
int vector(int channels) { return channels % 2 == 0 ? 2 : 1; }
int across(int channels) {
    const int cols = channels / vector(channels);
    int a = 1;
    while (a < 32 && a < cols) a *= 2;
    return a;
}
Args common(const fno_causal_conv_s &p, int run) {
    Args a{};
    a.length = (int)p.length;
    a.channels = p.channels;
    a.run = run;
    a.rows = p.batch * ceil_div(p.length, run);
    a.across = across(p.channels);
    a.silu = p.act == FNO_ACT_SILU;
    return a;
}

}  // namespace

extern "C" {

fno_status_t fno_causal_conv_plan(fno_causal_conv_t *out, int64_t batch, int64_t length,
                                  int32_t channels, int32_t width, fno_act_t act,
                                  fno_dtype_t dtype, uint32_t flags) {
    if (!out) return FNO_ERR_INVALID_ARG;
    *out = nullptr;
    if (batch < 1 || length < 1 || channels < 1 || width < 2 ||
        (act != FNO_ACT_NONE && act != FNO_ACT_SILU) || !valid_dtype(dtype) ||
        (flags & ~FNO_CAUSAL_CONV_BACKWARD))
        return FNO_ERR_INVALID_ARG;
    if (width > 8 || length > 2147483647 - 64 || (double)batch * (double)(length + width) * channels > kMaxElems)
        return FNO_ERR_UNSUPPORTED;
    if (inject("plan_alloc")) return FNO_ERR_OUT_OF_MEMORY;
    fno_causal_conv_s *p = new (std::nothrow) fno_causal_conv_s();
    if (!p) return FNO_ERR_OUT_OF_MEMORY;
    p->batch = batch;
    p->length = length;
    p->channels = channels;
    p->width = width;
    p->act = act;
    p->dtype = dtype;
    p->flags = flags;
    fno_status_t st = device_sms(&p->sms);
    if (st != FNO_OK) {
        delete p;
        return st;
    }
    // runs of 32 tokens, shorter ones (of 8 at least) while the threads do not fill the SMs;
    // backward of 64 (its runs reach over 2 width tokens more), a wave or two of blocks
    const int64_t cols = channels / vector(channels), want = (int64_t)p->sms * 1024;
    p->run = 32;
    while (p->run > 8 && batch * ceil_div(length, p->run) * cols < want) p->run /= 2;
    p->bwd_run = 64;
    while (p->bwd_run > 16 && batch * ceil_div(length, p->bwd_run) * cols < want) p->bwd_run /= 2;
    const int a = across(channels), down = kThreads / a;
    const int64_t blocks = ceil_div(batch * ceil_div(length, p->run), down);
    if (ceil_div(cols, a) > 65535 || blocks > 2147483647) {
        delete p;
        return FNO_ERR_UNSUPPORTED;
    }
    const int64_t most = ceil_div((int64_t)8 * p->sms, ceil_div(cols, a));
    const int64_t rows = ceil_div(batch * ceil_div(length, p->bwd_run), down);
    p->parts = (int)(most < rows ? most : rows);
    if (flags & FNO_CAUSAL_CONV_BACKWARD)
        p->workspace = (size_t)p->parts * (width + 1) * channels * 4;
    *out = p;
    return FNO_OK;
}

fno_status_t fno_causal_conv_workspace_size(fno_causal_conv_t p, size_t *bytes) {
    if (!p || !bytes) return FNO_ERR_INVALID_ARG;
    *bytes = p->workspace;
    return FNO_OK;
}

fno_status_t fno_causal_conv_forward(fno_causal_conv_t p, const void *x, const float *w,
                                     const float *bias, const int32_t *lengths, const void *s0,
                                     void *y, void *sT, fno_stream_t stream) {
    if (!p || !x || !w || !y) return FNO_ERR_INVALID_ARG;
    const Sizes n = sizes(*p, p->length);
    fno_status_t st = check_operands(
        {{x, n.row, false}, {w, n.w, false}, {bias, n.c, false}, {lengths, n.len, false},
         {s0, n.s, false}, {y, n.row, true}, {sT, n.s, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    Args a = common(*p, p->run);
    a.x = x, a.w = w, a.bias = bias, a.lengths = lengths, a.s0 = s0, a.y = y, a.sT = sT;
    const int v = vector(p->channels);
    const dim3 grid((unsigned)ceil_div(a.rows, kThreads / a.across),
                    (unsigned)ceil_div(p->channels / v, a.across));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        return with_width(p->width, [&](auto width) {
            constexpr int W = decltype(width)::value;
            if (v == 2) k_conv<T, 2, W><<<grid, kThreads, 0, s>>>(a);
            else k_conv<T, 1, W><<<grid, kThreads, 0, s>>>(a);
            return launched();
        });
    });
}

fno_status_t fno_causal_conv_backward(fno_causal_conv_t p, const void *x, const float *w,
                                      const float *bias, const int32_t *lengths, const void *s0,
                                      const void *dy, const void *dsT, void *dx, float *dw,
                                      float *dbias, void *ds0, void *workspace,
                                      fno_stream_t stream) {
    if (!p || !(p->flags & FNO_CAUSAL_CONV_BACKWARD) || !x || !w || !dy || !dx || !dw ||
        !workspace)
        return FNO_ERR_INVALID_ARG;
    const Sizes n = sizes(*p, p->length);
    fno_status_t st = check_operands(
        {{x, n.row, false}, {w, n.w, false}, {bias, n.c, false}, {lengths, n.len, false},
         {s0, n.s, false}, {dy, n.row, false}, {dsT, n.s, false}, {dx, n.row, true},
         {dw, n.w, true}, {dbias, n.c, true}, {ds0, n.s, true},
         {workspace, p->workspace, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    Args a = common(*p, p->bwd_run);
    a.x = x, a.w = w, a.bias = bias, a.lengths = lengths, a.s0 = s0, a.dy = dy, a.dsT = dsT;
    a.dx = dx, a.ds0 = ds0, a.part = static_cast<float *>(workspace);
    const int v = vector(p->channels);
    const dim3 grid((unsigned)p->parts, (unsigned)ceil_div(p->channels / v, a.across));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        return with_width(p->width, [&](auto width) {
            constexpr int W = decltype(width)::value;
            if (v == 2) k_conv_grad<T, 2, W><<<grid, kThreads, 0, s>>>(a);
            else k_conv_grad<T, 1, W><<<grid, kThreads, 0, s>>>(a);
            const int64_t outs = (int64_t)p->channels * (W + 1);
            k_conv_sum<<<(unsigned)ceil_div(outs, 32), dim3(32, kSumRows), 0, s>>>(
                a.part, dw, dbias, p->channels, W, p->parts);
            return launched();
        });
    });
}

fno_status_t fno_causal_conv_step(fno_causal_conv_t p, const void *x, const float *w,
                                  const float *bias, const int32_t *slots, int64_t num_slots,
                                  const void *state, void *new_state, void *y,
                                  fno_stream_t stream) {
    if (!p || !x || !w || !state || !new_state || !y || num_slots < 1 ||
        (!slots && num_slots < p->batch))
        return FNO_ERR_INVALID_ARG;
    if ((double)num_slots * (p->width - 1) * p->channels > kMaxElems) return FNO_ERR_UNSUPPORTED;
    const Sizes n = sizes(*p, 1);
    const size_t sb = (size_t)num_slots * (p->width - 1) * p->channels * elem_bytes(p->dtype);
    fno_status_t st = check_operands(
        {{x, n.row, false}, {w, n.w, false}, {bias, n.c, false}, {slots, n.len, false},
         {state, sb, false}, {new_state, sb, true, state}, {y, n.row, true}});
    if (st != FNO_OK) return st;
    return with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        return with_width(p->width, [&](auto width) {
            constexpr int W = decltype(width)::value, V = 2;
            const int v = p->channels % V == 0 ? V : 1;
            const int64_t blocks = ceil_div(p->batch * (p->channels / v), kThreads);
            if (blocks > 2147483647) return FNO_ERR_UNSUPPORTED;
            if (inject("launch")) return FNO_ERR_CUDA;
            const auto run = [&](auto kernel) {
                kernel<<<(unsigned)blocks, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
                    static_cast<const T *>(x), w, bias, slots, num_slots,
                    static_cast<const T *>(state), static_cast<T *>(new_state),
                    static_cast<T *>(y), p->batch, p->channels, p->act == FNO_ACT_SILU);
            };
            if (v == V) run(k_conv_step<T, V, W>);
            else run(k_conv_step<T, 1, W>);
            return launched();
        });
    });
}

fno_status_t fno_causal_conv_destroy(fno_causal_conv_t p) {
    delete p;
    return FNO_OK;
}

}  // extern "C"
