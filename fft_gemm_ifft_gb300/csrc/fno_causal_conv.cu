// fno_causal_conv.cu -- short causal convolutions of every channel along time, with their
// activation: whole sequences, gradients, single tokens.
//
// 2 width multiply-adds an element, an exponential and a quotient: bound by bytes and, at three
// quarters of the issue slots, nearly as much by instructions.  A thread takes two channels of a
// run of tokens with the last inputs in registers, so that an input is loaded once and the
// width - 1 in front of a run once more.  Two channels and no more: the weights, the window and
// the tokens loaded ahead then take few enough registers for the warps that keep enough loads
// on their way (4 x 8192 tokens of 2048 channels in bfloat16: 55 us, 4.9 TB/s; with eight
// channels a thread 2.7 times as long).
//
// The loads on their way are what the registers leave for them, of 16-bit types 8 tokens of 32
// warps an SM up to 4 taps, 32 KB, but 4 of 24 warps above, 12 KB, and the times follow them (the
// same tokens with 5, 6 and 8 taps: 88, 84 and 102 us a call, with 4 taps 63; 4 taps of float32,
// 88 us, are at 90 % of the copy rate).  Odd channel counts load single elements (2047: 149 us).
#include "fno_causal_conv.h"

using namespace fno;
using namespace fno::conv;

namespace {

template <typename T, bool WIDE, int W>
__global__ void __launch_bounds__(kThreads, W <= 4 ? 4 : 3)
k_conv(const Args p) {
    constexpr int U = W <= 4 ? 8 : 4;          // tokens whose loads are on their way
    const int lane = threadIdx.x % p.across, rank = threadIdx.x / p.across;
    const int c = (chunk(p) * p.across + lane) * 2, left = p.channels - c;
    const int64_t row = (int64_t)block(p) * (kThreads / p.across) + rank;
    if (row >= p.rows || left <= 0) return;
    const Run r(p, row);
    const int n = tokens(p, r.b), end = min(r.t1, n);
    float2 w[W], bias, win[W];                 // win: the last W inputs, oldest first
    load_weights<W>(p, c, left, w, bias);
    const int64_t at = (r.b * p.length + r.t0) * p.channels + c;
    T *y = static_cast<T *>(p.y) + at;
    const T *x = static_cast<const T *>(p.x) + at;
    Pair<T> next[U];
    const auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            next[k] = load_pair(x, WIDE, t + k < end ? left : 0);
            x += p.channels;
        }
    };
    if (r.t0 < end) {
        fetch(r.t0);
#pragma unroll
        for (int j = 1; j < W; ++j) win[j] = input<T, WIDE, W>(p, r.b, r.t0 - W + j, c, left);
    }
    for (int t = r.t0; t < end; t += U) {
        Pair<T> in[U];
#pragma unroll
        for (int k = 0; k < U; ++k) in[k] = next[k];
        if (t + U < end) fetch(t + U);
#pragma unroll
        for (int k = 0; k < U; ++k) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
            win[W - 1] = to_float2(in[k]);
            float2 s = taps<W>(w, win, bias);
            if (p.silu) s = make_float2(silu(s.x), silu(s.y));
            store_pair(y, s, WIDE, t + k < end ? left : 0);
            y += p.channels;
        }
    }
    y = static_cast<T *>(p.y) + at;
    for (int t = max(r.t0, end); t < r.t1; ++t)
        store_pair(y + (int64_t)(t - r.t0) * p.channels, f2(0.0f), WIDE, left);
    if (p.sT && r.t0 == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_pair(static_cast<T *>(p.sT) + (r.b * (W - 1) + j) * p.channels + c,
                       input<T, WIDE, W>(p, r.b, n - (W - 1) + j, c, left), WIDE, left);
    }
}

template <typename T, bool WIDE, int W>
__global__ void __launch_bounds__(kThreads)
k_conv_step(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
            const int32_t *__restrict__ slots, int64_t num_slots, const T *state, T *new_state,
            T *__restrict__ y, int channels, int blocks_a_row, bool act) {
    const int64_t b = blockIdx.x / blocks_a_row;
    const int c = ((int)(blockIdx.x - b * blocks_a_row) * kThreads + threadIdx.x) * 2;
    const int left = channels - c;
    if (left <= 0) return;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    float2 s = f2(0.0f);
    if (slot >= 0 && slot < num_slots) {
        Pair<T> in[W];
        const int64_t at = slot * (W - 1) * channels + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            in[j] = load_pair(state + at + (int64_t)j * channels, WIDE, left);
        in[W - 1] = load_pair(x + b * channels + c, WIDE, left);
        const float *from = w + (int64_t)c * W;
        if (bias) s = make_float2(bias[c], left > 1 ? bias[c + 1] : 0.0f);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float2 v = to_float2(in[j]);
            s.x = fmaf(from[j], v.x, s.x);
            if (left > 1) s.y = fmaf(from[W + j], v.y, s.y);
        }
        if (act) s = make_float2(silu(s.x), silu(s.y));
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_raw(new_state + at + (int64_t)j * channels, in[j + 1], WIDE, left);
    }
    store_pair(y + b * channels + c, s, WIDE, left);
}

struct Sizes {
    size_t row, w, c, s, len;    // bytes of x, w, bias, a state, lengths
};
Sizes sizes(const fno_causal_conv_s &p, int64_t length) {
    const size_t e = elem_bytes(p.dtype), n = (size_t)p.batch;
    return {n * length * p.channels * e, (size_t)p.channels * p.width * 4,
            (size_t)p.channels * 4, n * (p.width - 1) * p.channels * e, n * 4};
}

// Threads of a block over the channels.
int across(int channels) {
    int a = 1;
    while (a < 32 && 2 * a < channels) a *= 2;
    return a;
}
Args common(const fno_causal_conv_s &p, int run) {
    Args a{};
    a.length = (int)p.length;
    a.channels = p.channels;
    a.run = run;
    a.rows = p.batch * ceil_div(p.length, run);
    a.across = across(p.channels);
    a.chunks = (int)ceil_div(p.channels, 2 * a.across);
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
    if (width > 8 || length > 2147483647 - 64 ||
        (double)batch * (double)(length + width) * channels > kMaxElems)
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
    // runs of 32 tokens, shorter ones (of 8 at least) while the threads do not fill the SMs
    const int64_t cols = ceil_div(channels, 2), want = (int64_t)p->sms * 1024;
    p->run = 32;
    while (p->run > 8 && batch * ceil_div(length, p->run) * cols < want) p->run /= 2;
    const int a = across(channels), down = kThreads / a;
    // backward the shortest from 16 to 40 that make no more than a wave of blocks (4096
    // tokens of 2048 channels: 36 us, with runs of 32 44), or 64 for several waves (5 x 4099
    // tokens of 1001 channels, ragged: 51 us; 59 with 32, 65 with 96 in a wave)
    const int64_t wave = (int64_t)grad_blocks(width, (int)elem_bytes(dtype)) * p->sms;
    const auto backward_blocks = [&](int run) {
        return ceil_div(batch * ceil_div(length, run), down) * ceil_div(cols, a);
    };
    p->bwd_run = 16;
    while (p->bwd_run <= 40 && backward_blocks(p->bwd_run) > wave) p->bwd_run += 8;
    if (p->bwd_run > 40) p->bwd_run = 64;
    const int64_t blocks = ceil_div(batch * ceil_div(length, p->run), down);
    if ((double)ceil_div(cols, a) * (double)blocks > 2147483647.0 ||
        ceil_div(cols, a) > 65535) {
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
    const unsigned grid = (unsigned)(ceil_div(a.rows, kThreads / a.across) * a.chunks);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        return with_width(p->width, [&](auto width) {
            constexpr int W = decltype(width)::value;
            if (p->channels % 2) k_conv<T, false, W><<<grid, kThreads, 0, s>>>(a);
            else k_conv<T, true, W><<<grid, kThreads, 0, s>>>(a);
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
    return gradients(*p, a, dw, dbias, reinterpret_cast<cudaStream_t>(stream));
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
    const int64_t a_row = ceil_div(p->channels, 2 * kThreads);
    if ((double)a_row * (double)p->batch > 2147483647.0) return FNO_ERR_UNSUPPORTED;
    if (inject("launch")) return FNO_ERR_CUDA;
    return with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        return with_width(p->width, [&](auto width) {
            constexpr int W = decltype(width)::value;
            const auto run = [&](auto kernel) {
                kernel<<<(unsigned)(a_row * p->batch), kThreads, 0,
                         reinterpret_cast<cudaStream_t>(stream)>>>(
                    static_cast<const T *>(x), w, bias, slots, num_slots,
                    static_cast<const T *>(state), static_cast<T *>(new_state),
                    static_cast<T *>(y), p->channels, (int)a_row, p->act == FNO_ACT_SILU);
            };
            if (p->channels % 2) run(k_conv_step<T, false, W>);
            else run(k_conv_step<T, true, W>);
            return launched();
        });
    });
}

fno_status_t fno_causal_conv_destroy(fno_causal_conv_t p) {
    delete p;
    return FNO_OK;
}

}  // extern "C"
