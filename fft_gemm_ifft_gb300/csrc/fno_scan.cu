// fno_scan.cu -- the selective scan's plan and calls, the joining of its segments'
// states and its single-token step.
#include "fno_scan.h"

using namespace fno;
using namespace fno::ops;
using namespace fno::scan;

namespace fno {
namespace scan {
// instantiated in fno_scan_fwd_*.cu and fno_scan_bwd_*.cu
#define FNO_SCAN_EXTERN(T)                                                              \
    extern template fno_status_t forward_of<T>(const fno_scan_s &, Args, cudaStream_t); \
    extern template fno_status_t backward_of<T>(const fno_scan_s &, Args, cudaStream_t);
FNO_SCAN_EXTERN(float)
FNO_SCAN_EXTERN(__half)
FNO_SCAN_EXTERN(__nv_bfloat16)
}  // namespace scan
}  // namespace fno

namespace {

// A thread per (sequence, channel, state): the segments' local values are loaded eight
// at a time ahead of the chain of multiply-adds.
__global__ void __launch_bounds__(256)
k_scan_join(float *__restrict__ local, const float *__restrict__ steps,
            const float *__restrict__ A, const float *__restrict__ first, int64_t cn, int states,
            int channels, int segments, bool reverse) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, b = blockIdx.y;
    if (e >= cn) return;
    const int c = (int)(e / states);
    const float a2 = A[e] * kLog2e;
    float z = first ? first[b * cn + e] : 0.0f;
    const int64_t from = reverse ? segments - 1 : 0, dir = reverse ? -1 : 1;
    float *v = local + (b * segments + from) * cn + e;
    const float *d = steps + (b * segments + from) * channels + c;
    for (int s = 0; s < segments; s += 8) {
        float l[8], w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (s + k < segments) {
                l[k] = v[dir * (s + k) * cn];
                w[k] = d[dir * (s + k) * channels];
            }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (s + k < segments) {
                v[dir * (s + k) * cn] = z;
                z = fmaf(exp2_fast(a2 * w[k]), z, l[k]);
            }
    }
}

// One token.  `lanes` (a power of two) threads share a channel's states, V at a time
// (4 where the count allows); the states read and written once are all that it costs.
constexpr int kStepThreads = 128;

template <typename T, int V>
__global__ void __launch_bounds__(kStepThreads)
k_scan_step(const T *__restrict__ x, const T *__restrict__ dt, const float *__restrict__ A,
            const T *__restrict__ B, const T *__restrict__ C, const float *__restrict__ D,
            const T *__restrict__ z, const float *__restrict__ bias,
            const int32_t *__restrict__ slots, int64_t num_slots, const float *state,
            float *new_state, T *__restrict__ y, int channels, int per_group, int states, int lanes,
            int blocks_a_row, bool plus) {
    const int64_t b = blockIdx.x / blocks_a_row;
    const int c = (int)(blockIdx.x - b * blocks_a_row) * (kStepThreads / lanes) +
                  threadIdx.x / lanes;
    const int q = threadIdx.x & (lanes - 1);
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    const bool there = c < channels, live = there && slot >= 0 && slot < num_slots;
    const int64_t at = b * channels + c;
    float sum = 0.0f, xv = 0.0f;
    if (live) {
        const int64_t bc = (b * (channels / per_group) + c / per_group) * states;
        const int64_t cn = (int64_t)c * states, sn = slot * channels * states + cn;
        xv = Storage<T>::load(x + at);
        float d = Storage<T>::load(dt + at);
        if (bias) d += bias[c];
        if (plus) d = softplus(d);
        const float u = d * xv;
        for (int n = q * V; n < states; n += lanes * V) {
            Pack<float, V> h = *reinterpret_cast<const Pack<float, V> *>(state + sn + n);
            const Pack<float, V> a = *reinterpret_cast<const Pack<float, V> *>(A + cn + n);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                h.v[i] = fmaf(exp2_fast(a.v[i] * kLog2e * d), h.v[i],
                              u * Storage<T>::load(B + bc + n + i));
                sum = fmaf(Storage<T>::load(C + bc + n + i), h.v[i], sum);
            }
            *reinterpret_cast<Pack<float, V> *>(new_state + sn + n) = h;
        }
    }
    for (int o = lanes / 2; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (there && q == 0) {
        if (live) {
            if (D) sum = fmaf(D[c], xv, sum);
            if (z) {
                const float zv = Storage<T>::load(z + at);
                sum *= zv * logistic(zv);
            }
        }
        Storage<T>::store(y + at, live ? sum : 0.0f);
    }
}

// Bytes (16, 8, 4 or the element's) that divide every one of the sizes given in elements.
int vector_bytes(int e, std::initializer_list<int64_t> sizes) {
    for (int v = 16; v > e; v /= 2) {
        bool fits = true;
        for (int64_t n : sizes) fits = fits && n * e % v == 0;
        if (fits) return v;
    }
    return e;
}

struct Sizes {
    size_t row, bc, cn, c, s, len;    // bytes of x, B, A, D, a state, lengths
};
Sizes sizes(const fno_scan_desc_t &d, int64_t length) {
    const size_t e = elem_bytes(d.dtype), n = (size_t)d.batch * length;
    return {n * d.channels * e, n * d.groups * d.states * e, (size_t)d.channels * d.states * 4,
            (size_t)d.channels * 4, (size_t)d.batch * d.channels * d.states * 4,
            (size_t)d.batch * 4};
}

// Segments of the time axis, multiples of `unit` tokens: one where the sequences and
// channels alone give the SMs half of `warps` each, else as many as give them all, of 64
// tokens at least (a segment costs a second pass over its tokens).
void split(int64_t length, int64_t warps_there, int64_t warps, int unit, int64_t *seg_len,
           int *segments) {
    int64_t segs = 2 * warps_there >= warps ? 1 : warps / warps_there;
    const int64_t most = ceil_div(length, 64);
    segs = segs < most ? segs : most;
    *seg_len = ceil_div(ceil_div(length, segs), unit) * unit;
    *segments = (int)ceil_div(length, *seg_len);
}

Args common(const fno_scan_s &p) {
    const fno_scan_desc_t &d = p.d;
    Args a{};
    a.length = d.length;
    a.batch = (int)d.batch;
    a.channels = d.channels;
    a.per_group = d.channels / d.groups;
    a.groups = d.groups;
    a.states = d.states;
    a.softplus = d.softplus != 0;
    const int e = (int)elem_bytes(d.dtype);
    a.vec_c = vector_bytes(e, {d.channels, a.per_group});
    a.vec_n = vector_bytes(e, {d.states});
    return a;
}

int slabs(const fno_scan_s &p, int width, int warps) {
    const int per = p.d.channels / p.d.groups, nw = state_warps(p.d.states);
    int s = 1;
    while (2 * s * nw <= warps && s * width < per) s *= 2;
    return s;
}

}  // namespace

namespace fno {
namespace scan {

fno_status_t join(const Args &a, bool reverse, cudaStream_t s) {
    const int64_t cn = (int64_t)a.channels * a.states;
    const dim3 grid((unsigned)ceil_div(cn, 256), (unsigned)a.batch);
    k_scan_join<<<grid, 256, 0, s>>>(reverse ? a.gseg : a.hseg, a.dseg, a.A,
                                     reverse ? a.gsT : a.s0, cn, a.states, a.channels, a.segments,
                                     reverse);
    return launched();
}

BackwardParts backward_parts(const fno_scan_s &p) {
    const fno_scan_desc_t &d = p.d;
    const size_t cn = (size_t)d.channels * d.states, b = (size_t)d.batch;
    const size_t segs = b * p.bwd_segments, tiles = (size_t)ceil_div(d.length, kTile);
    const bool split = p.bwd_segments > 1, kept = tiles > 1;
    const int per = d.channels / d.groups;
    const size_t blocks = (size_t)ceil_div(per, 16 * backward_slabs(p));
    BackwardParts w{};
    size_t at = 0;
    const auto take = [&](size_t floats) {
        const size_t here = at;
        at += (floats * 4 + 255) & ~size_t(255);
        return here;
    };
    w.hseg = take(split ? segs * cn : 0);
    w.gseg = take(split ? segs * cn : 0);
    w.dseg = take(split ? segs * d.channels : 0);
    w.hchunk = take(kept ? b * tiles * cn : 0);
    w.dchunk = take(kept ? b * tiles * d.channels : 0);
    w.part_bc = take(blocks > 1 ? blocks * b * d.length * d.groups * 2 * d.states : 0);
    w.part_a = take(segs * cn);
    w.part_d = take(segs * 2 * d.channels);
    w.bytes = at;
    return w;
}

int forward_slabs(const fno_scan_s &p) { return slabs(p, 32, 4); }
int backward_slabs(const fno_scan_s &p) { return slabs(p, 16, 8); }

}  // namespace scan
}  // namespace fno

extern "C" {

fno_status_t fno_scan_plan(fno_scan_t *out, const fno_scan_desc_t *desc) {
    if (!out) return FNO_ERR_INVALID_ARG;
    *out = nullptr;
    if (!desc) return FNO_ERR_INVALID_ARG;
    const fno_scan_desc_t d = *desc;
    if (d.batch < 1 || d.length < 1 || d.channels < 1 || d.states < 1 || d.groups < 1 ||
        d.channels % d.groups || !valid_dtype(d.dtype) || (d.flags & ~FNO_SCAN_BACKWARD))
        return FNO_ERR_INVALID_ARG;
    const double wide = d.channels > (double)d.groups * d.states ? (double)d.channels
                                                                 : (double)d.groups * d.states;
    if (d.states > kMaxStates || (double)d.batch > 65535.0 * 1024.0 ||
        (double)d.batch * (double)d.length * wide > kMaxElems ||
        (double)d.batch * d.channels * d.states > kMaxElems)
        return FNO_ERR_UNSUPPORTED;
    if (inject("plan_alloc")) return FNO_ERR_OUT_OF_MEMORY;
    fno_scan_s *p = new (std::nothrow) fno_scan_s();
    if (!p) return FNO_ERR_OUT_OF_MEMORY;
    p->d = d;
    fno_status_t st = device_sms(&p->sms);
    if (st != FNO_OK) {
        delete p;
        return st;
    }
    const int per = d.channels / d.groups, nw = state_warps(d.states);
    const int fs = forward_slabs(*p), bs = backward_slabs(*p);
    const int64_t rows = d.batch * d.groups;
    split(d.length, rows * ceil_div(per, 32 * fs) * fs * nw, (int64_t)16 * p->sms, kTile,
          &p->seg_len, &p->segments);
    split(d.length, rows * ceil_div(per, 16 * bs) * bs * nw, (int64_t)16 * p->sms, kTile,
          &p->bwd_seg_len, &p->bwd_segments);
    const double blocks = (double)rows * (double)ceil_div(per, 16) *
                          (p->segments > p->bwd_segments ? p->segments : p->bwd_segments);
    if (blocks > 2147483647.0) {
        delete p;
        return FNO_ERR_UNSUPPORTED;
    }
    if (p->segments > 1)
        p->workspace = (size_t)d.batch * p->segments * d.channels * (d.states + 1) * 4;
    if (d.flags & FNO_SCAN_BACKWARD) {
        const size_t n = backward_parts(*p).bytes;
        if (n > p->workspace) p->workspace = n;
    }
    *out = p;
    return FNO_OK;
}

fno_status_t fno_scan_workspace_size(fno_scan_t p, size_t *bytes) {
    if (!p || !bytes) return FNO_ERR_INVALID_ARG;
    *bytes = p->workspace;
    return FNO_OK;
}

fno_status_t fno_scan_forward(fno_scan_t p, const void *x, const void *dt, const float *A,
                              const void *B, const void *C, const float *D, const void *z,
                              const float *dt_bias, const int32_t *lengths, const float *s0,
                              void *y, float *sT, void *workspace, fno_stream_t stream) {
    if (!p || !x || !dt || !A || !B || !C || !y || (p->workspace && !workspace))
        return FNO_ERR_INVALID_ARG;
    const Sizes n = sizes(p->d, p->d.length);
    fno_status_t st = check_operands(
        {{x, n.row, false}, {dt, n.row, false}, {A, n.cn, false}, {B, n.bc, false},
         {C, n.bc, false}, {D, n.c, false}, {z, n.row, false}, {dt_bias, n.c, false},
         {lengths, n.len, false}, {s0, n.s, false}, {y, n.row, true}, {sT, n.s, true},
         {workspace, p->workspace, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    Args a = common(*p);
    a.x = x, a.dt = dt, a.A = A, a.B = B, a.C = C, a.D = D, a.z = z, a.bias = dt_bias;
    a.lengths = lengths, a.s0 = s0, a.y = y, a.sT = sT;
    a.hseg = static_cast<float *>(workspace);
    a.dseg = a.hseg ? a.hseg + (size_t)p->d.batch * p->segments * p->d.channels * p->d.states
                    : nullptr;
    return with_storage(p->d.dtype, [&](auto t) {
        return forward_of<decltype(t)>(*p, a, reinterpret_cast<cudaStream_t>(stream));
    });
}

fno_status_t fno_scan_backward(fno_scan_t p, const void *x, const void *dt, const float *A,
                               const void *B, const void *C, const float *D, const void *z,
                               const float *dt_bias, const int32_t *lengths, const float *s0,
                               const void *dy, const float *dsT, void *dx, void *ddt, float *dA,
                               void *dB, void *dC, float *dD, void *dz, float *ddt_bias,
                               float *ds0, void *workspace, fno_stream_t stream) {
    if (!p || !(p->d.flags & FNO_SCAN_BACKWARD) || !x || !dt || !A || !B || !C || !dy || !dx ||
        !ddt || !dA || !dB || !dC || !z != !dz || (p->workspace && !workspace))
        return FNO_ERR_INVALID_ARG;
    const Sizes n = sizes(p->d, p->d.length);
    fno_status_t st = check_operands(
        {{x, n.row, false}, {dt, n.row, false}, {A, n.cn, false}, {B, n.bc, false},
         {C, n.bc, false}, {D, n.c, false}, {z, n.row, false}, {dt_bias, n.c, false},
         {lengths, n.len, false}, {s0, n.s, false}, {dy, n.row, false}, {dsT, n.s, false},
         {dx, n.row, true}, {ddt, n.row, true}, {dA, n.cn, true}, {dB, n.bc, true},
         {dC, n.bc, true}, {dD, n.c, true}, {dz, n.row, true}, {ddt_bias, n.c, true},
         {ds0, n.s, true}, {workspace, p->workspace, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    Args a = common(*p);
    a.x = x, a.dt = dt, a.A = A, a.B = B, a.C = C, a.D = D, a.z = z, a.bias = dt_bias;
    a.lengths = lengths, a.s0 = s0, a.dy = dy, a.gsT = dsT;
    a.dx = dx, a.ddt = ddt, a.dA = dA, a.dB = dB, a.dC = dC, a.dD = dD, a.dz = dz;
    a.dbias = ddt_bias, a.ds0 = ds0;
    const BackwardParts w = backward_parts(*p);
    const auto part = [&](size_t at) {
        return reinterpret_cast<float *>(static_cast<char *>(workspace) + at);
    };
    a.hseg = part(w.hseg), a.gseg = part(w.gseg), a.dseg = part(w.dseg);
    a.hchunk = part(w.hchunk), a.dchunk = part(w.dchunk);
    a.part_bc = part(w.part_bc), a.part_a = part(w.part_a), a.part_d = part(w.part_d);
    return with_storage(p->d.dtype, [&](auto t) {
        return backward_of<decltype(t)>(*p, a, reinterpret_cast<cudaStream_t>(stream));
    });
}

fno_status_t fno_scan_step(fno_scan_t p, const void *x, const void *dt, const float *A,
                           const void *B, const void *C, const float *D, const void *z,
                           const float *dt_bias, const int32_t *slots, int64_t num_slots,
                           const float *state, float *new_state, void *y, fno_stream_t stream) {
    if (!p || !x || !dt || !A || !B || !C || !state || !new_state || !y || num_slots < 1 ||
        (!slots && num_slots < p->d.batch))
        return FNO_ERR_INVALID_ARG;
    const fno_scan_desc_t &d = p->d;
    if ((double)num_slots * d.channels * d.states > kMaxElems) return FNO_ERR_UNSUPPORTED;
    const Sizes n = sizes(d, 1);
    const size_t sb = (size_t)num_slots * d.channels * d.states * 4;
    fno_status_t st = check_operands(
        {{x, n.row, false}, {dt, n.row, false}, {A, n.cn, false}, {B, n.bc, false},
         {C, n.bc, false}, {D, n.c, false}, {z, n.row, false}, {dt_bias, n.c, false},
         {slots, n.len, false}, {state, sb, false}, {new_state, sb, true, state},
         {y, n.row, true}});
    if (st != FNO_OK) return st;
    const int v = d.states % 4 == 0 ? 4 : 1;
    int lanes = 1;
    while (lanes < 32 && lanes * v < d.states) lanes *= 2;
    const int64_t a_row = ceil_div(d.channels, kStepThreads / lanes);
    if ((double)a_row * (double)d.batch > 2147483647.0) return FNO_ERR_UNSUPPORTED;
    if (inject("launch")) return FNO_ERR_CUDA;
    with_storage(d.dtype, [&](auto t) {
        using T = decltype(t);
        const auto run = [&](auto kernel) {
            kernel<<<(unsigned)(a_row * d.batch), kStepThreads, 0,
                     reinterpret_cast<cudaStream_t>(stream)>>>(
                static_cast<const T *>(x), static_cast<const T *>(dt), A,
                static_cast<const T *>(B), static_cast<const T *>(C), D,
                static_cast<const T *>(z), dt_bias, slots, num_slots, state, new_state,
                static_cast<T *>(y), d.channels, d.channels / d.groups, d.states, lanes,
                (int)a_row, d.softplus != 0);
        };
        if (v == 4) run(k_scan_step<T, 4>);
        else run(k_scan_step<T, 1>);
    });
    return launched();
}

fno_status_t fno_scan_destroy(fno_scan_t p) {
    delete p;
    return FNO_OK;
}

}  // extern "C"
