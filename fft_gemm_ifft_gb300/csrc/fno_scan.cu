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

// The joining of the segments: a lane per (sequence, channel, state), the segments over a
// block's warps.  Each warp puts its segments together, all warps go on from those in front
// of them, and each writes its segments' states (74 segments of 2 x 1024 x 16 with one thread
// for all of them: 20 us, all of it the latency of the reads).  The second half of the blocks
// joins the gradients, from the last segment.
constexpr int kJoinWarps = 8, kJoinHold = 16;
__global__ void __launch_bounds__(32 * kJoinWarps)
k_scan_join(const Args p) {
    __shared__ float2 ends[kJoinWarps][32];            // (local value, sum of the steps)
    const int np = p.shape.np, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const bool reverse = blockIdx.z != 0;
    const int64_t e = (int64_t)blockIdx.x * 32 + lane, b = blockIdx.y;
    const int64_t row = (int64_t)p.channels * np, c = over(e, np);
    const int n = (int)(e - c * np), each = (p.segments + kJoinWarps - 1) / kJoinWarps;
    const bool mine = e < row && n < p.states;
    const int64_t cn = c * p.states + n;
    const float a2 = mine ? p.A[cn] * kLog2e : 0.0f;
    const int first = w * each, count = mine ? max(0, min(each, p.segments - first)) : 0;
    const int64_t dir = reverse ? -1 : 1;
    const int64_t from = b * p.segments + (reverse ? p.segments - 1 - first : first);
    float *const v = (reverse ? p.gseg : p.hseg) + from * row + e;
    const float *const d = p.dseg + from * p.channels + c;
    const float *start = reverse ? p.gsT : p.s0;
    const float given = start && mine ? start[b * p.channels * p.states + cn] : 0.0f;
    const auto in_front = [&]() {                     // of this warp's segments
        float z = given;
        for (int k = 0; k < w; ++k) z = fmaf(exp2_fast(a2 * ends[k][lane].y), z, ends[k][lane].x);
        return z;
    };
    if (each <= kJoinHold) {
        float l[kJoinHold], t[kJoinHold], z = 0.0f, steps = 0.0f;
#pragma unroll
        for (int k = 0; k < kJoinHold; ++k)
            if (k < count) l[k] = v[dir * k * row], t[k] = d[dir * k * p.channels];
#pragma unroll
        for (int k = 0; k < kJoinHold; ++k)
            if (k < count) {
                steps += t[k];
                t[k] = exp2_fast(a2 * t[k]);
                z = fmaf(t[k], z, l[k]);
            }
        ends[w][lane] = make_float2(z, steps);
        __syncthreads();
        z = in_front();
#pragma unroll
        for (int k = 0; k < kJoinHold; ++k)
            if (k < count) {
                v[dir * k * row] = z;
                z = fmaf(t[k], z, l[k]);
            }
        return;
    }
    // more segments than a lane holds are read again
    float z = 0.0f, steps = 0.0f;
    for (int k = 0; k < count; ++k) {
        const float t = d[dir * k * p.channels];
        z = fmaf(exp2_fast(a2 * t), z, v[dir * k * row]);
        steps += t;
    }
    ends[w][lane] = make_float2(z, steps);
    __syncthreads();
    z = in_front();
    for (int k = 0; k < count; ++k) {
        const float l = v[dir * k * row];
        v[dir * k * row] = z;
        z = fmaf(exp2_fast(a2 * d[dir * k * p.channels]), z, l);
    }
}

// Sums over the blocks' parts, in the order of the parts, of dA (channels, padded states) and
// behind it of D's and the bias' gradients (2 x channels): COLS columns a block, its other
// threads over the parts, so that many parts of few columns (512 of 1024: 10 us by 32 rows)
// are read at once.
template <int COLS>
__global__ void __launch_bounds__(1024)
k_scan_sum(const Args p, int64_t parts) {
    constexpr int kRows = 1024 / COLS;
    __shared__ float s[kRows][COLS + 1];
    const int np = p.shape.np, col = threadIdx.x % COLS, r = threadIdx.x / COLS;
    const int64_t states = (int64_t)p.channels * np, more = 2 * (int64_t)p.channels;
    const int64_t i = (int64_t)blockIdx.x * COLS + col;
    const bool of_a = i < states;
    const float *in = of_a ? p.part_a + i : p.part_d + (i - states);
    const int64_t n = of_a ? states : more;
    float v = 0.0f;
    if (i < states + more) {
#pragma unroll 8
        for (int64_t k = r; k < parts; k += kRows) v += in[k * n];
    }
    s[r][col] = v;
    __syncthreads();
    // by 32 rows, then by one
    if (r < 32) {
        for (int k = r + 32; k < kRows; k += 32) v += s[k][col];
        s[r][col] = v;
    }
    __syncthreads();
    if (r || i >= states + more) return;
    for (int k = 1; k < 32; ++k) v += s[k][col];
    if (of_a) {
        const int64_t c = over(i, np);
        if (i - c * np < p.states) p.dA[c * p.states + (i - c * np)] = v;
    } else if (i - states < p.channels) {
        if (p.dD) p.dD[i - states] = v;
    } else if (p.dbias) {
        p.dbias[i - states - p.channels] = v;
    }
}

// One token.  `lanes` (a power of two) threads share a channel's states, V at a time (4 where
// the count allows); the states read and written once are all that it costs: 64 of 96 slots of
// 1024 x 16 states, 9 MB in 7.2 us, most of it the latency of a slot's number and its state.
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
    float sum = 0.0f, xv = 0.0f, d = 0.0f, zv = 0.0f, skip = 0.0f;
    if (there) {                       // (on their way with the slot's number)
        xv = Storage<T>::load(x + at);
        d = Storage<T>::load(dt + at);
        if (bias) d += bias[c];
        if (z) zv = Storage<T>::load(z + at);
        if (D) skip = D[c];
    }
    if (live) {
        const int64_t bc = (b * (channels / per_group) + c / per_group) * states;
        const int64_t cn = (int64_t)c * states, sn = slot * channels * states + cn;
        if (plus) d = softplus2(f2(d)).x;
        const float u = d * xv;
        for (int n = q * V; n < states; n += lanes * V) {
            Pack<float, V> h = *reinterpret_cast<const Pack<float, V> *>(state + sn + n);
            const Pack<float, V> a = *reinterpret_cast<const Pack<float, V> *>(A + cn + n);
            const Pack<T, V> bv = *reinterpret_cast<const Pack<T, V> *>(B + bc + n);
            const Pack<T, V> cv = *reinterpret_cast<const Pack<T, V> *>(C + bc + n);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                h.v[i] = fmaf(exp2_fast(a.v[i] * kLog2e * d), h.v[i],
                              u * Storage<T>::load(&bv.v[i]));
                sum = fmaf(Storage<T>::load(&cv.v[i]), h.v[i], sum);
            }
            *reinterpret_cast<Pack<float, V> *>(new_state + sn + n) = h;
        }
    }
    for (int o = lanes / 2; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (there && q == 0) {
        sum = fmaf(skip, xv, sum);
        if (z) sum *= zv * logistic2(f2(zv)).x;
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
// tokens at least (a segment costs a second pass over its tokens).  A call, forward and
// gradients, by the rule and in one segment, 16 states:
//   1 x 1000 tokens of 64 channels, bf16       16 segments:  63, 102 us; one: 444, 860
//   8 x 200 of 256, f32                         4 segments:  63, 110 us; one:  98, 198
//   16 x 300 of 512, bf16                       5 segments:  85, 165 us; one: 137, 281
//   32 x 512 of 1024, bf16                      3 segments: 263, 773 us; one: 235, 563
//   16 x 128 of 1024, bf16                      2 segments:  95, 198 us; one:  66, 131
//   64 x 100 of 512, bf16                       2 segments: 138, 306 us; one:  54, 128
// so four and more pay, and two or three, whose two passes are hardly shorter together than the
// one, lose.
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
    a.units = (int)ceil_div(a.per_group, 64);
    a.unit_shift = unit_shift(a.per_group);
    a.shape = forward_shape(d);
    a.seg_len = p.seg_len, a.segments = p.segments;
    a.span_len = p.span_len, a.spans = p.spans, a.rows = p.rows;
    return a;
}

}  // namespace

namespace fno {
namespace scan {

fno_status_t join(const Args &a, bool both, cudaStream_t s) {
    Args p = a;
    p.shape.np = padded_states(a.states);
    const dim3 grid((unsigned)ceil_div((int64_t)a.channels * p.shape.np, 32), (unsigned)a.batch,
                    both ? 2 : 1);
    k_scan_join<<<grid, 32 * kJoinWarps, 0, s>>>(p);
    return launched();
}

fno_status_t sum_parts(const Args &a, cudaStream_t s) {
    const int64_t parts = a.rows * a.spans, cols = (int64_t)a.channels * (a.shape.np + 2);
    if (parts >= 128) k_scan_sum<8><<<(unsigned)ceil_div(cols, 8), 1024, 0, s>>>(a, parts);
    else k_scan_sum<32><<<(unsigned)ceil_div(cols, 32), 1024, 0, s>>>(a, parts);
    return launched();
}

BackwardParts backward_parts(const fno_scan_s &p) {
    const fno_scan_desc_t &d = p.d;
    const size_t np = padded_states(d.states), b = (size_t)d.batch;
    const size_t states = (size_t)d.channels * np;
    const size_t segs = b * p.segments, tiles = (size_t)ceil_div(d.length, kTile);
    const size_t parts = (size_t)p.rows * p.spans;
    const bool split = p.segments > 1, kept = tiles > 2;
    const size_t blocks = (size_t)backward_shape(d).chblocks;
    const int per_group = d.channels / d.groups;
    const size_t kept_channels =
        (size_t)d.groups * ceil_div(per_group, 64) * (2 << unit_shift(per_group));
    BackwardParts w{};
    size_t at = 0;
    const auto take = [&](size_t floats) {
        const size_t here = at;
        at += (floats * 4 + 255) & ~size_t(255);
        return here;
    };
    w.hseg = take(split ? segs * states : 0);
    w.gseg = take(split ? segs * states : 0);
    w.dseg = take(split ? segs * d.channels : 0);
    w.htile = take(kept ? b * tiles * kept_channels * np : 0);
    w.dtile = take(kept ? b * tiles * d.channels : 0);
    w.part_bc = take(blocks > 1 ? blocks * b * d.length * d.groups * 2 * d.states : 0);
    w.part_a = take(parts * states);
    w.part_d = take(parts * 2 * d.channels);
    w.bytes = at;
    return w;
}

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
    // (a block's channels, up to 256 of them, are counted in 32 bits)
    if (d.states > kMaxStates || d.length > 2147483647 - 2 * kTile ||
        d.channels > 2147483647 - 256 ||
        (double)d.batch * (double)d.length * wide > kMaxElems ||
        (double)d.batch * d.channels * d.states > kMaxElems || d.batch >= (1 << 30) - 64)
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
    // warps that the sequences and channels make, and that the SMs hold
    const auto warps = [&](const Shape &s) {
        return ceil_div(d.batch * d.groups, s.seqs) * s.chblocks * ceil_div(s.threads(), 32);
    };
    const Shape fw = forward_shape(d), bw = backward_shape(d);
    const int held = scan_warps(scan_registers(lane_states(d.states)));
    split(d.length, warps(fw), (int64_t)held * p->sms, kTile, &p->seg_len, &p->segments);
    p->span_len = p->seg_len;
    p->rows = d.batch;
    if (p->segments > 1 && (d.flags & FNO_SCAN_BACKWARD)) {
        // the last pass of the backward has twice the registers, half the warps: its spans
        // are whole numbers of segments, a wave of blocks if they can
        int spans;
        split(d.length, warps(bw), (int64_t)8 * p->sms, kTile, &p->span_len, &spans);
        const int64_t each = ceil_div(p->segments, spans);
        p->seg_len = ceil_div(ceil_div(p->span_len, each), kTile) * kTile;
        p->span_len = each * p->seg_len;
        p->segments = (int)ceil_div(d.length, p->seg_len);
    } else if (p->segments == 1) {
        // a wave of its blocks, each of which goes on with further sequences, A's gradient in
        // registers; four, if a sequence's blocks make a quarter of one (64 x 20 tokens of 20000
        // channels: 868 us; 1181 by one and a bit)
        const int64_t wave = (int64_t)8 * p->sms, each = warps(bw) / d.batch;
        const int64_t most = ceil_div(4 * each > wave ? 4 * wave : wave, each);
        p->rows = ceil_div(d.batch, ceil_div(d.batch, most));
    }
    p->spans = (int)ceil_div(d.length, p->span_len);
    // (blocks of a launch; the padded states of all sequences)
    if ((double)warps(fw) * p->segments > 2147483647.0 ||
        (double)warps(bw) * p->spans > 2147483647.0 ||
        (double)d.batch * (d.channels + 63.0 * d.groups) * fw.np > 4.0 * kMaxElems) {
        delete p;
        return FNO_ERR_UNSUPPORTED;
    }
    if (p->segments > 1)
        p->workspace = (size_t)d.batch * p->segments * d.channels * (fw.np + 1) * 4;
    if (d.flags & FNO_SCAN_BACKWARD) {
        const size_t n = backward_parts(*p).bytes;
        if (n > p->workspace) p->workspace = n;
    }
    if ((double)p->workspace > kMaxElems) {           // (bytes that no GPU has)
        delete p;
        return FNO_ERR_UNSUPPORTED;
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
    a.dseg = a.hseg ? a.hseg + (size_t)p->d.batch * p->segments * p->d.channels * a.shape.np
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
    a.htile = part(w.htile), a.dtile = part(w.dtile);
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
