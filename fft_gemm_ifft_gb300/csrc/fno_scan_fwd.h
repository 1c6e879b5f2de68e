// fno_scan_fwd.h -- the selective scan forward, and the pass over the states that both
// directions make when the time axis is split.
//
// For each channel c and state n of a sequence
//   h_t = e^{d_t A} h_{t-1} + (d_t x_t) B_t,   y_t = sum_n C_t h_t,
// one exponential and four multiply-adds an element (c, n) and token, and no matrix
// product: the decay differs for every element.  So the exponentials and the issue
// slots bound it, not memory (16 states: 8 to 12 bytes a channel and token).
//
// A warp holds 32 channels x 4 NN states in registers: lane = 4 dl + nl has channels
// 4 dl .. 4 dl + 3 and the NN states from nl NN on, pairs of channels in one
// instruction.  The steps d and the inputs u = d x are computed once for each channel
// and token, by threads side by side, and read from shared memory as float4; B and C lie
// there twice each, as the packed products want them.  A token's sums over states take
// three shuffles for 16 elements: each lane ends with one channel.  More than 16 states
// are shared by several warps, whose sums meet in shared memory.
//
// When the sequences and channels do not fill the GPU, time is split into segments:
// one pass finds each segment's state from zero, a kernel joins them by
// e^{A sum d}, and the second pass starts from the joined states.
#pragma once

#include "fno_scan.h"

namespace fno {
namespace scan {

// The outputs; the segments' states; the segments' and tiles' states and the gradients'
// sums; the tiles' states of an unsplit time axis.
enum Mode { kFull, kStates, kBoth, kTiles };
constexpr bool with_c(Mode m) { return m == kFull || m == kBoth; }
constexpr int fields_of(Mode m) { return m == kFull ? 3 : m == kBoth ? 4 : 2; }

template <typename T>
struct ForwardShared {
    // raw tiles (two stages): x, dt, z (or dy, z backward), B, C; float tiles: the steps,
    // the inputs, the output's gradients, B and C twice each, the partial sums of y
    static __host__ __device__ size_t raw(int cb, int np, int fields) {
        return (size_t)kTile * (fields * cb + 2 * np) * sizeof(T);
    }
    static __host__ __device__ size_t bytes(int cb, int np, int warps, Mode m) {
        const int rows = 2 + (m == kFull ? warps : m == kBoth ? 1 : 0);
        return 2 * raw(cb, np, fields_of(m)) + (size_t)kTile * (rows * cb * 4 + np * 16);
    }
};

template <typename T, int NN, Mode M>
__global__ void __launch_bounds__(256, 2)
k_scan(const Args p) {
    using namespace ops;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
    const int cb = 32 * p.slabs, nw = threads / cb, np = 4 * NN * nw;
    const int slab = (tid >> 5) / nw, sub = (tid >> 5) - slab * nw;
    const int dl = lane >> 2, nl = lane & 3;
    int64_t at = blockIdx.x;
    const int seg = (int)(at % p.segments);
    at /= p.segments;
    const int chb = (int)(at % p.chblocks);
    at /= p.chblocks;
    const int grp = (int)(at % p.groups);
    const int64_t b = at / p.groups;
    const int c0 = chb * cb, cols = min(cb, p.per_group - c0);      // in the group
    const int64_t ch0 = (int64_t)grp * p.per_group + c0;            // of all channels
    const int64_t len = p.lengths ? max((int64_t)0, min((int64_t)p.lengths[b], p.length))
                                  : p.length;
    const int64_t t0 = seg * p.seg_len;
    const int64_t span = min(p.seg_len, p.length - t0);             // tokens of the segment
    const int64_t have = max((int64_t)0, min(span, len - t0));      // that are there
    constexpr int kFields = fields_of(M);
    const size_t raw_bytes = ForwardShared<T>::raw(cb, np, kFields);
    float *sd = reinterpret_cast<float *>(smem + 2 * raw_bytes);
    float *su = sd + kTile * cb;
    float *sy = su + kTile * cb;                                    // kBoth: dy silu(z)
    float4 *sbc = reinterpret_cast<float4 *>(sy + (M == kFull ? nw : M == kBoth ? 1 : 0) *
                                                      kTile * cb);

    const int64_t row0 = b * p.length + t0;
    const T *gx = static_cast<const T *>(p.x) + row0 * p.channels + ch0;
    const T *gdt = static_cast<const T *>(p.dt) + row0 * p.channels + ch0;
    const T *gz = p.z && with_c(M) ? static_cast<const T *>(p.z) + row0 * p.channels + ch0
                                      : nullptr;
    const T *gdy = M == kBoth ? static_cast<const T *>(p.dy) + row0 * p.channels + ch0 : nullptr;
    const int64_t bc_stride = (int64_t)p.groups * p.states;
    const T *gB = static_cast<const T *>(p.B) + row0 * bc_stride + (int64_t)grp * p.states;
    const T *gC = static_cast<const T *>(p.C) + row0 * bc_stride + (int64_t)grp * p.states;

    const auto fetch = [&](int stage_no, int64_t t) {
        const int valid = (int)min((int64_t)kTile, have - t);
        T *r = reinterpret_cast<T *>(smem + stage_no * raw_bytes);
        const int64_t o = t * p.channels;
        stage(r, gx + o, p.channels, kTile, valid, cols, cb, p.vec_c, tid, threads);
        stage(r + kTile * cb, gdt + o, p.channels, kTile, valid, cols, cb, p.vec_c, tid, threads);
        if (gz)
            stage(r + 2 * kTile * cb, gz + o, p.channels, kTile, valid, cols, cb, p.vec_c, tid,
                  threads);
        if (M == kBoth)
            stage(r + 3 * kTile * cb, gdy + o, p.channels, kTile, valid, cols, cb, p.vec_c, tid,
                  threads);
        T *rb = r + kFields * kTile * cb;
        stage(rb, gB + t * bc_stride, bc_stride, kTile, valid, p.states, np, p.vec_n, tid,
              threads);
        if (with_c(M))
            stage(rb + kTile * np, gC + t * bc_stride, bc_stride, kTile, valid, p.states, np,
                  p.vec_n, tid, threads);
        cp_async_commit();
    };

    // this lane's elements: channels cl + j, states n0 + i, as pairs of channels
    const int cl = slab * 32 + 4 * dl, n0 = (sub * 4 + nl) * NN;
    float2 a2[2][NN], h[2][NN], pr[2][NN], g[2][NN];
    float dsum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const auto each = [&](auto f) {                     // f(pair, half, state, index in (c, n))
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < NN; ++i)
                if (cl + j < cols && n0 + i < p.states)
                    f(j >> 1, j & 1, i, (ch0 + cl + j) * p.states + n0 + i);
    };
    const auto half = [](float2 &v, int k) -> float & { return k ? v.y : v.x; };
    const int64_t cn = (int64_t)p.channels * p.states;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NN; ++i) {
            a2[j][i] = h[j][i] = g[j][i] = f2(0.0f);
            pr[j][i] = f2(1.0f);
        }
    each([&](int j, int k, int i, int64_t e) { half(a2[j][i], k) = p.A[e] * kLog2e; });
    if (M == kFull) {
        const float *from = p.segments > 1 ? p.hseg + (b * p.segments + seg) * cn
                            : p.s0         ? p.s0 + b * cn
                                           : nullptr;
        if (from) each([&](int j, int k, int i, int64_t e) { half(h[j][i], k) = from[e]; });
    }

    // the pair of channels that this thread prepares and finishes, and its tokens
    const int pairs = cb / 2, pc = 2 * (tid & (pairs - 1)), pt = tid / pairs;
    const int pt_step = threads / pairs;
    const bool in0 = pc < cols, in1 = pc + 1 < cols;
    const bool wide = p.vec_c >= 2 * (int)sizeof(T);
    float2 bias = f2(0.0f), skip = f2(0.0f);
    if (p.bias) bias = make_float2(in0 ? p.bias[ch0 + pc] : 0.0f, in1 ? p.bias[ch0 + pc + 1] : 0.0f);
    if (M == kFull && p.D)
        skip = make_float2(in0 ? p.D[ch0 + pc] : 0.0f, in1 ? p.D[ch0 + pc + 1] : 0.0f);

    if (have > 0) fetch(0, 0);
    int stage_no = 0;
    for (int64_t t = 0; t < have; t += kTile, stage_no ^= 1) {
        const int valid = (int)min((int64_t)kTile, have - t);
        cp_async_wait<0>();
        __syncthreads();
        if (t + kTile < have) fetch(stage_no ^ 1, t + kTile);
        const T *r = reinterpret_cast<const T *>(smem + stage_no * raw_bytes);
        const T *rb = r + kFields * kTile * cb;
        for (int k = pt; k < kTile; k += pt_step) {
            const float2 xv = Storage<T>::load2(r + k * cb + pc);
            float2 d = Storage<T>::load2(r + (kTile + k) * cb + pc);
            d = add2(d, bias);
            if (p.softplus) d = make_float2(softplus(d.x), softplus(d.y));
            // (nothing lies beyond the last token or channel)
            if (k >= valid || !in0) d.x = 0.0f;
            if (k >= valid || !in1) d.y = 0.0f;
            *reinterpret_cast<float2 *>(sd + k * cb + pc) = d;
            *reinterpret_cast<float2 *>(su + k * cb + pc) = mul2(d, xv);
            if (M == kBoth) {
                float2 gy = Storage<T>::load2(r + (3 * kTile + k) * cb + pc);
                if (gz) {
                    const float2 zv = Storage<T>::load2(r + (2 * kTile + k) * cb + pc);
                    gy = make_float2(gy.x * zv.x * logistic(zv.x), gy.y * zv.y * logistic(zv.y));
                }
                *reinterpret_cast<float2 *>(sy + k * cb + pc) = gy;
            }
        }
        for (int i = tid; i < kTile * np; i += threads) {
            const float bv = Storage<T>::load(rb + i);
            const float cv = with_c(M) ? Storage<T>::load(rb + kTile * np + i) : 0.0f;
            sbc[i] = make_float4(bv, bv, cv, cv);
        }
        __syncthreads();
        if (M == kBoth || M == kTiles) {
            const int64_t ck = b * ((p.length + kTile - 1) / kTile) + (t0 + t) / kTile;
            each([&](int j, int k, int i, int64_t e) { p.hchunk[ck * cn + e] = half(h[j][i], k); });
            if (sub == 0 && nl == 0)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (cl + j < cols) p.dchunk[ck * p.channels + ch0 + cl + j] = dsum[j];
        }
#pragma unroll 2
        for (int k = 0; k < kTile; ++k) {
            if (k >= valid) break;
            const float4 d4 = *reinterpret_cast<const float4 *>(sd + k * cb + cl);
            const float4 u4 = *reinterpret_cast<const float4 *>(su + k * cb + cl);
            const float2 d[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
            const float2 u[2] = {make_float2(u4.x, u4.y), make_float2(u4.z, u4.w)};
            float2 gy[2];
            if (M == kBoth) {
                const float4 g4 = *reinterpret_cast<const float4 *>(sy + k * cb + cl);
                gy[0] = make_float2(g4.x, g4.y), gy[1] = make_float2(g4.z, g4.w);
            }
            if (M != kFull) dsum[0] += d4.x, dsum[1] += d4.y, dsum[2] += d4.z, dsum[3] += d4.w;
            float2 y[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
            for (int i = 0; i < NN; ++i) {
                const float4 bc = sbc[k * np + n0 + i];
                const float2 bv = make_float2(bc.x, bc.y), cv = make_float2(bc.z, bc.w);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 q = mul2(a2[j][i], d[j]);
                    const float2 a = make_float2(exp2_fast(q.x), exp2_fast(q.y));
                    h[j][i] = fma2(a, h[j][i], mul2(u[j], bv));
                    if (M == kFull) y[j] = fma2(cv, h[j][i], y[j]);
                    if (M == kBoth) {
                        pr[j][i] = mul2(pr[j][i], a);
                        g[j][i] = fma2(pr[j][i], mul2(cv, gy[j]), g[j][i]);
                    }
                }
            }
            if (M == kFull) {
                // the quad's sums: lane nl ends with channel 4 dl + nl
                const bool hi = nl & 2, odd = nl & 1;
                float2 keep = hi ? y[1] : y[0];
                const float2 send = hi ? y[0] : y[1];
                keep.x += __shfl_xor_sync(0xffffffffu, send.x, 2);
                keep.y += __shfl_xor_sync(0xffffffffu, send.y, 2);
                const float v = (odd ? keep.y : keep.x) +
                                __shfl_xor_sync(0xffffffffu, odd ? keep.x : keep.y, 1);
                sy[(sub * kTile + k) * cb + slab * 32 + lane] = v;
            }
        }
        if (M == kFull) {
            __syncthreads();
            T *out = static_cast<T *>(p.y) + (row0 + t) * p.channels + ch0 + pc;
            for (int k = pt; k < valid; k += pt_step) {
                float2 v = *reinterpret_cast<const float2 *>(sy + k * cb + pc);
                for (int w = 1; w < nw; ++w)
                    v = add2(v, *reinterpret_cast<const float2 *>(sy + (w * kTile + k) * cb + pc));
                v = fma2(skip, Storage<T>::load2(r + k * cb + pc), v);
                if (gz) {
                    const float2 zv = Storage<T>::load2(r + (2 * kTile + k) * cb + pc);
                    v = make_float2(v.x * zv.x * logistic(zv.x), v.y * zv.y * logistic(zv.y));
                }
                T *o = out + (int64_t)k * p.channels;
                if (wide && in0) {
                    Pack<T, 2> w2;
                    Storage<T>::store(&w2.v[0], v.x);
                    Storage<T>::store(&w2.v[1], v.y);
                    *reinterpret_cast<Pack<T, 2> *>(o) = w2;
                } else {
                    if (in0) Storage<T>::store(o, v.x);
                    if (in1) Storage<T>::store(o + 1, v.y);
                }
            }
        }
    }
    if (M == kFull) {
        T *out = static_cast<T *>(p.y) + row0 * p.channels + ch0 + pc;
        for (int64_t t = have + pt; t < span; t += pt_step) {
            if (in0) Storage<T>::store(out + t * p.channels, 0.0f);
            if (in1) Storage<T>::store(out + t * p.channels + 1, 0.0f);
        }
        if (p.sT && seg == p.segments - 1)
            each([&](int j, int k, int i, int64_t e) { p.sT[b * cn + e] = half(h[j][i], k); });
    } else if (M != kTiles) {
        const int64_t s = b * p.segments + seg;
        each([&](int j, int k, int i, int64_t e) { p.hseg[s * cn + e] = half(h[j][i], k); });
        if (M == kBoth)
            each([&](int j, int k, int i, int64_t e) { p.gseg[s * cn + e] = half(g[j][i], k); });
        if (sub == 0 && nl == 0)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (cl + j < cols) p.dseg[s * p.channels + ch0 + cl + j] = dsum[j];
    }
}

template <typename T, int NN, Mode M>
fno_status_t launch_scan(const Args &a, cudaStream_t s) {
    const int cb = 32 * a.slabs, nw = NN == 4 ? state_warps(a.states) : 1;
    const size_t bytes = ForwardShared<T>::bytes(cb, 4 * NN * nw, nw, M);
    const auto kernel = k_scan<T, NN, M>;
    if (bytes > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
            cudaSuccess) {
        cudaGetLastError();
        return FNO_ERR_CUDA;
    }
    const int64_t blocks = (int64_t)a.batch * a.groups * a.chblocks * a.segments;
    kernel<<<(unsigned)blocks, cb * nw, bytes, s>>>(a);
    return ops::launched();
}
template <typename T, Mode M>
fno_status_t scan_pass(Args a, int slabs, cudaStream_t s) {
    a.slabs = slabs;
    a.chblocks = (int)ops::ceil_div(a.per_group, 32 * slabs);
    switch (lane_states(a.states)) {
        case 1: return launch_scan<T, 1, M>(a, s);
        case 2: return launch_scan<T, 2, M>(a, s);
        default: return launch_scan<T, 4, M>(a, s);
    }
}

template <typename T>
fno_status_t forward_of(const fno_scan_s &p, Args a, cudaStream_t s) {
    const int slabs = forward_slabs(p);
    a.segments = p.segments;
    a.seg_len = p.seg_len;
    if (a.segments > 1) {
        fno_status_t st = scan_pass<T, kStates>(a, slabs, s);
        if (st == FNO_OK) st = join(a, false, s);
        if (st != FNO_OK) return st;
    }
    return scan_pass<T, kFull>(a, slabs, s);
}

}  // namespace scan
}  // namespace fno
