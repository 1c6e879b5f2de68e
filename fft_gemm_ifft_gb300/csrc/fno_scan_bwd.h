// fno_scan_bwd.h -- the selective scan's gradients.
//
// With a_t = e^{d_t A}, u = d x, w_t = dy_t silu(z_t) and g_t the gradient of h_t,
//   g_t = C_t w_t + a_{t+1} g_{t+1}
//   dC_t = sum_c w_t h_t        dB_t = sum_c g_t u_t         (over a group's channels)
//   e_t = a_t g_t h_{t-1}       dA = sum_t d_t e_t
//   S1 = sum_n B_t g_t          S2 = sum_n A e_t
//   dx = D w + d S1,  dd = x S1 + S2,  ddt = dd softplus',  dz = dy y silu'(z)
//
// Nothing is kept from the forward.  A first pass (fno_scan_fwd.h) leaves the state in
// front of every tile of 8 tokens, from zero at the segment's start, and, where time is
// split, what the segment adds to the gradient in front of it (sum over t of
// (a_1 .. a_t) C_t w_t); a kernel joins the segments in both directions.  The second pass
// walks the tiles backwards: it runs four tokens at a time forward with their states and
// decays in registers, then those four back.
//
// A warp holds 16 channels x 4 NN states: lane = 4 dl + nl has channels 2 dl and
// 2 dl + 1 as pairs, and NN states.  The sums over states go over the four nl lanes, the
// sums over channels over the eight dl lanes.  For the latter a lane's register i holds
// state i ^ (dl & (NN - 1)): the half of the registers that it sends then is the same in
// every lane, and no value has to be chosen.  The warps of a block add up their channels'
// parts of dB and dC in shared memory; blocks of channels meet in the workspace, always in
// the same order.
#pragma once

#include "fno_scan_fwd.h"

namespace fno {
namespace scan {

constexpr int kSub = kTile / 2;

template <typename T>
struct BackwardShared {
    static __host__ __device__ size_t raw(int cb, int np) {
        return (size_t)kTile * (4 * cb + 2 * np) * sizeof(T);
    }
    static __host__ __device__ size_t bytes(int cb, int np, int nw, int slabs) {
        return 2 * raw(cb, np) +
               (size_t)kTile * ((3 + 3 * nw) * cb * 4 + np * 16 + slabs * 2 * np * 4);
    }
};

template <typename T, int NN>
__global__ void __launch_bounds__(256, 1)
k_scan_grad(const Args p) {
    using namespace ops;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
    const int cb = 16 * p.slabs, nw = threads / (2 * cb), np = 4 * NN * nw;
    const int slab = (tid >> 5) / nw, sub = (tid >> 5) - slab * nw;
    const int dl = lane >> 2, nl = lane & 3, perm = dl & (NN - 1);
    int64_t at = blockIdx.x;
    const int seg = (int)(at % p.segments);
    at /= p.segments;
    const int chb = (int)(at % p.chblocks);
    at /= p.chblocks;
    const int grp = (int)(at % p.groups);
    const int64_t b = at / p.groups;
    const int c0 = chb * cb, cols = min(cb, p.per_group - c0);
    const int64_t ch0 = (int64_t)grp * p.per_group + c0;
    const int64_t len = p.lengths ? max((int64_t)0, min((int64_t)p.lengths[b], p.length))
                                  : p.length;
    const int64_t t0 = seg * p.seg_len;
    const int64_t span = min(p.seg_len, p.length - t0);
    const int64_t have = max((int64_t)0, min(span, len - t0));
    const size_t raw_bytes = BackwardShared<T>::raw(cb, np);
    float *sd = reinterpret_cast<float *>(smem + 2 * raw_bytes);
    float *su = sd + kTile * cb, *sw = su + kTile * cb;
    float *so = sw + kTile * cb;                       // S1, S2, y: [3][nw][kTile][cb]
    float4 *sbc = reinterpret_cast<float4 *>(so + 3 * nw * kTile * cb);
    float *sp = reinterpret_cast<float *>(sbc + kTile * np);    // [slabs][kTile][2][np]

    const int64_t row0 = b * p.length + t0, at0 = row0 * p.channels + ch0;
    const T *gx = static_cast<const T *>(p.x) + at0;
    const T *gdt = static_cast<const T *>(p.dt) + at0;
    const T *gdy = static_cast<const T *>(p.dy) + at0;
    const T *gz = p.z ? static_cast<const T *>(p.z) + at0 : nullptr;
    const int64_t bc_stride = (int64_t)p.groups * p.states;
    const int64_t bc0 = row0 * bc_stride + (int64_t)grp * p.states;
    const T *gB = static_cast<const T *>(p.B) + bc0;
    const T *gC = static_cast<const T *>(p.C) + bc0;

    const auto fetch = [&](int stage_no, int64_t t) {
        const int valid = (int)min((int64_t)kTile, have - t);
        T *r = reinterpret_cast<T *>(smem + stage_no * raw_bytes);
        const int64_t o = t * p.channels;
        stage(r, gx + o, p.channels, kTile, valid, cols, cb, p.vec_c, tid, threads);
        stage(r + kTile * cb, gdt + o, p.channels, kTile, valid, cols, cb, p.vec_c, tid, threads);
        if (gz)
            stage(r + 2 * kTile * cb, gz + o, p.channels, kTile, valid, cols, cb, p.vec_c, tid,
                  threads);
        stage(r + 3 * kTile * cb, gdy + o, p.channels, kTile, valid, cols, cb, p.vec_c, tid,
              threads);
        T *rb = r + 4 * kTile * cb;
        const int64_t ob = t * bc_stride;
        stage(rb, gB + ob, bc_stride, kTile, valid, p.states, np, p.vec_n, tid, threads);
        stage(rb + kTile * np, gC + ob, bc_stride, kTile, valid, p.states, np, p.vec_n, tid,
              threads);
        cp_async_commit();
    };

    const int cl = slab * 16 + 2 * dl, n0 = (sub * 4 + nl) * NN;
    const auto half = [](float2 &v, int k) -> float & { return k ? v.y : v.x; };
    const auto each = [&](auto f) {            // f(state register, channel of the pair, index)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < NN; ++i)
                if (cl + j < cols && n0 + (i ^ perm) < p.states)
                    f(i, j, (ch0 + cl + j) * p.states + n0 + (i ^ perm));
    };
    const int64_t cn = (int64_t)p.channels * p.states;
    float2 a2[NN], da[NN], gp[NN];             // log2 e A; its gradient; a_{t+1} g_{t+1}
#pragma unroll
    for (int i = 0; i < NN; ++i) a2[i] = da[i] = gp[i] = f2(0.0f);
    each([&](int i, int j, int64_t e) { half(a2[i], j) = p.A[e] * kLog2e; });
    {
        const float *from = p.segments > 1 ? p.gseg + (b * p.segments + seg) * cn
                            : p.gsT        ? p.gsT + b * cn
                                           : nullptr;
        if (from) each([&](int i, int j, int64_t e) { half(gp[i], j) = from[e]; });
    }
    const float *hin = p.segments > 1 ? p.hseg + (b * p.segments + seg) * cn
                       : p.s0         ? p.s0 + b * cn
                                      : nullptr;
    const int64_t tiles = (p.length + kTile - 1) / kTile;

    const int pairs = cb / 2, pc = 2 * (tid & (pairs - 1)), pt = tid / pairs;
    const int pt_step = threads / pairs;
    const bool in0 = pc < cols, in1 = pc + 1 < cols;
    const bool wide = p.vec_c >= 2 * (int)sizeof(T);
    float2 bias = f2(0.0f), skip = f2(0.0f), dskip = f2(0.0f), dbias = f2(0.0f);
    if (p.bias) bias = make_float2(in0 ? p.bias[ch0 + pc] : 0.0f, in1 ? p.bias[ch0 + pc + 1] : 0.0f);
    if (p.D) skip = make_float2(in0 ? p.D[ch0 + pc] : 0.0f, in1 ? p.D[ch0 + pc + 1] : 0.0f);
    const auto put = [&](void *out, int64_t t, float2 v) {
        T *o = static_cast<T *>(out) + at0 + t * p.channels + pc;
        if (wide && in0) {
            Pack<T, 2> w2;
            Storage<T>::store(&w2.v[0], v.x);
            Storage<T>::store(&w2.v[1], v.y);
            *reinterpret_cast<Pack<T, 2> *>(o) = w2;
        } else {
            if (in0) Storage<T>::store(o, v.x);
            if (in1) Storage<T>::store(o + 1, v.y);
        }
    };
    // dB and dC of the segment's token t, or this block's part of them
    const auto put_bc = [&](int64_t t, int which, int n, float v) {
        if (p.chblocks > 1) {
            const int64_t rows = (int64_t)p.batch * p.length * p.groups;
            const int64_t row = (row0 + t) * p.groups + grp;
            p.part_bc[((chb * rows + row) * 2 + which) * p.states + n] = v;
        } else {
            T *o = static_cast<T *>(which ? p.dC : p.dB);
            Storage<T>::store(o + bc0 + t * bc_stride + n, v);
        }
    };

    const int64_t last = have > 0 ? (have - 1) / kTile * kTile : -1;
    if (last >= 0) fetch(0, last);
    int stage_no = 0;
    for (int64_t t = last; t >= 0; t -= kTile, stage_no ^= 1) {
        const int valid = (int)min((int64_t)kTile, have - t);
        // the state in front of the tile
        float2 h0[NN];
#pragma unroll
        for (int i = 0; i < NN; ++i) h0[i] = f2(0.0f);
        if (tiles > 1) {
            const int64_t ck = b * tiles + (t0 + t) / kTile;
            each([&](int i, int j, int64_t e) { half(h0[i], j) = p.hchunk[ck * cn + e]; });
            if (hin) {
                float since[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    since[j] = cl + j < cols ? p.dchunk[ck * p.channels + ch0 + cl + j] : 0.0f;
                each([&](int i, int j, int64_t e) {
                    half(h0[i], j) =
                        fmaf(exp2_fast(half(a2[i], j) * since[j]), hin[e], half(h0[i], j));
                });
            }
        } else if (hin) {
            each([&](int i, int j, int64_t e) { half(h0[i], j) = hin[e]; });
        }
        cp_async_wait<0>();
        __syncthreads();
        if (t >= kTile) fetch(stage_no ^ 1, t - kTile);
        const T *r = reinterpret_cast<const T *>(smem + stage_no * raw_bytes);
        const T *rb = r + 4 * kTile * cb;
        for (int k = pt; k < kTile; k += pt_step) {
            const float2 xv = Storage<T>::load2(r + k * cb + pc);
            float2 d = add2(Storage<T>::load2(r + (kTile + k) * cb + pc), bias);
            float2 w = Storage<T>::load2(r + (3 * kTile + k) * cb + pc);
            if (p.softplus) d = make_float2(softplus(d.x), softplus(d.y));
            if (k >= valid || !in0) d.x = 0.0f;
            if (k >= valid || !in1) d.y = 0.0f;
            if (gz) {
                const float2 zv = Storage<T>::load2(r + (2 * kTile + k) * cb + pc);
                w = make_float2(w.x * zv.x * logistic(zv.x), w.y * zv.y * logistic(zv.y));
            }
            *reinterpret_cast<float2 *>(sd + k * cb + pc) = d;
            *reinterpret_cast<float2 *>(su + k * cb + pc) = mul2(d, xv);
            *reinterpret_cast<float2 *>(sw + k * cb + pc) = w;
        }
        for (int i = tid; i < kTile * np; i += threads) {
            const float bv = Storage<T>::load(rb + i), cv = Storage<T>::load(rb + kTile * np + i);
            sbc[i] = make_float4(bv, bv, cv, cv);
        }
        __syncthreads();

        // a tile's tokens beyond the last have d = u = w = 0: they change nothing
        const auto step = [&](int k, float2 *a, const float2 *from, float2 *to) {
            const float2 d = *reinterpret_cast<const float2 *>(sd + k * cb + cl);
            const float2 u = *reinterpret_cast<const float2 *>(su + k * cb + cl);
#pragma unroll
            for (int i = 0; i < NN; ++i) {
                const float2 bv = *reinterpret_cast<const float2 *>(sbc + k * np + n0 + (i ^ perm));
                const float2 q = mul2(a2[i], d);
                a[i] = make_float2(exp2_fast(q.x), exp2_fast(q.y));
                to[i] = fma2(a[i], from[i], mul2(u, bv));
            }
        };
        float2 hm[NN];
#pragma unroll
        for (int i = 0; i < NN; ++i) hm[i] = h0[i];
#pragma unroll
        for (int k = 0; k < kSub; ++k) {
            float2 a[NN];
            step(k, a, hm, hm);
        }
#pragma unroll 1
        for (int part = 1; part >= 0; --part) {
            const int k0 = part * kSub;
            float2 a[kSub][NN], h[kSub + 1][NN];
#pragma unroll
            for (int i = 0; i < NN; ++i) h[0][i] = part ? hm[i] : h0[i];
#pragma unroll
            for (int k = 0; k < kSub; ++k) step(k0 + k, a[k], h[k], h[k + 1]);
#pragma unroll
            for (int k = kSub - 1; k >= 0; --k) {
                const int kk = k0 + k;
                const float2 d = *reinterpret_cast<const float2 *>(sd + kk * cb + cl);
                const float2 u = *reinterpret_cast<const float2 *>(su + kk * cb + cl);
                const float2 w = *reinterpret_cast<const float2 *>(sw + kk * cb + cl);
                float2 s1 = f2(0.0f), s2 = f2(0.0f), y = f2(0.0f);
                float vb[NN], vc[NN];
#pragma unroll
                for (int i = 0; i < NN; ++i) {
                    const float4 bc = sbc[kk * np + n0 + (i ^ perm)];
                    const float2 bv = make_float2(bc.x, bc.y), cv = make_float2(bc.z, bc.w);
                    const float2 g = fma2(cv, w, gp[i]);
                    s1 = fma2(g, bv, s1);
                    y = fma2(cv, h[k + 1][i], y);
                    const float2 pb = mul2(g, u), pw = mul2(w, h[k + 1][i]);
                    vb[i] = pb.x + pb.y;
                    vc[i] = pw.x + pw.y;
                    gp[i] = mul2(a[k][i], g);
                    const float2 e = mul2(gp[i], h[k][i]);
                    s2 = fma2(a2[i], e, s2);
                    da[i] = fma2(d, e, da[i]);
                }
                // over the channels: a lane ends with one state of dB or of dC
                if (NN == 4) {
#pragma unroll
                    for (int i = 0; i < NN / 2; ++i) {
                        vb[i] += __shfl_xor_sync(0xffffffffu, vb[i + NN / 2], 8);
                        vc[i] += __shfl_xor_sync(0xffffffffu, vc[i + NN / 2], 8);
                    }
                }
                if (NN >= 2) {
                    vb[0] += __shfl_xor_sync(0xffffffffu, vb[NN / 2 == 2 ? 1 : NN - 1], 4);
                    vc[0] += __shfl_xor_sync(0xffffffffu, vc[NN / 2 == 2 ? 1 : NN - 1], 4);
                }
                const bool second = dl & 4;
                float v = (second ? vc[0] : vb[0]) +
                          __shfl_xor_sync(0xffffffffu, second ? vb[0] : vc[0], 16);
                if (NN < 4) v += __shfl_xor_sync(0xffffffffu, v, 8);
                if (NN < 2) v += __shfl_xor_sync(0xffffffffu, v, 4);
                if ((dl & 3) < NN)
                    sp[((slab * kTile + kk) * 2 + (dl >> 2)) * np + n0 + perm] = v;
                // over the states: even lanes the first channel, odd ones the second
                const bool odd = nl & 1;
                float o1 = (odd ? s1.y : s1.x) +
                           __shfl_xor_sync(0xffffffffu, odd ? s1.x : s1.y, 1);
                float o2 = (odd ? s2.y : s2.x) +
                           __shfl_xor_sync(0xffffffffu, odd ? s2.x : s2.y, 1);
                float o3 = (odd ? y.y : y.x) + __shfl_xor_sync(0xffffffffu, odd ? y.x : y.y, 1);
                o1 += __shfl_xor_sync(0xffffffffu, o1, 2);
                o2 += __shfl_xor_sync(0xffffffffu, o2, 2);
                o3 += __shfl_xor_sync(0xffffffffu, o3, 2);
                if (nl < 2) {
                    float *o = so + (sub * kTile + kk) * cb + cl + nl;
                    o[0] = o1;
                    o[nw * kTile * cb] = o2;
                    o[2 * nw * kTile * cb] = o3;
                }
            }
        }
        __syncthreads();
        for (int k = pt; k < valid; k += pt_step) {
            const float *o = so + k * cb + pc;
            float2 v[3];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                v[q] = *reinterpret_cast<const float2 *>(o + q * nw * kTile * cb);
                for (int w = 1; w < nw; ++w)
                    v[q] = add2(v[q], *reinterpret_cast<const float2 *>(
                                          o + (q * nw + w) * kTile * cb));
            }
            const float2 xv = Storage<T>::load2(r + k * cb + pc);
            const float2 d = *reinterpret_cast<const float2 *>(sd + k * cb + pc);
            const float2 w = *reinterpret_cast<const float2 *>(sw + k * cb + pc);
            put(p.dx, t + k, fma2(skip, w, mul2(d, v[0])));
            dskip = fma2(w, xv, dskip);
            float2 dd = fma2(xv, v[0], mul2(v[1], f2(kLn2)));
            if (p.softplus) {
                const float2 dtv = add2(Storage<T>::load2(r + (kTile + k) * cb + pc), bias);
                dd = mul2(dd, make_float2(logistic(dtv.x), logistic(dtv.y)));
            }
            put(p.ddt, t + k, dd);
            dbias = add2(dbias, dd);
            if (gz) {
                const float2 zv = Storage<T>::load2(r + (2 * kTile + k) * cb + pc);
                const float2 gy = Storage<T>::load2(r + (3 * kTile + k) * cb + pc);
                const float2 y = fma2(skip, xv, v[2]);
                const float2 l = make_float2(logistic(zv.x), logistic(zv.y));
                put(p.dz, t + k,
                    make_float2(gy.x * y.x * l.x * fmaf(zv.x, 1.0f - l.x, 1.0f),
                                gy.y * y.y * l.y * fmaf(zv.y, 1.0f - l.y, 1.0f)));
            }
        }
        for (int i = tid; i < valid * 2 * np; i += threads) {
            const int n = i & (np - 1), which = (i / np) & 1, k = i / (2 * np);
            if (n >= p.states) continue;
            float v = 0.0f;
            for (int s = 0; s < p.slabs; ++s) v += sp[((s * kTile + k) * 2 + which) * np + n];
            put_bc(t + k, which, n, v);
        }
    }
    for (int64_t t = have + pt; t < span; t += pt_step) {
        put(p.dx, t, f2(0.0f));
        put(p.ddt, t, f2(0.0f));
        if (gz) put(p.dz, t, f2(0.0f));
    }
    for (int64_t i = have * 2 * np + tid; i < span * 2 * np; i += threads) {
        const int n = (int)(i & (np - 1));
        if (n < p.states) put_bc(i / (2 * np), (int)(i / np) & 1, n, 0.0f);
    }
    const int64_t s = b * p.segments + seg;
    each([&](int i, int j, int64_t e) { p.part_a[s * cn + e] = half(da[i], j); });
    if (p.ds0 && seg == 0)
        each([&](int i, int j, int64_t e) { p.ds0[b * cn + e] = half(gp[i], j); });
    // the bias' and D's gradients: the threads that share a pair of channels
    __syncthreads();
    float4 *sum = reinterpret_cast<float4 *>(so);
    sum[tid] = make_float4(dskip.x, dskip.y, dbias.x, dbias.y);
    __syncthreads();
    if (pt == 0) {
        float4 v = sum[tid];
        for (int k = 1; k < pt_step; ++k) {
            const float4 o = sum[tid + k * pairs];
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        float *o = p.part_d + s * 2 * p.channels + ch0 + pc;
        if (in0) o[0] = v.x, o[p.channels] = v.z;
        if (in1) o[1] = v.y, o[p.channels + 1] = v.w;
    }
}

// dB and dC: the sum of the blocks' parts (rows of 2 x states) of the tokens there.
template <typename T>
__global__ void __launch_bounds__(256)
k_scan_sum_bc(const Args p) {
    const int64_t rows = (int64_t)p.batch * p.length * p.groups, n = rows * 2 * p.states;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = p.part_bc[i];
    for (int k = 1; k < p.chblocks; ++k) v += p.part_bc[k * n + i];
    const int64_t row = i / (2 * p.states);
    const int e = (int)(i - row * 2 * p.states);
    T *o = static_cast<T *>(e >= p.states ? p.dC : p.dB);
    Storage<T>::store(o + row * p.states + (e >= p.states ? e - p.states : e), v);
}

// out[i] = the sum of `parts` values n apart: 32 columns a block, its 16 rows of threads
// over the parts; scaled (dA's pairs carry no factor, so 1).
constexpr int kSumRows = 16;
template <int kOuts>
__global__ void __launch_bounds__(32 * kSumRows)
k_scan_sum(const float *__restrict__ in, float *__restrict__ out0, float *__restrict__ out1,
           int64_t n, int64_t parts) {
    __shared__ float s[kSumRows][33];
    const int64_t i = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float v = 0.0f;
    if (i < n) {
#pragma unroll 8
        for (int64_t k = threadIdx.y; k < parts; k += kSumRows) v += in[k * n + i];
    }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y || i >= n) return;
    for (int k = 1; k < kSumRows; ++k) v += s[k][threadIdx.x];
    if (kOuts == 1) out0[i] = v;
    else if (i < n / 2) { if (out0) out0[i] = v; }
    else if (out1) out1[i - n / 2] = v;
}

template <typename T, int NN>
fno_status_t launch_grad(const Args &a, cudaStream_t s) {
    const int nw = NN == 4 ? state_warps(a.states) : 1, cb = 16 * a.slabs;
    const size_t bytes = BackwardShared<T>::bytes(cb, 4 * NN * nw, nw, a.slabs);
    const auto kernel = k_scan_grad<T, NN>;
    if (bytes > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
            cudaSuccess) {
        cudaGetLastError();
        return FNO_ERR_CUDA;
    }
    const int64_t blocks = (int64_t)a.batch * a.groups * a.chblocks * a.segments;
    kernel<<<(unsigned)blocks, 2 * cb * nw, bytes, s>>>(a);
    return ops::launched();
}

template <typename T>
fno_status_t backward_of(const fno_scan_s &p, Args a, cudaStream_t s) {
    using ops::ceil_div;
    a.segments = p.bwd_segments;
    a.seg_len = p.bwd_seg_len;
    fno_status_t st = FNO_OK;
    if (a.segments > 1) {
        st = scan_pass<T, kBoth>(a, forward_slabs(p), s);
        if (st == FNO_OK) st = join(a, false, s);
        if (st == FNO_OK) st = join(a, true, s);
    } else if (a.length > kTile) {
        st = scan_pass<T, kTiles>(a, forward_slabs(p), s);
    }
    if (st != FNO_OK) return st;
    a.slabs = backward_slabs(p);
    a.chblocks = (int)ceil_div(a.per_group, 16 * a.slabs);
    switch (lane_states(a.states)) {
        case 1: st = launch_grad<T, 1>(a, s); break;
        case 2: st = launch_grad<T, 2>(a, s); break;
        default: st = launch_grad<T, 4>(a, s); break;
    }
    if (st != FNO_OK) return st;
    if (a.chblocks > 1) {
        const int64_t n = (int64_t)a.batch * a.length * a.groups * 2 * a.states;
        k_scan_sum_bc<T><<<(unsigned)ceil_div(n, 256), 256, 0, s>>>(a);
    }
    const int64_t cn = (int64_t)a.channels * a.states, parts = (int64_t)a.batch * a.segments;
    const dim3 threads(32, kSumRows);
    k_scan_sum<1><<<(unsigned)ceil_div(cn, 32), threads, 0, s>>>(a.part_a, a.dA, nullptr, cn,
                                                                 parts);
    if (a.dD || a.dbias)
        k_scan_sum<2><<<(unsigned)ceil_div(2 * a.channels, 32), threads, 0, s>>>(
            a.part_d, a.dD, a.dbias, 2 * (int64_t)a.channels, parts);
    return ops::launched();
}

}  // namespace scan
}  // namespace fno
