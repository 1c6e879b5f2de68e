// fno_scan_fwd.h -- the selective scan forward, and the pass over the states that both
// directions make when the time axis is split.
//
// For each channel c and state n of a sequence
//   h_t = e^{d_t A} h_{t-1} + (d_t x_t) B_t,   y_t = sum_n C_t h_t,
// one exponential and four multiply-adds an element (c, n) and token, and no matrix
// product: the decay differs for every element.  So instructions bound it, not device memory
// (16 states: 8 to 12 bytes a channel and token).  With everything in registers this loop takes
// 1.7 cycles of an SM for 32 elements (a packed multiply-add occupies two issue slots, as two
// single ones do); the kernel, with softplus, gates, loads and stores, takes 3.2 (4096 tokens
// of 2048 channels and 16 states in bfloat16: 47 us), half of the issue slots at 12 warps an SM.
//
// A lane holds two channels x up to 16 states in registers, so that nothing is summed over
// lanes: its channels' steps, inputs and outputs stay in its registers, from and to global
// memory.  B and C, which all channels share, lie in shared memory as floats, and a whole warp
// reads the same ones at once.  (Four channels x four states a lane read four addresses a warp,
// for which shared memory takes four times as long, and staged the steps there as well: 62 us;
// pairs of lanes sharing 16 states, 20 warps an SM in place of 12: 59 us.)  More than 16 states
// are shared by several warps, whose sums meet in shared memory.
//
// When the sequences and channels do not fill the GPU, time is split into segments:
// one pass finds each segment's state from zero, a kernel joins them by
// e^{A sum d}, and the second pass starts from the joined states.
#pragma once

#include "fno_scan.h"

namespace fno {
namespace scan {

// The outputs from the states in front of the segments; the states at the segments' ends
// and in front of the tiles (each if wanted); from the last token, what each segment adds to
// the gradient of the state in front of it: r_t = a_t (r_{t+1} + C_t w_t), w = dy silu(z).
enum Mode { kFull, kStates, kBack };
// At 168 registers an SM holds 12 warps (4096 tokens of 2048 channels: 47 us; at 128 registers
// and 16 warps 51 us); short sequences, which are mostly the latency of their first loads, take
// the 16 warps (4096 x 12 tokens of 64 channels in float32: 42 us; 48 us at 168).
constexpr int kShort = 32;
template <typename T, int NS, Mode M, int REGS>
__global__ void __maxnreg__(REGS)
k_scan(const Args p) {
    using namespace ops;
    constexpr int G = M == kFull ? 1 : 2;             // tokens worked on together
    constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;    // pairs of B or C fetched ahead
    extern __shared__ __align__(16) float sbc[];      // [2][seqs][kTile][2][np], sums of y
    const int tid = threadIdx.x, threads = blockDim.x;
    const Shape s = p.shape;
    const int np = s.np;
    const Unit u(tid, s);
    int64_t at = blockIdx.x;
    const int seg = (int)(at % p.segments);
    at /= p.segments;
    const int chb = (int)(at % s.chblocks);
    const int64_t seq0 = at / s.chblocks * s.seqs, all = (int64_t)p.batch * p.groups;
    const int64_t seq = seq0 + u.seq, b = min(seq, all - 1) / p.groups;
    const int grp = (int)(min(seq, all - 1) - b * p.groups);
    const int c = ((chb * s.slabs + u.slab) * s.lanes + u.lane) * 2;     // in the group
    const int left = seq < all ? p.per_group - c : 0;
    const int64_t ch = (int64_t)grp * p.per_group + c;
    const int64_t t0 = seg * p.seg_len;
    const int span = (int)min(p.seg_len, p.length - t0);
    const auto tokens = [&](int64_t sequence) {       // of the segment that are there
        const int64_t n = p.lengths ? max(0, p.lengths[sequence]) : p.length;
        return (int)max((int64_t)0, min((int64_t)span, n - t0));
    };
    const int have = tokens(b);
    int most = have, least = have;                    // of any sequence of the block
    for (int k = 0; k < s.seqs && p.lengths; ++k) {
        const int n = tokens(min(seq0 + k, all - 1) / p.groups);
        most = max(most, n);
        least = min(least, n);
    }
    const int64_t row0 = b * p.length + t0;
    const bool wide = p.vec_c >= 2 * (int)sizeof(T);
    const bool whole_block = wide && (chb + 1) * s.slabs * s.lanes * 2 <= p.per_group &&
                             seq0 + s.seqs <= all;

    // B and C of a tile: a thread has one pair of states of one of them (of a sequence) and
    // every bc_step-th token
    const int combos = s.seqs * np;                   // (no more than there are threads)
    const int bc_step = threads / combos, bc_k = tid / combos, bc_tile = 2 * kTile * combos;
    const T *bc_from;
    int bc_to, bc_have, bc_left;
    {
        const int i = tid - bc_k * combos, q = i / np, which = (i - q * np) / (np / 2);
        const int n = 2 * (i - q * np - which * (np / 2));
        const int64_t sq = min(seq0 + q, all - 1), bb = sq / p.groups;
        bc_have = p.lengths ? tokens(bb) : span;
        bc_from = static_cast<const T *>(which || M == kBack ? p.C : p.B) +
                  ((bb * p.length + t0 + (M == kBack ? bc_have - 1 - bc_k : bc_k)) * p.groups +
                   (sq - bb * p.groups)) * p.states + n;
        bc_to = ((q * kTile + bc_k) * 2 + which) * np + n;
        bc_left = bc_k < bc_step && (!which || M == kFull) ? p.states - n : 0;
    }
    const bool bc_wide = p.vec_n >= 2 * (int)sizeof(T);
    const int64_t bc_row = (M == kBack ? -1 : 1) * (int64_t)p.groups * p.states;
    // the thread's m-th pair of the tile at t
    const auto bc_load = [&](int m, int t) {
        const int k = bc_k + m * bc_step;
        return load_pair(bc_from + (int64_t)(t + m * bc_step) * bc_row, bc_wide,
                         k < kTile && t + k < bc_have ? bc_left : 0);
    };
    const auto bc_store = [&](int buffer, int m, Pair<T> v) {
        if (bc_k + m * bc_step < kTile && bc_k < bc_step)
            *reinterpret_cast<float2 *>(sbc + buffer * bc_tile + bc_to + m * bc_step * 2 * np) =
                to_float2(v);
    };

    float2 a2[2][NS / 2], h[2][NS / 2], dsum = f2(0.0f);
    const int n0 = u.sub * NS;
    load_states<NS>(p.A + ch * p.states + n0, left, p.states - n0, p.states, a2);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NS / 2; ++i) {
            a2[j][i] = mul2(a2[j][i], f2(kLog2e));
            h[j][i] = f2(0.0f);
        }
    float2 bias = f2(0.0f), skip = f2(0.0f);
    if (p.bias) bias = make_float2(left > 0 ? p.bias[ch] : 0.0f, left > 1 ? p.bias[ch + 1] : 0.0f);
    if (M == kFull && p.D)
        skip = make_float2(left > 0 ? p.D[ch] : 0.0f, left > 1 ? p.D[ch + 1] : 0.0f);
    if (M == kFull && left > 0) {
        if (p.segments > 1)
            load_states<NS>(p.hseg + ((b * p.segments + seg) * p.channels + ch) * np + n0, left, NS,
                            np, h);
        else if (p.s0)
            load_states<NS>(p.s0 + (b * p.channels + ch) * p.states + n0, left, p.states - n0,
                            p.states, h);
    }

    const bool gated = M != kStates && p.z;
    const int64_t o0 = row0 * p.channels + ch;
    // x (back: dy), dt and z of the next G tokens
    const T *const xs = static_cast<const T *>(M == kBack ? p.dy : p.x);
    const int64_t row = M == kBack ? -(int64_t)p.channels : (int64_t)p.channels;
    Pair<T> xr[G], dr[G], zr[G];
    int64_t next = o0 + (M == kBack ? (have - 1) * (int64_t)p.channels : 0);
    // (WHOLE: every token and channel is there, and pairs lie on their size)
    const auto fetch = [&](int t, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const int n = WHOLE ? 2 : t + k < have ? left : 0;
            xr[k] = load_pair(xs + next, WHOLE || wide, n);
            dr[k] = load_pair(static_cast<const T *>(p.dt) + next, WHOLE || wide, n);
            if (gated) zr[k] = load_pair(static_cast<const T *>(p.z) + next, WHOLE || wide, n);
            next += row;
        }
    };
    if (most > 0) {
        for (int m = 0; m * bc_step < kTile; ++m) bc_store(0, m, bc_load(m, 0));
        fetch(0, std::false_type());
    }
    float2 *sy = reinterpret_cast<float2 *>(sbc + 2 * bc_tile) + tid;     // [kTile][threads]
    T *out = M == kFull ? static_cast<T *>(p.y) + o0 : nullptr;
    int buffer = 0;
    for (int t = 0; t < most; t += kTile, buffer ^= 1) {
        __syncthreads();
        const bool more = t + kTile < most;
        Pair<T> ahead[kAhead];
        if (more) {
#pragma unroll
            for (int m = 0; m < kAhead; ++m) ahead[m] = bc_load(m, t + kTile);
        }
        if (M == kStates && p.htile && t < have && left > 0) {
            const int64_t tile = b * ((p.length + kTile - 1) / kTile) + (t0 + t) / kTile;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < NS / 4; ++q) {
                    const float2 v = h[j][2 * q], w = h[j][2 * q + 1];
                    *tile_at(p, tile, grp, c, j, n0 + 4 * q) = make_float4(v.x, v.y, w.x, w.y);
                }
            if (u.sub == 0) {
                float *d = p.dtile + tile * p.channels + ch;
                d[0] = dsum.x;
                if (left > 1) d[1] = dsum.y;
            }
        }
        const float *bc = sbc + buffer * bc_tile + u.seq * kTile * 2 * np + n0;
        const auto tokens_of = [&](auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll 1
            for (int k0 = 0; k0 < kTile && (WHOLE || t + k0 < most); k0 += G) {
                float2 d[G], x[G], z[G];
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    x[k] = to_float2(xr[k]);
                    d[k] = add2(to_float2(dr[k]), bias);
                    if (p.softplus) d[k] = softplus2(d[k]);
                    if (!WHOLE && t + k0 + k >= have) d[k] = f2(0.0f);
                    if (gated) z[k] = to_float2(zr[k]);
                    if (M == kBack && gated) x[k] = mul2(x[k], mul2(z[k], logistic2(z[k])));
                }
                fetch(t + k0 + G, whole);
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    // (back: the output's gradient in the input's place, C in B's)
                    const float2 du = M == kBack ? x[k] : mul2(d[k], x[k]);
                    if (M == kStates) dsum = add2(dsum, d[k]);
                    float2 y[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
                    for (int q = 0; q < NS / 4; ++q) {
                        const float4 bq = *reinterpret_cast<const float4 *>(bc + 4 * q);
                        float4 cq;
                        if (M == kFull) cq = *reinterpret_cast<const float4 *>(bc + np + 4 * q);
#pragma unroll
                        for (int i = 2 * q; i < 2 * q + 2; ++i) {
                            const float2 bv =
                                i & 1 ? make_float2(bq.z, bq.w) : make_float2(bq.x, bq.y);
                            const float2 cv =
                                i & 1 ? make_float2(cq.z, cq.w) : make_float2(cq.x, cq.y);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                // (the packed product would want d twice, in two registers)
                                const float2 a = exp2_fast2(
                                    M == kFull ? make_float2(a2[j][i].x * (j ? d[k].y : d[k].x),
                                                             a2[j][i].y * (j ? d[k].y : d[k].x))
                                               : mul2(a2[j][i], f2(j ? d[k].y : d[k].x)));
                                const float2 uv = f2(j ? du.y : du.x);
                                if (M == kBack) h[j][i] = mul2(a, fma2(uv, bv, h[j][i]));
                                else h[j][i] = fma2(a, h[j][i], mul2(uv, bv));
                                if (M == kFull) y[j] = fma2(cv, h[j][i], y[j]);
                            }
                        }
                    }
                    bc += 2 * np;
                    if (M == kFull) {
                        float2 v = make_float2(y[0].x + y[0].y, y[1].x + y[1].y);
                        if (s.warps > 1) {
                            sy[(k0 + k) * threads] = v;
                            continue;
                        }
                        v = fma2(skip, x[k], v);
                        if (gated) v = mul2(v, mul2(z[k], logistic2(z[k])));
                        store_pair(out, v, WHOLE || wide,
                                   WHOLE ? 2 : t + k0 + k < have ? left : 0);
                        out += p.channels;
                    }
                }
            }
        };
        if (whole_block && t + kTile + G <= least) tokens_of(std::true_type());
        else tokens_of(std::false_type());
        if (M == kFull && s.warps > 1) {
            // the warps that share these channels' states take the tokens in turns
            __syncthreads();
            for (int k = u.sub; k < kTile && t + k < have; k += s.warps) {
                float2 v = f2(0.0f);
                for (int i = 0; i < s.warps; ++i)
                    v = add2(v, sy[k * threads + (i - u.sub) * s.lanes]);
                const int64_t o = o0 + (int64_t)(t + k) * p.channels;
                const float2 xv = to_float2(load_pair(static_cast<const T *>(p.x) + o, wide, left));
                v = fma2(skip, xv, v);
                if (gated) {
                    const float2 zv =
                        to_float2(load_pair(static_cast<const T *>(p.z) + o, wide, left));
                    v = mul2(v, mul2(zv, logistic2(zv)));
                }
                store_pair(static_cast<T *>(p.y) + o, v, wide, left);
            }
        }
        if (more) {
#pragma unroll
            for (int m = 0; m < kAhead; ++m) bc_store(buffer ^ 1, m, ahead[m]);
            for (int m = kAhead; m * bc_step < kTile; ++m)
                bc_store(buffer ^ 1, m, bc_load(m, t + kTile));
        }
    }
    if (M == kFull) {
        for (int t = have + u.sub; t < span; t += s.warps)
            store_pair(static_cast<T *>(p.y) + o0 + (int64_t)t * p.channels, f2(0.0f), wide, left);
        if (p.sT && seg == p.segments - 1)
            store_states<NS>(p.sT + (b * p.channels + ch) * p.states + n0, left, p.states - n0,
                             p.states, h);
    } else if (p.segments > 1) {
        const int64_t r = (b * p.segments + seg) * p.channels + ch;
        store_states<NS>((M == kBack ? p.gseg : p.hseg) + r * np + n0, left, NS, np, h);
        if (M == kStates && u.sub == 0) {
            if (left > 0) p.dseg[r] = dsum.x;
            if (left > 1) p.dseg[r + 1] = dsum.y;
        }
    }
}

template <typename T, int NS, Mode M, int REGS = 168>
fno_status_t launch_scan(const Args &a, cudaStream_t s) {
    const Shape &h = a.shape;
    const int threads = h.threads();
    const int bytes = h.seqs * kTile * h.np * 16 +
                      (M == kFull && h.warps > 1 ? kTile * threads * 8 : 0);
    const auto kernel = k_scan<T, NS, M, REGS>;
    if (bytes > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
            cudaSuccess) {
        cudaGetLastError();
        return FNO_ERR_CUDA;
    }
    const int64_t blocks = ops::ceil_div((int64_t)a.batch * a.groups, h.seqs) * h.chblocks *
                           a.segments;
    kernel<<<(unsigned)blocks, threads, bytes, s>>>(a);
    return ops::launched();
}
template <typename T, Mode M>
fno_status_t scan_pass(const fno_scan_s &p, Args a, cudaStream_t s) {
    a.shape = forward_shape(p.d);
    switch (lane_states(a.states)) {
        case 4: return launch_scan<T, 4, M>(a, s);
        case 8: return launch_scan<T, 8, M>(a, s);
        default: break;
    }
    if constexpr (M == kFull)
        if (a.length <= kShort) return launch_scan<T, 16, M, 128>(a, s);
    return launch_scan<T, 16, M>(a, s);
}

template <typename T>
fno_status_t forward_of(const fno_scan_s &p, Args a, cudaStream_t s) {
    a.htile = nullptr;
    if (a.segments > 1) {
        fno_status_t st = scan_pass<T, kStates>(p, a, s);
        if (st == FNO_OK) st = join(a, false, s);
        if (st != FNO_OK) return st;
    }
    return scan_pass<T, kFull>(p, a, s);
}

}  // namespace scan
}  // namespace fno
