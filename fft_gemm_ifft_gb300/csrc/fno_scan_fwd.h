// fno_scan_fwd.h -- the selective scan forward, and the pass over the states that both
// directions make when the time axis is split.
//
// For each channel c and state n of a sequence
//   h_t = e^{d_t A} h_{t-1} + (d_t x_t) B_t,   y_t = sum_n C_t h_t,
// one exponential and four multiply-adds an element (c, n) and token, and no matrix
// product: the decay differs for every element.  So instructions bound it, not device memory
// (16 states: 8 to 12 bytes a channel and token).  With everything in registers this loop takes
// 1.7 cycles of an SM for 32 elements (a packed multiply-add occupies two issue slots, as two
// single ones do); the kernel, with softplus, gates, loads and stores, takes 3.0 (8191 tokens
// of 2048 channels and 16 states in bfloat16: 87 us), half of the issue slots at 12 warps an SM.
//
// The decay is the multi-function unit's power of two of (A log2 e) d, so what is rounded to
// float32 before it, log2 e (1.4e-8) and two products (2^-24 each), is 1.4e-7 |d A| of the
// result, and the unit adds 1.5e-7.  Carrying the products' remainders along would add two
// multiply-adds or more to an element's five instructions.
//
// A lane holds two channels x up to 16 states in registers, so that nothing is summed over
// lanes: its channels' steps, inputs and outputs stay in its registers, from and to global
// memory.  B and C, which all channels share, lie in shared memory as floats, and a whole warp
// reads the same ones at once.  (Four channels x four states a lane read four addresses a warp,
// for which shared memory takes four times as long, and staged the steps there as well: 125 us;
// pairs of lanes sharing 16 states, 20 warps an SM in place of 12: 118 us.)  More than 16 states
// are shared by several warps, whose sums meet in shared memory.
//
// When the sequences and channels do not fill the GPU, time is split into segments:
// one pass finds each segment's state from zero, a kernel joins them by
// e^{A sum d}, and the second pass starts from the joined states.
#pragma once

#include "fno_scan.h"

#include <numeric>

namespace fno {
namespace scan {

// The outputs from the states in front of the segments; the states at the segments' ends
// and in front of the tiles (each if wanted); from the last token, what each segment adds to
// the gradient of the state in front of it: r_t = a_t (r_{t+1} + C_t w_t), w = dy silu(z).
enum Mode { kFull, kStates, kBack };
// 16 states take 168 registers, so an SM holds 12 warps; at 128 registers and 16 warps some are
// spilled (8191 tokens of 2048 channels: a call of 192 us; 165 at 168).  Short sequences, which
// are mostly the latency of their first loads, take the 16 warps all the same (2048 x 12 tokens of
// 64 channels in float32: 26 us, at 168 28; 4096 x 30 of 32: 50 and 67; 512 x 20 of 256 in
// bfloat16: 31 and 32; but 64 x 30 of 4096: 64 and 58; 1024 x 64 of 64: 63 and 43).  Fewer states
// have less to hold: 8 in 112 registers, 4 in 96 (8191 tokens of 2048 channels, 8 states: 123 us,
// with 168 registers 159; 4 in float32: 108 us, 177).
constexpr int kShort = 32;
template <typename T, int NS, Mode M, int REGS>
__global__ void __maxnreg__(REGS)
k_scan(const Args p) {
    using namespace ops;
    constexpr int G = M == kFull ? 1 : 2;             // tokens worked on together, and loaded ahead
    constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;    // pairs of B or C fetched ahead
    extern __shared__ __align__(16) float sbc[];      // [2][seqs][kTile][2][np], sums of y
    const int tid = threadIdx.x, threads = blockDim.x;
    const Shape s = p.shape;
    const int np = s.np;
    const Unit u(tid, s);
    unsigned at = blockIdx.x;
    const int seg = (int)(at % p.segments);
    at /= p.segments;
    const int chb = (int)(at % s.chblocks);
    // the block's sequences (of any group), and those `step` sequences of the batch further on
    int64_t seq0 = (int64_t)(at / s.chblocks) * s.seqs;
    const int64_t all = (int64_t)p.batch * p.groups;
    const int step = p.step;
    int b = (int)over(seq0 + u.seq, p.groups);
    const int grp = (int)(seq0 + u.seq - (int64_t)b * p.groups);
    const int c = ((chb * s.slabs + u.slab) * s.lanes + u.lane) * 2;     // in the group
    const int there = p.per_group - c;
    int left = b < p.batch ? there : 0;
    const int64_t ch = (int64_t)grp * p.per_group + c;
    const int64_t t0 = seg * p.seg_len;
    const int span = (int)min(p.seg_len, p.length - t0);
    // tokens of the segment that are there: a lane has those of one of the block's sequences
    // (none of those that do not exist)
    const unsigned warp = threads < 32 ? (1u << threads) - 1 : 0xffffffffu;
    int lane_b = (int)over(seq0 + (tid & (s.seqs - 1)), p.groups);
    const auto length_of = [&](int sequence) {
        return sequence >= p.batch ? 0 : p.lengths ? p.lengths[sequence] : (int)p.length;
    };
    const auto tokens = [&](int n) { return (int)max((int64_t)0, min((int64_t)span, n - t0)); };
    int lens = tokens(length_of(lane_b));
    int have = __shfl_sync(warp, lens, u.seq);
    int most = __reduce_max_sync(warp, lens), least = __reduce_min_sync(warp, lens);
    const bool wide = p.vec_c >= 2 * (int)sizeof(T);
    const bool whole_block = wide && (chb + 1) * s.slabs * s.lanes * 2 <= p.per_group;

    // B and C of a tile: a thread has one pair of states of one of them (of a sequence) and
    // every bc_step-th token
    const int combos = s.seqs * np;                   // (no more than there are threads)
    const int bc_step = threads / combos, bc_k = tid / combos, bc_tile = 2 * kTile * combos;
    const T *bc_from;
    int bc_to, bc_seq, bc_left;
    {
        const int i = tid - bc_k * combos, r = i & (np - 1), which = r / (np / 2);
        const int n = 2 * (r - which * (np / 2));
        bc_seq = min(i / np, s.seqs - 1);
        const int64_t sq = seq0 + bc_seq, bb = over(sq, p.groups);
        const int n_bb = __shfl_sync(warp, lens, bc_seq);
        bc_from = static_cast<const T *>(which || M == kBack ? p.C : p.B) +
                  ((bb * p.length + t0 + (M == kBack ? n_bb - 1 - bc_k : bc_k)) * p.groups +
                   (sq - bb * p.groups)) * p.states + n;
        bc_to = ((bc_seq * kTile + bc_k) * 2 + which) * np + n;
        bc_left = bc_k < bc_step && (!which || M == kFull) ? p.states - n : 0;
    }
    int bc_have = __shfl_sync(warp, lens, bc_seq);
    const bool bc_wide = p.vec_n >= 2 * (int)sizeof(T);
    const int64_t bc_row = (M == kBack ? -1 : 1) * (int64_t)p.groups * p.states;
    // the thread's m-th pair of the tile at `from` that has `n` tokens
    const auto bc_load = [&](int m, const T *from, int n) {
        const int k = bc_k + m * bc_step;
        return load_pair(from + (int64_t)(m * bc_step) * bc_row, bc_wide,
                         k < kTile && k < n ? bc_left : 0);
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
    const auto first_states = [&]() {
        if (p.segments > 1)
            load_states<NS>(p.hseg + (((int64_t)b * p.segments + seg) * p.channels + ch) * np + n0,
                            left, NS, np, h);
        else if (p.s0)
            load_states<NS>(p.s0 + ((int64_t)b * p.channels + ch) * p.states + n0, left,
                            p.states - n0, p.states, h);
    };

    const bool gated = M != kStates && p.z;
    int64_t o0 = ((int64_t)b * p.length + t0) * p.channels + ch;
    const int64_t o_step = (int64_t)step * p.length * p.channels;
    // x (back: dy), dt and z of the next tokens
    const T *const xs = static_cast<const T *>(M == kBack ? p.dy : p.x);
    const int64_t row = M == kBack ? -(int64_t)p.channels : (int64_t)p.channels;
    Pair<T> xr[G], dr[G], zr[G];
    int64_t next = o0 + (M == kBack ? (have - 1) * (int64_t)p.channels : 0);
    int have_next = 0;                                // tokens of the next sequence
    // (WHOLE: every token and channel is there, and pairs lie on their size)
    // (t of `most`: the first of the next sequence)
    const auto fetch = [&](int t, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
        for (int k = 0; k < G; ++k) {
            int n = WHOLE ? 2 : t + k < have ? there : 0;
            if (M == kFull && !WHOLE && t >= most) {
                n = have_next > 0 ? there : 0;
                next = o0 + o_step;
            }
            xr[k] = load_pair(xs + next, WHOLE || wide, n);
            dr[k] = load_pair(static_cast<const T *>(p.dt) + next, WHOLE || wide, n);
            if (gated) zr[k] = load_pair(static_cast<const T *>(p.z) + next, WHOLE || wide, n);
            next += row;
        }
    };
    // x, dt and z of the `n` next tokens of a tile, from token 0's place `from` on, into L2: the
    // lanes take a line of 128 bytes each.  A token's registers are loaded one token ahead, which
    // is enough for L2 but not for device memory (300 x 500 tokens of 256 channels in float32:
    // a call of 250 us; 357 without; loaded two tokens ahead no less).
    const auto call_for = [&](int64_t from, int n) {
        constexpr int kLines = sizeof(T) == 4 ? 2 : 1, kLine = 128 / sizeof(T);
        if (u.sub) return;
        for (int i = u.lane; i < kTile * kLines * (gated ? 3 : 2); i += s.lanes) {
            const int k = i % kTile, line = i / kTile, part = line % kLines * kLine;
            const T *base = line < kLines ? xs : static_cast<const T *>(
                                                     line < 2 * kLines ? p.dt : p.z);
            if (k < n && part < there + 2 * u.lane)
                prefetch_l2(base + from - 2 * u.lane + k * row + part);
        }
    };
    float2 *sy = reinterpret_cast<float2 *>(sbc + 2 * bc_tile) + tid;     // [kTile][threads]
    int buffer = 0;
    bool ready = false;             // the first tile and token are there or on their way
    for (;;) {
        if (M == kFull && left > 0) first_states();
        if (most > 0 && !ready) {
            for (int m = 0; m * bc_step < kTile; ++m)
                bc_store(buffer, m, bc_load(m, bc_from, bc_have));
            call_for(next, have);
            fetch(0, std::false_type());
        }
        // (looked at where this sequence ends)
        const int length_next = M == kFull ? length_of(lane_b + step) : 0;
        T *out = M == kFull ? static_cast<T *>(p.y) + o0 : nullptr;
        for (int t = 0; t < most; t += kTile, buffer ^= 1) {
            __syncthreads();
            // the next tile: of this sequence or the first of the next one
            bool more = t + kTile < most;
            const T *bc_next = bc_from + (t + kTile) * bc_row;
            int bc_n = bc_have - t - kTile;
            if (M == kFull && !more) {
                const int n = seq0 + (int64_t)step * p.groups < all ? tokens(length_next) : 0;
                have_next = __shfl_sync(warp, n, u.seq);
                bc_n = __shfl_sync(warp, n, bc_seq);
                bc_next = bc_from + (int64_t)step * p.length * p.groups * p.states;
                more = __reduce_max_sync(warp, n) > 0;
            }
            Pair<T> ahead[kAhead];
            if (more) {
#pragma unroll
                for (int m = 0; m < kAhead; ++m) ahead[m] = bc_load(m, bc_next, bc_n);
                if (t + kTile < most) call_for(next + (kTile - G) * row, have - t - kTile);
                else call_for(o0 + o_step, have_next);
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
            const auto tokens_of = [&](int from, int to, auto whole) {
                constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll 1
                for (int k0 = from; k0 < to; k0 += G) {
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
            // without checks as far as every sequence has them and those loaded ahead
            const int whole = whole_block ? max(0, min(kTile, least - t - G)) / G * G : 0;
            tokens_of(0, whole, std::true_type());
            tokens_of(whole, min(kTile, most - t), std::false_type());
            if (M == kFull && s.warps > 1) {
                // the warps that share these channels' states take the tokens in turns
                __syncthreads();
                for (int k = u.sub; k < kTile && t + k < have; k += s.warps) {
                    float2 v = f2(0.0f);
                    for (int i = 0; i < s.warps; ++i)
                        v = add2(v, sy[k * threads + (i - u.sub) * s.lanes]);
                    const int64_t o = o0 + (int64_t)(t + k) * p.channels;
                    const float2 xv =
                        to_float2(load_pair(static_cast<const T *>(p.x) + o, wide, left));
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
                    bc_store(buffer ^ 1, m, bc_load(m, bc_next, bc_n));
            }
            ready = more;
        }
        if (M == kFull) {
            for (int t = have + u.sub; t < span; t += s.warps)
                store_pair(static_cast<T *>(p.y) + o0 + (int64_t)t * p.channels, f2(0.0f), wide,
                           left);
            if (p.sT && seg == p.segments - 1)
                store_states<NS>(p.sT + ((int64_t)b * p.channels + ch) * p.states + n0, left,
                                 p.states - n0, p.states, h);
        } else if (p.segments > 1) {
            const int64_t r = ((int64_t)b * p.segments + seg) * p.channels + ch;
            store_states<NS>((M == kBack ? p.gseg : p.hseg) + r * np + n0, left, NS, np, h);
            if (M == kStates && u.sub == 0) {
                if (left > 0) p.dseg[r] = dsum.x;
                if (left > 1) p.dseg[r + 1] = dsum.y;
            }
        }
        // the next sequence of the same channels
        seq0 += (int64_t)step * p.groups;
        if (M != kFull || seq0 >= all) break;
        ready = ready && most > 0;
        b += step, lane_b += step;
        left = b < p.batch ? there : 0;
        lens = tokens(length_next);
        have = __shfl_sync(warp, lens, u.seq);
        most = __reduce_max_sync(warp, lens), least = __reduce_min_sync(warp, lens);
        bc_from += (int64_t)step * p.length * p.groups * p.states;
        bc_have = __shfl_sync(warp, lens, bc_seq);
        o0 += o_step;
        if (!ready) next = o0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < NS / 2; ++i) h[j][i] = f2(0.0f);
    }
}

template <typename T, int NS, Mode M, int REGS = scan_registers(NS)>
fno_status_t launch_scan(const Args &a, int sms, cudaStream_t s) {
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
    const int64_t all = (int64_t)a.batch * a.groups;
    int64_t across = ops::ceil_div(all, h.seqs);
    Args b = a;
    b.step = a.batch;
    if (M == kFull && a.segments == 1) {
        // a wave of blocks, which go on with further sequences (of the same groups) and load
        // their first tokens ahead (16384 x 4 tokens, 32 channels, float32: 41 us as many blocks,
        // 34 so), where whole rounds of channels and groups nearly make one (64 x 30 tokens, 300
        // groups of 128 channels: 434 us by many blocks, 620 by a wave and a third)
        const int64_t wave = 65536 / ((int64_t)REGS * threads) * sms;
        const int64_t unit = a.groups / std::gcd(a.groups, h.seqs);
        const int64_t some = wave / h.chblocks / unit * unit;
        if (4 * some * h.chblocks >= 3 * wave && some < across) {
            across = some;
            b.step = (int)(across * h.seqs / a.groups);
        }
    }
    kernel<<<(unsigned)(across * h.chblocks * a.segments), threads, bytes, s>>>(b);
    return ops::launched();
}
template <typename T, Mode M>
fno_status_t scan_pass(const fno_scan_s &p, Args a, cudaStream_t s) {
    a.shape = forward_shape(p.d);
    switch (lane_states(a.states)) {
        case 4: return launch_scan<T, 4, M>(a, p.sms, s);
        case 8: return launch_scan<T, 8, M>(a, p.sms, s);
        default: break;
    }
    if constexpr (M == kFull)
        if (a.length <= kShort) return launch_scan<T, 16, M, 128>(a, p.sms, s);
    return launch_scan<T, 16, M>(a, p.sms, s);
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
