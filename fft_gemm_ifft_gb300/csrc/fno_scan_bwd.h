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
// split, a second one what each segment adds to the gradient in front of it; a kernel joins
// the segments in both directions.  The last pass walks the tiles backwards: it runs a tile
// forward with the state in front of every second token put aside in shared memory, then goes
// back by two tokens at a time, whose states and decays it works out again into registers.
//
// Bound by the latency of its instructions: they fill 45 % of the issue slots (2 x 4096 tokens,
// 1024 channels, 16 states, gated, in bfloat16: 180 us of the call's 290).  It needs 255
// registers, so 8 warps an SM; at 168 registers and 12 warps values loaded ahead are spilled,
// which waits for their loads: 310 us.  Four states a lane and 16 warps: 190 us.
//
// A lane holds two channels x 8 states.  The warps that share a channel's states prepare and
// finish its tokens in turns and add up S1, S2 and y in shared memory.  dB and dC are summed
// over a warp's lanes by shuffles that halve the values at each step: the upper half of the
// lanes holds its two quads of states exchanged, so that all lanes send the same registers
// first.  Blocks of channels meet in the workspace, always in the same order.
#pragma once

#include "fno_scan_fwd.h"

namespace fno {
namespace scan {

constexpr int kSub = 2;                     // tokens whose states are in registers
constexpr int kSubs = kTile / kSub;

// Shared memory of a block: WARPS warps that share the states of 64 channels.
template <typename T, int NS, int WARPS>
struct BackwardShared {
    static constexpr int kThreads = 32 * WARPS, kNp = NS * WARPS;
    float4 du[kTile][32];                             // steps and inputs
    float4 kept[kSubs - 1][NS / 2][kThreads];         // states in front of pairs of tokens
    float2 w[kTile][32];                              // output gradients
    float2 out[3][WARPS][kTile][32];                  // S1, S2, y
    Pair<T> raw[4][kTile][32];                        // x, dt, dy, z
    float bc[kTile][2][kNp];
    float sums[kTile][2][kNp];                        // dB, dC
};

// AHEAD: sequences of up to two tiles, whose states the first pass did not leave: the second
// tile's by a run over the first one (2048 x 12 tokens, 64 channels: a pass of 18 us less).
template <typename T, int NS, int WARPS, bool AHEAD>
__global__ void __launch_bounds__(32 * WARPS)
k_scan_grad(const Args p) {
    using namespace ops;
    using Shared = BackwardShared<T, NS, WARPS>;
    constexpr int NP = NS / 2, kThreads = Shared::kThreads, np = Shared::kNp;
    constexpr int kOwn = WARPS < kTile ? kTile / WARPS : 1;      // tokens a thread prepares
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &sm = *reinterpret_cast<Shared *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, sub = tid >> 5;
    unsigned at = blockIdx.x;
    const int part = (int)(at % p.spans);
    at /= p.spans;
    const int chblocks = p.shape.chblocks, chb = (int)(at % chblocks);
    at /= chblocks;
    const int grp = (int)(at % p.groups);
    const int64_t first_row = at / p.groups;
    const int c = (chb * 32 + lane) * 2;              // in the group
    const int left = p.per_group - c;
    const int64_t ch = (int64_t)grp * p.per_group + c;
    const int flip = NS == 8 ? lane >> 4 : 0, n0 = sub * NS;
    const int64_t t0 = part * p.span_len;
    const int span = (int)min(p.span_len, p.length - t0);
    const int64_t bc_stride = (int64_t)p.groups * p.states;      // (may pass 2^31)
    const bool wide = p.vec_c >= 2 * (int)sizeof(T), gated = p.z != nullptr;
    const int64_t tiles = (p.length + kTile - 1) / kTile;
    const bool kept_tiles = !AHEAD && p.htile && left > 0, before = p.segments > 1 || p.s0;

    float2 a2[2][NP], da[2][NP];                      // log2 e A, and A's gradient
    load_states<NS>(p.A + ch * p.states + n0, left, p.states - n0, p.states, a2, flip);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            a2[j][i] = mul2(a2[j][i], f2(kLog2e));
            da[j][i] = f2(0.0f);
        }
    float2 bias = f2(0.0f), skip = f2(0.0f), dskip = f2(0.0f), dbias = f2(0.0f);
    if (p.bias) bias = make_float2(left > 0 ? p.bias[ch] : 0.0f, left > 1 ? p.bias[ch + 1] : 0.0f);
    if (p.D) skip = make_float2(left > 0 ? p.D[ch] : 0.0f, left > 1 ? p.D[ch + 1] : 0.0f);
    // B and C of a tile, and their gradients: a thread has one state of one of them and every
    // kRows-th token
    constexpr int kMost = kThreads / (2 * np), kRows = kMost < kTile ? kMost : kTile;
    constexpr int kRounds = kTile / kRows;
    static_assert(kRows >= 1 && kTile % kRows == 0, "a block's threads cover B and C");
    const int bc_k = tid / (2 * np), bc_at = tid % (2 * np), bc_which = bc_at / np;
    const int bc_n = bc_at % np;
    const bool bc_mine = bc_k < kRows && bc_n < p.states;

    for (int64_t b = first_row; b < p.batch; b += p.rows) {
        const int64_t len = p.lengths ? max(0, p.lengths[b]) : p.length;
        const int have = (int)max((int64_t)0, min((int64_t)span, len - t0));
        const int last = have > 0 ? (have - 1) / kTile * kTile : -1;
        const int64_t row0 = b * p.length + t0, o0 = row0 * p.channels + ch;
        const int64_t bc0 = row0 * bc_stride + (int64_t)grp * p.states;
        // dB and dC of the span's token t, or this block's part of them
        const auto put_bc = [&](int64_t t, float v) {
            if (chblocks > 1) {
                const int64_t all = (int64_t)p.batch * p.length * p.groups;
                const int64_t row = (row0 + t) * p.groups + grp;
                p.part_bc[((chb * all + row) * 2 + bc_which) * p.states + bc_n] = v;
            } else {
                T *o = static_cast<T *>(bc_which ? p.dC : p.dB);
                Storage<T>::store(o + bc0 + t * bc_stride + bc_n, v);
            }
        };
        // what the tile at t takes from memory
        Pair<T> raw[4][kOwn];
        T bc_raw[kRounds];
        float2 h[2][NP], hin[2][NP], since;
        const auto fetch = [&](int t) {
#pragma unroll
            for (int m = 0; m < kOwn; ++m) {
                const int k = t + sub + m * WARPS;
                const int n = k < have ? left : 0;
                const int64_t o = o0 + (int64_t)k * p.channels;
                raw[0][m] = load_pair(static_cast<const T *>(p.x) + o, wide, n);
                raw[1][m] = load_pair(static_cast<const T *>(p.dt) + o, wide, n);
                raw[2][m] = load_pair(static_cast<const T *>(p.dy) + o, wide, n);
                if (gated) raw[3][m] = load_pair(static_cast<const T *>(p.z) + o, wide, n);
            }
            const T *from = static_cast<const T *>(bc_which ? p.C : p.B) + bc0 + bc_n;
#pragma unroll
            for (int m = 0; m < kRounds; ++m) {
                const int k = t + bc_k + m * kRows;
                Storage<T>::store(&bc_raw[m], 0.0f);
                if (bc_mine && k < have) bc_raw[m] = from[k * bc_stride];
            }
            if (p.segments > 1)
                load_states<NS>(
                    p.hseg + ((b * p.segments + over(t0 + t, (int)p.seg_len)) * p.channels + ch) *
                                 np + n0,
                    left, NS, np, hin, flip);
            else if (p.s0)
                load_states<NS>(p.s0 + (b * p.channels + ch) * p.states + n0, left, p.states - n0,
                                p.states, hin, flip);
            if (kept_tiles) {
                const int64_t tile = b * tiles + (t0 + t) / kTile;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < NS / 4; ++q) {
                        const float4 v = *tile_at(p, tile, grp, c, j, n0 + 4 * (q ^ flip));
                        h[j][2 * q] = make_float2(v.x, v.y);
                        h[j][2 * q + 1] = make_float2(v.z, v.w);
                    }
                if (before) {
                    const float *d = p.dtile + tile * p.channels + ch;
                    since = make_float2(d[0], left > 1 ? d[1] : 0.0f);
                }
            }
        };
        bool ahead = AHEAD && last > 0;
        if (last >= 0) fetch(ahead ? 0 : last);
        float2 gp[2][NP];                             // a_{t+1} g_{t+1}
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < NP; ++i) gp[j][i] = f2(0.0f);
        if (p.segments > 1)
            load_states<NS>(p.gseg + ((b * p.segments + (t0 + span - 1) / p.seg_len) * p.channels +
                                      ch) * np + n0,
                            left, NS, np, gp, flip);
        else if (p.gsT)
            load_states<NS>(p.gsT + (b * p.channels + ch) * p.states + n0, left, p.states - n0,
                            p.states, gp, flip);
        for (int t = ahead ? 0 : last; t >= 0; t -= kTile) {
            const int valid = min(kTile, have - t);
            // the steps, inputs and output gradients of this thread's tokens; beyond the last
            // token they are zero and change nothing
#pragma unroll
            for (int m = 0; m < kOwn; ++m) {
                const int k = sub + m * WARPS;
                const float2 x = to_float2(raw[0][m]);
                float2 d = add2(to_float2(raw[1][m]), bias), w = to_float2(raw[2][m]);
                if (p.softplus) d = softplus2(d);
                if (k >= valid) d = f2(0.0f);
                if (gated) {
                    const float2 z = to_float2(raw[3][m]);
                    w = mul2(w, mul2(z, logistic2(z)));
                    sm.raw[3][k][lane] = raw[3][m];
                }
                const float2 du = mul2(d, x);
                sm.du[k][lane] = make_float4(d.x, d.y, du.x, du.y);
                sm.w[k][lane] = w;
#pragma unroll
                for (int f = 0; f < 3; ++f) sm.raw[f][k][lane] = raw[f][m];
            }
#pragma unroll
            for (int m = 0; m < kRounds; ++m)
                if (bc_k < kRows)
                    sm.bc[bc_k + m * kRows][bc_which][bc_n] = Storage<T>::load(&bc_raw[m]);
            // the state in front of the tile
            const auto put_aside = [&](int r) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < NS / 4; ++q)
                        sm.kept[r][j * (NS / 4) + q][tid] =
                            make_float4(h[j][2 * q].x, h[j][2 * q].y, h[j][2 * q + 1].x,
                                        h[j][2 * q + 1].y);
            };
            const auto take_back = [&](int r) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < NS / 4; ++q) {
                        const float4 v = sm.kept[r][j * (NS / 4) + q][tid];
                        h[j][2 * q] = make_float2(v.x, v.y);
                        h[j][2 * q + 1] = make_float2(v.z, v.w);
                    }
            };
            if (!kept_tiles) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < NP; ++i) h[j][i] = before ? hin[j][i] : f2(0.0f);
                if (AHEAD && t > 0) take_back(0);
            } else if (before) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < NP; ++i)
                        h[j][i] = fma2(hin[j][i],
                                       exp2_fast2(mul2(a2[j][i], f2(j ? since.y : since.x))),
                                       h[j][i]);
            }
            __syncthreads();

            const auto step = [&](int k, float2 (&a)[2][NP], const float2 (&from)[2][NP],
                                  float2 (&to)[2][NP]) {
                const float4 e = sm.du[k][lane];
#pragma unroll
                for (int q = 0; q < NS / 4; ++q) {
                    const float4 bq =
                        *reinterpret_cast<const float4 *>(&sm.bc[k][0][n0 + 4 * (q ^ flip)]);
#pragma unroll
                    for (int i = 2 * q; i < 2 * q + 2; ++i) {
                        const float2 bv = i & 1 ? make_float2(bq.z, bq.w) : make_float2(bq.x, bq.y);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float dv = j ? e.y : e.x;
                            a[j][i] = exp2_fast2(make_float2(a2[j][i].x * dv, a2[j][i].y * dv));
                            to[j][i] = fma2(a[j][i], from[j][i], mul2(f2(j ? e.w : e.z), bv));
                        }
                    }
                }
            };
            if (AHEAD && ahead) {
#pragma unroll 2
                for (int k = 0; k < kTile; ++k) {
                    float2 a[2][NP];
                    step(k, a, h, h);
                }
                put_aside(0);
                ahead = false;
                t = last + kTile;
                fetch(last);
                __syncthreads();
                continue;
            }
            const int subs = (valid + kSub - 1) / kSub;
#pragma unroll 1
            for (int r = 0; r < subs - 1; ++r) {
                put_aside(r);
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
                    float2 a[2][NP];
                    step(r * kSub + k, a, h, h);
                }
            }
#pragma unroll 1
            for (int r = subs - 1; r >= 0; --r) {
                float2 a[kSub][2][NP], hs[kSub][2][NP];
                if (r < subs - 1) take_back(r);
                step(r * kSub, a[0], h, hs[0]);
#pragma unroll
                for (int k = 1; k < kSub; ++k) step(r * kSub + k, a[k], hs[k - 1], hs[k]);
#pragma unroll
                for (int k = kSub - 1; k >= 0; --k) {
                    const int kk = r * kSub + k;
                    const float4 e = sm.du[kk][lane];
                    const float2 w = sm.w[kk][lane];
                    float2 s1[2], s2[2], y[2], vb[NP], vc[NP];
#pragma unroll
                    for (int j = 0; j < 2; ++j) s1[j] = s2[j] = y[j] = f2(0.0f);
#pragma unroll
                    for (int q = 0; q < NS / 4; ++q) {
                        const float4 bq =
                            *reinterpret_cast<const float4 *>(&sm.bc[kk][0][n0 + 4 * (q ^ flip)]);
                        const float4 cq =
                            *reinterpret_cast<const float4 *>(&sm.bc[kk][1][n0 + 4 * (q ^ flip)]);
#pragma unroll
                        for (int i = 2 * q; i < 2 * q + 2; ++i) {
                            const float2 bv =
                                i & 1 ? make_float2(bq.z, bq.w) : make_float2(bq.x, bq.y);
                            const float2 cv =
                                i & 1 ? make_float2(cq.z, cq.w) : make_float2(cq.x, cq.y);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float2 dv = f2(j ? e.y : e.x), uv = f2(j ? e.w : e.z);
                                const float2 wv = f2(j ? w.y : w.x);
                                const float2 earlier = k ? hs[k ? k - 1 : 0][j][i] : h[j][i];
                                const float2 g = fma2(cv, wv, gp[j][i]);
                                s1[j] = fma2(g, bv, s1[j]);
                                y[j] = fma2(cv, hs[k][j][i], y[j]);
                                vb[i] = j ? fma2(g, uv, vb[i]) : mul2(g, uv);
                                vc[i] = j ? fma2(wv, hs[k][j][i], vc[i]) : mul2(wv, hs[k][j][i]);
                                gp[j][i] = mul2(a[k][j][i], g);
                                const float2 m = mul2(gp[j][i], earlier);
                                s2[j] = fma2(a2[j][i], m, s2[j]);
                                da[j][i] = fma2(dv, m, da[j][i]);
                            }
                        }
                    }
                    sm.out[0][sub][kk][lane] = make_float2(s1[0].x + s1[0].y, s1[1].x + s1[1].y);
                    sm.out[1][sub][kk][lane] = make_float2(s2[0].x + s2[0].y, s2[1].x + s2[1].y);
                    sm.out[2][sub][kk][lane] = make_float2(y[0].x + y[0].y, y[1].x + y[1].y);
                    // over the lanes: quads, then dB or dC, then pairs, then one state
                    const auto add_from = [](float2 v, float2 send, int mask) {
                        return add2(v, make_float2(__shfl_xor_sync(0xffffffffu, send.x, mask),
                                                   __shfl_xor_sync(0xffffffffu, send.y, mask)));
                    };
                    if constexpr (NS == 8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            vb[i] = add_from(vb[i], vb[i + 2], 16);
                            vc[i] = add_from(vc[i], vc[i + 2], 16);
                        }
                    }
                    const bool is_c = lane & 8, second = lane & 4, odd = lane & 2;
                    float2 v[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        v[i] = add_from(is_c ? vc[i] : vb[i], is_c ? vb[i] : vc[i], 8);
                    const float2 m = add_from(second ? v[1] : v[0], second ? v[0] : v[1], 4);
                    float one = (odd ? m.y : m.x) +
                                __shfl_xor_sync(0xffffffffu, odd ? m.x : m.y, 2);
                    one += __shfl_xor_sync(0xffffffffu, one, 1);
                    if constexpr (NS == 4) one += __shfl_xor_sync(0xffffffffu, one, 16);
                    if (!(lane & (NS == 8 ? 1 : 17)))
                        sm.sums[kk][is_c ? 1 : 0]
                               [n0 + 4 * flip + (second ? 2 : 0) + (odd ? 1 : 0)] = one;
                }
            }
            __syncthreads();
            if (t > 0) fetch(t - kTile);
#pragma unroll 1
            for (int m = 0; m < kOwn; ++m) {
                const int k = sub + m * WARPS;
                if (k >= valid) break;
                float2 v[3];
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    v[q] = sm.out[q][0][k][lane];
#pragma unroll
                    for (int i = 1; i < WARPS; ++i) v[q] = add2(v[q], sm.out[q][i][k][lane]);
                }
                const float2 x = to_float2(sm.raw[0][k][lane]), w = sm.w[k][lane];
                const float4 e = sm.du[k][lane];
                const int64_t o = o0 + (int64_t)(t + k) * p.channels;
                store_pair(static_cast<T *>(p.dx) + o,
                           fma2(skip, w, mul2(make_float2(e.x, e.y), v[0])), wide, left);
                dskip = fma2(w, x, dskip);
                float2 dd = fma2(x, v[0], mul2(v[1], f2(kLn2)));
                if (p.softplus)
                    dd = mul2(dd, logistic2(add2(to_float2(sm.raw[1][k][lane]), bias)));
                store_pair(static_cast<T *>(p.ddt) + o, dd, wide, left);
                dbias = add2(dbias, dd);
                if (gated) {
                    const float2 z = to_float2(sm.raw[3][k][lane]), l = logistic2(z);
                    const float2 gy = to_float2(sm.raw[2][k][lane]), y = fma2(skip, x, v[2]);
                    // silu' = l (1 + z (1 - l))
                    store_pair(static_cast<T *>(p.dz) + o,
                               mul2(mul2(gy, y), mul2(l, fma2(z, sub2(f2(1.0f), l), f2(1.0f)))),
                               wide, left);
                }
            }
            if (bc_mine) {
#pragma unroll
                for (int m = 0; m < kRounds; ++m) {
                    const int k = bc_k + m * kRows;
                    if (k >= valid) break;
                    put_bc(t + k, sm.sums[k][bc_which][bc_n]);
                }
            }
        }
        for (int t = have + sub; t < span; t += WARPS) {
            const int64_t o = o0 + (int64_t)t * p.channels;
            store_pair(static_cast<T *>(p.dx) + o, f2(0.0f), wide, left);
            store_pair(static_cast<T *>(p.ddt) + o, f2(0.0f), wide, left);
            if (gated) store_pair(static_cast<T *>(p.dz) + o, f2(0.0f), wide, left);
        }
        if (bc_mine)
            for (int t = have + bc_k; t < span; t += kRows) put_bc(t, 0.0f);
        if (p.ds0 && part == 0)
            store_states<NS>(p.ds0 + (b * p.channels + ch) * p.states + n0, left, p.states - n0,
                             p.states, gp, flip);
        __syncthreads();          // (shared memory is read before the next sequence writes it)
    }
    const int64_t r = first_row * p.spans + part;
    store_states<NS>(p.part_a + (r * p.channels + ch) * np + n0, left, NS, np, da, flip);
    // the bias' and D's gradients: the warps that share these channels
    sm.out[0][sub][0][lane] = dskip;
    sm.out[1][sub][0][lane] = dbias;
    __syncthreads();
    if (sub == 0) {
#pragma unroll
        for (int i = 1; i < WARPS; ++i) {
            dskip = add2(dskip, sm.out[0][i][0][lane]);
            dbias = add2(dbias, sm.out[1][i][0][lane]);
        }
        float *o = p.part_d + r * 2 * p.channels + ch;
        if (left > 0) o[0] = dskip.x, o[p.channels] = dbias.x;
        if (left > 1) o[1] = dskip.y, o[p.channels + 1] = dbias.y;
    }
}

// dB and dC: the sum of the blocks' parts (rows of 2 x states).
template <typename T>
__global__ void __launch_bounds__(256)
k_scan_sum_bc(const Args p) {
    const int64_t rows = (int64_t)p.batch * p.length * p.groups, n = rows * 2 * p.states;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = p.part_bc[i];
#pragma unroll 8
    for (int k = 1; k < p.shape.chblocks; ++k) v += p.part_bc[k * n + i];
    const int64_t row = over(i, 2 * p.states);
    const int e = (int)(i - row * 2 * p.states);
    T *o = static_cast<T *>(e >= p.states ? p.dC : p.dB);
    Storage<T>::store(o + row * p.states + (e >= p.states ? e - p.states : e), v);
}

template <typename T, int NS, int WARPS, bool AHEAD>
fno_status_t launch_grad(const Args &a, cudaStream_t s) {
    using Shared = BackwardShared<T, NS, WARPS>;
    const auto kernel = k_scan_grad<T, NS, WARPS, AHEAD>;
    if (sizeof(Shared) > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Shared)) != cudaSuccess) {
        cudaGetLastError();
        return FNO_ERR_CUDA;
    }
    const int64_t blocks = a.rows * a.groups * a.shape.chblocks * a.spans;
    kernel<<<(unsigned)blocks, Shared::kThreads, sizeof(Shared), s>>>(a);
    return ops::launched();
}
// The kernel of the plan's states.
template <typename T, bool AHEAD>
fno_status_t grad_pass(const Args &a, cudaStream_t s) {
    switch (a.shape.np) {
        case 4: return launch_grad<T, 4, 1, AHEAD>(a, s);
        case 8: return launch_grad<T, 8, 1, AHEAD>(a, s);
        case 16: return launch_grad<T, 8, 2, AHEAD>(a, s);
        case 32: return launch_grad<T, 8, 4, AHEAD>(a, s);
        default: return launch_grad<T, 8, 8, AHEAD>(a, s);
    }
}

template <typename T>
fno_status_t backward_of(const fno_scan_s &p, Args a, cudaStream_t s) {
    using ops::ceil_div;
    fno_status_t st = FNO_OK;
    // (up to two tiles the last pass works out for itself)
    if (a.length <= 2 * kTile) a.htile = nullptr;
    if (a.segments > 1 || a.htile) st = scan_pass<T, kStates>(p, a, s);
    if (a.segments > 1) {
        if (st == FNO_OK) st = scan_pass<T, kBack>(p, a, s);
        if (st == FNO_OK) st = join(a, true, s);
    }
    if (st != FNO_OK) return st;
    a.shape = backward_shape(p.d);
    st = a.segments == 1 && !a.htile ? grad_pass<T, true>(a, s) : grad_pass<T, false>(a, s);
    if (st != FNO_OK) return st;
    if (a.shape.chblocks > 1) {
        const int64_t n = (int64_t)a.batch * a.length * a.groups * 2 * a.states;
        k_scan_sum_bc<T><<<(unsigned)ceil_div(n, 256), 256, 0, s>>>(a);
    }
    return sum_parts(a, s);
}

}  // namespace scan
}  // namespace fno
