// fno_scan.h -- what the selective scan's translation units share.
#pragma once

#include "fno_ops_internal.h"

struct fno_scan_s {
    fno_scan_desc_t d;
    int sms;
    // the time axis in `segments` parts that run side by side; for the last pass of the
    // backward, `spans` of several segments each, and the sequences that run side by side
    int64_t seg_len, span_len;
    int segments, spans;
    int64_t rows;
    size_t workspace;
};

namespace fno {
namespace scan {

constexpr int kMaxStates = 64;
constexpr int kTile = 8;       // tokens staged at a time, and between two states kept for
                               // the backward

// How a kernel's block divides its work: `seqs` sequences (and groups) x `slabs` of 2 lanes
// channels x `warps` that share a channel's states x `lanes` of two channels each.
struct Shape {
    int seqs, slabs, warps, lanes;
    int chblocks;              // blocks of channels in a group
    int np;                    // states, padded to whole lanes' shares
    __host__ __device__ int threads() const { return seqs * slabs * warps * lanes; }
};

// The operands of a scan, and where its work lies in the workspace.
struct Args {
    const void *x, *dt, *B, *C, *z, *dy;
    const float *A, *D, *bias, *s0, *gsT;
    const int32_t *lengths;
    void *y, *dx, *ddt, *dB, *dC, *dz;
    float *sT, *dA, *dD, *dbias, *ds0;
    // per (sequence, segment), (channels, padded states): states at its end and, after the
    // joining, in front of it; likewise the gradients that reach its end; the sums of the
    // steps (channels)
    float *hseg, *gseg, *dseg;
    // per (sequence, tile): the state in front of it from zero at the segment's start (in
    // the order of tile_at), and the sum of the steps since then
    float *htile, *dtile;
    // partial sums of the gradients: of B and C per block of channels, of A (channels,
    // padded states), D and the bias per (row of blocks, span)
    float *part_bc, *part_a, *part_d;
    int64_t length, seg_len;
    int64_t span_len, rows;    // last pass backward: tokens and sequences side by side
    int batch, channels, per_group, groups, states, segments, spans;
    int units, unit_shift;     // kept states: units of up to 64 channels in a group, and
                               // the channel pairs of one as a power of two
    int step;                  // forward: sequences between those of a block, of one group
    bool softplus;
    int vec_c, vec_n;          // bytes that rows of channels and of states may be moved in
    Shape shape;
};

// What a plan needs of the workspace for the backward, and its parts.
struct BackwardParts {
    size_t hseg, gseg, dseg, htile, dtile, part_bc, part_a, part_d, bytes;
};
BackwardParts backward_parts(const fno_scan_s &p);

template <typename T> fno_status_t forward_of(const fno_scan_s &p, Args a, cudaStream_t s);
template <typename T> fno_status_t backward_of(const fno_scan_s &p, Args a, cudaStream_t s);
// The states in front of the segments from the local ones at their ends, in place (both:
// and the gradients that reach the segments' ends, from the last one).
fno_status_t join(const Args &a, bool both, cudaStream_t s);
// dA, dD and the bias' gradient from the blocks' parts.
fno_status_t sum_parts(const Args &a, cudaStream_t s);

inline int pow2_at_least(int64_t n) {
    int v = 1;
    while (v < n) v *= 2;
    return v;
}
// States of a lane forward, and padded to a power of two.
inline int lane_states(int states) { return states <= 4 ? 4 : states <= 8 ? 8 : 16; }
// Registers of a thread of the forward kernels (see there), and the warps an SM then holds.
constexpr int scan_registers(int lane_states) {
    return lane_states == 4 ? 96 : lane_states == 8 ? 112 : 168;
}
constexpr int scan_warps(int registers) { return 65536 / (32 * registers) / 4 * 4; }
inline int padded_states(int states) { return pow2_at_least(states < 4 ? 4 : states); }
// Blocks of four warps (as many as share a channel's states, if more).  Groups of up to 32
// channels take half a warp, so that a block holds more sequences instead.
inline Shape forward_shape(const fno_scan_desc_t &d) {
    const int per = d.channels / d.groups;
    Shape s{};
    s.np = padded_states(d.states);
    s.warps = s.np / lane_states(d.states);
    s.lanes = s.warps > 1 || per > 32 ? 32 : 16;
    const int64_t slabs = ops::ceil_div(per, 2 * s.lanes), all = d.batch * d.groups;
    s.slabs = s.warps >= 4 ? 1 : 4 / s.warps;
    while (s.slabs / 2 >= slabs) s.slabs /= 2;
    s.seqs = 1;
    while (2 * s.seqs * s.slabs * s.warps * s.lanes <= 128 && s.seqs < all) s.seqs *= 2;
    s.chblocks = (int)ops::ceil_div(slabs, s.slabs);
    return s;
}
// Backward a lane has eight states (four of four), and a block the warps that share the states
// of 64 channels.
inline Shape backward_shape(const fno_scan_desc_t &d) {
    Shape s{};
    s.np = padded_states(d.states);
    s.warps = s.np <= 4 ? 1 : s.np / 8;
    s.lanes = 32;
    s.seqs = s.slabs = 1;
    s.chblocks = (int)ops::ceil_div(d.channels / d.groups, 64);
    return s;
}

// a / b of counts; in 32 bits, a fifth of the instructions, where a has no more.
__device__ __forceinline__ int64_t over(int64_t a, int b) {
    return (uint64_t)a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// ---------------------------------------------------------------------------
// a thread's elements
// ---------------------------------------------------------------------------
// Its place in the block: two channels from 2 lane on of its slab.
struct Unit {
    int lane, sub, slab, seq;
    __device__ Unit(int tid, const Shape &s) {
        const int r = tid / s.lanes, q = r / s.warps;
        lane = tid - r * s.lanes;
        sub = r - q * s.warps;
        seq = q / s.slabs;
        slab = q - seq * s.slabs;
    }
};

// NS states of two channels from rows `pitch` apart, where `left` channels and `there`
// states are left; zero where there are none.  `flip` exchanges the two quads of eight.
template <int NS>
__device__ __forceinline__ void read_states(const float *at, int left, int there, int pitch,
                                            float (&v)[2][NS], int flip) {
    const bool quads = pitch % 4 == 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < NS / 4; ++q) {
            const int n = 4 * (q ^ flip);
            const float *p = at + (int64_t)j * pitch + n;
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (j < left) {
                if (quads) {
                    if (n < there) f = *reinterpret_cast<const float4 *>(p);
                } else {
                    if (n < there) f.x = p[0];
                    if (n + 1 < there) f.y = p[1];
                    if (n + 2 < there) f.z = p[2];
                    if (n + 3 < there) f.w = p[3];
                }
            }
            v[j][4 * q] = f.x, v[j][4 * q + 1] = f.y, v[j][4 * q + 2] = f.z, v[j][4 * q + 3] = f.w;
        }
}
template <int NS>
__device__ __forceinline__ void write_states(float *at, int left, int there, int pitch,
                                             const float (&v)[2][NS], int flip) {
    const bool quads = pitch % 4 == 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < NS / 4; ++q) {
            const int n = 4 * (q ^ flip);
            float *p = at + (int64_t)j * pitch + n;
            const float *f = v[j] + 4 * q;
            if (j >= left) continue;
            if (quads) {
                if (n < there) *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < there) p[i] = f[i];
            }
        }
}
// The same as pairs of states.
template <int NS>
__device__ __forceinline__ void load_states(const float *at, int left, int there, int pitch,
                                            float2 (&v)[2][NS / 2], int flip = 0) {
    float f[2][NS];
    read_states<NS>(at, left, there, pitch, f, flip);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NS / 2; ++i) v[j][i] = make_float2(f[j][2 * i], f[j][2 * i + 1]);
}
template <int NS>
__device__ __forceinline__ void store_states(float *at, int left, int there, int pitch,
                                             const float2 (&v)[2][NS / 2], int flip = 0) {
    float f[2][NS];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NS / 2; ++i) f[j][2 * i] = v[j][i].x, f[j][2 * i + 1] = v[j][i].y;
    write_states<NS>(at, left, there, pitch, f, flip);
}
// A unit of the kept states has 32 channel pairs, or as many (a power of two) as a group of fewer
// channels, so that many small groups keep little more than their own states.
inline int unit_shift(int per_group) {
    int s = 0;
    while (s < 5 && (2 << s) < per_group) ++s;
    return s;
}
// The tiles' states: by units, their quads of states by channel pair, so that a warp's accesses
// are whole lines.  The quad of channel c + j (of its group) from state n.
__device__ __forceinline__ float4 *tile_at(const Args &p, int64_t tile, int grp, int c, int j,
                                           int n) {
    const int np = p.shape.np;
    const int64_t unit = (tile * p.groups + grp) * p.units + c / 64;
    return reinterpret_cast<float4 *>(p.htile) +
           ((unit * (np / 2) + j * (np / 4) + n / 4) << p.unit_shift) + (c % 64) / 2;
}

// ---------------------------------------------------------------------------
// functions
// ---------------------------------------------------------------------------
using ops::exp2_fast;
using ops::kLn2;
using ops::kLog2e;
using ops::load_pair;
using ops::Pair;
using ops::rcp_fast;
using ops::store_pair;
using ops::to_float2;

__device__ __forceinline__ float2 exp2_fast2(float2 x) {
    return make_float2(exp2_fast(x.x), exp2_fast(x.y));
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^{-|v|} in (0, 1], and
//   log(1 + e) = 2 artanh(w) = w p(w^2),  w = e / (2 + e) <= 1/3,
// p by a polynomial fitted to 2 artanh(w) / w over w^2 in [0, 1/9] (4e-9); small e keeps its
// digits.  The product of v with log2 e is taken in two parts, so that the error does not
// grow with |v|.
__device__ __forceinline__ float2 softplus2(float2 v) {
    using namespace ops;
    const float2 m = make_float2(max_nan(-fabsf(v.x), -100.0f), max_nan(-fabsf(v.y), -100.0f));
    const float2 nt = mul2(m, f2(-kLog2e));
    const float2 r = fma2(m, f2(1.92596299e-8f), fma2(m, f2(kLog2e), nt));
    float2 e = make_float2(exp2_fast(-nt.x), exp2_fast(-nt.y));
    e = fma2(e, mul2(r, f2(kLn2)), e);
    const float2 d = add2(e, f2(2.0f));
    const float2 w = mul2(e, make_float2(rcp_fast(d.x), rcp_fast(d.y))), q = mul2(w, w);
    float2 s = fma2(q, f2(0.2817833f), f2(0.27960604f));
    s = fma2(s, q, f2(0.4002491f));
    s = fma2(s, q, f2(0.66666317f));
    s = fma2(s, q, f2(2.0f));
    return fma2(w, s, make_float2(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
}
// 1 / (1 + e^{-v}), to 1e-6 for |v| up to 10
__device__ __forceinline__ float2 logistic2(float2 v) {
    using namespace ops;
    const float2 d = add2(exp2_fast2(mul2(v, f2(-kLog2e))), f2(1.0f));
    return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}

}  // namespace scan
}  // namespace fno
