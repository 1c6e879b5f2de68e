// fno_scan.h -- what the selective scan's translation units share.
#pragma once

#include "fno_ops_internal.h"

struct fno_scan_s {
    fno_scan_desc_t d;
    int sms;
    // forward: the time axis in `segments` parts that run side by side
    int64_t seg_len;
    int segments;
    // backward: parts of the time axis, in whole chunks
    int64_t bwd_seg_len;
    int bwd_segments;
    size_t workspace;
};

namespace fno {
namespace scan {

constexpr int kMaxStates = 128;
constexpr int kTile = 8;       // tokens staged at a time, and between two states kept for the backward

// The operands of a scan, and where its work lies in the workspace.
struct Args {
    const void *x, *dt, *B, *C, *z, *dy;
    const float *A, *D, *bias, *s0, *gsT;
    const int32_t *lengths;
    void *y, *dx, *ddt, *dB, *dC, *dz;
    float *sT, *dA, *dD, *dbias, *ds0;
    // per (sequence, segment): states at its end and, after the joining, in front of
    // it; likewise the gradients that reach its end; the sum of the steps
    float *hseg, *gseg, *dseg;
    // per (sequence, chunk): the state in front of it from zero at the segment's
    // start, and the sum of the steps since then
    float *hchunk, *dchunk;
    // partial sums of the gradients: of B and C per block of channels, of A, D and the
    // bias per (sequence, segment)
    float *part_bc, *part_a, *part_d;
    int64_t length, seg_len;
    int batch, channels, per_group, groups, states, segments, chblocks;
    int slabs;                 // of channels in a block
    bool softplus;
    int vec_c, vec_n;          // bytes that rows of channels and of states may be moved in
};

// What a plan needs of the workspace for the backward, and its parts.
struct BackwardParts {
    size_t hseg, gseg, dseg, hchunk, dchunk, part_bc, part_a, part_d, bytes;
};
BackwardParts backward_parts(const fno_scan_s &p);

template <typename T> fno_status_t forward_of(const fno_scan_s &p, Args a, cudaStream_t s);
template <typename T> fno_status_t backward_of(const fno_scan_s &p, Args a, cudaStream_t s);
// The states in front of the segments from the local ones at their ends, in place
// (reverse: the gradients that reach the segments' ends, from the last one).
fno_status_t join(const Args &a, bool reverse, cudaStream_t s);

// States per lane of a quad (1, 2 or 4) and warps that share a slab's states.
inline int lane_states(int states) { return states <= 4 ? 1 : states <= 8 ? 2 : 4; }
inline int state_warps(int states) {
    int w = 1;
    while (16 * w < states) w *= 2;
    return w;
}
inline int padded_states(int states) { return 4 * lane_states(states) * state_warps(states); }
int forward_slabs(const fno_scan_s &p);
int backward_slabs(const fno_scan_s &p);

// ---------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e^{-|v|}: the product with log2 e in two parts, so that the error does not grow
// with |v|
__device__ __forceinline__ float exp_neg_abs(float v) {
    const float m = -fabsf(v);
    const float t = m * kLog2e;
    const float r = fmaf(m, 1.92596299e-8f, fmaf(m, kLog2e, -t));
    const float e = exp2_fast(t);
    return m < -100.0f ? 0.0f : fmaf(e, r * kLn2, e);      // (an infinity's r is a NaN)
}
// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^{-|v|} in (0, 1], and
//   log(1 + e) = 2 artanh(w) = 2 w (1 + w^2/3 + w^4/5 + ...),  w = e / (2 + e) <= 1/3
// (the terms left out are below 2e-8 of the sum; small e keeps its digits)
__device__ __forceinline__ float softplus(float v) {
    const float e = exp_neg_abs(v);
    const float w = __fdividef(e, 2.0f + e), q = w * w;
    float s = 1.0f / 13.0f;
    s = fmaf(s, q, 1.0f / 11.0f);
    s = fmaf(s, q, 1.0f / 9.0f);
    s = fmaf(s, q, 1.0f / 7.0f);
    s = fmaf(s, q, 1.0f / 5.0f);
    s = fmaf(s, q, 1.0f / 3.0f);
    s = fmaf(s, q, 1.0f);
    return fmaxf(v, 0.0f) + 2.0f * w * s;
}
// 1 / (1 + e^{-v})
__device__ __forceinline__ float logistic(float v) {
    const float e = exp_neg_abs(v);
    return __fdividef(v < 0.0f ? e : 1.0f, 1.0f + e);
}

// Rows of a tile from global to shared memory: `rows` of them (the first `valid` are
// there, the others become zero) of `cols` elements, zero beyond up to `pitch` (a power
// of two); rows are `stride` elements apart in memory.  By asynchronous copies of `vec`
// bytes, which rows, strides and cols are multiples of (2: element by element), or of as
// many as a row holds here.
template <typename T>
__device__ __forceinline__ void stage(T *dst, const T *src, int64_t stride, int rows, int valid,
                                      int cols, int pitch, int vec, int tid, int threads) {
    vec = min(vec, pitch * (int)sizeof(T));
    const int per = vec / (int)sizeof(T), shift = 31 - __clz(pitch / per);
#pragma unroll 1
    for (int i = tid; i < rows << shift; i += threads) {
        const int t = i >> shift, c = (i - (t << shift)) * per;
        T *to = dst + t * pitch + c;
        if (t < valid && c < cols) {
            const T *from = src + t * stride + c;
            const uint32_t at = ops::smem_u32(to);
            if (vec == 16) ops::cp_async16(at, from);
            else if (vec == 8) ops::cp_async8(at, from);
            else if (vec == 4) ops::cp_async4(at, from);
            else *to = *from;
        } else {
            for (int k = 0; k < per; ++k) Storage<T>::store(to + k, 0.0f);
        }
    }
}

}  // namespace scan
}  // namespace fno
