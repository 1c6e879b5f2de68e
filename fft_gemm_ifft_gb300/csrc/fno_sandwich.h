// fno_sandwich.h -- what the sandwich norm's translation units share: the plan,
// the kernels' arguments, the gate, and the entry points of the variants.
#pragma once

#include "fno_ops_internal.h"

namespace fno {
namespace sandwich {
// How a call runs: by the kernels for any size, by tiles held in registers, by
// token rows, by tiles staged in shared memory, or by tiles read again for each
// round of sums.
enum { kAny = 0, kTiles = 1, kRows = 2, kStaged = 3, kWide = 4 };
// vec: elements of a thread's loads, parts of a warp for kStaged; per: a thread's
// channels (tiles) or runs (rows); warps: of a CTA; group: warps of a row, stages
// of kStaged; lanes: of a row within one warp.
struct Way {
    int kind, vec, per, warps, group, lanes;
};
}  // namespace sandwich
}  // namespace fno

struct fno_sandwich_s {
    fno_sandwich_desc_t d;
    int sms;
    fno::sandwich::Way fwd, bwd;
    int segs;                // sums kept apart: samples for a gate per channel, else 1
    int64_t seg_points;      // points of a segment
    int splits;              // shares of a segment's points in the parameter sums
    size_t part_off, workspace;
};

namespace fno {
namespace sandwich {

constexpr int kStats = 8;    // per point: norm 1 (shift, mean, r), mean(d), mean(d N), norm 2
constexpr int kSums = 4;     // per channel: A, B, sum du N, sum du

// The operands of a call, as the kernels take them.
struct Args {
    const void *x, *f, *gate, *dy, *du;    // x: the stream (forward) or y (backward)
    const float *s, *w2, *b2, *w1, *b1;
    const int8_t *f8;
    const float *f8_scale;
    void *y, *u, *dx, *df, *dgate;         // dgate: of a full gate
    float *stats, *part;
    int64_t batch, points;
    int channels;
    bool layer, sigmoid;
    int gate_kind;
    float eps;
    int splits;
    int64_t seg_points;
};

// (the fast exponential and quotient, 1e-6 relative for |g| up to 10: the exact
// quotient alone is a dozen instructions and a branch)
__device__ __forceinline__ float sigmoid(float g) {
    return __fdividef(1.0f, 1.0f + __expf(-g));
}

// a and da/dg of a gate value
__device__ __forceinline__ float gate_value(float g, bool sig) { return sig ? sigmoid(g) : g; }
__device__ __forceinline__ float gate_slope(float a, bool sig) { return sig ? a * (1.0f - a) : 1.0f; }

// A gradient times its norm's weight, rounded on its own: contracted into the
// subtraction of the mean it would differ from the mean's terms by a rounding,
// which r (up to 1 / sqrt(eps)) magnifies where the difference should vanish.
__device__ __forceinline__ float weighted(float g, float w) { return __fmul_rn(g, w); }
// (two scalar products: the packed one is contracted into a packed sum)
__device__ __forceinline__ float2 weighted2(float2 g, float w) {
    return make_float2(__fmul_rn(g.x, w), __fmul_rn(g.y, w));
}

// The variant of a layout for a description (kAny: the kernels for any size).
Way grid_forward_way(const fno_sandwich_desc_t &d);
Way grid_backward_way(const fno_sandwich_desc_t &d);
Way rows_way(const fno_sandwich_desc_t &d, bool backward);
// The forward of p.fwd, which must be the layout's; *packed: f was kept in 8
// bits on the way (f8 may be NULL).
fno_status_t grid_forward(const fno_sandwich_s &p, const Args &a, int8_t *f8, float *f8_scale,
                          bool *packed, cudaStream_t s);
fno_status_t rows_forward(const fno_sandwich_s &p, const Args &a, int8_t *f8, float *f8_scale,
                          bool *packed, cudaStream_t s);
// The backward of p.bwd: p.segs x p.splits CTAs.
fno_status_t grid_backward(const fno_sandwich_s &p, const Args &a, cudaStream_t s);
fno_status_t rows_backward(const fno_sandwich_s &p, const Args &a, cudaStream_t s);
// CTAs of the backward that an SM holds, and the most shares a segment divides into.
fno_status_t grid_shares(const fno_sandwich_s &p, int *ctas, int64_t *most);
fno_status_t rows_shares(const fno_sandwich_s &p, int *ctas, int64_t *most);

// f(a, b) with the two flags as constants
template <class F>
void with_bools(bool a, bool b, F &&f) {
    const std::true_type yes;
    const std::false_type no;
    if (a && b) f(yes, yes);
    else if (a) f(yes, no);
    else if (b) f(no, yes);
    else f(no, no);
}

// CTAs of a kernel that an SM holds
template <class K>
fno_status_t occupancy(K kernel, int threads, size_t smem, int *ctas) {
    if (raise_smem_limit(kernel, smem) == cudaSuccess &&
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kernel, threads, smem) ==
            cudaSuccess && *ctas > 0)
        return FNO_OK;
    cudaGetLastError();
    return FNO_ERR_CUDA;
}

}  // namespace sandwich
}  // namespace fno
