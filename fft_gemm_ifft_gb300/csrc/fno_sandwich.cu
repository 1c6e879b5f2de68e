// fno_sandwich.cu -- norms before and after a block, fused with the block's
// gate, residual scale and residual sum, and their gradients.
//
// Forward, over the channels c of each point:
//   y_c = x_c + s_c a_c (n2(f)_c w2_c + b2_c),   u_c = n1(y)_c w1_c + b1_c,
//   n(v) = (v - mu) r,  mu = 0 (RMS) or mean v,  r = 1 / sqrt(mean (v - mu)^2 + eps).
// Backward, with N = n1(y), M = n2(f) and d = du w1:
//   dY = dy + r1 (d - mean(d) [LayerNorm] - N mean(d N)),       dx = dY
//   t = dY s a,  e = t w2:  df = r2 (e - mean(e) [LayerNorm] - M mean(e M))
//   A = sum dY a M, B = sum dY a  (over the points):
//   ds = w2 A + b2 B,  dw2 = s A,  db2 = s B,  dw1 = sum du N,  db1 = sum du
//   dg = dY s (M w2 + b2) a'(g), summed over the points for a gate per channel.
// A gate per (sample, channel) multiplies whole sums, so A and B are then kept
// per sample without it and it is applied in the last step.
#include <cfloat>

#include "fno_ops_internal.h"

using namespace fno;
using namespace fno::ops;

// How a call runs: by tiles (grid layout), by rows (tokens), or by the kernels
// for any size.  vec: elements of a thread's loads; per: a thread's channels
// (tiles) or runs (rows); warps: of a CTA; group: warps of a row.
enum { kAny = 0, kTiles = 1, kRows = 2, kStaged = 3 };
struct Way {
    int kind, vec, per, warps, group;    // (group of kStaged: its stages)
};

struct fno_sandwich_s {
    fno_sandwich_desc_t d;
    int sms;
    Way fwd, bwd;
    int segs;                // sums kept apart: samples for a gate per channel, else 1
    int64_t seg_points;      // points of a segment
    int splits;              // shares of a segment's points in the parameter sums
    size_t part_off, workspace;
};

namespace {

constexpr int kThreads = 256;
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

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

// a and da/dg of a gate value
__device__ __forceinline__ float gate_value(float g, bool sig) { return sig ? sigmoid(g) : g; }
__device__ __forceinline__ float gate_slope(float a, bool sig) { return sig ? a * (1.0f - a) : 1.0f; }

// A gradient times its norm's weight, rounded on its own: contracted into the
// subtraction of the mean it would differ from the mean's terms by a rounding,
// which r (up to 1 / sqrt(eps)) magnifies where the difference should vanish.
__device__ __forceinline__ float weighted(float g, float w) { return __fmul_rn(g, w); }

// A point's norm: n(v) = ((v - shift) - mean) r.  For LayerNorm the shift is the
// value of channel 0, so that a mean far above the spread costs no digits.
struct Norm {
    float shift, mean, r;
    __device__ __forceinline__ float operator()(float v) const { return ((v - shift) - mean) * r; }
};

// Running mean and sum of squared deviations (Welford), joined by Chan's rule:
// no cancellation when the mean is large against the spread.
struct Moments {
    float n, mean, m2;
    __device__ __forceinline__ void add(float v) {
        n += 1.0f;
        const float d = v - mean;
        mean += d / n;
        m2 = fmaf(d, v - mean, m2);
    }
    __device__ __forceinline__ void join(float n2, float mean2, float m22) {
        const float t = n + n2;
        if (t == 0.0f) return;
        const float d = mean2 - mean, f = n2 / t;
        mean = fmaf(d, f, mean);
        m2 += m22 + d * d * n * f;
        n = t;
    }
};

// Where the elements of point (b, p) are: channel c at base + c * stride.
template <bool GRID>
struct Point {
    int64_t base, stride;
    __device__ __forceinline__ Point(const Args &a, int64_t pt) {
        if (GRID) {
            const int64_t b = pt / a.points;
            base = b * a.channels * a.points + (pt - b * a.points);
            stride = a.points;
        } else {
            base = pt * a.channels;
            stride = 1;
        }
    }
    __device__ __forceinline__ int64_t at(int c) const { return base + c * stride; }
};

// The value of f at element `at` (point pt, channel c): stored, or a code's.
template <typename T, bool GRID>
__device__ __forceinline__ float load_f(const Args &a, int64_t at, int64_t pt, int c) {
    if (a.f) return Storage<T>::load(static_cast<const T *>(a.f) + at);
    int64_t sc;
    if (GRID) {
        const int64_t b = pt / a.points, p = pt - b * a.points;
        sc = (b * a.channels + c) * ((a.points + kGroup - 1) / kGroup) + p / kGroup;
    } else {
        sc = pt * ((a.channels + kGroup - 1) / kGroup) + c / kGroup;
    }
    return (float)a.f8[at] * a.f8_scale[sc];
}

template <typename T, bool GRID>
__device__ __forceinline__ float load_gate(const Args &a, int64_t at, int64_t pt, int c) {
    if (a.gate_kind == FNO_GATE_NONE) return 1.0f;
    const float g = a.gate_kind == FNO_GATE_FULL
                        ? Storage<T>::load(static_cast<const T *>(a.gate) + at)
                        : static_cast<const float *>(a.gate)[pt / a.points * a.channels + c];
    return gate_value(g, a.sigmoid);
}

// A team works on one point: a thread for GRID (neighbouring threads on
// neighbouring points), a warp for TOKENS (the lanes on neighbouring channels).
template <bool GRID>
struct Team {
    static constexpr int kSize = GRID ? 1 : 32;
    __device__ static int lane() { return GRID ? 0 : threadIdx.x & 31; }
    __device__ static int64_t first() {
        return ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kSize;
    }
    __device__ static int64_t step() { return (int64_t)gridDim.x * kThreads / kSize; }
    __device__ static float sum(float v) {
        if (!GRID)
#pragma unroll
            for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        return v;
    }
    // the norm of the values (less shift) that the team added up
    __device__ static Norm norm(Moments q, float shift, const Args &a) {
        if (!GRID)
#pragma unroll
            for (int m = 16; m; m >>= 1) {
                const float n = __shfl_xor_sync(0xffffffffu, q.n, m);
                const float mean = __shfl_xor_sync(0xffffffffu, q.mean, m);
                const float m2 = __shfl_xor_sync(0xffffffffu, q.m2, m);
                q.join(n, mean, m2);
            }
        const float var = a.layer ? q.m2 / q.n : q.m2 / q.n + q.mean * q.mean;
        return {shift, a.layer ? q.mean : 0.0f, rsqrtf(var + a.eps)};
    }
};

template <typename T, bool GRID>
__global__ void __launch_bounds__(kThreads) k_sandwich_fwd(Args a) {
    using W = Team<GRID>;
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y), *u = static_cast<T *>(a.u);
    for (int64_t pt = W::first(); pt < a.batch * a.points; pt += W::step()) {
        const Point<GRID> P(a, pt);
        Norm n2 = {0.0f, 0.0f, 0.0f}, n1 = n2;
        if (a.f) {
            Moments q = {0.0f, 0.0f, 0.0f};
            const float shift = a.layer ? load_f<T, GRID>(a, P.at(0), pt, 0) : 0.0f;
            for (int c = W::lane(); c < a.channels; c += W::kSize)
                q.add(load_f<T, GRID>(a, P.at(c), pt, c) - shift);
            n2 = W::norm(q, shift, a);
        }
        const auto value = [&](int c) {
            const int64_t at = P.at(c);
            const float v = Storage<T>::load(x + at);
            if (!a.f) return v;
            const float m = n2(load_f<T, GRID>(a, at, pt, c));
            const float z = a.layer ? fmaf(m, a.w2[c], a.b2[c]) : m * a.w2[c];
            return fmaf(a.s[c] * load_gate<T, GRID>(a, at, pt, c), z, v);
        };
        if (a.u) {
            Moments q = {0.0f, 0.0f, 0.0f};
            const float shift = a.layer ? value(0) : 0.0f;
            for (int c = W::lane(); c < a.channels; c += W::kSize) q.add(value(c) - shift);
            n1 = W::norm(q, shift, a);
        }
        if (!GRID) __syncwarp();      // y may be x: channel 0 is read by every lane
        for (int c = W::lane(); c < a.channels; c += W::kSize) {
            const float v = value(c);
            if (a.u) {
                const float n = n1(v);
                Storage<T>::store(u + P.at(c), a.layer ? fmaf(n, a.w1[c], a.b1[c]) : n * a.w1[c]);
            }
            if (a.y) Storage<T>::store(y + P.at(c), v);
        }
    }
}

template <typename T, bool GRID>
__global__ void __launch_bounds__(kThreads) k_sandwich_bwd(Args a) {
    using W = Team<GRID>;
    const T *y = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    const T *du = static_cast<const T *>(a.du);
    const bool block = a.f || a.f8;
    const float inv = 1.0f / (float)a.channels;
    for (int64_t pt = W::first(); pt < a.batch * a.points; pt += W::step()) {
        const Point<GRID> P(a, pt);
        Norm n1 = {0.0f, 0.0f, 0.0f}, n2 = n1;
        float d0 = 0.0f, d1 = 0.0f;
        if (a.du) {
            Moments q = {0.0f, 0.0f, 0.0f};
            const float shift = a.layer ? Storage<T>::load(y + P.at(0)) : 0.0f;
            for (int c = W::lane(); c < a.channels; c += W::kSize)
                q.add(Storage<T>::load(y + P.at(c)) - shift);
            n1 = W::norm(q, shift, a);
            for (int c = W::lane(); c < a.channels; c += W::kSize) {
                const float d = weighted(Storage<T>::load(du + P.at(c)), a.w1[c]);
                d0 += d;
                d1 = fmaf(d, n1(Storage<T>::load(y + P.at(c))), d1);
            }
            d0 = a.layer ? W::sum(d0) * inv : 0.0f;
            d1 = W::sum(d1) * inv;
        }
        const auto grad = [&](int c) {
            float g = a.dy ? Storage<T>::load(dy + P.at(c)) : 0.0f;
            if (a.du) {
                const float d = weighted(Storage<T>::load(du + P.at(c)), a.w1[c]);
                g = fmaf(n1.r, d - d0 - n1(Storage<T>::load(y + P.at(c))) * d1, g);
            }
            return g;
        };
        float e0 = 0.0f, e1 = 0.0f;
        if (block) {
            Moments q = {0.0f, 0.0f, 0.0f};
            const float shift = a.layer ? load_f<T, GRID>(a, P.at(0), pt, 0) : 0.0f;
            for (int c = W::lane(); c < a.channels; c += W::kSize)
                q.add(load_f<T, GRID>(a, P.at(c), pt, c) - shift);
            n2 = W::norm(q, shift, a);
            for (int c = W::lane(); c < a.channels; c += W::kSize) {
                const float t = grad(c) * a.s[c] * load_gate<T, GRID>(a, P.at(c), pt, c);
                const float e = weighted(t, a.w2[c]);
                e0 += e;
                e1 = fmaf(e, n2(load_f<T, GRID>(a, P.at(c), pt, c)), e1);
            }
            e0 = a.layer ? W::sum(e0) * inv : 0.0f;
            e1 = W::sum(e1) * inv;
        }
        for (int c = W::lane(); c < a.channels; c += W::kSize) {
            const int64_t at = P.at(c);
            const float g = grad(c);
            if (block) {
                const float m = n2(load_f<T, GRID>(a, at, pt, c));
                const float av = load_gate<T, GRID>(a, at, pt, c);
                const float t = g * a.s[c];
                if (a.dgate) {
                    const float z = a.layer ? fmaf(m, a.w2[c], a.b2[c]) : m * a.w2[c];
                    Storage<T>::store(static_cast<T *>(a.dgate) + at,
                                      t * z * gate_slope(av, a.sigmoid));
                }
                Storage<T>::store(static_cast<T *>(a.df) + at,
                                  n2.r * (weighted(t * av, a.w2[c]) - e0 - m * e1));
            }
        }
        if (W::lane() == 0) {
            float *st = a.stats + pt * kStats;
            st[0] = n1.shift;
            st[1] = n1.mean;
            st[2] = n1.r;
            st[3] = d0;
            st[4] = d1;
            st[5] = n2.shift;
            st[6] = n2.mean;
            st[7] = n2.r;
        }
    }
}

// dx and the sums A, B, sum du N, sum du of each channel over one share of one
// segment's points.  Block (32 channels, share, segment); GRID: a warp per
// channel, the lanes on points; TOKENS: the lanes on channels, warps on points.
// It runs after k_sandwich_bwd and writes dx last, so that dx may be dy.
template <typename T, bool GRID>
__global__ void __launch_bounds__(kThreads) k_sandwich_sums(Args a) {
    __shared__ float sm[kSums][8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int seg = blockIdx.z;
    const int64_t first = seg * a.seg_points;
    const int64_t per = (a.seg_points + a.splits - 1) / a.splits;
    const int64_t p0 = first + min(a.seg_points, blockIdx.y * per);
    const int64_t p1 = first + min(a.seg_points, (blockIdx.y + 1) * per);
    const bool block = a.f || a.f8;
    float *out = a.part + ((int64_t)seg * a.splits + blockIdx.y) * kSums * a.channels;
    for (int k = 0; k < (GRID ? 4 : 1); ++k) {
        const int c = blockIdx.x * 32 + (GRID ? w + 8 * k : lane);
        float sum[kSums] = {};
        if (c < a.channels) {
            for (int64_t pt = p0 + (GRID ? lane : w); pt < p1; pt += GRID ? 32 : 8) {
                const int64_t at = Point<GRID>(a, pt).at(c);
                const float *st = a.stats + pt * kStats;
                float g = a.dy ? Storage<T>::load(static_cast<const T *>(a.dy) + at) : 0.0f;
                if (a.du) {
                    const float d = Storage<T>::load(static_cast<const T *>(a.du) + at);
                    const float n =
                        Norm{st[0], st[1], st[2]}(Storage<T>::load(static_cast<const T *>(a.x) + at));
                    g = fmaf(st[2], weighted(d, a.w1[c]) - st[3] - n * st[4], g);
                    sum[2] = fmaf(d, n, sum[2]);
                    sum[3] += d;
                }
                if (block) {
                    const float m = Norm{st[5], st[6], st[7]}(load_f<T, GRID>(a, at, pt, c));
                    const float t = a.gate_kind == FNO_GATE_FULL
                                        ? g * load_gate<T, GRID>(a, at, pt, c) : g;
                    sum[0] = fmaf(t, m, sum[0]);
                    sum[1] += t;
                }
                Storage<T>::store(static_cast<T *>(a.dx) + at, g);
            }
        }
        if (GRID) {
#pragma unroll
            for (int j = 0; j < kSums; ++j) {
#pragma unroll
                for (int m = 16; m; m >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], m);
                if (lane == 0 && c < a.channels) out[j * a.channels + c] = sum[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSums; ++j) sm[j][w][lane] = sum[j];
            __syncthreads();
            if (w < kSums && c < a.channels) {
                float t = 0.0f;
#pragma unroll
                for (int r = 0; r < 8; ++r) t += sm[w][r][lane];
                out[w * a.channels + c] = t;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Grid layout, up to 512 channels: a CTA holds a tile of 32 V points by every
// channel in registers, so that each field is read once.  Warp w takes the
// channels w, w + warps, ... (CPT of them at most), lane l the V consecutive
// points l V ...; a norm's sums go over a thread's channels in registers and
// over the warps through shared memory.
// ---------------------------------------------------------------------------
constexpr int kMaxWarps = 16;

template <int V> __device__ __forceinline__ void store_row(float *at, const float (&v)[V]) {
    Pack<float, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.v[i] = v[i];
    *reinterpret_cast<Pack<float, V> *>(at) = p;
}

// mean and r of every point of the tile (2 barriers): the warps leave the mean
// and the squared deviations of their own channels, one thread a point joins
// them.  x(j) is the thread's channel j less its shift.
template <int V, int CPT, bool LAYER, class X>
__device__ __forceinline__ void tile_norm(X &&x, int mine, int channels, float eps, float *red,
                                          float *fin, float (&mean)[V], float (&r)[V]) {
    constexpr int PT = 32 * V;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float m[V] = {}, q[V] = {};
    if (LAYER) {
#pragma unroll
        for (int j = 0; j < CPT; ++j)
            if (j < mine)
#pragma unroll
                for (int i = 0; i < V; ++i) m[i] += x(j, i);
        const float inv = mine > 0 ? 1.0f / (float)mine : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] *= inv;
        store_row<V>(red + w * PT + lane * V, m);
    }
#pragma unroll
    for (int j = 0; j < CPT; ++j)
        if (j < mine)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = x(j, i) - m[i];
                q[i] = fmaf(d, d, q[i]);
            }
    store_row<V>(red + (warps + w) * PT + lane * V, q);
    __syncthreads();
    for (int p = threadIdx.x; p < PT; p += blockDim.x) {
        const float inv = 1.0f / (float)channels;
        const int base = channels / warps, more = channels - base * warps;   // warps with one more
        float mu = 0.0f, ss = 0.0f;
        if (LAYER) {
            for (int k = 0; k < warps; ++k)
                mu = fmaf((float)(base + (k < more)), red[k * PT + p], mu);
            mu *= inv;
        }
        for (int k = 0; k < warps; ++k) {
            ss += red[(warps + k) * PT + p];
            if (LAYER) {
                const float d = red[k * PT + p] - mu;
                ss = fmaf((float)(base + (k < more)), d * d, ss);
            }
        }
        fin[p] = mu;
        fin[PT + p] = rsqrtf(fmaf(ss, inv, eps));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        mean[i] = fin[lane * V + i];
        r[i] = fin[PT + lane * V + i];
    }
}

// Sums over the channels of a thread's points of two quantities (1 barrier).
template <int V>
__device__ __forceinline__ void tile_sum2(float (&a)[V], float (&b)[V], float *red) {
    constexpr int PT = 32 * V;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    store_row<V>(red + w * PT + lane * V, a);
    store_row<V>(red + (warps + w) * PT + lane * V, b);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = b[i] = 0.0f;
    for (int k = 0; k < warps; ++k) {
        const Pack<float, V> pa = *reinterpret_cast<Pack<float, V> *>(red + k * PT + lane * V);
        const Pack<float, V> pb =
            *reinterpret_cast<Pack<float, V> *>(red + (warps + k) * PT + lane * V);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] += pa.v[i];
            b[i] += pb.v[i];
        }
    }
}

// Shared memory of a grid kernel: per channel (s w2, s b2, w1, b1), then the
// sums' rows, then the norms' results.
size_t grid_smem(int channels, int V, int warps, int sums) {
    return (size_t)channels * 16 + (size_t)(sums * 2 * warps + 4) * 32 * V * 4;
}

template <typename T, int V, int CPT, bool LAYER>
__global__ void __launch_bounds__(512)
k_sandwich_fwd_grid(Args a, int8_t *f8, float *f8_scale) {
    constexpr int PT = 32 * V;
    extern __shared__ float4 sm[];
    float4 *par = sm;
    float *red = reinterpret_cast<float *>(sm + a.channels);
    float *fin = red + 2 * (blockDim.x >> 5) * PT;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int mine = (a.channels - w + warps - 1) / warps;
    const int64_t tiles = (a.points + PT - 1) / PT;
    const int64_t b = blockIdx.x / tiles, p = (blockIdx.x - b * tiles) * PT + lane * V;
    const bool on = p < a.points;
    const int64_t at = (b * a.channels + w) * a.points + p, step = warps * a.points;
    const T *x = static_cast<const T *>(a.x) + at, *f = static_cast<const T *>(a.f) + at;
    T *y = static_cast<T *>(a.y) + at, *u = static_cast<T *>(a.u) + at;
    const bool block = a.f != nullptr;
    float v[CPT][V];             // f, then y
    Pack<T, V> xs[CPT] = {};
    float shift[V] = {};
    if (block) {
        Pack<T, V> fs[CPT] = {}, f0 = {};
#pragma unroll
        for (int j = 0; j < CPT; ++j)
            if (on && j < mine) fs[j] = *reinterpret_cast<const Pack<T, V> *>(f + j * step);
        if (LAYER && on) f0 = *reinterpret_cast<const Pack<T, V> *>(f - w * a.points);
#pragma unroll
        for (int j = 0; j < CPT; ++j)
            if (on && j < mine) xs[j] = *reinterpret_cast<const Pack<T, V> *>(x + j * step);
        for (int c = threadIdx.x; c < a.channels; c += blockDim.x)
            par[c] = make_float4(a.s[c] * a.w2[c], LAYER ? a.s[c] * a.b2[c] : 0.0f,
                                 a.u ? a.w1[c] : 0.0f, LAYER && a.u ? a.b1[c] : 0.0f);
        if (f8) {                // V = 4: the warp's 128 points of a channel are one group
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                if (j >= mine) break;
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) m = max(m, abs_bits(Storage<T>::load(&fs[j].v[i])));
                m = __reduce_max_sync(0xffffffffu, m);
                const Group8 s = group8(m);
                Pack<int8_t, V> q;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    q.v[i] = (int8_t)code8(Storage<T>::load(&fs[j].v[i]), s.inv);
                if (on) *reinterpret_cast<Pack<int8_t, V> *>(f8 + at + j * step) = q;
                if (lane == 0)
                    f8_scale[(b * a.channels + w + j * warps) * tiles + blockIdx.x - b * tiles] =
                        s.scale;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) shift[i] = LAYER ? Storage<T>::load(&f0.v[i]) : 0.0f;
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) v[j][i] = Storage<T>::load(&fs[j].v[i]) - shift[i];
        float mean[V], r[V];
        tile_norm<V, CPT, LAYER>([&](int j, int i) { return v[j][i]; }, mine, a.channels, a.eps,
                                 red, fin, mean, r);
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            if (j >= mine) break;
            const int c = w + j * warps;
            const float4 q = par[c];
            float g[V];
            if (a.gate_kind == FNO_GATE_FULL) {
                Pack<T, V> gs = {};
                if (on)
                    gs = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.gate) +
                                                               at + j * step);
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] = gate_value(Storage<T>::load(&gs.v[i]), a.sigmoid);
            } else {
                const float gv = a.gate_kind == FNO_GATE_CHANNEL
                                     ? gate_value(static_cast<const float *>(a.gate)[b * a.channels + c],
                                                  a.sigmoid)
                                     : 1.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] = gv;
            }
            Pack<T, V> ys;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float m = (v[j][i] - mean[i]) * r[i];
                v[j][i] = fmaf(g[i], LAYER ? fmaf(m, q.x, q.y) : m * q.x,
                               Storage<T>::load(&xs[j].v[i]));
                Storage<T>::store(&ys.v[i], v[j][i]);
            }
            if (on) *reinterpret_cast<Pack<T, V> *>(y + j * step) = ys;
        }
        if (!a.u) return;
    } else {
        for (int c = threadIdx.x; c < a.channels; c += blockDim.x)
            par[c] = make_float4(0.0f, 0.0f, a.w1[c], LAYER ? a.b1[c] : 0.0f);
#pragma unroll
        for (int j = 0; j < CPT; ++j)
            if (on && j < mine) xs[j] = *reinterpret_cast<const Pack<T, V> *>(x + j * step);
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) v[j][i] = Storage<T>::load(&xs[j].v[i]);
    }
    // the shift of y's norm: channel 0 (its warp's first), by way of `fin`
    float mean[V], r[V];
    if (LAYER) {
        if (w == 0) store_row<V>(fin + 2 * PT + lane * V, v[0]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) shift[i] = fin[2 * PT + lane * V + i];
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) v[j][i] -= shift[i];
    }
    tile_norm<V, CPT, LAYER>([&](int j, int i) { return v[j][i]; }, mine, a.channels, a.eps, red,
                             fin, mean, r);
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
        if (j >= mine || !on) break;
        const float4 q = par[w + j * warps];
        Pack<T, V> us;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float n = (v[j][i] - mean[i]) * r[i];
            Storage<T>::store(&us.v[i], LAYER ? fmaf(n, q.z, q.w) : n * q.z);
        }
        *reinterpret_cast<Pack<T, V> *>(u + j * step) = us;
    }
}

// Backward on the same tiles; a CTA walks the tiles share, share + splits, ...
// of one segment (the tiles of a sample, or of all) and keeps its channels'
// sums in registers.  Each field is converted once, into the normalised value
// or the gradient that is used from there on: what bounds this kernel next to
// the bytes is the number of instructions an element.
template <typename T, int V, int CPT, bool LAYER, bool F8>
__global__ void __launch_bounds__(512)
k_sandwich_bwd_grid(Args a) {
    constexpr int PT = 32 * V;
    using TF = typename std::conditional<F8, int8_t, T>::type;
    extern __shared__ float4 sm[];
    float4 *par = sm;            // s a w2, s a, s b2, w1 (a of a gate per channel, else 1)
    float *red = reinterpret_cast<float *>(sm + a.channels);
    float *fin = red + 3 * 2 * (blockDim.x >> 5) * PT;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int mine = (a.channels - w + warps - 1) / warps;
    const int64_t tiles = (a.points + PT - 1) / PT, seg_tiles = a.batch / gridDim.y * tiles;
    const int64_t groups = (a.points + kGroup - 1) / kGroup;
    const bool block = F8 || a.f != nullptr, full = block && a.gate_kind == FNO_GATE_FULL;
    const float inv = 1.0f / (float)a.channels;
    for (int c = threadIdx.x; c < a.channels; c += blockDim.x) {
        float sa = block ? a.s[c] : 0.0f;
        const float sb = block && LAYER ? sa * a.b2[c] : 0.0f;
        if (block && a.gate_kind == FNO_GATE_CHANNEL)      // one sample a segment
            sa *= gate_value(static_cast<const float *>(a.gate)[blockIdx.y * a.channels + c],
                             a.sigmoid);
        par[c] = make_float4(block ? sa * a.w2[c] : 0.0f, sa, sb, a.du ? a.w1[c] : 0.0f);
    }
    __syncthreads();
    float acc[kSums][CPT] = {};
    for (int64_t t = blockIdx.x; t < seg_tiles; t += gridDim.x) {
        const int64_t tt = blockIdx.y * seg_tiles + t, b = tt / tiles;
        const int64_t p = (tt - b * tiles) * PT + lane * V;
        const bool on = p < a.points;
        const int64_t at = (b * a.channels + w) * a.points + p, step = warps * a.points;
        Pack<T, V> ys[CPT] = {}, us[CPT] = {}, gs[CPT] = {};
        Pack<TF, V> fs[CPT] = {};
        float fsc[F8 ? CPT : 1] = {}, shift1[V] = {}, shift2[V] = {};
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            if (!on || j >= mine) break;
            const int64_t e = at + j * step;
            if (a.du) {
                ys[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.x) + e);
                us[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.du) + e);
            }
            if (a.dy) gs[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.dy) + e);
            if (F8) {
                fs[j] = *reinterpret_cast<const Pack<TF, V> *>(a.f8 + e);
                fsc[j] = a.f8_scale[(b * a.channels + w + j * warps) * groups + p / kGroup];
            } else if (block) {
                fs[j] = *reinterpret_cast<const Pack<TF, V> *>(static_cast<const TF *>(a.f) + e);
            }
        }
        if (LAYER && on) {       // channel 0 of the point
            const int64_t e = at - w * a.points;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (a.du) shift1[i] = Storage<T>::load(static_cast<const T *>(a.x) + e + i);
                if (!block) continue;
                if constexpr (F8)
                    shift2[i] = (float)a.f8[e + i] *
                                a.f8_scale[b * a.channels * groups + p / kGroup];
                else
                    shift2[i] = Storage<T>::load(static_cast<const T *>(a.f) + e + i);
            }
        }
        float n1[CPT][V], n2[CPT][V], dY[CPT][V];
        float r1[V] = {}, r2[V] = {}, mu[V], d0[V] = {}, d1[V] = {};
        if (a.du) {
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) n1[j][i] = Storage<T>::load(&ys[j].v[i]) - shift1[i];
            tile_norm<V, CPT, LAYER>([&](int j, int i) { return n1[j][i]; }, mine, a.channels,
                                     a.eps, red, fin, mu, r1);
#pragma unroll
            for (int i = 0; i < V; ++i) r1[i] = on ? r1[i] : 0.0f;
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                if (j >= mine) break;
                const float w1 = par[w + j * warps].w;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float du = Storage<T>::load(&us[j].v[i]);
                    n1[j][i] = (n1[j][i] - mu[i]) * r1[i];
                    dY[j][i] = weighted(du, w1);
                    d0[i] += dY[j][i];
                    d1[i] = fmaf(dY[j][i], n1[j][i], d1[i]);
                    acc[2][j] = fmaf(du, n1[j][i], acc[2][j]);
                    if (LAYER) acc[3][j] += du;
                }
            }
            tile_sum2<V>(d0, d1, red + 4 * warps * PT);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                d0[i] = LAYER ? d0[i] * inv : 0.0f;
                d1[i] *= inv;
            }
        }
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            if (j >= mine) break;
            Pack<T, V> xs;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float g = Storage<T>::load(&gs[j].v[i]);
                if (a.du) g = fmaf(r1[i], dY[j][i] - d0[i] - n1[j][i] * d1[i], g);
                dY[j][i] = g;
                Storage<T>::store(&xs.v[i], g);
            }
            if (on) *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.dx) + at + j * step) = xs;
        }
        if (block) {
            float e0[V] = {}, e1[V] = {};
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float f;
                    if constexpr (F8) f = (float)fs[j].v[i] * fsc[j];
                    else f = Storage<T>::load(&fs[j].v[i]);
                    n2[j][i] = f - shift2[i];
                }
            tile_norm<V, CPT, LAYER>([&](int j, int i) { return n2[j][i]; }, mine, a.channels,
                                     a.eps, red + 2 * warps * PT, fin + 2 * PT, mu, r2);
#pragma unroll
            for (int i = 0; i < V; ++i) r2[i] = on ? r2[i] : 0.0f;
            // from here dY is the gradient of a (n2 w2 + b2) s, a of a full gate
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                if (j >= mine) break;
                const float4 q = par[w + j * warps];
                Pack<T, V> gate = {}, dg;
                if (full && on)
                    gate = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.gate) +
                                                                 at + j * step);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    n2[j][i] = (n2[j][i] - mu[i]) * r2[i];
                    if (full) {
                        const float av = gate_value(Storage<T>::load(&gate.v[i]), a.sigmoid);
                        Storage<T>::store(&dg.v[i], dY[j][i] * fmaf(n2[j][i], q.x, q.z) *
                                                        gate_slope(av, a.sigmoid));
                        dY[j][i] *= av;
                    }
                    acc[0][j] = fmaf(dY[j][i], n2[j][i], acc[0][j]);
                    if (LAYER) acc[1][j] += dY[j][i];
                    dY[j][i] = weighted(dY[j][i], q.x);
                    e0[i] += dY[j][i];
                    e1[i] = fmaf(dY[j][i], n2[j][i], e1[i]);
                }
                if (a.dgate && on)
                    *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.dgate) + at + j * step) = dg;
            }
            tile_sum2<V>(e0, e1, red);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                e0[i] = LAYER ? e0[i] * inv : 0.0f;
                e1[i] *= inv;
            }
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                if (j >= mine || !on) break;
                Pack<T, V> out;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    Storage<T>::store(&out.v[i], r2[i] * (dY[j][i] - e0[i] - n2[j][i] * e1[i]));
                *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.df) + at + j * step) = out;
            }
        }
        __syncthreads();         // the next tile's sums reuse the rows
    }
    float *out = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kSums * a.channels;
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
        if (j >= mine) break;
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
            float v = acc[k][j];
#pragma unroll
            for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            if (lane == 0) out[k * a.channels + w + j * warps] = v;
        }
    }
}

// ---------------------------------------------------------------------------
// Backward on tiles of 64 points by every channel (up to 128), for even point
// counts.  The fields' tiles come to shared memory asynchronously, the next
// tile's over the work on this one where two fit; warp w takes the 8 channels
// w, w + warps, ..., lane l the points 2 l and 2 l + 1, and all arithmetic is on
// the pair (f32x2): what bounds the kernel next to the bytes is the number of
// instructions, so sums are taken in two rounds (both norms' moments and
// sum d, sum d N in the first, sum e, sum e M in the second), and a normalised
// value is one subtraction and one multiply-add wherever it is needed.
//
// Moments.  A thread sums x - x0 and (x - x0)^2 over its channels, x0 its first
// channel; sum (x - mean)^2 = S2 - S1^2 / n loses at most a factor n + 1 of the
// digits, because x0's own deviation is part of it.  The warps' means are then
// joined relative to channel 0 of the point, so that a large mean cancels in
// exact differences.
// ---------------------------------------------------------------------------
constexpr int kTileP = 64, kTileC = 8;

template <typename T> __device__ __forceinline__ float2 load_pair(const T *p) {
    return Storage<T>::load2(p);
}
template <typename T> __device__ __forceinline__ void store_pair(T *p, float2 v);
template <> __device__ __forceinline__ void store_pair<float>(float *p, float2 v) {
    *reinterpret_cast<float2 *>(p) = v;
}
template <> __device__ __forceinline__ void store_pair<__half>(__half *p, float2 v) {
    *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(v.x, v.y);
}
template <> __device__ __forceinline__ void store_pair<__nv_bfloat16>(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ float2 code_pair(const int8_t *p) {
    const uint32_t w = (uint32_t)*reinterpret_cast<const uint16_t *>(p) ^ 0x8080u;
    return add2(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)),
                            __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441))),
                f2(-8388736.0f));
}

// bytes of a stage (the fields' tiles and the codes' scales) and of the rest
__host__ __device__ inline int tile_stage(int channels, int elem, bool f8, bool du, bool dy,
                                          bool block, bool full) {
    const int n = channels * kTileP;
    return n * elem * ((du ? 2 : 0) + dy + full + (block && !f8)) +
           (f8 ? n + (channels * 4 + 15) / 16 * 16 : 0);
}
__host__ __device__ inline int tile_rest(int channels, int warps) {
    return channels * 16 + 8 * warps * kTileP * 4 + 8 * kTileP * 4;
}

// WHOLE: every operand is there but a full gate, the points are a multiple of
// 64 and the channels of 8, so that no element needs a check.
template <typename T, bool LAYER, bool F8, bool WHOLE>
__global__ void __launch_bounds__(512)
k_sandwich_bwd_tile(Args a, int stages) {
    extern __shared__ float4 sm[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int C = a.channels, mine = WHOLE ? kTileC : (C - w + warps - 1) / warps;
    const bool block = F8 || WHOLE || a.f != nullptr;
    const bool full = !WHOLE && block && a.gate_kind == FNO_GATE_FULL;
    const bool has_du = WHOLE || a.du != nullptr, has_dy = WHOLE || a.dy != nullptr;
    float4 *par = sm;            // s a w2, s a, s b2, w1 (a of a gate per channel, else 1)
    float *rows = reinterpret_cast<float *>(sm + C);
    float *fin = rows + 8 * warps * kTileP;
    char *buf = reinterpret_cast<char *>(fin + 8 * kTileP);
    const int tile_n = C * kTileP, stage = tile_stage(C, sizeof(T), F8, has_du, has_dy, block, full);
    // offsets of the fields in a stage
    const int oy = 0, ou = oy + (has_du ? tile_n * (int)sizeof(T) : 0),
              og = ou + (has_du ? tile_n * (int)sizeof(T) : 0),
              oa = og + (has_dy ? tile_n * (int)sizeof(T) : 0),
              of = oa + (full ? tile_n * (int)sizeof(T) : 0), os = of + tile_n;
    const int64_t tiles = (a.points + kTileP - 1) / kTileP, seg_tiles = a.batch / gridDim.y * tiles;
    const int64_t groups = (a.points + kGroup - 1) / kGroup;
    const float inv = 1.0f / (float)C;
    const bool wide = WHOLE || a.points % (16 / sizeof(T)) == 0;
    const bool wide8 = WHOLE || a.points % 16 == 0;
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
        float sa = block ? a.s[c] : 0.0f;
        const float sb = block && LAYER ? sa * a.b2[c] : 0.0f;
        if (block && a.gate_kind == FNO_GATE_CHANNEL)      // one sample a segment
            sa *= gate_value(static_cast<const float *>(a.gate)[blockIdx.y * C + c], a.sigmoid);
        par[c] = make_float4(block ? sa * a.w2[c] : 0.0f, sa, sb, has_du ? a.w1[c] : 0.0f);
    }
    // a field's tile, 64 points of every channel (what lies past the row's end is
    // left as it is: those points are worked on and not stored)
    const auto fetch_field = [&](const void *src, int elem, bool by16, uint32_t dst, int64_t base,
                                 int np) {
        const char *s = static_cast<const char *>(src);
        if (WHOLE) {             // 16 warps at most: a thread's pieces are some rows apart
            const int per = kTileP * elem / 16, c = threadIdx.x / per;
            const int o = threadIdx.x % per * 16, hop = blockDim.x / per;
            const char *at = s + (base + (int64_t)c * a.points) * elem + o;
            const int64_t step = (int64_t)hop * a.points * elem;
            dst += c * kTileP * elem + o;
            const int n = C * per / blockDim.x;          // (C = 8 warps: 1, 2, 4 pieces)
#pragma unroll 4
            for (int i = 0; i < n; ++i, at += step, dst += hop * kTileP * elem)
                cp_async16(dst, at);
            return;
        }
        const int row = kTileP * elem, piece = by16 ? 16 : 4, per = row / piece;
        const int sh = 31 - __clz(per);                    // (a power of two)
        for (int i = threadIdx.x; i < C * per; i += blockDim.x) {
            const int c = i >> sh, o = (i & (per - 1)) * piece;
            if (o >= np * elem) continue;
            const char *at = s + (base + (int64_t)c * a.points) * elem + o;
            if (by16) cp_async16(dst + c * row + o, at);
            else if (elem > 1 || np * elem - o >= 4) cp_async4(dst + c * row + o, at);
        }
    };
    const auto fetch = [&](int64_t t, int k) {
        const int64_t tt = blockIdx.y * seg_tiles + t, b = tt / tiles, p = (tt - b * tiles) * kTileP;
        const int64_t base = b * C * a.points + p;
        const int np = (int)min((int64_t)kTileP, a.points - p);
        char *st = buf + k * stage;
        const uint32_t u = smem_u32(st);
        if (has_du) {
            fetch_field(a.x, sizeof(T), wide, u + oy, base, np);
            fetch_field(a.du, sizeof(T), wide, u + ou, base, np);
        }
        if (has_dy) fetch_field(a.dy, sizeof(T), wide, u + og, base, np);
        if (full) fetch_field(a.gate, sizeof(T), wide, u + oa, base, np);
        if (F8) {
            // rows of an even length start on 2 bytes: 4-byte copies need 4
            if (WHOLE || a.points % 4 == 0) {
                fetch_field(a.f8, 1, wide8, u + of, base, np);
            } else {
                for (int i = threadIdx.x; i < C * (kTileP / 2); i += blockDim.x) {
                    const int c = i / (kTileP / 2), o = i % (kTileP / 2) * 2;
                    if (o < np)
                        *reinterpret_cast<uint16_t *>(st + of + c * kTileP + o) =
                            *reinterpret_cast<const uint16_t *>(a.f8 + base +
                                                                (int64_t)c * a.points + o);
                }
            }
            for (int c = threadIdx.x; c < C; c += blockDim.x)
                cp_async4(u + os + c * 4, a.f8_scale + (b * C + c) * groups + p / kGroup);
        } else if (block) {
            fetch_field(a.f, sizeof(T), wide, u + of, base, np);
        }
    };
    float acc[kSums][kTileC] = {};
    int k = 0;
    if (blockIdx.x < seg_tiles) fetch(blockIdx.x, 0);
    cp_async_commit();
    for (int64_t t = blockIdx.x; t < seg_tiles; t += gridDim.x) {
        const int64_t tt = blockIdx.y * seg_tiles + t, b = tt / tiles;
        const int64_t p = (tt - b * tiles) * kTileP + lane * 2;
        const bool on = WHOLE || p < a.points;
        const int64_t at = (b * C + w) * a.points + p, step = warps * a.points;
        if (stages > 1) {
            if (t + gridDim.x < seg_tiles) fetch(t + gridDim.x, k ^ 1);
            cp_async_commit();
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        const char *st = buf + k * stage;
        const int first = w * kTileP + lane * 2, hop = warps * kTileP;
        const T *sy = reinterpret_cast<const T *>(st + oy) + first;
        const T *su = reinterpret_cast<const T *>(st + ou) + first;
        const T *sg = reinterpret_cast<const T *>(st + og) + first;
        const T *sa = reinterpret_cast<const T *>(st + oa) + first;
        const auto f_at = [&](int j) {
            if constexpr (F8) {
                const float s = reinterpret_cast<const float *>(st + os)[w + j * warps];
                return mul2(code_pair(reinterpret_cast<const int8_t *>(st + of) + first + j * hop),
                            f2(s));
            } else {
                return load_pair(reinterpret_cast<const T *>(st + of) + first + j * hop);
            }
        };
        float2 fv[kTileC];       // f
        // round 1: each warp's moments of y and f, sum d and sum d (y - y0)
        {
            float2 y0 = f2(0.0f), y1 = y0, y2 = y0, g0 = y0, g1 = y0, f0 = y0, f1 = y0, fq = y0;
#pragma unroll
            for (int j = 0; j < kTileC; ++j) {
                if (j >= mine) break;
                if (has_du) {
                    const float2 y = load_pair(sy + j * hop);
                    if (j == 0 && LAYER) y0 = y;
                    const float2 v = LAYER ? sub2(y, y0) : y;
                    const float2 d = mul2(load_pair(su + j * hop), f2(par[w + j * warps].w));
                    if (LAYER) y1 = add2(y1, v);
                    y2 = fma2(v, v, y2);
                    g0 = add2(g0, d);
                    g1 = fma2(d, v, g1);
                }
                if (block) {
                    fv[j] = f_at(j);
                    if (j == 0 && LAYER) f0 = fv[j];
                    const float2 v = LAYER ? sub2(fv[j], f0) : fv[j];
                    if (LAYER) f1 = add2(f1, v);
                    fq = fma2(v, v, fq);
                }
            }
            float *r = rows + w * kTileP + lane * 2;
            const int line = warps * kTileP;
            if (has_du) {
                if (LAYER) {
                    *reinterpret_cast<float2 *>(r) = y0;
                    *reinterpret_cast<float2 *>(r + line) = y1;
                }
                *reinterpret_cast<float2 *>(r + 2 * line) = y2;
                *reinterpret_cast<float2 *>(r + 3 * line) = g0;
                *reinterpret_cast<float2 *>(r + 4 * line) = g1;
            }
            if (block) {
                if (LAYER) {
                    *reinterpret_cast<float2 *>(r + 5 * line) = f0;
                    *reinterpret_cast<float2 *>(r + 6 * line) = f1;
                }
                *reinterpret_cast<float2 *>(r + 7 * line) = fq;
            }
        }
        __syncthreads();
        // joined by one thread for each (point, norm)
        for (int i = threadIdx.x; i < 2 * kTileP; i += blockDim.x) {
            const int q = i & (kTileP - 1), line = warps * kTileP;
            const bool second = i >= kTileP;
            if (second ? !block : !has_du) continue;
            const float *r = rows + q + (second ? 5 * line : 0);
            const int base = C / warps, more = C - base * warps;
            float ref = 0.0f, mean = 0.0f, ss = 0.0f, e0 = 0.0f, e1 = 0.0f;
            if (LAYER) {
                ref = r[0];
#pragma unroll 4
                for (int v = 0; v < warps; ++v)
                    mean += fmaf((float)(base + (v < more)), r[v * kTileP] - ref,
                                 r[line + v * kTileP]);
                mean *= inv;
            }
#pragma unroll 4
            for (int v = 0; v < warps; ++v) {
                ss += r[2 * line + v * kTileP];
                float off = 0.0f;
                if (LAYER) {
                    const float nv = (float)(base + (v < more)), s1 = r[line + v * kTileP];
                    off = r[v * kTileP] - ref;
                    const float m = __fdividef(s1, nv), d = off + m - mean;
                    ss += nv * d * d - m * s1;
                }
                if (!second) {
                    e0 += r[3 * line + v * kTileP];
                    e1 += fmaf(off, r[3 * line + v * kTileP], r[4 * line + v * kTileP]);
                }
            }
            const float rr = rsqrtf(fmaf(fmaxf(ss, 0.0f), inv, a.eps));
            float *o = fin + q + (second ? 5 * kTileP : 0);
            o[0] = ref;
            o[kTileP] = -mean * rr;
            o[2 * kTileP] = rr;
            if (!second) {
                o[3 * kTileP] = LAYER ? -e0 * inv : 0.0f;
                o[4 * kTileP] = -rr * (e1 - mean * e0) * inv;
            }
        }
        __syncthreads();
        const auto fin_at = [&](int i) {
            return *reinterpret_cast<const float2 *>(fin + i * kTileP + lane * 2);
        };
        // round 2: dY and dx, the channels' sums, sum e and sum e M
        const float2 ref1 = fin_at(0), mr1 = fin_at(1), r1 = fin_at(2), d0 = fin_at(3),
                     d1 = fin_at(4), ref2 = fin_at(5), mr2 = fin_at(6), r2 = fin_at(7);
        float2 e[kTileC], e0 = f2(0.0f), e1 = e0;
        T *dx = static_cast<T *>(a.dx) + at, *df = static_cast<T *>(a.df) + at;
#pragma unroll
        for (int j = 0; j < kTileC; ++j) {
            if (j >= mine) break;
            const float4 q = par[w + j * warps];
            float2 g = has_dy ? load_pair(sg + j * hop) : f2(0.0f);
            if (has_du) {
                const float2 y = load_pair(sy + j * hop), u = load_pair(su + j * hop);
                const float2 n = fma2(LAYER ? sub2(y, ref1) : y, r1, mr1);
                float2 d = mul2(u, f2(q.w));
                if (LAYER) d = add2(d, d0);
                g = fma2(fma2(n, d1, d), r1, g);
                const float2 un = mul2(u, n);
                if (on) {
                    acc[2][j] += un.x + un.y;
                    if (LAYER) acc[3][j] += u.x + u.y;
                }
            }
            if (on) store_pair(dx, g);
            dx += step;
            if (block) {
                const float2 m = fma2(LAYER ? sub2(fv[j], ref2) : fv[j], r2, mr2);
                fv[j] = m;       // M from here on
                if (full) {
                    const float2 gate = load_pair(sa + j * hop);
                    const float ax = gate_value(gate.x, a.sigmoid), ay = gate_value(gate.y, a.sigmoid);
                    if (a.dgate && on)
                        store_pair(static_cast<T *>(a.dgate) + at + j * step,
                                   mul2(mul2(g, fma2(m, f2(q.x), f2(q.z))),
                                        make_float2(gate_slope(ax, a.sigmoid),
                                                    gate_slope(ay, a.sigmoid))));
                    g = mul2(g, make_float2(ax, ay));
                }
                const float2 gm = mul2(g, m);
                if (on) {
                    acc[0][j] += gm.x + gm.y;
                    if (LAYER) acc[1][j] += g.x + g.y;
                }
                e[j] = mul2(g, f2(q.x));
                e0 = add2(e0, e[j]);
                e1 = fma2(e[j], m, e1);
            }
        }
        if (block) {
            float *r = rows + w * kTileP + lane * 2;
            const int line = warps * kTileP;
            if (LAYER) *reinterpret_cast<float2 *>(r) = e0;
            *reinterpret_cast<float2 *>(r + line) = e1;
            __syncthreads();
            e0 = e1 = f2(0.0f);
#pragma unroll 4
            for (int v = 0; v < warps; ++v) {
                const float *s = rows + v * kTileP + lane * 2;
                if (LAYER) e0 = add2(e0, *reinterpret_cast<const float2 *>(s));
                e1 = add2(e1, *reinterpret_cast<const float2 *>(s + line));
            }
            e0 = mul2(e0, f2(-inv));
            e1 = mul2(e1, f2(-inv));
#pragma unroll
            for (int j = 0; j < kTileC; ++j) {
                if (j >= mine || !on) break;
                float2 v = LAYER ? add2(e[j], e0) : e[j];
                v = mul2(fma2(fv[j], e1, v), r2);
                store_pair(df, v);
                df += step;
            }
        }
        __syncthreads();         // the next tile reuses the rows and the stage
        if (stages > 1) {
            k ^= 1;
        } else {
            if (t + gridDim.x < seg_tiles) fetch(t + gridDim.x, 0);
            cp_async_commit();
        }
    }
    float *out = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kSums * C;
#pragma unroll
    for (int j = 0; j < kTileC; ++j) {
        if (j >= mine) break;
#pragma unroll
        for (int q = 0; q < kSums; ++q) {
            float v = acc[q][j];
#pragma unroll
            for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            if (lane == 0) out[q * C + w + j * warps] = v;
        }
    }
}

// ---------------------------------------------------------------------------
// Token layout: G warps hold a row in registers, each thread J runs of V
// consecutive channels; a CTA of R = warps / G rows.
// ---------------------------------------------------------------------------
// the sum of N values over the G warps of a row
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int G, float (*red)[kMaxWarps]) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int m = 16; m; m >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
    if (G == 1) return;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();             // the last sum's readers are done
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) red[k][w] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = lane < G ? red[k][w / G * G + lane] : 0.0f;
#pragma unroll
        for (int m = 16; m; m >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
    }
}

// mean and r of a row whose values less the shift are x[.]; entries beyond the
// row's channels are excluded by `have`.
template <int N, bool LAYER, class Have>
__device__ __forceinline__ void row_norm(const float (&x)[N], Have &&have, int channels, float eps,
                                         int G, float (*red)[kMaxWarps], float &mean, float &r) {
    const float inv = 1.0f / (float)channels;
    mean = 0.0f;
    if (LAYER) {
        float s[1] = {};
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += x[i];          // absent entries are 0
        row_sum<1>(s, G, red);
        mean = s[0] * inv;
    }
    float q[1] = {};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = have(i) ? x[i] - mean : 0.0f;
        q[0] = fmaf(d, d, q[0]);
    }
    row_sum<1>(q, G, red);
    r = rsqrtf(fmaf(q[0], inv, eps));
}

template <typename T, int V, int J, bool LAYER>
__global__ void __launch_bounds__(512)
k_sandwich_fwd_rows(Args a, int G, int8_t *f8, float *f8_scale) {
    constexpr int N = V * J;
    __shared__ float red[1][kMaxWarps];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, R = (blockDim.x >> 5) / G;
    const int64_t rows = a.batch * a.points;
    const int64_t row = (int64_t)blockIdx.x * R + w / G;
    const bool on = row < rows;
    const int c0 = ((w % G) * 32 + lane) * V, cs = G * 32 * V;     // run j at c0 + j cs
    const int64_t base = row * a.channels;
    const auto have = [&](int i) { return c0 + i / V * cs < a.channels; };
    const bool block = a.f != nullptr;
    Pack<T, V> xs[J] = {};
    float v[N];
#pragma unroll
    for (int j = 0; j < J; ++j)
        if (on && have(j * V))
            xs[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.x) + base + c0 +
                                                          j * cs);
    if (block) {
        Pack<T, V> fs[J] = {};
        float shift = 0.0f, mean, r;
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (on && have(j * V))
                fs[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.f) + base +
                                                              c0 + j * cs);
        if (LAYER && on) shift = Storage<T>::load(static_cast<const T *>(a.f) + base);
        if (f8) {
            // a group is V L lanes' runs: 32 lanes for V = 4, 16 for 8; for V = 1
            // four runs of 32 lanes (G = 1 run j, or neighbouring warps): then
            // the caller packs by itself
            constexpr int L = V > 1 ? kGroup / V : 32;
            const uint32_t mask = L == 32 ? 0xffffffffu : 0xffffu << (lane & 16);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) m = max(m, abs_bits(Storage<T>::load(&fs[j].v[i])));
                m = __reduce_max_sync(mask, m);
                const Group8 s = group8(m);
                Pack<int8_t, V> q;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    q.v[i] = (int8_t)code8(Storage<T>::load(&fs[j].v[i]), s.inv);
                if (on && have(j * V)) {
                    const int c = c0 + j * cs;
                    *reinterpret_cast<Pack<int8_t, V> *>(f8 + base + c) = q;
                    if (lane % L == 0)
                        f8_scale[row * ((a.channels + kGroup - 1) / kGroup) + c / kGroup] = s.scale;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = have(i) ? Storage<T>::load(&fs[i / V].v[i % V]) - shift : 0.0f;
        row_norm<N, LAYER>(v, have, a.channels, a.eps, G, red, mean, r);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!on || !have(j * V)) continue;
            const int c = c0 + j * cs;
            const auto s = *reinterpret_cast<const Pack<float, V> *>(a.s + c);
            const auto w2 = *reinterpret_cast<const Pack<float, V> *>(a.w2 + c);
            Pack<float, V> b2 = {}, gf = {};
            Pack<T, V> gs = {}, ys;
            if (LAYER) b2 = *reinterpret_cast<const Pack<float, V> *>(a.b2 + c);
            if (a.gate_kind == FNO_GATE_FULL)
                gs = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.gate) + base + c);
            if (a.gate_kind == FNO_GATE_CHANNEL)
                gf = *reinterpret_cast<const Pack<float, V> *>(
                    static_cast<const float *>(a.gate) + row / a.points * a.channels + c);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float g = 1.0f;
                if (a.gate_kind != FNO_GATE_NONE)
                    g = gate_value(a.gate_kind == FNO_GATE_FULL ? Storage<T>::load(&gs.v[i])
                                                                : gf.v[i], a.sigmoid);
                const float m = (v[j * V + i] - mean) * r;
                const float z = LAYER ? fmaf(m, w2.v[i], b2.v[i]) : m * w2.v[i];
                v[j * V + i] = fmaf(s.v[i] * g, z, Storage<T>::load(&xs[j].v[i]));
                Storage<T>::store(&ys.v[i], v[j * V + i]);
            }
            *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.y) + base + c) = ys;
        }
        if (!a.u) return;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = have(i) ? Storage<T>::load(&xs[i / V].v[i % V]) : 0.0f;
    }
    float mean, r;
    if (LAYER) {                 // shift by the row's channel 0
        __shared__ float first[kMaxWarps];
        if (w % G == 0 && lane == 0) first[w / G] = v[0];
        __syncthreads();
        const float shift = first[w / G];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = have(i) ? v[i] - shift : 0.0f;
    }
    row_norm<N, LAYER>(v, have, a.channels, a.eps, G, red, mean, r);
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (!on || !have(j * V)) continue;
        const int c = c0 + j * cs;
        const auto w1 = *reinterpret_cast<const Pack<float, V> *>(a.w1 + c);
        Pack<float, V> b1 = {};
        if (LAYER) b1 = *reinterpret_cast<const Pack<float, V> *>(a.b1 + c);
        Pack<T, V> us;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float n = (v[j * V + i] - mean) * r;
            Storage<T>::store(&us.v[i], LAYER ? fmaf(n, w1.v[i], b1.v[i]) : n * w1.v[i]);
        }
        *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.u) + base + c) = us;
    }
}

template <typename T, int V, int J, bool LAYER, bool F8>
__global__ void __launch_bounds__(512)
k_sandwich_bwd_rows(Args a, int G) {
    constexpr int N = V * J;
    using TF = typename std::conditional<F8, int8_t, T>::type;
    __shared__ float red[2][kMaxWarps];
    extern __shared__ float4 sm[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, R = (blockDim.x >> 5) / G;
    const int c0 = ((w % G) * 32 + lane) * V, cs = G * 32 * V;
    const auto have = [&](int i) { return c0 + i / V * cs < a.channels; };
    const bool block = F8 || a.f != nullptr;
    const float inv = 1.0f / (float)a.channels;
    const int64_t groups = (a.channels + kGroup - 1) / kGroup;
    float acc[kSums][N] = {};
    for (int64_t t = (int64_t)blockIdx.x * R; t < a.seg_points; t += (int64_t)gridDim.x * R) {
        const bool on = t + w / G < a.seg_points;
        const int64_t row = blockIdx.y * a.seg_points + t + w / G, base = row * a.channels;
        Pack<T, V> ys[J] = {}, us[J] = {}, gs[J] = {}, gates[J] = {};
        Pack<TF, V> fs[J] = {};
        float fsc[F8 ? J : 1] = {};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!on || !have(j * V)) continue;
            const int64_t e = base + c0 + j * cs;
            if (a.du) {
                ys[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.x) + e);
                us[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.du) + e);
            }
            if (a.dy) gs[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.dy) + e);
            if (F8) {
                fs[j] = *reinterpret_cast<const Pack<TF, V> *>(a.f8 + e);
                fsc[j] = a.f8_scale[row * groups + (c0 + j * cs) / kGroup];
            } else if (block) {
                fs[j] = *reinterpret_cast<const Pack<TF, V> *>(static_cast<const TF *>(a.f) + e);
            }
            if (a.gate_kind == FNO_GATE_FULL && block)
                gates[j] =
                    *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.gate) + e);
        }
        float n1[N], m2[N], dY[N], mean, r1 = 0.0f, r2 = 0.0f, d[2] = {};
        if (a.du) {
            const float shift = LAYER && on ? Storage<T>::load(static_cast<const T *>(a.x) + base)
                                            : 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
                n1[i] = have(i) ? Storage<T>::load(&ys[i / V].v[i % V]) - shift : 0.0f;
            row_norm<N, LAYER>(n1, have, a.channels, a.eps, G, red, mean, r1);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                Pack<float, V> w1 = {};
                if (have(j * V)) w1 = *reinterpret_cast<const Pack<float, V> *>(a.w1 + c0 + j * cs);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int k = j * V + i;
                    n1[k] = have(k) ? (n1[k] - mean) * r1 : 0.0f;
                    const float du = Storage<T>::load(&us[j].v[i]);
                    acc[2][k] = fmaf(du, n1[k], acc[2][k]);
                    acc[3][k] += du;
                    dY[k] = weighted(du, w1.v[i]);
                    d[0] += dY[k];
                    d[1] = fmaf(dY[k], n1[k], d[1]);
                }
            }
            row_sum<2>(d, G, red);
            d[0] = LAYER ? d[0] * inv : 0.0f;
            d[1] *= inv;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            Pack<T, V> xs;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int k = j * V + i;
                float g = Storage<T>::load(&gs[j].v[i]);
                if (a.du) g = fmaf(r1, dY[k] - d[0] - n1[k] * d[1], g);
                dY[k] = have(k) ? g : 0.0f;
                Storage<T>::store(&xs.v[i], g);
            }
            if (on && have(j * V))
                *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.dx) + base + c0 + j * cs) = xs;
        }
        if (!block) continue;
        float shift = 0.0f;
        if constexpr (F8) {
            if (LAYER && on) shift = (float)a.f8[base] * a.f8_scale[row * groups];
        } else {
            if (LAYER && on) shift = Storage<T>::load(static_cast<const T *>(a.f) + base);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float f;
            if constexpr (F8) f = (float)fs[i / V].v[i % V] * fsc[i / V];
            else f = Storage<T>::load(&fs[i / V].v[i % V]);
            m2[i] = have(i) ? f - shift : 0.0f;
        }
        row_norm<N, LAYER>(m2, have, a.channels, a.eps, G, red, mean, r2);
        float e[2] = {}, ev[N];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = c0 + j * cs;
            Pack<float, V> s = {}, w2 = {}, b2 = {}, gf = {};
            Pack<T, V> dg;
            if (have(j * V)) {
                s = *reinterpret_cast<const Pack<float, V> *>(a.s + c);
                w2 = *reinterpret_cast<const Pack<float, V> *>(a.w2 + c);
                if (LAYER) b2 = *reinterpret_cast<const Pack<float, V> *>(a.b2 + c);
                if (a.gate_kind == FNO_GATE_CHANNEL)
                    gf = *reinterpret_cast<const Pack<float, V> *>(
                        static_cast<const float *>(a.gate) + blockIdx.y * a.channels + c);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int k = j * V + i;
                m2[k] = have(k) ? (m2[k] - mean) * r2 : 0.0f;
                float av = 1.0f;
                if (a.gate_kind != FNO_GATE_NONE)
                    av = gate_value(a.gate_kind == FNO_GATE_FULL ? Storage<T>::load(&gates[j].v[i])
                                                                 : gf.v[i], a.sigmoid);
                const float ga = a.gate_kind == FNO_GATE_FULL ? dY[k] * av : dY[k];
                acc[0][k] = fmaf(ga, m2[k], acc[0][k]);
                acc[1][k] += ga;
                const float ts = dY[k] * s.v[i];
                Storage<T>::store(&dg.v[i], ts * (LAYER ? fmaf(m2[k], w2.v[i], b2.v[i])
                                                        : m2[k] * w2.v[i]) *
                                                gate_slope(av, a.sigmoid));
                ev[k] = weighted(ts * av, w2.v[i]);
                e[0] += ev[k];
                e[1] = fmaf(ev[k], m2[k], e[1]);
            }
            if (a.dgate && on && have(j * V))
                *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.dgate) + base + c) = dg;
        }
        row_sum<2>(e, G, red);
        e[0] = LAYER ? e[0] * inv : 0.0f;
        e[1] *= inv;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!on || !have(j * V)) continue;
            Pack<T, V> out;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int k = j * V + i;
                Storage<T>::store(&out.v[i], r2 * (ev[k] - e[0] - m2[k] * e[1]));
            }
            *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.df) + base + c0 + j * cs) = out;
        }
    }
    // the CTA's rows joined in order, one of the four sums at a time
    float *join = reinterpret_cast<float *>(sm);        // [R][channels]
    float *out = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kSums * a.channels;
#pragma unroll
    for (int q = 0; q < kSums; ++q) {
        if (R > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (have(i)) join[(w / G) * a.channels + c0 + i / V * cs + i % V] = acc[q][i];
            __syncthreads();
            for (int c = threadIdx.x; c < a.channels; c += blockDim.x) {
                float t = 0.0f;
                for (int k = 0; k < R; ++k) t += join[k * a.channels + c];
                out[q * a.channels + c] = t;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (have(i)) out[q * a.channels + c0 + i / V * cs + i % V] = acc[q][i];
        }
    }
}

// The parameter gradients from the partial sums: 32 channels a block, 32 warps
// over the shares (and segments), joined in a fixed order.
__global__ void __launch_bounds__(1024)
k_sandwich_params(const float *__restrict__ part, int channels, int segs, int splits,
                  const float *s, const float *w2, const float *b2, const float *gate,
                  bool sig, float *ds, float *dw2, float *db2, float *dw1, float *db1,
                  float *dgate) {
    __shared__ float sm[kSums][32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const bool on = c < channels;
    float tot[kSums] = {};
    // warps of a segment: all 32 for one segment, fewer (a power of two) for more
    int per = 32;
    while (per > 1 && per * segs > 32) per >>= 1;
    const int r = w % per;
    for (int s0 = 0; s0 < segs; s0 += 32 / per) {
        const int seg = s0 + w / per;
        float v[kSums] = {};
        if (on && seg < segs)
            for (int k = r; k < splits; k += per)
#pragma unroll
                for (int j = 0; j < kSums; ++j)
                    v[j] += part[(((int64_t)seg * splits + k) * kSums + j) * channels + c];
        if (per > 1) {
#pragma unroll
            for (int j = 0; j < kSums; ++j) sm[j][w][lane] = v[j];
            __syncthreads();
            if (r == 0)
                for (int k = 1; k < per; ++k)
#pragma unroll
                    for (int j = 0; j < kSums; ++j) v[j] += sm[j][w + k][lane];
            __syncthreads();
        }
        if (r == 0 && on && seg < segs) {
            float a = 1.0f;
            if (gate) {
                a = gate_value(gate[(int64_t)seg * channels + c], sig);
                if (dgate)
                    dgate[(int64_t)seg * channels + c] =
                        s[c] * fmaf(w2[c], v[0], b2 ? b2[c] * v[1] : 0.0f) * gate_slope(a, sig);
            }
            tot[0] = fmaf(a, v[0], tot[0]);
            tot[1] = fmaf(a, v[1], tot[1]);
            tot[2] += v[2];
            tot[3] += v[3];
        }
    }
#pragma unroll
    for (int j = 0; j < kSums; ++j) sm[j][w][lane] = tot[j];
    __syncthreads();
    if (w == 0 && on) {
        for (int k = per; k < 32; k += per)
#pragma unroll
            for (int j = 0; j < kSums; ++j) tot[j] += sm[j][k][lane];
        if (ds) ds[c] = fmaf(w2[c], tot[0], b2 ? b2[c] * tot[1] : 0.0f);
        if (dw2) dw2[c] = s[c] * tot[0];
        if (db2) db2[c] = s[c] * tot[1];
        if (dw1) dw1[c] = tot[2];
        if (db1) db1[c] = tot[3];
    }
}

Args common_args(const fno_sandwich_s &p) {
    Args a = {};
    a.batch = p.d.batch;
    a.points = p.d.points;
    a.channels = p.d.channels;
    a.layer = p.d.norm == FNO_NORM_LAYER;
    a.sigmoid = p.d.gate_sigmoid != 0;
    a.gate_kind = p.d.gate;
    a.eps = p.d.eps;
    a.splits = p.splits;
    a.seg_points = p.seg_points;
    return a;
}

template <class F>
void with_layout(const fno_sandwich_s &p, F &&f) {
    with_storage(p.d.dtype, [&](auto t) {
        if (p.d.layout == FNO_LAYOUT_GRID) f(t, std::true_type());
        else f(t, std::false_type());
    });
}

constexpr int kSmemPerSm = 228 * 1024;

// The variant for a shape.  Vectors need the last axis (where every row
// starts) to be a multiple of them; registers bound a thread's elements (32 of
// each field forward, 16 to 32 of up to four backward), and with 16 warps a
// CTA's channels; longer rows take the kernels for any size, which read each
// field up to four times.
Way choose_way(const fno_sandwich_desc_t &d, bool backward) {
    const int c = d.channels, big = d.dtype == FNO_F32 ? 4 : 8;
    if (d.layout == FNO_LAYOUT_GRID) {
        const auto tiles = [&](int vec, int per) {
            return Way{kTiles, vec, per, (int)ceil_div(c, per), 0};
        };
        if (backward) {
            if (c <= 128 && d.points % 2 == 0) {
                const int warps = (int)ceil_div(c, kTileC);
                const int stage = tile_stage(c, (int)elem_bytes(d.dtype), false, true, true, true,
                                             d.gate == FNO_GATE_FULL);
                const int most = (kSmemPerSm / 2 - 1024 - tile_rest(c, warps)) / stage;
                return Way{kStaged, 2, kTileC, warps, most >= 2 ? 2 : 1};
            }
            if (c <= 128) return tiles(1, 8);
            if (c <= 256) return tiles(1, 16);
        } else {
            if (c <= 128) return tiles(d.points % 4 == 0 ? 4 : 1, 8);
            if (c <= 256 && d.points % 2 == 0) return tiles(2, 16);
            if (c <= 512) return tiles(1, 32);
        }
        return Way{kAny, 0, 0, 0, 0};
    }
    const int vec = c % big == 0 ? big : 1, each = backward ? 8 : 16;
    int group = 1;
    while (group <= 16 && group * 32 * each < c) group *= 2;
    if (group > 16) return Way{kAny, 0, 0, 0, 0};
    return Way{kRows, vec, each / vec, group > 8 ? group : 8, group};
}

// Calls f with the storage type and the variant's constants.
template <bool BACKWARD, class F>
void with_tiles(const fno_sandwich_s &p, const Way &way, F &&f) {
    with_storage(p.d.dtype, [&](auto t) {
        const auto layer = [&](auto v, auto per) {
            if (p.d.norm == FNO_NORM_LAYER) f(t, v, per, std::true_type());
            else f(t, v, per, std::false_type());
        };
        constexpr std::integral_constant<int, BACKWARD ? 1 : 4> wide;
        constexpr std::integral_constant<int, 1> one;
        constexpr std::integral_constant<int, 2> two;
        constexpr std::integral_constant<int, 8> few;
        constexpr std::integral_constant<int, BACKWARD ? 16 : 32> most;
        if (way.per == 8 && way.vec > 1) layer(wide, few);
        else if (way.per == 8) layer(one, few);
        else if (way.vec == 1) layer(one, most);
        else if constexpr (!BACKWARD) layer(two, std::integral_constant<int, 16>());
    });
}
template <int EACH, class F>
void with_rows(const fno_sandwich_s &p, const Way &way, F &&f) {
    using std::integral_constant;
    with_storage(p.d.dtype, [&](auto t) {
        const auto layer = [&](auto v, auto j) {
            if (p.d.norm == FNO_NORM_LAYER) f(t, v, j, std::true_type());
            else f(t, v, j, std::false_type());
        };
        constexpr int V = kVec<decltype(t)>;
        if (way.vec > 1) layer(integral_constant<int, V>(), integral_constant<int, EACH / V>());
        else layer(integral_constant<int, 1>(), integral_constant<int, EACH>());
    });
}

// The backward kernel of a plan as a function for Args, by its way.
template <class F>
void with_backward(const fno_sandwich_s &p, bool f8, bool whole, F &&f) {
    if (p.bwd.kind == kStaged) {
        with_storage(p.d.dtype, [&](auto t) {
            using T = decltype(t);
            const bool layer = p.d.norm == FNO_NORM_LAYER;
            const auto pick = [&](auto l, auto q) {
                constexpr bool L = decltype(l)::value, Q = decltype(q)::value;
                if (whole) f(k_sandwich_bwd_tile<T, L, Q, true>);
                else f(k_sandwich_bwd_tile<T, L, Q, false>);
            };
            if (layer && f8) pick(std::true_type(), std::true_type());
            else if (layer) pick(std::true_type(), std::false_type());
            else if (f8) pick(std::false_type(), std::true_type());
            else pick(std::false_type(), std::false_type());
        });
    } else if (p.bwd.kind == kTiles) {
        with_tiles<true>(p, p.bwd, [&](auto t, auto v, auto per, auto layer) {
            using T = decltype(t);
            constexpr int V = decltype(v)::value, CPT = decltype(per)::value;
            if (f8) f(k_sandwich_bwd_grid<T, V, CPT, decltype(layer)::value, true>);
            else f(k_sandwich_bwd_grid<T, V, CPT, decltype(layer)::value, false>);
        });
    } else {
        with_rows<8>(p, p.bwd, [&](auto t, auto v, auto j, auto layer) {
            using T = decltype(t);
            constexpr int V = decltype(v)::value, J = decltype(j)::value;
            if (f8) f(k_sandwich_bwd_rows<T, V, J, decltype(layer)::value, true>);
            else f(k_sandwich_bwd_rows<T, V, J, decltype(layer)::value, false>);
        });
    }
}

// (with_backward's kernels take Args and, but for kTiles, the way's `group`)
fno_status_t launch_backward(void (*k)(Args), dim3 grid, const Way &way, size_t smem,
                             cudaStream_t s, const Args &a) {
    k<<<grid, way.warps * 32, smem, s>>>(a);
    return launched();
}
fno_status_t launch_backward(void (*k)(Args, int), dim3 grid, const Way &way, size_t smem,
                             cudaStream_t s, const Args &a) {
    if (raise_smem_limit(k, smem) != cudaSuccess) return FNO_ERR_CUDA;
    k<<<grid, way.warps * 32, smem, s>>>(a, way.group);
    return launched();
}

// Shared memory of a call (of the largest call, for a plan: every operand there).
size_t backward_smem(const fno_sandwich_s &p, bool f8 = false, bool du = true, bool dy = true,
                     bool block = true) {
    const Way &way = p.bwd;
    const int c = p.d.channels;
    if (way.kind == kStaged)
        return tile_rest(c, way.warps) +
               (size_t)way.group * tile_stage(c, (int)elem_bytes(p.d.dtype), f8, du, dy, block,
                                              block && p.d.gate == FNO_GATE_FULL);
    if (way.kind == kTiles) return grid_smem(c, way.vec, way.warps, 3);
    const int rows = way.warps / way.group;
    return rows > 1 ? (size_t)rows * c * 4 : 0;
}

int team_blocks(const fno_sandwich_s &p) {
    const int64_t teams = p.d.batch * p.d.points;
    const int64_t per = p.d.layout == FNO_LAYOUT_GRID ? kThreads : kThreads / 32;
    const int64_t b = ceil_div(teams, per);
    return (int)(b < p.sms * 16 ? b : p.sms * 16);
}

struct Bytes {
    size_t field, vec, gate, f8, f8_scale;
};
Bytes bytes_of(const fno_sandwich_s &p) {
    const size_t n = (size_t)p.d.batch * p.d.channels * p.d.points;
    const bool grid = p.d.layout == FNO_LAYOUT_GRID;
    const size_t rows = (size_t)p.d.batch * (grid ? p.d.channels : p.d.points);
    return {n * elem_bytes(p.d.dtype), (size_t)p.d.channels * 4,
            p.d.gate == FNO_GATE_FULL ? n * elem_bytes(p.d.dtype)
                                      : (size_t)p.d.batch * p.d.channels * 4,
            n, rows * (size_t)ceil_div(grid ? p.d.points : p.d.channels, kGroup) * 4};
}

}  // namespace

extern "C" {

fno_status_t fno_sandwich_plan(fno_sandwich_t *out, const fno_sandwich_desc_t *d) {
    if (!out) return FNO_ERR_INVALID_ARG;
    *out = nullptr;
    if (!d || d->batch < 1 || d->points < 1 || d->channels < 1 || !valid_dtype(d->dtype) ||
        (d->layout != FNO_LAYOUT_GRID && d->layout != FNO_LAYOUT_TOKENS) ||
        (d->norm != FNO_NORM_RMS && d->norm != FNO_NORM_LAYER) ||
        (d->gate != FNO_GATE_NONE && d->gate != FNO_GATE_CHANNEL && d->gate != FNO_GATE_FULL) ||
        !(d->eps >= 0.0f) || !(d->eps <= FLT_MAX))
        return FNO_ERR_INVALID_ARG;
    if (d->channels > 65536 || (double)d->batch * d->channels * (double)d->points > kMaxElems ||
        (d->gate == FNO_GATE_CHANNEL && d->batch > 65535))
        return FNO_ERR_UNSUPPORTED;
    if (inject("plan_alloc")) return FNO_ERR_OUT_OF_MEMORY;
    fno_sandwich_s *p = new (std::nothrow) fno_sandwich_s();
    if (!p) return FNO_ERR_OUT_OF_MEMORY;
    p->d = *d;
    const fno_status_t st = device_sms(&p->sms);
    if (st != FNO_OK) {
        delete p;
        return st;
    }
    const int64_t points = d->batch * d->points;
    p->segs = d->gate == FNO_GATE_CHANNEL ? (int)d->batch : 1;
    p->seg_points = points / p->segs;
    p->fwd = choose_way(*d, false);
    p->bwd = choose_way(*d, true);
    int64_t want, most;      // shares of a segment: one wave of CTAs, or its tiles or rows
    if (p->bwd.kind == kAny) {
        want = ceil_div(4 * p->sms, ceil_div(d->channels, 32) * p->segs);
        most = ceil_div(p->seg_points, 32);
        p->part_off = ((size_t)points * kStats * 4 + 255) & ~size_t(255);
    } else {
        int ctas = 1;
        cudaError_t e = cudaSuccess;
        with_backward(*p, false, false, [&](auto kernel) {
            e = raise_smem_limit(kernel, backward_smem(*p));
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                    &ctas, kernel, p->bwd.warps * 32, backward_smem(*p));
        });
        if (e != cudaSuccess || ctas < 1) {
            cudaGetLastError();
            delete p;
            return FNO_ERR_CUDA;
        }
        want = (int64_t)p->sms * ctas / p->segs;
        if (want < 1) want = 1;
        most = p->bwd.kind == kRows ? ceil_div(p->seg_points, p->bwd.warps / p->bwd.group)
                                    : d->batch / p->segs * ceil_div(d->points, 32 * p->bwd.vec);
    }
    p->splits = (int)(want < most ? want : most);
    p->workspace = p->part_off + (size_t)p->segs * p->splits * kSums * d->channels * 4;
    *out = p;
    return FNO_OK;
}

fno_status_t fno_sandwich_workspace_size(fno_sandwich_t p, size_t *bytes) {
    if (!p || !bytes) return FNO_ERR_INVALID_ARG;
    *bytes = p->workspace;
    return FNO_OK;
}

fno_status_t fno_sandwich_forward(fno_sandwich_t p, const void *x, const void *f,
                                  const void *gate, const float *s, const float *w2,
                                  const float *b2, const float *w1, const float *b1, void *y,
                                  void *u, int8_t *f8, float *f8_scale, fno_stream_t stream) {
    if (!p || !x || (!f && !u)) return FNO_ERR_INVALID_ARG;
    const bool layer = p->d.norm == FNO_NORM_LAYER;
    if (f ? (!y || !s || !w2 || layer != !!b2 || (p->d.gate != FNO_GATE_NONE) != !!gate)
          : (y || s || w2 || b2 || gate || f8))
        return FNO_ERR_INVALID_ARG;
    if (u ? (!w1 || layer != !!b1) : (w1 || b1)) return FNO_ERR_INVALID_ARG;
    if (!f8 != !f8_scale) return FNO_ERR_INVALID_ARG;
    const Bytes n = bytes_of(*p);
    fno_status_t st = check_operands(
        {{x, n.field, false}, {f, n.field, false}, {gate, n.gate, false}, {s, n.vec, false},
         {w2, n.vec, false}, {b2, n.vec, false}, {w1, n.vec, false}, {b1, n.vec, false},
         {y, n.field, true, x}, {u, n.field, true}, {f8, n.f8, true},
         {f8_scale, n.f8_scale, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    Args a = common_args(*p);
    a.x = x;
    a.f = f;
    a.gate = gate;
    a.s = s;
    a.w2 = w2;
    a.b2 = b2;
    a.w1 = w1;
    a.b1 = b1;
    a.y = y;
    a.u = u;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const Way &way = p->fwd;
    // the checkpoint's groups lie within a warp's loads in these two variants
    const bool inside = way.kind == kTiles ? way.vec == 4 : way.kind == kRows && way.vec > 1;
    if (way.kind == kTiles) {
        with_tiles<false>(*p, way, [&](auto t, auto v, auto per, auto layer) {
            constexpr int V = decltype(v)::value, CPT = decltype(per)::value;
            k_sandwich_fwd_grid<decltype(t), V, CPT, decltype(layer)::value>
                <<<(unsigned)(p->d.batch * ceil_div(p->d.points, 32 * V)), way.warps * 32,
                   grid_smem(a.channels, V, way.warps, 1), cs>>>(a, inside ? f8 : nullptr,
                                                                 f8_scale);
        });
    } else if (way.kind == kRows) {
        with_rows<16>(*p, way, [&](auto t, auto v, auto j, auto layer) {
            k_sandwich_fwd_rows<decltype(t), decltype(v)::value, decltype(j)::value,
                                decltype(layer)::value>
                <<<(unsigned)ceil_div(p->d.batch * p->d.points, way.warps / way.group),
                   way.warps * 32, 0, cs>>>(a, way.group, inside ? f8 : nullptr, f8_scale);
        });
    } else {
        with_layout(*p, [&](auto t, auto grid) {
            k_sandwich_fwd<decltype(t), decltype(grid)::value>
                <<<team_blocks(*p), kThreads, 0, cs>>>(a);
        });
    }
    st = launched();
    if (st != FNO_OK || !f8 || inside) return st;
    const bool g = p->d.layout == FNO_LAYOUT_GRID;
    return fno_act8_pack(p->d.batch * (g ? p->d.channels : p->d.points),
                         g ? p->d.points : p->d.channels, p->d.dtype, f, f8, f8_scale, stream);
}

fno_status_t fno_sandwich_backward(fno_sandwich_t p, const void *y, const void *f,
                                   const int8_t *f8, const float *f8_scale, const void *gate,
                                   const float *s, const float *w2, const float *b2,
                                   const float *w1, const void *dy, const void *du, void *dx,
                                   void *df, void *dgate, float *ds, float *dw2, float *db2,
                                   float *dw1, float *db1, void *workspace, fno_stream_t stream) {
    if (!p || !y || !dx || !workspace || (!dy && !du) || (f && f8) || !f8 != !f8_scale)
        return FNO_ERR_INVALID_ARG;
    const bool layer = p->d.norm == FNO_NORM_LAYER, block = f || f8;
    if (block ? (!df || !s || !w2 || layer != !!b2 || (p->d.gate != FNO_GATE_NONE) != !!gate ||
                 (dgate && !gate) || (db2 && !layer))
              : (df || s || w2 || b2 || gate || dgate || ds || dw2 || db2))
        return FNO_ERR_INVALID_ARG;
    if (du ? (!w1 || (db1 && !layer)) : (w1 || dw1 || db1)) return FNO_ERR_INVALID_ARG;
    const Bytes n = bytes_of(*p);
    fno_status_t st = check_operands(
        {{y, n.field, false}, {f, n.field, false}, {f8, n.f8, false},
         {f8_scale, n.f8_scale, false}, {gate, n.gate, false}, {s, n.vec, false},
         {w2, n.vec, false}, {b2, n.vec, false}, {w1, n.vec, false}, {dy, n.field, false},
         {du, n.field, false}, {dx, n.field, true, dy}, {df, n.field, true},
         {dgate, n.gate, true}, {ds, n.vec, true}, {dw2, n.vec, true}, {db2, n.vec, true},
         {dw1, n.vec, true}, {db1, n.vec, true}, {workspace, p->workspace, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    Args a = common_args(*p);
    a.x = y;
    a.f = f;
    a.f8 = f8;
    a.f8_scale = f8_scale;
    a.gate = gate;
    a.s = s;
    a.w2 = w2;
    a.b2 = b2;
    a.w1 = w1;
    a.dy = dy;
    a.du = du;
    a.dx = dx;
    a.df = df;
    a.dgate = p->d.gate == FNO_GATE_FULL ? dgate : nullptr;
    a.stats = static_cast<float *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + p->part_off);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const dim3 sums((unsigned)ceil_div(a.channels, 32), (unsigned)p->splits, (unsigned)p->segs);
    if (p->bwd.kind == kAny) {
        with_layout(*p, [&](auto t, auto grid) {
            using T = decltype(t);
            constexpr bool G = decltype(grid)::value;
            k_sandwich_bwd<T, G><<<team_blocks(*p), kThreads, 0, cs>>>(a);
            k_sandwich_sums<T, G><<<sums, kThreads, 0, cs>>>(a);
        });
    } else {
        const dim3 shares((unsigned)p->splits, (unsigned)p->segs);
        const bool whole = block && du && dy && p->d.gate != FNO_GATE_FULL &&
                           p->d.points % kTileP == 0 && p->d.channels % kTileC == 0;
        with_backward(*p, f8 != nullptr, whole, [&](auto kernel) {
            st = launch_backward(kernel, shares, p->bwd,
                                 backward_smem(*p, f8 != nullptr, du != nullptr, dy != nullptr,
                                               block),
                                 cs, a);
        });
        if (st != FNO_OK) return st;
    }
    const bool per_channel = block && p->d.gate == FNO_GATE_CHANNEL;
    k_sandwich_params<<<(unsigned)ceil_div(a.channels, 32), 1024, 0, cs>>>(
        a.part, a.channels, p->segs, p->splits, s, w2, b2,
        per_channel ? static_cast<const float *>(gate) : nullptr, a.sigmoid, ds, dw2, db2, dw1,
        db1, per_channel ? static_cast<float *>(dgate) : nullptr);
    return launched();
}

fno_status_t fno_sandwich_destroy(fno_sandwich_t p) {
    delete p;
    return FNO_OK;
}

}  // extern "C"
