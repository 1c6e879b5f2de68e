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

#include "fno_sandwich.h"

using namespace fno;
using namespace fno::ops;
using namespace fno::sandwich;

namespace {

constexpr int kThreads = 256;

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
        (double)d->batch * d->points > 8.0 * 2147483647.0 ||       // (a grid of 8 rows a block)
        (d->gate == FNO_GATE_CHANNEL && d->batch > 65535))
        return FNO_ERR_UNSUPPORTED;
    if (inject("plan_alloc")) return FNO_ERR_OUT_OF_MEMORY;
    fno_sandwich_s *p = new (std::nothrow) fno_sandwich_s();
    if (!p) return FNO_ERR_OUT_OF_MEMORY;
    p->d = *d;
    fno_status_t st = device_sms(&p->sms);
    if (st != FNO_OK) {
        delete p;
        return st;
    }
    const int64_t points = d->batch * d->points;
    p->segs = d->gate == FNO_GATE_CHANNEL ? (int)d->batch : 1;
    p->seg_points = points / p->segs;
    const bool grid = d->layout == FNO_LAYOUT_GRID;
    p->fwd = grid ? grid_forward_way(*d) : rows_way(*d, false);
    p->bwd = grid ? grid_backward_way(*d) : rows_way(*d, true);
    int64_t want, most;      // shares of a segment: one wave of CTAs, or its tiles or rows
    if (p->bwd.kind == kAny) {
        want = ceil_div(4 * p->sms, ceil_div(d->channels, 32) * p->segs);
        most = ceil_div(p->seg_points, 32);
        p->part_off = ((size_t)points * kStats * 4 + 255) & ~size_t(255);
    } else {
        int ctas = 1;
        st = grid ? grid_shares(*p, &ctas, &most) : rows_shares(*p, &ctas, &most);
        if (st != FNO_OK) {
            delete p;
            return st;
        }
        want = (int64_t)p->sms * ctas / p->segs;
        if (want < 1) want = 1;
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
    bool packed = false;
    if (p->fwd.kind == kTiles) {
        st = grid_forward(*p, a, f8, f8_scale, &packed, cs);
    } else if (p->fwd.kind == kRows) {
        st = rows_forward(*p, a, f8, f8_scale, &packed, cs);
    } else {
        with_layout(*p, [&](auto t, auto grid) {
            k_sandwich_fwd<decltype(t), decltype(grid)::value>
                <<<team_blocks(*p), kThreads, 0, cs>>>(a);
        });
        st = launched();
    }
    if (st != FNO_OK || !f8 || packed) return st;
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
        st = p->bwd.kind == kRows ? rows_backward(*p, a, cs) : grid_backward(*p, a, cs);
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
