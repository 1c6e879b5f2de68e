// fno_rotary.cu -- rotary positions: every pair of a head's first elements turned by an
// angle that grows with the token's position.
//
// The angle of pair i at position p is p f_i.  In float32 a far position would lose it
// (p = 10^6 leaves an error of 0.06 radians), so the plan keeps f_i as the turns a
// position takes in 64-bit fixed point: p times that, modulo 2^64, is the fraction of a
// turn, exactly, for any 32-bit p (a negative one too), and its upper 32 bits go to the
// sine and cosine.
//
// Bound by bytes: each element is read and written once.  A thread keeps the sines and
// cosines of the pairs in one 16-byte vector (half layout: of two vectors, which hold the
// pairs' two sides) and goes over the token's heads, so that they cost a few percent.
#include "fno_ops_internal.h"

#include <cmath>

using namespace fno;
using namespace fno::ops;

struct fno_rotary_s {
    fno_rotary_desc_t d;
    float magnitude;
    int sms;
    uint64_t turns[128];       // a position's turns of each pair, times 2^64
};

namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 128;

struct Turns {
    uint64_t v[kMaxPairs];
};
struct Args {
    const void *q, *k;
    void *qo, *ko;
    const int32_t *positions, *offsets;
    int64_t rows, length;
    int heads, kv_heads, dim, rotary;
    int units, lanes;          // vectors of a head; threads that share a token's heads
    float magnitude;
    bool transpose;
};

// HALF: a thread turns V elements of the first side with V of the second; interleaved: the
// pairs in a run of max(V, 2) elements.  The units beyond the pairs are V elements copied.
// V divides the rotary part's sides (half) or the rotary part, and the head.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads)
k_rotary(const Args p, const __grid_constant__ Turns turns) {
    constexpr int R = HALF || V > 1 ? V : 2, N = HALF ? V : R / 2;      // a run, its pairs
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int per_token = p.units * p.lanes;
    const int64_t row = id / per_token;
    if (row >= p.rows) return;
    const int rest = (int)(id - row * per_token), first = rest / p.units;
    const int unit = rest - first * p.units;
    const int half = p.rotary / 2;
    const int turning = HALF ? half / V : p.rotary / R;        // units that turn
    const int heads = p.heads + p.kv_heads;
    const int64_t base = row * p.heads * p.dim, kbase = row * p.kv_heads * p.dim;
    const auto head = [&](int h, const T *&from, T *&to) {
        if (h < p.heads) {
            from = static_cast<const T *>(p.q) + base + (int64_t)h * p.dim;
            to = static_cast<T *>(p.qo) + base + (int64_t)h * p.dim;
        } else {
            const int64_t o = kbase + (int64_t)(h - p.heads) * p.dim;
            from = static_cast<const T *>(p.k) + o;
            to = static_cast<T *>(p.ko) + o;
        }
    };
    if (unit >= turning) {
        if (p.q == p.qo && p.k == p.ko) return;
        const int at = p.rotary + (unit - turning) * V;
#pragma unroll 2
        for (int h = first; h < heads; h += p.lanes) {
            const T *from;
            T *to;
            head(h, from, to);
            *reinterpret_cast<Pack<T, V> *>(to + at) =
                *reinterpret_cast<const Pack<T, V> *>(from + at);
        }
        return;
    }
    int64_t pos = row;
    if (p.positions) {
        pos = p.positions[row];
    } else {
        const int64_t b = row / p.length;
        pos = row - b * p.length;
        if (p.offsets) pos += p.offsets[b];
    }
    float co[N], si[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint64_t turn = (uint64_t)pos * turns.v[unit * N + i];
        // the upper half as a signed number: -1/2 .. 1/2 of a turn
        const float x = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;    // 2^-31
        float s, c;
        sincospif(x, &s, &c);
        co[i] = p.magnitude * c;
        si[i] = p.transpose ? -p.magnitude * s : p.magnitude * s;
    }
    const int at = unit * R;
#pragma unroll 2
    for (int h = first; h < heads; h += p.lanes) {
        const T *from;
        T *to;
        head(h, from, to);
        if constexpr (HALF) {
            const Pack<T, V> a = *reinterpret_cast<const Pack<T, V> *>(from + at);
            const Pack<T, V> b = *reinterpret_cast<const Pack<T, V> *>(from + half + at);
            Pack<T, V> x, y;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float av = Storage<T>::load(&a.v[i]), bv = Storage<T>::load(&b.v[i]);
                Storage<T>::store(&x.v[i], fmaf(av, co[i], -(bv * si[i])));
                Storage<T>::store(&y.v[i], fmaf(bv, co[i], av * si[i]));
            }
            *reinterpret_cast<Pack<T, V> *>(to + at) = x;
            *reinterpret_cast<Pack<T, V> *>(to + half + at) = y;
        } else {
            Pack<T, V> a[R / V];
#pragma unroll
            for (int i = 0; i < R / V; ++i)
                a[i] = *reinterpret_cast<const Pack<T, V> *>(from + at + i * V);
            T *e = a[0].v;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float av = Storage<T>::load(e + 2 * i), bv = Storage<T>::load(e + 2 * i + 1);
                Storage<T>::store(e + 2 * i, fmaf(av, co[i], -(bv * si[i])));
                Storage<T>::store(e + 2 * i + 1, fmaf(bv, co[i], av * si[i]));
            }
#pragma unroll
            for (int i = 0; i < R / V; ++i) *reinterpret_cast<Pack<T, V> *>(to + at + i * V) = a[i];
        }
    }
}

template <typename T, int V>
fno_status_t launch(const fno_rotary_s &plan, Args a, const Turns &turns, cudaStream_t s) {
    const bool half = plan.d.layout == FNO_ROTARY_HALF;
    const int turning = half ? a.rotary / 2 / V : a.rotary / (V > 1 ? V : 2);
    a.units = turning + (a.dim - a.rotary) / V;
    // a token's heads go over as many threads as it takes to fill the SMs, so that the
    // sines are worked out as few times as that allows
    const int heads = a.heads + a.kv_heads;
    const int64_t want = (int64_t)plan.sms * 1024;
    int lanes = 1;
    while (lanes < heads && a.rows * a.units * lanes < want) lanes *= 2;
    a.lanes = lanes < heads ? lanes : heads;
    const int64_t blocks = ceil_div(a.rows * a.units * a.lanes, kThreads);
    if (blocks > 2147483647) return FNO_ERR_UNSUPPORTED;
    if (half) k_rotary<T, V, true><<<(unsigned)blocks, kThreads, 0, s>>>(a, turns);
    else k_rotary<T, V, false><<<(unsigned)blocks, kThreads, 0, s>>>(a, turns);
    return launched();
}

}  // namespace

extern "C" {

fno_status_t fno_rotary_plan(fno_rotary_t *out, const fno_rotary_desc_t *desc) {
    if (!out) return FNO_ERR_INVALID_ARG;
    *out = nullptr;
    if (!desc) return FNO_ERR_INVALID_ARG;
    const fno_rotary_desc_t d = *desc;
    if (d.batch < 1 || d.length < 1 || d.heads < 1 || d.kv_heads < 0 || d.dim < 1 ||
        d.rotary_dim < 2 || d.rotary_dim % 2 || d.rotary_dim > d.dim ||
        (d.layout != FNO_ROTARY_HALF && d.layout != FNO_ROTARY_INTERLEAVED) ||
        !valid_dtype(d.dtype) || !(d.base > 1.0) || !std::isfinite(d.base))
        return FNO_ERR_INVALID_ARG;
    if (d.scaling < FNO_ROTARY_NONE || d.scaling > FNO_ROTARY_RAMP) return FNO_ERR_INVALID_ARG;
    if (d.scaling != FNO_ROTARY_NONE && !(d.factor >= 1.0 && std::isfinite(d.factor)))
        return FNO_ERR_INVALID_ARG;
    if (d.scaling == FNO_ROTARY_BASE && d.rotary_dim == 2) return FNO_ERR_INVALID_ARG;
    if (d.scaling == FNO_ROTARY_RAMP &&
        !(d.original > 0.0 && std::isfinite(d.original) && d.slow >= 0.0 && d.fast > d.slow &&
          std::isfinite(d.fast)))
        return FNO_ERR_INVALID_ARG;
    if (d.dim > 1024 || d.rotary_dim > 2 * kMaxPairs ||
        (double)d.batch * (double)d.length * ((double)d.heads + d.kv_heads) * d.dim > kMaxElems)
        return FNO_ERR_UNSUPPORTED;
    if (inject("plan_alloc")) return FNO_ERR_OUT_OF_MEMORY;
    fno_rotary_s *p = new (std::nothrow) fno_rotary_s();
    if (!p) return FNO_ERR_OUT_OF_MEMORY;
    p->d = d;
    p->magnitude = 1.0f;
    fno_status_t st = device_sms(&p->sms);
    if (st != FNO_OK) {
        delete p;
        return st;
    }
    const double pi = 3.14159265358979323846, r = d.rotary_dim;
    double base = d.base;
    if (d.scaling == FNO_ROTARY_BASE) base *= std::pow(d.factor, r / (r - 2.0));
    if (d.scaling == FNO_ROTARY_RAMP) p->magnitude = (float)(1.0 + 0.1 * std::log(d.factor));
    for (int i = 0; i < d.rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / r);
        if (d.scaling == FNO_ROTARY_LINEAR) f /= d.factor;
        if (d.scaling == FNO_ROTARY_RAMP) {
            const double turns = d.original * f / (2.0 * pi);
            double keep = (turns - d.slow) / (d.fast - d.slow);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f *= keep + (1.0 - keep) / d.factor;
        }
        // f <= 1 radian: less than a sixth of a turn a position
        p->turns[i] = (uint64_t)std::ldexp(f / (2.0 * pi), 64);
    }
    *out = p;
    return FNO_OK;
}

fno_status_t fno_rotary_apply(fno_rotary_t p, const void *q, const void *k,
                              const int32_t *positions, const int32_t *offsets,
                              int32_t transpose, void *qo, void *ko, fno_stream_t stream) {
    if (!p || !q || !qo || (positions && offsets)) return FNO_ERR_INVALID_ARG;
    const fno_rotary_desc_t &d = p->d;
    if (d.kv_heads ? !k || !ko : k || ko) return FNO_ERR_INVALID_ARG;
    const size_t e = elem_bytes(d.dtype), n = (size_t)d.batch * d.length;
    const size_t qb = n * d.heads * d.dim * e, kb = n * d.kv_heads * d.dim * e;
    fno_status_t st = check_operands({{q, qb, false}, {k, kb, false}, {positions, n * 4, false},
                                      {offsets, (size_t)d.batch * 4, false}, {qo, qb, true, q},
                                      {ko, kb, true, k}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    Args a{q, k, qo, ko, positions, offsets, (int64_t)n, d.length, d.heads, d.kv_heads, d.dim,
           d.rotary_dim, 0, 0, p->magnitude, transpose != 0};
    Turns turns;
    std::memcpy(turns.v, p->turns, sizeof turns.v);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // the widest vectors (16 bytes at most) that the head and the pairs' sides divide into
    const int side = d.layout == FNO_ROTARY_HALF ? d.rotary_dim / 2 : d.rotary_dim;
    const auto fits = [&](int v) { return side % v == 0 && d.dim % v == 0; };
    return with_storage(d.dtype, [&](auto t) {
        using T = decltype(t);
        if constexpr (sizeof(T) == 2)
            if (fits(8)) return launch<T, 8>(*p, a, turns, s);
        if (fits(4)) return launch<T, 4>(*p, a, turns, s);
        if (fits(2)) return launch<T, 2>(*p, a, turns, s);
        return launch<T, 1>(*p, a, turns, s);
    });
}

fno_status_t fno_rotary_destroy(fno_rotary_t p) {
    delete p;
    return FNO_OK;
}

}  // extern "C"
