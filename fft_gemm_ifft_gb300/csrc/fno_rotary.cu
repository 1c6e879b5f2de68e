// fno_rotary.cu -- rotary positions: every pair of a head's first elements turned by an
// angle that grows with the token's position.
//
// The angle of pair i at position p is p f_i.  In float32 a far position would lose it
// (p = 10^6 leaves an error of 0.06 radians), so the plan keeps f_i as the turns a
// position takes in 64-bit fixed point: p times that, modulo 2^64, is the fraction of a
// turn, exactly, for any 32-bit p (a negative one too), and its upper 32 bits go to the
// sine and cosine.
//
// Bound by bytes: each element is read and written once.  A block works out the cosines and
// sines of its tokens' positions once, into shared memory, and then goes over all heads of
// these tokens, vector after vector as they lie in memory (4 x 8192 tokens, 20 heads of 128 in
// bfloat16: 58 us, 5.8 TB/s; 3 x 4097, 24 heads of 80 in float32: 30 us, 6.3 TB/s, where a
// thread for one vector of every head, with the sines in registers, takes 1.4 times as long).
// A vector is as wide as divides the head and the pairs' sides, so that sides of an odd count
// take one element a vector and twice an odd count two, which costs time (4 x 8192, 20 heads of
// 64 in bfloat16: 40 us a call with all 64 turned, 97 with 42; heads of 80: 53 with all turned,
// 73 with 52).
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

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

struct Turns {
    uint64_t v[kMaxPairs];
};
// i / d for i below 2^16, d at most 2^16, by a product: ceil(2^32 / d) is off by less than
// one, i times which stays below 2^32 / d.
struct Divisor {
    uint32_t d, m;
    explicit Divisor(int n) : d((uint32_t)n), m((uint32_t)((0x100000000ull + n - 1) / n)) {}
    __device__ uint32_t div(uint32_t i) const { return d == 1 ? i : __umulhi(i, m); }
};
struct Args {
    const void *q, *k;
    void *qo, *ko;
    const int32_t *positions, *offsets;
    int64_t rows, length;
    int heads, kv_heads, dim, rotary;
    int tokens;                // of a block
    Divisor units, token;      // vectors of a head; of all heads of a token
    float magnitude;
    bool transpose;
};

// Cosine and sine of x half turns, |x| <= 1.  For 16-bit types by the multi-function unit:
// off by 2^-20 at most, which their roundings (2^-11, 2^-8) hide.
template <typename T>
__device__ __forceinline__ void cos_sin(float x, float *c, float *s) {
    if constexpr (sizeof(T) == 4) sincospif(x, s, c);
    else __sincosf(3.14159265f * x, s, c);
}
// Two pairs (a, b) turned; two neighbouring elements as one pair.
template <typename T>
__device__ __forceinline__ Pair<T> from_float2(float2 v) {
    Pair<T> r;
    store_pair(reinterpret_cast<T *>(&r), v, true, 2);
    return r;
}
template <typename T>
__device__ __forceinline__ void turn2(Pair<T> &a, Pair<T> &b, float2 c, float2 s) {
    const float2 av = to_float2(a), bv = to_float2(b);
    const float2 bs = mul2(bv, s);
    a = from_float2<T>(fma2(av, c, make_float2(-bs.x, -bs.y)));
    b = from_float2<T>(fma2(bv, c, mul2(av, s)));
}
template <typename T>
__device__ __forceinline__ void turn1(T &a, T &b, float c, float s) {
    const float av = Storage<T>::load(&a), bv = Storage<T>::load(&b);
    Storage<T>::store(&a, fmaf(av, c, -(bv * s)));
    Storage<T>::store(&b, fmaf(bv, c, av * s));
}

// HALF: a vector of V elements of the first side turns with one of the second; interleaved:
// the pairs in a run of max(V, 2) elements.  The units beyond the pairs are V elements copied.
// V divides the rotary part's sides (half) or the rotary part, and the head.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads)
k_rotary(const Args p, const __grid_constant__ Turns turns) {
    constexpr int R = HALF || V > 1 ? V : 2, N = HALF ? V : R / 2;      // a run, its pairs
    constexpr int kUnroll = HALF ? 2 : 4;      // units of a thread whose loads are on their way
    extern __shared__ __align__(16) float table[];     // [tokens][2][pairs]: cosines, sines
    const int half = p.rotary / 2;
    const int turning = HALF ? half / V : p.rotary / R;                 // units that turn
    const int64_t row0 = (int64_t)blockIdx.x * p.tokens;
    const int tokens = (int)min((int64_t)p.tokens, p.rows - row0);
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int k = i / half, pair = i - k * half;
        const int64_t row = row0 + k;
        int64_t pos;
        if (p.positions) {
            pos = p.positions[row];
        } else {
            const int64_t b = p.rows <= 0xffffffffll
                                  ? (int64_t)((uint32_t)row / (uint32_t)p.length)
                                  : row / p.length;
            pos = row - b * p.length;
            if (p.offsets) pos += p.offsets[b];
        }
        const uint64_t turn = (uint64_t)pos * turns.v[pair];
        // the upper half as a signed number: -1/2 .. 1/2 of a turn
        const float x = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;    // 2^-31
        float s, c;
        cos_sin<T>(x, &c, &s);
        table[2 * k * half + pair] = p.magnitude * c;
        table[(2 * k + 1) * half + pair] = p.transpose ? -p.magnitude * s : p.magnitude * s;
    }
    __syncthreads();
    const bool copies = p.q != p.qo || p.k != p.ko;
    const uint32_t all = (uint32_t)tokens * p.token.d;
    for (uint32_t i0 = threadIdx.x; i0 < all; i0 += kThreads * kUnroll) {
        Pack<T, R> a[kUnroll];                         // (in R / V pieces)
        Pack<T, V> b[kUnroll];
        T *to[kUnroll];
        int unit[kUnroll], at_table[kUnroll];          // unit -1: nothing
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t i = i0 + u * kThreads;
            unit[u] = -1;
            if (i >= all) continue;
            const uint32_t k = p.token.div(i), rest = i - k * p.token.d;
            const uint32_t head = p.units.div(rest), n = rest - head * p.units.d;
            if ((int)n >= turning && !copies) continue;
            unit[u] = (int)n;
            const bool is_q = (int)head < p.heads;
            const int at = (int)n < turning ? n * R : p.rotary + (n - turning) * V;
            const int64_t o = (is_q ? ((row0 + k) * p.heads + head)
                                    : ((row0 + k) * p.kv_heads + (head - p.heads))) * p.dim + at;
            const T *from = static_cast<const T *>(is_q ? p.q : p.k) + o;
            to[u] = static_cast<T *>(is_q ? p.qo : p.ko) + o;
            at_table[u] = 2 * k * half + n * N;
#pragma unroll
            for (int j = 0; j < R / V; ++j)
                if (j == 0 || (int)n < turning)
                    *reinterpret_cast<Pack<T, V> *>(a[u].v + j * V) =
                        *reinterpret_cast<const Pack<T, V> *>(from + j * V);
            if (HALF && (int)n < turning) b[u] = *reinterpret_cast<const Pack<T, V> *>(from + half);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (unit[u] < 0) continue;
            if (unit[u] < turning) {
                const float *at = table + at_table[u];
                const Pack<float, N> c = *reinterpret_cast<const Pack<float, N> *>(at);
                const Pack<float, N> s = *reinterpret_cast<const Pack<float, N> *>(at + half);
                T *e = a[u].v;
                if constexpr (HALF && V > 1) {
                    Pair<T> *first = reinterpret_cast<Pair<T> *>(e);
                    Pair<T> *second = reinterpret_cast<Pair<T> *>(b[u].v);
#pragma unroll
                    for (int j = 0; j < V / 2; ++j)
                        turn2(first[j], second[j], make_float2(c.v[2 * j], c.v[2 * j + 1]),
                              make_float2(s.v[2 * j], s.v[2 * j + 1]));
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        turn1(HALF ? e[j] : e[2 * j], HALF ? b[u].v[j] : e[2 * j + 1], c.v[j],
                              s.v[j]);
                }
                if (HALF) *reinterpret_cast<Pack<T, V> *>(to[u] + half) = b[u];
            }
#pragma unroll
            for (int j = 0; j < R / V; ++j)
                if (j == 0 || unit[u] < turning)
                    *reinterpret_cast<Pack<T, V> *>(to[u] + j * V) =
                        *reinterpret_cast<const Pack<T, V> *>(a[u].v + j * V);
        }
    }
}

template <typename T, int V>
fno_status_t launch(const fno_rotary_s &plan, Args a, const Turns &turns, cudaStream_t s) {
    const bool half = plan.d.layout == FNO_ROTARY_HALF;
    const int turning = half ? a.rotary / 2 / V : a.rotary / (V > 1 ? V : 2);
    a.units = Divisor(turning + (a.dim - a.rotary) / V);
    a.token = Divisor((int)a.units.d * (a.heads + a.kv_heads));
    // up to 2048 vectors and 32 tokens a block, fewer while there are less than four blocks, half
    // of the threads that it holds, for every SM
    a.tokens = 32;
    while (a.tokens > 1 && (a.tokens * (int64_t)a.token.d > 2048 ||
                            ceil_div(a.rows, a.tokens) < 4 * plan.sms))
        a.tokens /= 2;
    const int64_t blocks = ceil_div(a.rows, a.tokens);
    if (blocks > 2147483647) return FNO_ERR_UNSUPPORTED;
    const size_t bytes = (size_t)a.tokens * a.rotary * 4;
    if (half) k_rotary<T, V, true><<<(unsigned)blocks, kThreads, bytes, s>>>(a, turns);
    else k_rotary<T, V, false><<<(unsigned)blocks, kThreads, bytes, s>>>(a, turns);
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
    const double r = d.rotary_dim;
    double base = d.base;
    if (d.scaling == FNO_ROTARY_BASE) {
        if (d.rotary_dim == 2) return FNO_ERR_INVALID_ARG;
        base *= std::pow(d.factor, r / (r - 2.0));
        if (!std::isfinite(base)) return FNO_ERR_INVALID_ARG;
    }
    if (d.scaling == FNO_ROTARY_RAMP &&
        !(d.original > 0.0 && std::isfinite(d.original) && d.slow >= 0.0 && d.fast > d.slow &&
          std::isfinite(d.fast)))
        return FNO_ERR_INVALID_ARG;
    if (d.dim > 1024 || d.rotary_dim > 2 * kMaxPairs ||
        ((double)d.heads + d.kv_heads) * d.dim > 65536.0 ||
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
    const double pi = 3.14159265358979323846;
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
           d.rotary_dim, 1, Divisor(1), Divisor(1), p->magnitude, transpose != 0};
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
