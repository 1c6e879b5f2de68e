// fno_sandwich_rows.cu -- the sandwich norm on token rows, forward up to 8192
// channels and backward up to 4096.
#include "fno_sandwich.h"

using namespace fno;
using namespace fno::ops;
using namespace fno::sandwich;

namespace {

constexpr int kMaxWarps = 16;

// ---------------------------------------------------------------------------
// Token layout: a row lies in registers, with G whole warps or (SMALL) with 2^k
// lanes of one; each thread holds J runs of V consecutive channels.
// ---------------------------------------------------------------------------
template <bool SMALL>
struct Team {
    int lanes, warps;        // of a row
    int row, rows;           // this thread's among the CTA's
    int member;              // this thread's place in its row
    int first, slot;         // the row's and this warp's entries of a buffer of sums
    __device__ __forceinline__ Team(int G, int L) {
        const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
        lanes = SMALL ? L : 32;
        warps = SMALL ? 1 : G;
        row = SMALL ? (int)threadIdx.x / L : w / G;
        rows = SMALL ? (int)blockDim.x / L : (int)(blockDim.x >> 5) / G;
        member = SMALL ? lane & (L - 1) : w % G * 32 + lane;
        first = w / G * (G > 2 ? (G + 3) & ~3 : G);
        slot = first + w % G;
    }
    // the entries behind a row's last, for its sums' vector reads
    template <int N> __device__ __forceinline__ void clear(float (*buf)[kMaxWarps]) const {
        if constexpr (!SMALL)
            if (warps > 2 && member == 32 * warps - 1)
                for (int i = slot + 1; i & 3; ++i)
                    for (int k = 0; k < N; ++k) buf[k][i] = 0.0f;
    }
};

// The sums of N values over a row.  `buf` ([N][kMaxWarps]) is this sum's own: a
// buffer may be used again once another sum came in between, whose barrier every
// reader of this one has passed.
template <int N, bool SMALL>
__device__ __forceinline__ void row_sum(float (&v)[N], const Team<SMALL> &team,
                                        float (*buf)[kMaxWarps]) {
#pragma unroll
    for (int m = 16; m; m >>= 1)
        if (!SMALL || m < team.lanes)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
    if (SMALL || team.warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) buf[k][team.slot] = v[k];
    __syncthreads();
    if (team.warps == 2) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float2 x = *reinterpret_cast<const float2 *>(&buf[k][team.first]);
            v[k] = x.x + x.y;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = 0.0f;
    for (int i = 0; i < team.warps; i += 4)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(&buf[k][team.first + i]);
            v[k] += (x.x + x.y) + (x.z + x.w);
        }
}

// mean and r of a row whose values less the shift are x[.]; entries beyond the
// row's channels are excluded by `have`.
template <int N, bool LAYER, bool SMALL, class Have>
__device__ __forceinline__ void row_norm(const float (&x)[N], Have &&have, int channels, float eps,
                                         const Team<SMALL> &team, float (*red)[1][kMaxWarps],
                                         float &mean, float &r) {
    const float inv = 1.0f / (float)channels;
    mean = 0.0f;
    if (LAYER) {
        float s[1] = {};
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += x[i];          // absent entries are 0
        row_sum<1, SMALL>(s, team, red[0]);
        mean = s[0] * inv;
    }
    float q[1] = {};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = have(i) ? x[i] - mean : 0.0f;
        q[0] = fmaf(d, d, q[0]);
    }
    row_sum<1, SMALL>(q, team, red[1]);
    r = rsqrtf(fmaf(q[0], inv, eps));
}

template <typename T, int V, int J, bool LAYER, bool SMALL>
// (80 registers, three CTAs of 8 warps an SM: 3 x 10922 x 1024 fp16 with a sigmoid gate
// an element 123 us, with as many as it takes 159)
__global__ void __maxnreg__(80)
k_sandwich_fwd_rows(Args a, int G, int L, int8_t *f8, float *f8_scale) {
    constexpr int N = V * J;
    __shared__ alignas(16) float red[4][1][kMaxWarps];
    const Team<SMALL> team(G, L);
#pragma unroll
    for (int k = 0; k < 4; ++k) team.clear<1>(red[k]);
    const int lane = threadIdx.x & 31;
    const int64_t rows = a.batch * a.points;
    const int64_t row = (int64_t)blockIdx.x * team.rows + team.row;
    const bool on = row < rows;
    const int c0 = team.member * V, cs = (SMALL ? L : G * 32) * V;                // run j at c0 + j cs
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
            // a group is 128 / V lanes' runs, which are the row's lanes or fewer
            // (for V <= 2 the caller packs by itself)
            constexpr int S = V > 2 ? kGroup / V : 32;
            const uint32_t mask = S == 32 ? 0xffffffffu : 0xffffu << (lane & 16);
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
                    if (lane % S == 0)
                        f8_scale[row * ((a.channels + kGroup - 1) / kGroup) + c / kGroup] = s.scale;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = have(i) ? Storage<T>::load(&fs[i / V].v[i % V]) - shift : 0.0f;
        row_norm<N, LAYER, SMALL>(v, have, a.channels, a.eps, team, red, mean, r);
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
        float shift = __shfl_sync(0xffffffffu, v[0], SMALL ? lane & -L : 0);
        if (!SMALL && G > 1) {
            if (team.member == 0) first[team.row] = shift;
            __syncthreads();
            shift = first[team.row];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = have(i) ? v[i] - shift : 0.0f;
    }
    row_norm<N, LAYER, SMALL>(v, have, a.channels, a.eps, team, red + 2, mean, r);
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

// The pair of elements 2 k, 2 k + 1 of a thread's runs.
template <typename T, int V, int J>
__device__ __forceinline__ float2 pair_of(const Pack<T, V> (&x)[J], int k) {
    return make_float2(Storage<T>::load(&x[2 * k / V].v[2 * k % V]),
                       Storage<T>::load(&x[(2 * k + 1) / V].v[(2 * k + 1) % V]));
}
template <int V, int J>
__device__ __forceinline__ float2 pair_of(const Pack<int8_t, V> (&x)[J], const float (&scale)[J],
                                          int k) {
    return make_float2((float)x[2 * k / V].v[2 * k % V] * scale[2 * k / V],
                       (float)x[(2 * k + 1) / V].v[(2 * k + 1) % V] * scale[(2 * k + 1) / V]);
}
template <typename T, int V, int J>
__device__ __forceinline__ void set_pair(Pack<T, V> (&x)[J], int k, float2 v) {
    Storage<T>::store(&x[2 * k / V].v[2 * k % V], v.x);
    Storage<T>::store(&x[(2 * k + 1) / V].v[(2 * k + 1) % V], v.y);
}

// Backward: G warps walk the rows of a share, and keep their channels' sums in
// registers.  The arithmetic is on pairs of elements (f32x2).  3 x 4099 x 1024 fp16
// with a sigmoid gate an element (201 MB): 72 us, of which the three rounds of
// row sums with their barriers are a third; 106 us with six rounds and the row's
// loads at its start, 593 us reading each field for each sum.  A row in the lanes that
// it needs: 3 x 174762 x 64 fp16 131 us, with a warp to a row 484.
template <typename T, int V, int J, bool LAYER, bool F8, bool SMALL>
__global__ void __launch_bounds__(512)
k_sandwich_bwd_rows(Args a, int G, int L) {
    constexpr int N = V * J, H = N / 2;
    using TF = typename std::conditional<F8, int8_t, T>::type;
    // three rounds of sums a row: the means; the squared deviations, sum d and
    // sum d N; sum e and sum e M
    __shared__ alignas(16) float red1[2][kMaxWarps], red2[4][kMaxWarps], red3[2][kMaxWarps];
    extern __shared__ float4 sm[];
    const Team<SMALL> team(G, L);
    team.clear<2>(red1);
    team.clear<4>(red2);
    team.clear<2>(red3);
    const int R = team.rows, c0 = team.member * V, cs = (SMALL ? L : G * 32) * V;
    const bool block = F8 || a.f != nullptr, full = block && a.gate_kind == FNO_GATE_FULL;
    const bool has_du = a.du != nullptr, has_dy = a.dy != nullptr;
    const float inv = 1.0f / (float)a.channels;
    const int64_t groups = (a.channels + kGroup - 1) / kGroup;
    bool have[J];
    float one[J];                // 1 for a run within the row, else 0
#pragma unroll
    for (int j = 0; j < J; ++j) {
        have[j] = c0 + j * cs < a.channels;
        one[j] = have[j] ? 1.0f : 0.0f;
    }
    const auto ones = [&](int k) { return make_float2(one[2 * k / V], one[(2 * k + 1) / V]); };
    float2 acc[kSums][H] = {};
    // The next row's vectors are on their way over the work on this one: each
    // thread copies its own into its own slots of shared memory (two rows' worth),
    // which takes no registers and no barrier.  (Pairs of
    // fp16 so, 3 x 21592 x 518: 391 us, loaded when they are needed 611; but single
    // float32, 3 x 21760 x 257: 297 us, loaded 243.)
    constexpr int kPiece = V * (int)sizeof(T);
    constexpr bool AHEAD = V > 1 && (!F8 || V >= 4);
    constexpr int kFields = F8 ? 4 : 5;                    // y, du, dy, gate, (f)
    char *slots = reinterpret_cast<char *>(sm) + (size_t)(R > 1 ? R : 0) * a.channels * 4 +
                  threadIdx.x * kPiece;
    const int slot = blockDim.x * kPiece, stage = (kFields * J + (F8 ? 1 : 0)) * slot;
    const int64_t hop = (int64_t)gridDim.x * R;
    // the next row's channel 0, as stored (a conversion would wait for the load)
    T next1 = T(0.0f);
    TF next2 = TF(0);
    float next_scale = 0.0f;
    const auto ahead = [&](int64_t t, int k) {
        const int64_t row = blockIdx.y * a.seg_points + t + team.row, base = row * a.channels + c0;
        if (t + team.row < a.seg_points) {
            char *at = slots + k * stage;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!have[j]) continue;
                const int64_t e = base + j * cs;
                const auto fetch = [&](int f, const void *src) {
                    const uint32_t to = smem_u32(at + (f * J + j) * slot);
                    const T *from = static_cast<const T *>(src) + e;
                    if constexpr (kPiece == 16) cp_async16(to, from);
                    else if constexpr (kPiece == 8) cp_async8(to, from);
                    else cp_async4(to, from);
                };
                if (has_du) {
                    fetch(0, a.x);
                    fetch(1, a.du);
                }
                if (has_dy) fetch(2, a.dy);
                if (full) fetch(3, a.gate);
                if (F8) {
                    // codes at the front of the slots of J runs, their scales behind
                    const uint32_t to = smem_u32(at + kFields * J * slot + j * 8);
                    if (V == 8) cp_async8(to, a.f8 + e);
                    else cp_async4(to, a.f8 + e);
                } else if (block) {
                    fetch(4, a.f);
                }
            }
            if (LAYER) {
                if (has_du) next1 = static_cast<const T *>(a.x)[base - c0];
                if (F8) {
                    next2 = static_cast<const TF *>(static_cast<const void *>(a.f8))[base - c0];
                    next_scale = a.f8_scale[row * groups];
                } else if (block) {
                    next2 = static_cast<const TF *>(a.f)[base - c0];
                }
            }
        }
        cp_async_commit();
    };
    int k = 0;
    if (AHEAD) ahead((int64_t)blockIdx.x * R, 0);
    for (int64_t t = (int64_t)blockIdx.x * R; t < a.seg_points; t += hop, k ^= 1) {
        const bool on = t + team.row < a.seg_points;
        const int64_t row = blockIdx.y * a.seg_points + t + team.row, base = row * a.channels + c0;
        Pack<T, V> ys[J] = {}, us[J] = {}, gs[J] = {}, gates[J] = {}, out[J], out2[J];
        Pack<TF, V> fs[J] = {};
        float fsc[J] = {};
        float mean[2] = {}, q[4] = {}, shift1 = 0.0f, shift2 = 0.0f;
        if (AHEAD) {
            if (LAYER) {
                shift1 = Storage<T>::load(&next1);
                if constexpr (F8) shift2 = (float)next2 * next_scale;
                else shift2 = Storage<T>::load(&next2);
            }
            if (F8)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (on && have[j]) fsc[j] = a.f8_scale[row * groups + (c0 + j * cs) / kGroup];
            ahead(t + hop, k ^ 1);
            cp_async_wait<1>();
            const char *at = slots + k * stage;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!on || !have[j]) continue;
                const auto get = [&](int f) {
                    return *reinterpret_cast<const Pack<T, V> *>(at + (f * J + j) * slot);
                };
                if (has_du) {
                    ys[j] = get(0);
                    us[j] = get(1);
                }
                if (has_dy) gs[j] = get(2);
                if (full) gates[j] = get(3);
                if constexpr (F8)
                    fs[j] = *reinterpret_cast<const Pack<TF, V> *>(at + kFields * J * slot + j * 8);
                else if (block)
                    fs[j] = get(4);
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (AHEAD || !on || !have[j]) continue;
            const int64_t e = base + j * cs;
            if (has_du) {
                ys[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.x) + e);
                us[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.du) + e);
            }
            if (has_dy)
                gs[j] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.dy) + e);
            if (F8) {
                fs[j] = *reinterpret_cast<const Pack<TF, V> *>(a.f8 + e);
                fsc[j] = a.f8_scale[row * groups + (c0 + j * cs) / kGroup];
            } else if (block) {
                fs[j] = *reinterpret_cast<const Pack<TF, V> *>(static_cast<const TF *>(a.f) + e);
            }
            if (full)
                gates[j] =
                    *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.gate) + e);
        }
        if (!on) shift1 = shift2 = 0.0f;
        if (!AHEAD && LAYER && on) {
            if (has_du) shift1 = Storage<T>::load(static_cast<const T *>(a.x) + base - c0);
            if constexpr (F8) {
                shift2 = (float)a.f8[base - c0] * a.f8_scale[row * groups];
            } else {
                if (block) shift2 = Storage<T>::load(static_cast<const T *>(a.f) + base - c0);
            }
        }
        float2 n[H], m[H], dY[H];
        {
            float2 s1 = f2(0.0f), s2 = s1;
#pragma unroll
            for (int k = 0; k < H; ++k) {
                n[k] = pair_of<T, V, J>(ys, k);
                if constexpr (F8) m[k] = pair_of<V, J>(fs, fsc, k);
                else m[k] = pair_of<T, V, J>(fs, k);
                if (LAYER) {
                    n[k] = fma2(ones(k), f2(-shift1), n[k]);
                    m[k] = fma2(ones(k), f2(-shift2), m[k]);
                    s1 = add2(s1, n[k]);
                    s2 = add2(s2, m[k]);
                }
            }
            mean[0] = s1.x + s1.y;
            mean[1] = s2.x + s2.y;
        }
        if (LAYER) {
            row_sum<2, SMALL>(mean, team, red1);
            mean[0] *= -inv;
            mean[1] *= -inv;
        }
        // q: sum (y - mean)^2, sum (f - mean)^2, sum d, sum d (y - mean)
        {
            Pack<float, V> w1[J] = {};
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (has_du && have[j])
                    w1[j] = *reinterpret_cast<const Pack<float, V> *>(a.w1 + c0 + j * cs);
            float2 q0 = f2(0.0f), q1 = q0, q2 = q0, q3 = q0;
#pragma unroll
            for (int k = 0; k < H; ++k) {
                if (LAYER) {
                    n[k] = fma2(ones(k), f2(mean[0]), n[k]);
                    m[k] = fma2(ones(k), f2(mean[1]), m[k]);
                }
                const float2 u = pair_of<T, V, J>(us, k), wk = pair_of<float, V, J>(w1, k);
                dY[k] = make_float2(weighted(u.x, wk.x), weighted(u.y, wk.y));
                q0 = fma2(n[k], n[k], q0);
                q1 = fma2(m[k], m[k], q1);
                q2 = add2(q2, dY[k]);
                q3 = fma2(dY[k], n[k], q3);
            }
            q[0] = q0.x + q0.y;
            q[1] = q1.x + q1.y;
            q[2] = q2.x + q2.y;
            q[3] = q3.x + q3.y;
        }
        row_sum<4, SMALL>(q, team, red2);
        const float r1 = on && has_du ? rsqrtf(fmaf(q[0], inv, a.eps)) : 0.0f;
        const float r2 = on ? rsqrtf(fmaf(q[1], inv, a.eps)) : 0.0f;
        const float2 d0 = f2(LAYER ? -q[2] * inv : 0.0f), d1 = f2(-q[3] * r1 * inv);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            float2 g = pair_of<T, V, J>(gs, k);
            if (has_du) {
                const float2 u = pair_of<T, V, J>(us, k);
                n[k] = mul2(n[k], f2(r1));
                acc[2][k] = fma2(u, n[k], acc[2][k]);
                if (LAYER) acc[3][k] = add2(acc[3][k], u);
                const float2 d = LAYER ? add2(dY[k], d0) : dY[k];
                g = fma2(fma2(n[k], d1, d), f2(r1), g);
            }
            set_pair<T, V, J>(out, k, g);
            dY[k] = mul2(g, ones(k));
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (on && have[j])
                *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.dx) + base + j * cs) = out[j];
        if (!block) {
            // red2 is the only sum of such a row without the means' own: every warp of
            // the row has read it before the next row's is written
            if (!LAYER && !SMALL && team.warps > 1) __syncthreads();
            continue;
        }
        // dY becomes e
        Pack<float, V> s[J] = {}, w2[J] = {}, b2[J] = {}, gf[J] = {};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = c0 + j * cs;
            if (!have[j]) continue;
            s[j] = *reinterpret_cast<const Pack<float, V> *>(a.s + c);
            w2[j] = *reinterpret_cast<const Pack<float, V> *>(a.w2 + c);
            if (LAYER && full) b2[j] = *reinterpret_cast<const Pack<float, V> *>(a.b2 + c);
            if (a.gate_kind == FNO_GATE_CHANNEL)
                gf[j] = *reinterpret_cast<const Pack<float, V> *>(
                    static_cast<const float *>(a.gate) + blockIdx.y * a.channels + c);
        }
        float2 e0 = f2(0.0f), e1 = e0;
#pragma unroll
        for (int k = 0; k < H; ++k) {
            m[k] = mul2(m[k], f2(r2));
            const float2 w2k = pair_of<float, V, J>(w2, k);
            float2 ts = mul2(dY[k], pair_of<float, V, J>(s, k));
            if (full) {
                const float2 gate = pair_of<T, V, J>(gates, k);
                const float2 av = make_float2(gate_value(gate.x, a.sigmoid),
                                              gate_value(gate.y, a.sigmoid));
                const float2 slope = make_float2(gate_slope(av.x, a.sigmoid),
                                                 gate_slope(av.y, a.sigmoid));
                const float2 z = LAYER ? fma2(m[k], w2k, pair_of<float, V, J>(b2, k))
                                       : mul2(m[k], w2k);
                set_pair<T, V, J>(out2, k, mul2(mul2(ts, z), slope));
                ts = mul2(ts, av);
                dY[k] = mul2(dY[k], av);
            } else if (a.gate_kind == FNO_GATE_CHANNEL) {
                const float2 gate = pair_of<float, V, J>(gf, k);
                ts = mul2(ts, make_float2(gate_value(gate.x, a.sigmoid),
                                          gate_value(gate.y, a.sigmoid)));
            }
            acc[0][k] = fma2(dY[k], m[k], acc[0][k]);
            if (LAYER) acc[1][k] = add2(acc[1][k], dY[k]);
            dY[k] = make_float2(weighted(ts.x, w2k.x), weighted(ts.y, w2k.y));
            e0 = add2(e0, dY[k]);
            e1 = fma2(dY[k], m[k], e1);
        }
        float e[2] = {e0.x + e0.y, e1.x + e1.y};
        row_sum<2, SMALL>(e, team, red3);
        e0 = f2(LAYER ? -e[0] * inv : 0.0f);
        e1 = f2(-e[1] * inv);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            const float2 d = LAYER ? add2(dY[k], e0) : dY[k];
            set_pair<T, V, J>(out, k, mul2(fma2(m[k], e1, d), f2(r2)));
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!on || !have[j]) continue;
            *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.df) + base + j * cs) = out[j];
            if (a.dgate)
                *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.dgate) + base + j * cs) =
                    out2[j];
        }
    }
    // the CTA's rows joined in order, one of the four sums at a time
    float *join = reinterpret_cast<float *>(sm);        // [R][channels]
    float *part = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kSums * a.channels;
#pragma unroll
    for (int q = 0; q < kSums; ++q) {
        float *to = R > 1 ? join + team.row * a.channels : part + q * a.channels;
        if (R > 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (have[i / V]) to[c0 + i / V * cs + i % V] = i % 2 ? acc[q][i / 2].y : acc[q][i / 2].x;
        if (R > 1) {
            __syncthreads();
            for (int c = threadIdx.x; c < a.channels; c += blockDim.x) {
                float v = 0.0f;
                for (int k = 0; k < R; ++k) v += join[k * a.channels + c];
                part[q * a.channels + c] = v;
            }
        }
    }
}

// Calls f with the storage type, the variant's constants, and whether a row has
// less than a warp.
template <int EACH, class F>
void with_rows(const fno_sandwich_s &p, const Way &way, F &&f) {
    using std::integral_constant;
    with_storage(p.d.dtype, [&](auto t) {
        const auto rows = [&](auto v, auto j) {
            with_bools(p.d.norm == FNO_NORM_LAYER, way.lanes < 32,
                       [&](auto layer, auto small) { f(t, v, j, layer, small); });
        };
        constexpr int V = kVec<decltype(t)>;
        if (way.vec > 2) rows(integral_constant<int, V>(), integral_constant<int, EACH / V>());
        else if (way.vec == 2) rows(integral_constant<int, 2>(), integral_constant<int, EACH / 2>());
        else rows(integral_constant<int, 1>(), integral_constant<int, EACH>());
    });
}

// Calls f with the backward kernel.
template <class F>
void with_kernel(const fno_sandwich_s &p, bool f8, F &&f) {
    with_rows<8>(p, p.bwd, [&](auto t, auto v, auto j, auto layer, auto small) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value, J = decltype(j)::value;
        constexpr bool LAYER = decltype(layer)::value, SMALL = decltype(small)::value;
        if (f8) f(k_sandwich_bwd_rows<T, V, J, LAYER, true, SMALL>);
        else f(k_sandwich_bwd_rows<T, V, J, LAYER, false, SMALL>);
    });
}
int rows_of(const Way &way) { return way.warps / way.group * (32 / way.lanes); }

// the rows' sums joined in shared memory, and two rows' pieces (as many as the
// float32 codes' case takes: y, du, dy, gate, f)
size_t smem_of(const fno_sandwich_s &p) {
    const int rows = rows_of(p.bwd);
    const size_t join = rows > 1 ? (size_t)rows * p.d.channels * 4 : 0;
    const size_t piece = p.bwd.vec * elem_bytes(p.d.dtype);
    return join + (p.bwd.vec > 1 ? 2 * 5 * piece * p.bwd.per * p.bwd.warps * 32 : 0);
}

}  // namespace

namespace fno {
namespace sandwich {

// Vectors need the channel count (where every row starts) to be a multiple of
// them; registers bound a thread's elements (16 forward, 8 backward), and 16
// warps a row.  A row has the fewest lanes that hold it, or warps if it is longer,
// so that few lie beyond its end.
Way rows_way(const fno_sandwich_desc_t &d, bool backward) {
    const int c = d.channels, big = d.dtype == FNO_F32 ? 4 : 8;
    const int vec = c % big == 0 ? big : c % 2 == 0 ? 2 : 1, each = backward ? 8 : 16;
    const int group = (int)ceil_div(c, 32 * each);
    if (group > kMaxWarps) return Way{kAny, 0, 0, 0, 0};
    int lanes = 32;
    while (group == 1 && lanes > 1 && lanes / 2 * each >= c) lanes /= 2;
    return Way{kRows, vec, each / vec, group * (group < 8 ? 8 / group : 1), group, lanes};
}

fno_status_t rows_forward(const fno_sandwich_s &p, const Args &a, int8_t *f8, float *f8_scale,
                          bool *packed, cudaStream_t s) {
    Way way = p.fwd;
    *packed = f8 && way.vec > 2;         // a group lies within a warp's loads
    int8_t *q = *packed ? f8 : nullptr;
    if (q && way.lanes < kGroup / way.vec) way.lanes = kGroup / way.vec;
    with_rows<16>(p, way, [&](auto t, auto v, auto j, auto layer, auto small) {
        k_sandwich_fwd_rows<decltype(t), decltype(v)::value, decltype(j)::value,
                            decltype(layer)::value, decltype(small)::value>
            <<<(unsigned)ceil_div(p.d.batch * p.d.points, rows_of(way)), way.warps * 32,
               0, s>>>(a, way.group, way.lanes, q, f8_scale);
    });
    return launched();
}

fno_status_t rows_shares(const fno_sandwich_s &p, int *ctas, int64_t *most) {
    *most = ceil_div(p.seg_points, rows_of(p.bwd));
    fno_status_t st = FNO_OK;
    with_kernel(p, false,
                [&](auto k) { st = occupancy(k, p.bwd.warps * 32, smem_of(p), ctas); });
    return st;
}

fno_status_t rows_backward(const fno_sandwich_s &p, const Args &a, cudaStream_t s) {
    fno_status_t st = FNO_OK;
    with_kernel(p, a.f8 != nullptr, [&](auto k) {
        if (raise_smem_limit(k, smem_of(p)) != cudaSuccess) {
            st = FNO_ERR_CUDA;
            return;
        }
        k<<<dim3((unsigned)p.splits, (unsigned)p.segs), p.bwd.warps * 32, smem_of(p), s>>>(
            a, p.bwd.group, p.bwd.lanes);
        st = launched();
    });
    return st;
}

}  // namespace sandwich
}  // namespace fno
