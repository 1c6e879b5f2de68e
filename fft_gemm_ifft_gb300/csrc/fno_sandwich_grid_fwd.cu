// fno_sandwich_grid_fwd.cu -- the sandwich norm's forward on channels-first
// fields, up to 512 channels.
#include "fno_sandwich.h"

using namespace fno;
using namespace fno::ops;
using namespace fno::sandwich;

namespace {

// ---------------------------------------------------------------------------
// Grid layout, up to 512 channels: a CTA holds a tile of 32 V points by every
// channel in registers, so that each field is read once.  Warp w takes the
// channels w, w + warps, ... (CPT of them at most), lane l the V consecutive
// points l V ...; a norm's sums go over a thread's channels in registers and
// over the warps through shared memory.  Bound by bytes: 60 us for 16 x 64 x 128^2
// float32 with the 8-bit checkpoint (302 MB, 5.0 TB/s; the kernel that reads each
// field for each sum 297 us); the rest is the two norms' barriers.
// ---------------------------------------------------------------------------

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

// TIGHT keeps to 80 registers, so that an SM holds more CTAs of up to 12 warps: 17 x
// 289 x 6560 fp16 314 us against 505, 79 x 64 x 6560 fp16 127 against 142.  With more
// warps only the spills are left (500 channels 390 us against 350), and the float32
// tiles of 4 points spill most (84 against 83).  Those of one point and 8 channels
// always keep to 64, for two CTAs of 16 warps (39 x 128 x 6557 fp16 221 us against 397).
constexpr int kTightWarps = 12;
template <typename T, int V, int CPT>
constexpr bool tight_pays = !(V == 4 && sizeof(T) == 4) && V * CPT > 8;

// Shared memory of a grid kernel: per channel (s w2, s b2, w1, b1), then the
// sums' rows, then the norms' results.
size_t grid_smem(int channels, int V, int warps) {
    return (size_t)channels * 16 + (size_t)(2 * warps + 4) * 32 * V * 4;
}

template <typename T, int V, int CPT, bool LAYER, bool TIGHT>
__global__ void __launch_bounds__(TIGHT ? kTightWarps * 32 : 512,
                                  TIGHT || V * CPT == 8 ? 2 : 1)
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

// Calls f with the storage type and the variant's constants.
template <class F>
void with_tiles(const fno_sandwich_s &p, const Way &way, F &&f) {
    with_storage(p.d.dtype, [&](auto t) {
        const auto layer = [&](auto v, auto per) {
            if (p.d.norm == FNO_NORM_LAYER) f(t, v, per, std::true_type());
            else f(t, v, per, std::false_type());
        };
        constexpr std::integral_constant<int, 1> one;
        constexpr std::integral_constant<int, 8> few;
        if (way.per == 8 && way.vec == 4) layer(std::integral_constant<int, 4>(), few);
        else if (way.per == 8 && way.vec == 2) layer(std::integral_constant<int, 2>(), few);
        else if (way.per == 8) layer(one, few);
        else if (way.vec == 1) layer(one, std::integral_constant<int, 32>());
        else layer(std::integral_constant<int, 2>(), std::integral_constant<int, 16>());
    });
}
}  // namespace

namespace fno {
namespace sandwich {

// Vectors need the point count (where every channel's row starts) to be a
// multiple of them; registers bound a thread's elements (32 of each field), and
// 16 warps a CTA's channels.  A launch has a CTA a tile: more tiles than a grid has
// room for (billions of samples of a few points) take the kernel for any size.
Way grid_forward_way(const fno_sandwich_desc_t &d) {
    const int c = d.channels;
    const auto tiles = [&](int vec, int per) {
        if (d.batch * ceil_div(d.points, 32 * vec) > 0x7fffffffll) return Way{kAny, 0, 0, 0, 0};
        return Way{kTiles, vec, per, (int)ceil_div(c, per), 0};
    };
    if (c <= 128 && d.points % 4 == 0) return tiles(4, 8);
    if (c <= 8 * kTightWarps && d.points % 2 == 0) return tiles(2, 8);
    if (c <= 128) return tiles(1, 8);
    if (c <= 256 && d.points % 2 == 0) return tiles(2, 16);
    if (c <= 512) return tiles(1, 32);
    return Way{kAny, 0, 0, 0, 0};
}

fno_status_t grid_forward(const fno_sandwich_s &p, const Args &a, int8_t *f8, float *f8_scale,
                          bool *packed, cudaStream_t s) {
    const Way &way = p.fwd;
    *packed = f8 && way.vec == 4;        // a warp's 128 points are one group
    int8_t *q = *packed ? f8 : nullptr;
    with_tiles(p, way, [&](auto t, auto v, auto per, auto layer) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value, CPT = decltype(per)::value;
        constexpr bool LAYER = decltype(layer)::value;
        const auto run = [&](auto kernel) {
            kernel<<<(unsigned)(p.d.batch * ceil_div(p.d.points, 32 * V)), way.warps * 32,
                     grid_smem(a.channels, V, way.warps), s>>>(a, q, f8_scale);
        };
        if constexpr (tight_pays<T, V, CPT>) {
            if (way.warps <= kTightWarps)
                return run(k_sandwich_fwd_grid<T, V, CPT, LAYER, true>);
        }
        run(k_sandwich_fwd_grid<T, V, CPT, LAYER, false>);
    });
    return launched();
}

}  // namespace sandwich
}  // namespace fno
