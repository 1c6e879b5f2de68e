// fno_sandwich_grid_bwd.h -- the sandwich norm's backward on channels-first
// fields, up to kWideC channels: the kernels, instantiated for one storage type
// in each of three translation units.
#pragma once

#include "fno_sandwich.h"

namespace fno {
namespace sandwich {

using namespace ops;

template <typename T> fno_status_t grid_backward_of(const fno_sandwich_s &p, const Args &a,
                                                    cudaStream_t s);
template <typename T> fno_status_t grid_shares_of(const fno_sandwich_s &p, int *ctas);


// ---------------------------------------------------------------------------
// Backward on tiles of 64 points by every channel.  The fields' tiles come to shared memory asynchronously, the next
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
//
// Measured for 32 x 64 x 256^2 bfloat16 from the 8-bit checkpoint (1.48 GB): 470 us,
// 3.2 TB/s (float32 5.0 TB/s); with the checks of ragged tiles 784 us, with the
// fields held in registers and six rounds of sums 1892 us, reading each field for
// each sum 4225 us.  1400 warp instructions a tile and warp are what is left
// over the bytes.
// ---------------------------------------------------------------------------
constexpr int kTileP = 64, kTileC = 8;
constexpr int kSmemPerSm = 228 * 1024;

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

// Joins the warps' rows of round 1 for one point of a tile of `pt` (norm 1, or
// `second`) and leaves what the tile needs of it: the shift, -mean r, r, and for
// norm 1 also -mean(d) [LayerNorm] and -mean(d N).  Rows: y0, S1, S2, sum d,
// sum d (y - y0), f0, S1, S2, each [warps][pt].
template <bool LAYER>
__device__ __forceinline__ void join_moments(const float *rows, float *fin, int q, bool second,
                                             int pt, int warps, int C, float eps) {
    const int line = warps * pt;
    const float *r = rows + q + (second ? 5 * line : 0);
    const int base = C / warps, more = C - base * warps;       // warps with a channel more
    const float inv = 1.0f / (float)C;
    float ref = 0.0f, mean = 0.0f, ss = 0.0f, e0 = 0.0f, e1 = 0.0f;
    if (LAYER) {
        ref = r[0];
#pragma unroll 4
        for (int v = 0; v < warps; ++v) {
            const float nv = (float)(base + (v < more));
            mean += nv > 0.0f ? fmaf(nv, r[v * pt] - ref, r[line + v * pt]) : 0.0f;
        }
        mean *= inv;
    }
#pragma unroll 4
    for (int v = 0; v < warps; ++v) {
        ss += r[2 * line + v * pt];
        float off = 0.0f;
        if (LAYER) {
            const float nv = (float)(base + (v < more)), s1 = r[line + v * pt];
            off = r[v * pt] - ref;
            const float m = nv > 0.0f ? __fdividef(s1, nv) : 0.0f, d = off + m - mean;
            ss += nv > 0.0f ? nv * d * d - m * s1 : 0.0f;
        }
        if (!second) {
            e0 += r[3 * line + v * pt];
            e1 += fmaf(off, r[3 * line + v * pt], r[4 * line + v * pt]);
        }
    }
    // (a NaN stays one; fmaxf would make it 0)
    const float rr = rsqrtf(fmaf(ss < 0.0f ? 0.0f : ss, inv, eps));
    float *o = fin + q + (second ? 5 * pt : 0);
    o[0] = ref;
    o[pt] = -mean * rr;
    o[2 * pt] = rr;
    if (!second) {
        o[3 * pt] = LAYER ? -e0 * inv : 0.0f;
        o[4 * pt] = -rr * (e1 - mean * e0) * inv;
    }
}

__device__ __forceinline__ void st_shared8(uint32_t at, unsigned char v) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"((uint32_t)v) : "memory");
}

// A field's row of a tile takes points x elem bytes in a stage.  Rows that do not
// start on 4 bytes come as the aligned words that hold them, one word more, and
// keep their offset in the first word.  The others come in the widest pieces on
// which every row starts: 17 x 289 x 6558 fp16 708 us, by words a warp a row 1885.
__host__ __device__ inline bool row_shifted(int64_t points, int elem) {
    return points * elem % 4 != 0;
}
__host__ __device__ inline int row_pitch(int64_t points, int tile, int elem) {
    return tile * elem + (row_shifted(points, elem) ? 4 : 0);
}
// bytes of a stage (the fields' tiles and the codes' scales) and of the rest
__host__ __device__ inline int tile_stage(int channels, int64_t points, int tile, int elem, bool f8,
                                          bool du, bool dy, bool block, bool full) {
    const int field = channels * row_pitch(points, tile, elem);
    const int codes = channels * row_pitch(points, tile, 1);
    return (field * ((du ? 2 : 0) + dy + full + (block && !f8)) + (f8 ? codes + channels * 4 : 0) +
            15) / 16 * 16;
}
__host__ __device__ inline int tile_rest(int channels, int warps) {
    return channels * 16 + 8 * warps * kTileP * 4 + 8 * kTileP * 4;
}

// S parts of a warp work as warps of their own, on tiles of 64 / S points: 128 S
// channels at most.
template <typename T, bool LAYER, bool F8, bool WHOLE, int S>
__global__ void __launch_bounds__(512)
k_sandwich_bwd_tile(Args a, int stages) {
    constexpr int TP = kTileP / S, TL = 32 / S;
    extern __shared__ float4 sm[];
    const int lane = threadIdx.x % TL, w = threadIdx.x / TL, warps = blockDim.x / TL;
    const int C = a.channels, mine = WHOLE ? kTileC : (C - w + warps - 1) / warps;
    const bool block = F8 || WHOLE || a.f != nullptr;
    const bool full = !WHOLE && block && a.gate_kind == FNO_GATE_FULL;
    const bool has_du = WHOLE || a.du != nullptr, has_dy = WHOLE || a.dy != nullptr;
    float4 *par = sm;            // s a w2, s a, s b2, w1 (a of a gate per channel, else 1)
    float *rows = reinterpret_cast<float *>(sm + C);
    float *fin = rows + 8 * warps * TP;
    char *buf = reinterpret_cast<char *>(fin + 8 * TP);
    const int stage = tile_stage(C, a.points, TP, sizeof(T), F8, has_du, has_dy, block, full);
    // rows and offsets of the fields in a stage
    const bool odd = !WHOLE && row_shifted(a.points, sizeof(T));
    const bool odd8 = !WHOLE && row_shifted(a.points, 1);
    const int pitch = WHOLE ? TP * (int)sizeof(T) : row_pitch(a.points, TP, sizeof(T));
    const int pitch8 = WHOLE ? TP : row_pitch(a.points, TP, 1);
    const int oy = 0, ou = oy + (has_du ? C * pitch : 0), og = ou + (has_du ? C * pitch : 0),
              oa = og + (has_dy ? C * pitch : 0), of = oa + (full ? C * pitch : 0),
              os = of + C * pitch8;
    const int64_t tiles = (a.points + TP - 1) / TP, seg_tiles = a.batch / gridDim.y * tiles;
    const int64_t groups = (a.points + kGroup - 1) / kGroup;
    const float inv = 1.0f / (float)C;
    // bytes on which every row starts, 16 at most
    const int starts = (int)(a.points & 15) * (int)sizeof(T) | 16;
    const int starts8 = (int)(a.points & 15) | 16;
    const int piece = starts & -starts, piece8 = starts8 & -starts8;
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
        float sa = block ? a.s[c] : 0.0f;
        const float sb = block && LAYER ? sa * a.b2[c] : 0.0f;
        if (block && a.gate_kind == FNO_GATE_CHANNEL)      // one sample a segment
            sa *= gate_value(static_cast<const float *>(a.gate)[blockIdx.y * C + c], a.sigmoid);
        par[c] = make_float4(block ? sa * a.w2[c] : 0.0f, sa, sb, has_du ? a.w1[c] : 0.0f);
    }
    // a field's tile, TP points of every channel (what lies past the row's end is
    // left as it is: those points are worked on and not stored)
    const auto fetch_field = [&](const void *src, int elem, int piece, uint32_t dst, int64_t base,
                                 int np) {
        const char *s = static_cast<const char *>(src);
        if (WHOLE) {             // a thread's pieces are some rows apart
            const int per = TP * elem / 16, c = threadIdx.x / per;
            const int o = threadIdx.x % per * 16, hop = blockDim.x / per;
            const char *at = s + (base + (int64_t)c * a.points) * elem + o;
            const int64_t step = (int64_t)hop * a.points * elem;
            dst += c * TP * elem + o;
            const int n = C * per / blockDim.x;          // (C = 8 warps: as many as bytes)
#pragma unroll 4
            for (int i = 0; i < n; ++i, at += step, dst += hop * TP * elem)
                cp_async16(dst, at);
            return;
        }
        const auto pieces = [&](auto bytes) {
            constexpr int B = decltype(bytes)::value;
            const int row = TP * elem, sh = 31 - __clz(row / B);           // (a power of two)
            for (int i = threadIdx.x; i < C << sh; i += blockDim.x) {
                const int c = i >> sh, o = (i - (c << sh)) * B;
                if (o >= np * elem) continue;
                const uint32_t to = dst + c * row + o;
                const char *from = s + (base + (int64_t)c * a.points) * elem + o;
                if constexpr (B == 16) cp_async16(to, from);
                else if constexpr (B == 8) cp_async8(to, from);
                else cp_async4(to, from);
            }
        };
        if (piece == 16) return pieces(std::integral_constant<int, 16>());
        if (piece == 8) return pieces(std::integral_constant<int, 8>());
        if (piece == 4) return pieces(std::integral_constant<int, 4>());
        // as many lanes a row as it has words, or a warp
        const char *end = s + a.batch * C * a.points * elem;
        const int row = row_pitch(a.points, TP, elem);
        const int sub = min(32, TP * elem / 4), sh = 31 - __clz(sub);
        for (int c = threadIdx.x >> sh; c < C; c += blockDim.x >> sh) {
            const char *at = s + (base + (int64_t)c * a.points) * elem;
            const int mis = (int)(reinterpret_cast<uintptr_t>(at) & 3), n = mis + np * elem;
            for (int o = (threadIdx.x & (sub - 1)) * 4; o < n; o += 4 * sub) {
                const char *from = at - mis + o;
                if (from + 4 <= end) {
                    cp_async4(dst + c * row + o, from);
                } else {
                    for (int k = 0; k < 4; ++k)
                        if (from + k < end)
                            st_shared8(dst + c * row + o + k,
                                       *reinterpret_cast<const unsigned char *>(from + k));
                }
            }
        }
    };
    const auto fetch = [&](int64_t t, int k) {
        const int64_t tt = blockIdx.y * seg_tiles + t, b = tt / tiles, p = (tt - b * tiles) * TP;
        const int64_t base = b * C * a.points + p;
        const int np = (int)min((int64_t)TP, a.points - p);
        char *st = buf + k * stage;
        const uint32_t u = smem_u32(st);
        if (has_du) {
            fetch_field(a.x, sizeof(T), piece, u + oy, base, np);
            fetch_field(a.du, sizeof(T), piece, u + ou, base, np);
        }
        if (has_dy) fetch_field(a.dy, sizeof(T), piece, u + og, base, np);
        if (full) fetch_field(a.gate, sizeof(T), piece, u + oa, base, np);
        if (F8) {
            fetch_field(a.f8, 1, piece8, u + of, base, np);
            for (int c = threadIdx.x; c < C; c += blockDim.x)
                cp_async4(u + os + c * 4, a.f8_scale + (b * C + c) * groups + p / kGroup);
        } else if (block) {
            fetch_field(a.f, sizeof(T), piece, u + of, base, np);
        }
    };
    float acc[kSums][kTileC] = {};
    int k = 0;
    if (blockIdx.x < seg_tiles) fetch(blockIdx.x, 0);
    cp_async_commit();
    for (int64_t t = blockIdx.x; t < seg_tiles; t += gridDim.x) {
        const int64_t tt = blockIdx.y * seg_tiles + t, b = tt / tiles;
        const int64_t p = (tt - b * tiles) * TP + lane * 2;
        const bool on = WHOLE || p < a.points, on2 = WHOLE || p + 1 < a.points;
        const auto store = [&](T *to, float2 v) {
            if (WHOLE || a.points % 2 == 0) {
                if (on) store_pair(to, v);
            } else {
                if (on) Storage<T>::store(to, v.x);
                if (on2) Storage<T>::store(to + 1, v.y);
            }
        };
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
        // where the tile starts in the tensors; only its low bits are used
        const uint32_t low = (uint32_t)(b * C * a.points + (tt - b * tiles) * TP);
        const auto pair_at = [&](int o, int j) {
            const int c = w + j * warps;
            const T *r = reinterpret_cast<const T *>(st + o + c * pitch) + lane * 2;
            if (!odd) return load_pair(r);
            r += ((low + (uint32_t)c * (uint32_t)a.points) * (uint32_t)sizeof(T) & 3u) / sizeof(T);
            return make_float2(Storage<T>::load(r), Storage<T>::load(r + 1));
        };
        const auto f_at = [&](int j) {
            if constexpr (F8) {
                const int c = w + j * warps;
                const int8_t *r = reinterpret_cast<const int8_t *>(st + of + c * pitch8) + lane * 2;
                const float2 s = f2(reinterpret_cast<const float *>(st + os)[c]);
                if (!odd8) return mul2(code_pair(r), s);
                r += (low + (uint32_t)c * (uint32_t)a.points) & 3u;
                return mul2(make_float2((float)r[0], (float)r[1]), s);
            } else {
                return pair_at(of, j);
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
                    const float2 y = pair_at(oy, j);
                    if (j == 0 && LAYER) y0 = y;
                    const float2 v = LAYER ? sub2(y, y0) : y;
                    const float2 d = weighted2(pair_at(ou, j), par[w + j * warps].w);
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
            float *r = rows + w * TP + lane * 2;
            const int line = warps * TP;
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
        for (int i = threadIdx.x; i < 2 * TP; i += blockDim.x) {
            const bool second = i >= TP;
            if (second ? block : has_du)
                join_moments<LAYER>(rows, fin, i & (TP - 1), second, TP, warps, C, a.eps);
        }
        __syncthreads();
        const auto fin_at = [&](int i) {
            return *reinterpret_cast<const float2 *>(fin + i * TP + lane * 2);
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
            float2 g = has_dy ? pair_at(og, j) : f2(0.0f);
            if (has_du) {
                const float2 y = pair_at(oy, j), u = pair_at(ou, j);
                const float2 n = fma2(LAYER ? sub2(y, ref1) : y, r1, mr1);
                float2 d = weighted2(u, q.w);
                if (LAYER) d = add2(d, d0);
                g = fma2(fma2(n, d1, d), r1, g);
                const float2 un = mul2(u, n);
                if (on) {
                    acc[2][j] += un.x + (on2 ? un.y : 0.0f);
                    if (LAYER) acc[3][j] += u.x + (on2 ? u.y : 0.0f);
                }
            }
            store(dx, g);
            dx += step;
            if (block) {
                const float2 m = fma2(LAYER ? sub2(fv[j], ref2) : fv[j], r2, mr2);
                fv[j] = m;       // M from here on
                if (full) {
                    const float2 gate = pair_at(oa, j);
                    const float ax = gate_value(gate.x, a.sigmoid), ay = gate_value(gate.y, a.sigmoid);
                    if (a.dgate)
                        store(static_cast<T *>(a.dgate) + at + j * step,
                                   mul2(mul2(g, fma2(m, f2(q.x), f2(q.z))),
                                        make_float2(gate_slope(ax, a.sigmoid),
                                                    gate_slope(ay, a.sigmoid))));
                    g = mul2(g, make_float2(ax, ay));
                }
                const float2 gm = mul2(g, m);
                if (on) {
                    acc[0][j] += gm.x + (on2 ? gm.y : 0.0f);
                    if (LAYER) acc[1][j] += g.x + (on2 ? g.y : 0.0f);
                }
                e[j] = weighted2(g, q.x);
                e0 = add2(e0, e[j]);
                e1 = fma2(e[j], m, e1);
            }
        }
        if (block) {
            float *r = rows + w * TP + lane * 2;
            const int line = warps * TP;
            if (LAYER) *reinterpret_cast<float2 *>(r) = e0;
            *reinterpret_cast<float2 *>(r + line) = e1;
            __syncthreads();
            e0 = e1 = f2(0.0f);
#pragma unroll 4
            for (int v = 0; v < warps; ++v) {
                const float *s = rows + v * TP + lane * 2;
                if (LAYER) e0 = add2(e0, *reinterpret_cast<const float2 *>(s));
                e1 = add2(e1, *reinterpret_cast<const float2 *>(s + line));
            }
            e0 = mul2(e0, f2(-inv));
            e1 = mul2(e1, f2(-inv));
#pragma unroll
            for (int j = 0; j < kTileC; ++j) {
                if (j >= mine) break;
                float2 v = LAYER ? add2(e[j], e0) : e[j];
                v = mul2(fma2(fv[j], e1, v), r2);
                store(df, v);
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
    for (int j = 0; j < kTileC; ++j)
#pragma unroll
        for (int q = 0; q < kSums; ++q) {
            // every lane of the warp, whose parts need not have as many channels (a
            // channel that a part has not is a sum of 0)
            float v = acc[q][j];
#pragma unroll
            for (int m = TL / 2; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            if (lane == 0 && j < mine) out[q * C + w + j * warps] = v;
        }
}

// The sums over the lanes of four values: lanes 0-7, 8-15, 16-23 and 24-31 get
// the totals of s[0], s[1], s[2] and s[3].
__device__ __forceinline__ float lanes_sum4(const float (&s)[kSums]) {
    const int lane = threadIdx.x & 31;
    const bool hi = lane & 16, odd = lane & 8;
    float k0 = hi ? s[2] : s[0], k1 = hi ? s[3] : s[1];
    k0 += __shfl_xor_sync(0xffffffffu, hi ? s[0] : s[2], 16);
    k1 += __shfl_xor_sync(0xffffffffu, hi ? s[1] : s[3], 16);
    float t = odd ? k1 : k0;
    t += __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 8);
#pragma unroll
    for (int m = 4; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    return t;
}

// The same two rounds for any point count and up to kWideC channels, where the
// channels of a tile do not fit registers: 32 V points a tile (V = 2 for even
// counts), each round reads the fields again (from L1 or L2), and the channels'
// sums are kept in shared memory by the warp that owns the channel.  2 x 1023 x
// 256^2 bfloat16: 0.3 to 0.5 TB/s, where the point-by-point kernels take twice the
// time; 2 x 512 x 256^2 takes the staged tiles at 0.7 TB/s.
constexpr int kWideWarps = 16, kWideC = 4096;

template <typename T, bool LAYER, bool F8, int V>
__global__ void __launch_bounds__(kWideWarps * 32)
k_sandwich_bwd_wide(Args a) {
    constexpr int PT = 32 * V, W = kWideWarps;
    extern __shared__ float4 sm[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, C = a.channels;
    float *rows = reinterpret_cast<float *>(sm), *fin = rows + 8 * W * PT, *sums = fin + 8 * PT;
    const bool block = F8 || a.f != nullptr, full = block && a.gate_kind == FNO_GATE_FULL;
    const bool has_du = a.du != nullptr, has_dy = a.dy != nullptr;
    const int64_t tiles = (a.points + PT - 1) / PT, seg_tiles = a.batch / gridDim.y * tiles;
    const int64_t groups = (a.points + kGroup - 1) / kGroup;
    const float inv = 1.0f / (float)C;
    for (int i = threadIdx.x; i < kSums * C; i += blockDim.x) sums[i] = 0.0f;
    __syncthreads();
    for (int64_t t = blockIdx.x; t < seg_tiles; t += gridDim.x) {
        const int64_t tt = blockIdx.y * seg_tiles + t, b = tt / tiles;
        const int64_t p = (tt - b * tiles) * PT + lane * V;
        const bool on = p < a.points;
        const int64_t base = b * C * a.points + p;
        const auto field = [&](const void *src, int c) {
            const T *at = static_cast<const T *>(src) + base + c * a.points;
            if (!on) return f2(0.0f);
            if constexpr (V == 2) return load_pair(at);
            else return make_float2(Storage<T>::load(at), 0.0f);
        };
        const auto put = [&](void *dst, int c, float2 v) {
            T *at = static_cast<T *>(dst) + base + c * a.points;
            if (!on) return;
            if constexpr (V == 2) store_pair(at, v);
            else Storage<T>::store(at, v.x);
        };
        const auto f_at = [&](int c) {
            if constexpr (F8) {
                if (!on) return f2(0.0f);
                const int8_t *at = a.f8 + base + c * a.points;
                const float s = a.f8_scale[(b * C + c) * groups + p / kGroup];
                if constexpr (V == 2) return mul2(code_pair(at), f2(s));
                else return make_float2((float)*at * s, 0.0f);
            } else {
                return field(a.f, c);
            }
        };
        const auto gate_at = [&](int c) {
            float2 g = f2(1.0f);
            if (full) {
                g = field(a.gate, c);
                g = make_float2(gate_value(g.x, a.sigmoid), gate_value(g.y, a.sigmoid));
            }
            return g;
        };
        float2 y0 = f2(0.0f), y1 = y0, y2 = y0, g0 = y0, g1 = y0, f0 = y0, f1 = y0, fq = y0;
#pragma unroll 4
        for (int c = w; c < C; c += W) {
            if (has_du) {
                const float2 y = field(a.x, c);
                if (c == w && LAYER) y0 = y;
                const float2 v = LAYER ? sub2(y, y0) : y;
                const float2 d = weighted2(field(a.du, c), a.w1[c]);
                y1 = add2(y1, v);
                y2 = fma2(v, v, y2);
                g0 = add2(g0, d);
                g1 = fma2(d, v, g1);
            }
            if (block) {
                const float2 f = f_at(c);
                if (c == w && LAYER) f0 = f;
                const float2 v = LAYER ? sub2(f, f0) : f;
                f1 = add2(f1, v);
                fq = fma2(v, v, fq);
            }
        }
        const auto row = [&](int q, float2 v) {
            float *r = rows + (q * W + w) * PT + lane * V;
            r[0] = v.x;
            if (V == 2) r[V - 1] = v.y;
        };
        row(0, y0);
        row(1, y1);
        row(2, y2);
        row(3, g0);
        row(4, g1);
        row(5, f0);
        row(6, f1);
        row(7, fq);
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * PT; i += blockDim.x) {
            join_moments<LAYER>(rows, fin, i % PT, i >= PT, PT, W, C, a.eps);
        }
        __syncthreads();
        const auto fin_at = [&](int i) {
            const float *r = fin + i * PT + lane * V;
            return make_float2(r[0], V == 2 ? r[V - 1] : 0.0f);
        };
        const float2 ref1 = fin_at(0), mr1 = fin_at(1), r1 = fin_at(2), d0 = fin_at(3),
                     d1 = fin_at(4), ref2 = fin_at(5), mr2 = fin_at(6), r2 = fin_at(7);
        const auto n_at = [&](float2 y) { return fma2(LAYER ? sub2(y, ref1) : y, r1, mr1); };
        const auto grad = [&](int c, float2 u, float2 n) {
            float2 g = has_dy ? field(a.dy, c) : f2(0.0f);
            if (!has_du) return g;
            float2 d = weighted2(u, a.w1[c]);
            if (LAYER) d = add2(d, d0);
            return fma2(fma2(n, d1, d), r1, g);
        };
        const auto weight = [&](int c) {                   // s a w2, a of a gate per channel
            float s = a.s[c];
            if (a.gate_kind == FNO_GATE_CHANNEL)
                s *= gate_value(static_cast<const float *>(a.gate)[b * C + c], a.sigmoid);
            return s * a.w2[c];
        };
        const auto m_at = [&](int c) {
            const float2 f = f_at(c);
            return fma2(LAYER ? sub2(f, ref2) : f, r2, mr2);
        };
        float2 e0 = f2(0.0f), e1 = e0;
#pragma unroll 2
        for (int c = w; c < C; c += W) {
            float2 u = f2(0.0f), n = u;
            if (has_du) {
                u = field(a.du, c);
                n = n_at(field(a.x, c));
            }
            float2 g = grad(c, u, n);
            float s[kSums] = {};
            s[2] = on ? fmaf(u.x, n.x, V == 2 ? u.y * n.y : 0.0f) : 0.0f;
            s[3] = u.x + (V == 2 ? u.y : 0.0f);
            if (block) {
                const float2 m = m_at(c), av = gate_at(c);
                if (full && a.dgate)
                    put(a.dgate, c,
                        mul2(mul2(mul2(g, f2(a.s[c])),
                                  fma2(m, f2(a.w2[c]), f2(LAYER ? a.b2[c] : 0.0f))),
                             make_float2(gate_slope(av.x, a.sigmoid),
                                         gate_slope(av.y, a.sigmoid))));
                const float2 ga = full ? mul2(g, av) : g;
                s[0] = on ? fmaf(ga.x, m.x, V == 2 ? ga.y * m.y : 0.0f) : 0.0f;
                s[1] = on ? ga.x + (V == 2 ? ga.y : 0.0f) : 0.0f;
                const float2 e = weighted2(ga, weight(c));
                e0 = add2(e0, e);
                e1 = fma2(e, m, e1);
            }
            const float q = lanes_sum4(s);
            if ((lane & 7) == 0) sums[(lane >> 3) * C + c] += q;
            if (!block) put(a.dx, c, g);
        }
        if (block) {
            row(0, e0);
            row(1, e1);
            __syncthreads();
            e0 = e1 = f2(0.0f);
#pragma unroll 4
            for (int v = 0; v < W; ++v) {
                const float *r = rows + v * PT + lane * V;
                e0 = add2(e0, make_float2(r[0], r[V - 1]));
                e1 = add2(e1, make_float2(r[W * PT], r[W * PT + V - 1]));
            }
            e0 = LAYER ? mul2(e0, f2(-inv)) : f2(0.0f);
            e1 = mul2(e1, f2(-inv));
            // dx is written where dy was last read: it may be dy
#pragma unroll 2
            for (int c = w; c < C; c += W) {
                float2 u = f2(0.0f), n = u;
                if (has_du) {
                    u = field(a.du, c);
                    n = n_at(field(a.x, c));
                }
                const float2 g = grad(c, u, n);
                put(a.dx, c, g);
                const float2 ga = full ? mul2(g, gate_at(c)) : g;
                const float2 e = add2(weighted2(ga, weight(c)), e0);
                put(a.df, c, mul2(fma2(m_at(c), e1, e), r2));
            }
        }
        __syncthreads();
    }
    float *out = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kSums * C;
    for (int i = threadIdx.x; i < kSums * C; i += blockDim.x) out[i] = sums[i];
}

// Calls f with the kernel of a call: f8 as given, or every operand a plan allows for.
template <typename T, class F>
void with_kernel(const fno_sandwich_s &p, bool f8, bool whole, F &&f) {
    with_bools(p.d.norm == FNO_NORM_LAYER, f8, [&](auto l, auto q) {
        constexpr bool L = decltype(l)::value, Q = decltype(q)::value;
        if (p.bwd.kind == kWide && p.bwd.vec == 2) f(k_sandwich_bwd_wide<T, L, Q, 2>);
        else if (p.bwd.kind == kWide) f(k_sandwich_bwd_wide<T, L, Q, 1>);
        else if (p.bwd.vec == 4) f(k_sandwich_bwd_tile<T, L, Q, false, 4>);
        else if (p.bwd.vec == 2) f(k_sandwich_bwd_tile<T, L, Q, false, 2>);
        else if (whole) f(k_sandwich_bwd_tile<T, L, Q, true, 1>);
        else f(k_sandwich_bwd_tile<T, L, Q, false, 1>);
    });
}
inline void launch(void (*k)(Args), dim3 grid, int threads, size_t smem, cudaStream_t s, const Args &a,
            int) {
    k<<<grid, threads, smem, s>>>(a);
}
inline void launch(void (*k)(Args, int), dim3 grid, int threads, size_t smem, cudaStream_t s,
            const Args &a, int stages) {
    k<<<grid, threads, smem, s>>>(a, stages);
}

inline size_t smem_of(const fno_sandwich_s &p, bool f8, bool du, bool dy, bool block) {
    const Way &way = p.bwd;
    const int c = p.d.channels;
    if (way.kind == kWide)
        return (size_t)8 * (kWideWarps + 1) * 32 * way.vec * 4 + (size_t)kSums * c * 4;
    return tile_rest(c, way.warps) +
           (size_t)way.group * tile_stage(c, p.d.points, kTileP / way.vec,
                                          (int)elem_bytes(p.d.dtype), f8, du, dy, block,
                                          block && p.d.gate == FNO_GATE_FULL);
}

template <typename T>
fno_status_t grid_shares_of(const fno_sandwich_s &p, int *ctas) {
    fno_status_t st = FNO_OK;
    with_kernel<T>(p, false, false, [&](auto k) {
        st = occupancy(k, p.bwd.warps * 32, smem_of(p, false, true, true, true), ctas);
    });
    return st;
}

template <typename T>
fno_status_t grid_backward_of(const fno_sandwich_s &p, const Args &a, cudaStream_t s) {
    const bool f8 = a.f8 != nullptr, block = a.f || f8;
    const bool whole = block && a.du && a.dy && p.d.gate != FNO_GATE_FULL &&
                       p.d.points % kTileP == 0 && p.d.channels % kTileC == 0;
    const size_t smem = smem_of(p, f8, a.du, a.dy, block);
    fno_status_t st = FNO_OK;
    with_kernel<T>(p, f8, whole, [&](auto k) {
        if (raise_smem_limit(k, smem) != cudaSuccess) {
            st = FNO_ERR_CUDA;
            return;
        }
        launch(k, dim3((unsigned)p.splits, (unsigned)p.segs), p.bwd.warps * 32, smem, s, a,
               p.bwd.group);
        st = launched();
    });
    return st;
}

}  // namespace sandwich
}  // namespace fno
