// fno_linattn_chunk.h -- the scans of the linear attention: the kernels,
// instantiated for one storage type in each of three translation units.
#pragma once

#include <cmath>

#include "fno_linattn.h"

namespace fno {
namespace linattn {

using namespace ops;

// One scan of the recurrence  Z = gamma Z + kw k_t v_t^T,  o_t = qw q_t Z + ...
// over one (sequence, query head, slice of 8 value columns): a warp per value
// column, the lanes over the key rows.  REV walks the tokens backwards and
// decays after the token instead of before it.
template <typename T, typename TO, bool REV>
__global__ void __launch_bounds__(256) k_linattn_scan(ScanArgs a) {
    const int lane = threadIdx.x & 31, e = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int h = blockIdx.x % a.heads;
    const int64_t b = blockIdx.x / a.heads;
    if (e >= a.dv) return;
    // gamma - 1 keeps the digits of a slow decay: gamma itself, rounded, would
    // be off by 2^-25 at every step, the same way each time
    const float gm1 = expm1f(a.log_decay[h]);
    int64_t n = a.length;
    if (a.lengths) n = max((int64_t)0, min((int64_t)a.lengths[b], n));
    const int nq = a.heads / a.gq, nk = a.heads / a.gk, nv = a.heads / a.gv;
    const T *q = static_cast<const T *>(a.q) + (b * a.length * nq + h / a.gq) * a.dk;
    const T *k = static_cast<const T *>(a.k) + (b * a.length * nk + h / a.gk) * a.dk;
    const T *v = static_cast<const T *>(a.v) + (b * a.length * nv + h / a.gv) * a.dv + e;
    TO *o = static_cast<TO *>(a.o) + (b * a.length * a.heads + h) * a.dv + e;
    const int64_t sbase = (b * a.heads + h) * (int64_t)a.dk * a.dv;
    constexpr int R = kMaxWidth / 32;
    float z[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int d = lane + 32 * r;
        z[r] = d < a.dk && a.s0
                   ? a.s0[sbase + (a.s_transposed ? (int64_t)e * a.dk + d : (int64_t)d * a.dv + e)]
                   : 0.0f;
    }
    for (int64_t i = 0; i < n; ++i) {
        const int64_t t = REV ? n - 1 - i : i;
        const float ve = a.scale_k * Storage<T>::load(v + t * nv * a.dv);
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int d = lane + 32 * r;
            if (d >= a.dk) continue;
            if (!REV) z[r] = fmaf(z[r], gm1, z[r]);
            z[r] = fmaf(Storage<T>::load(k + t * nk * a.dk + d), ve, z[r]);
            s = fmaf(Storage<T>::load(q + t * nq * a.dk + d), z[r], s);
            if (REV) z[r] = fmaf(z[r], gm1, z[r]);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (lane == 0) Storage<TO>::store(o + t * a.heads * a.dv, a.scale_o * s);
    }
    for (int64_t t = n + lane; t < a.length; t += 32)
        Storage<TO>::store(o + t * a.heads * a.dv, 0.0f);
    if (a.sT) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int d = lane + 32 * r;
            if (d < a.dk)
                a.sT[sbase + (a.s_transposed ? (int64_t)e * a.dk + d : (int64_t)d * a.dv + e)] =
                    z[r];
        }
    }
}

// ---------------------------------------------------------------------------
// The scan in chunks of 64 tokens, on the tensor cores.  Within a chunk, with
// Z the state in front of it and g_i = gamma^i,
//   O = diag(g_{i+1}) Q Z + (Q K^T * [i >= j] g_{i-j}) V
//   Z <- gamma^64 Z + sum_j g_{63-j} k_j v_j^T
// (a reversed scan: g_i in the first, g_{64-j} in the last).  Every exponent is
// >= 0, so nothing overflows.
//
// Numbers.  Operands are sums of bfloat16 terms: 1 for bfloat16 inputs, 2 for
// fp16 (exact: 11 bits in 16), 3 for float32 (24 bits), and products of terms
// below the result's own rounding are left out (i + j > L).  All sums are
// float32.  For bfloat16 the chunk's weights and the state in front of it are two
// terms (16 bits, under the output's own 8); the state itself is carried in float32
// and its update takes the decayed values in three terms, so that a final state has
// float32's digits.
//
// A warp owns 16 rows of the transposed state Z^T (value columns x key rows) in
// registers, in the accumulator layout, which is also the layout of the left
// operand of O^T = Z^T Q^T: the state never leaves the registers.  V^T is the
// other left operand, of O^T += V^T P^T and of the update, read with a
// transposing ldmatrix; the chunk's weights P go through shared memory.
//
// These kernels take what fno_linattn_tc.cu does not: fp16 and float32 wider than
// 64, and widths that are not multiples of 8.  Measured for 2 x 4096 tokens, 8 heads:
// 128 wide 234 us in float32 and 195 in fp16 (bfloat16 on tcgen05: 73), keys of 48
// and values of 80 columns 150 and 114 (49), 50 wide 97, 72 and, in bfloat16, 63.
// mma.sync peaks at 1024 multiply-adds a cycle and SM, and the latency of its chains
// keeps it at a third of that.
// ---------------------------------------------------------------------------
struct ChunkArgs {
    ScanArgs s;
    float *states;             // [b, h, segment][e][a]: local, then initial states
    int segments;
    int64_t seg_len;
    float scale_p;             // of a chunk's weights
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two floats as the next bfloat16 term; they keep what it leaves
__device__ __forceinline__ uint32_t take_term(float &x, float &y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    x -= f.x;
    y -= f.y;
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}
__device__ __forceinline__ float2 term_value(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

template <typename T> constexpr int kTerms = std::is_same<T, float>::value ? 3
                                             : std::is_same<T, __half>::value ? 2 : 1;
// of the chunk's weights and of the state in front of it
template <typename T> constexpr int kInner = kTerms<T> == 1 ? 2 : kTerms<T>;

// 16 bytes, or zeros
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}

// Rows t0 .. t0 + m - 1 (in scan order), w columns, of a (length, heads, full)
// tensor into kTerms planes of 64 x W (+ 8) bfloat16; the rest zeros.  Every
// head's rows start on 16 bytes when `full` is a multiple of 8.  bfloat16 rows
// that do are copied asynchronously (the caller waits); others go through
// registers, four vectors' loads in flight.
template <typename T, bool REV>
__device__ __forceinline__ void load_rows(__nv_bfloat16 *dst, const T *src, int64_t stride,
                                          int64_t n, int64_t t0, int m, int w, int full, int W,
                                          bool async) {
    constexpr int NT = kTerms<T>, U = 4;
    const int plane = kC * (W + 8), vecs = W / 8;
    const bool fast = full % 8 == 0;
    if (NT == 1 && async) {
        for (int i = threadIdx.x; i < kC * vecs; i += blockDim.x) {
            const int r = i / vecs, c = (i - r * vecs) * 8;
            const bool have = r < m && c < w;
            const T *at = have ? src + (REV ? n - 1 - (t0 + r) : t0 + r) * stride + c : src;
            cp_async16_or_zero(smem_u32(dst + r * (W + 8) + c), at, have);
        }
        return;
    }
    for (int i0 = threadIdx.x; i0 < kC * vecs; i0 += U * blockDim.x) {
        Pack<T, 8> x[U] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * blockDim.x, r = i / vecs, c = (i - r * vecs) * 8;
            if (r < m && c < w) {
                const T *at = src + (REV ? n - 1 - (t0 + r) : t0 + r) * stride + c;
                if (fast) {
                    x[u] = *reinterpret_cast<const Pack<T, 8> *>(at);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (c + k < w) x[u].v[k] = at[k];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * blockDim.x, r = i / vecs, c = (i - r * vecs) * 8;
            if (i >= kC * vecs) break;
            if constexpr (NT == 1) {
                *reinterpret_cast<Pack<T, 8> *>(dst + r * (W + 8) + c) = x[u];
            } else {
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = Storage<T>::load(&x[u].v[k]);
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    uint4 t;
                    t.x = take_term(f[0], f[1]);
                    t.y = take_term(f[2], f[3]);
                    t.z = take_term(f[4], f[5]);
                    t.w = take_term(f[6], f[7]);
                    *reinterpret_cast<uint4 *>(dst + q * plane + r * (W + 8) + c) = t;
                }
            }
        }
    }
}

// D += sum over the terms' products i + j <= L.  The leading product's sum and
// the others' are kept apart: the tensor cores truncate what they add to a sum,
// which costs the leading sum a digit for every small product added to it.
template <int NA, int NB, int L>
__device__ __forceinline__ void mma_terms(float (&hi)[2][4], float (&lo)[2][4],
                                          const uint32_t (&A)[NA][4], const uint32_t (&B)[NB][4]) {
#pragma unroll
    for (int x = 0; x < NA; ++x)
#pragma unroll
        for (int y = 0; y < NB; ++y) {
            if (x + y > L) continue;
            mma16816(x + y ? lo[0] : hi[0], A[x], B[y][0], B[y][1]);
            mma16816(x + y ? lo[1] : hi[1], A[x], B[y][2], B[y][3]);
        }
}

// O: outputs (false: only the segment's local state).  KT: terms of the decayed
// values in the state's update.
template <typename T, typename TO, int AP, bool REV, bool O, int KT>
__global__ void __launch_bounds__(256) k_linattn_chunk(ChunkArgs ca) {
    constexpr int NT = kTerms<T>, LA = AP + 8, PL = kC * LA, LP = kC + 8, PP = kC * LP;
    constexpr int PT = kInner<T>, L = PT - 1;
    extern __shared__ __align__(16) char smem_chunk[];
    const ScanArgs &p = ca.s;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int ET = warps * 16, LE = ET + 8, PE = kC * LE;
    // weights, then one (two with asynchronous copies) of k, v, q
    __nv_bfloat16 *sp = reinterpret_cast<__nv_bfloat16 *>(smem_chunk);
    __nv_bfloat16 *sbuf = sp + (O ? PT * PP : 0);
    const int buf = NT * (PL + PE + (O ? PL : 0));
    __shared__ float pw[kC + 2];
    const int seg = blockIdx.x % ca.segments;
    if (!O && seg == ca.segments - 1) return;      // no segment starts from its state
    const int64_t bh = blockIdx.x / ca.segments;
    const int h = (int)(bh % p.heads);
    const int64_t b = bh / p.heads;
    const int e0 = blockIdx.y * ET;
    int64_t n = p.length;
    if (p.lengths) n = max((int64_t)0, min((int64_t)p.lengths[b], n));
    const int64_t first = seg * ca.seg_len, last = min(n, first + ca.seg_len);
    const int nq = p.heads / p.gq, nk = p.heads / p.gk, nv = p.heads / p.gv;
    const T *q = static_cast<const T *>(p.q) + (b * p.length * nq + h / p.gq) * p.dk;
    const T *k = static_cast<const T *>(p.k) + (b * p.length * nk + h / p.gk) * p.dk;
    const T *v = static_cast<const T *>(p.v) + (b * p.length * nv + h / p.gv) * p.dv + e0;
    const int ew = min(ET, p.dv - e0);
    const float ld = p.log_decay[h];
    for (int i = threadIdx.x; i < kC + 2; i += blockDim.x) pw[i] = i ? expf(ld * (float)i) : 1.0f;
    const int g = lane >> 2, c2 = (lane & 3) * 2;
    const int er = w * 16 + g;                     // the lane's rows er, er + 8 of the tile
    const int64_t sbase = bh * (int64_t)p.dk * p.dv;
    float *seg_state = ca.states + (bh * ca.segments + seg) * (int64_t)p.dk * p.dv;
    // element (e, a) of a state: the segment's own layout, or the caller's
    const auto own = [&](int e, int a) { return (int64_t)(e0 + e) * p.dk + a; };
    const auto caller = [&](int e, int a) {
        return p.s_transposed ? (int64_t)(e0 + e) * p.dk + a : (int64_t)a * p.dv + e0 + e;
    };
    float Z[AP / 8][4];
    bool zero = true;                              // Z is known to be 0
    {
        const float *src = nullptr;
        bool mine = false;
        if (O && ca.segments > 1) {
            src = seg_state;
            mine = true;
        } else if (O && p.s0) {
            src = p.s0 + sbase;
        }
        zero = !src;
#pragma unroll
        for (int j = 0; j < AP / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = er + (i >> 1) * 8, a = j * 8 + c2 + (i & 1);
                Z[j][i] = src && e < ew && a < p.dk ? src[mine ? own(e, a) : caller(e, a)] : 0.0f;
            }
    }
    // ldmatrix rows of a 16 x 16 block: left operand / transposed right operand
    // (rows 0-7, 8-15 of column 0, then of column 8), and right operand
    const int ra = lane & 15, ka = (lane >> 4) * 8;
    const int rb = (lane & 7) + (lane >> 4) * 8, kb = ((lane >> 3) & 1) * 8;
    const uint32_t up = smem_u32(sp);
    const bool async = NT == 1 && p.dk % 8 == 0 && p.dv % 8 == 0;
    const auto load = [&](int64_t t0, int which) {
        const int m = (int)min((int64_t)kC, last - t0);
        __nv_bfloat16 *d = sbuf + which * buf;
        load_rows<T, REV>(d, k, (int64_t)nk * p.dk, n, t0, m, p.dk, p.dk, AP, async);
        load_rows<T, REV>(d + NT * PL, v, (int64_t)nv * p.dv, n, t0, m, ew, p.dv, ET, async);
        if (O)
            load_rows<T, REV>(d + NT * (PL + PE), q, (int64_t)nq * p.dk, n, t0, m, p.dk, p.dk, AP,
                              async);
    };
    if (async && first < last) {
        load(first, 0);
        cp_async_commit();
    }
    int which = 0;
    for (int64_t t0 = first; t0 < last; t0 += kC) {
        const int m = (int)min((int64_t)kC, last - t0), blocks = (m + 15) / 16;
        __syncthreads();                           // the last chunk's readers are done
        if (async) {
            if (t0 + kC < last) load(t0 + kC, which ^ 1);
            cp_async_commit();
            cp_async_wait<1>();
        } else {
            load(t0, 0);
        }
        __syncthreads();
        const uint32_t uk = smem_u32(sbuf + which * buf), uv = uk + 2 * NT * PL,
                       uq = uv + 2 * NT * PE;
        which ^= async;
        if (O) {
            // the chunk's weights, in 16 x 16 blocks on and below the diagonal
            for (int u = w; u < blocks * (blocks + 1) / 2; u += warps) {
                int i = 0;
                while ((i + 1) * (i + 2) / 2 <= u) ++i;
                const int j = u - i * (i + 1) / 2;
                float s[2][4] = {}, sl[2][4] = {};
#pragma unroll
                for (int kk = 0; kk < AP; kk += 16) {
                    uint32_t A[NT][4], B[NT][4];
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        ldsm4(A[x], uq + 2 * (x * PL + (i * 16 + ra) * LA + kk + ka));
                        ldsm4(B[x], uk + 2 * (x * PL + (j * 16 + rb) * LA + kk + kb));
                    }
                    mma_terms<NT, NT, L>(s, sl, A, B);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[y][x] += sl[y][x];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int t = i * 16 + g + 8 * x, sc = j * 16 + y * 8 + c2;
                        float f0 = t >= sc ? s[y][2 * x] * (pw[max(0, t - sc)] * ca.scale_p) : 0.0f;
                        float f1 = t > sc
                                       ? s[y][2 * x + 1] * (pw[max(0, t - sc - 1)] * ca.scale_p)
                                       : 0.0f;
#pragma unroll
                        for (int z = 0; z < PT; ++z)
                            *reinterpret_cast<uint32_t *>(sp + z * PP + t * LP + sc) =
                                take_term(f0, f1);
                    }
            }
            __syncthreads();
            float acc[kC / 16][2][4] = {}, acl[kC / 16][2][4] = {};
            if (!zero) {
#pragma unroll
                for (int kk = 0; kk < AP / 16; ++kk) {
                    uint32_t A[PT][4];
                    float z[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        z[i] = Z[2 * kk][i];
                        z[4 + i] = Z[2 * kk + 1][i];
                    }
#pragma unroll
                    for (int x = 0; x < PT; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i) A[x][i] = take_term(z[2 * i], z[2 * i + 1]);
#pragma unroll
                    for (int tb = 0; tb < kC / 16; ++tb) {
                        if (tb >= blocks) break;
                        uint32_t B[NT][4];
#pragma unroll
                        for (int x = 0; x < NT; ++x)
                            ldsm4(B[x], uq + 2 * (x * PL + (tb * 16 + rb) * LA + kk * 16 + kb));
                        mma_terms<PT, NT, L>(acc[tb], acl[tb], A, B);
                    }
                }
#pragma unroll
                for (int j = 0; j < kC / 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float f = pw[j * 8 + c2 + (i & 1) + !REV];
                        acc[j / 2][j % 2][i] *= f;
                        acl[j / 2][j % 2][i] *= f;
                    }
            }
#pragma unroll
            for (int sb = 0; sb < kC / 16; ++sb) {
                if (sb >= blocks) break;
                uint32_t A[NT][4];
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    uint32_t r[4];
                    ldsm4t(r, uv + 2 * (x * PE + (sb * 16 + ra) * LE + w * 16 + ka));
                    A[x][0] = r[0];
                    A[x][1] = r[2];
                    A[x][2] = r[1];
                    A[x][3] = r[3];
                }
#pragma unroll
                for (int tb = 0; tb < kC / 16; ++tb) {
                    if (tb < sb || tb >= blocks) continue;
                    uint32_t B[PT][4];
#pragma unroll
                    for (int x = 0; x < PT; ++x)
                        ldsm4(B[x], up + 2 * (x * PP + (tb * 16 + rb) * LP + sb * 16 + kb));
                    mma_terms<NT, PT, L>(acc[tb], acl[tb], A, B);
                }
            }
            TO *o = static_cast<TO *>(p.o) + (b * p.length * p.heads + h) * p.dv + e0;
#pragma unroll
            for (int j = 0; j < kC / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = j * 8 + c2 + (i & 1), e = er + (i >> 1) * 8;
                    if (r < m && e < ew)
                        Storage<TO>::store(
                            o + (REV ? n - 1 - (t0 + r) : t0 + r) * p.heads * p.dv + e,
                            p.scale_o * (acc[j / 2][j % 2][i] + acl[j / 2][j % 2][i]));
                }
        }
        // the state after the chunk: the chunk's own sum is made apart and added
        // rounded, so that the tensor cores' truncation does not pile up in Z
        uint32_t A[kC / 16][KT][4];
#pragma unroll
        for (int sb = 0; sb < kC / 16; ++sb) {
            float f[8] = {};
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                uint32_t r[4];
                ldsm4t(r, uv + 2 * (x * PE + (sb * 16 + ra) * LE + w * 16 + ka));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 t = term_value(r[i == 1 ? 2 : i == 2 ? 1 : i]);
                    f[2 * i] += t.x;
                    f[2 * i + 1] += t.y;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = sb * 16 + (i >> 1) * 8 + c2;
                f[2 * i] *= pw[max(0, m - 1 - s + REV)] * p.scale_k;
                f[2 * i + 1] *= pw[max(0, m - 2 - s + REV)] * p.scale_k;
            }
#pragma unroll
            for (int x = 0; x < KT; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) A[sb][x][i] = take_term(f[2 * i], f[2 * i + 1]);
        }
        const float carry = pw[m];
        zero = false;
#pragma unroll
        for (int ab = 0; ab < AP / 16; ++ab) {
            float hi[2][4] = {}, lo[2][4] = {};
#pragma unroll
            for (int sb = 0; sb < kC / 16; ++sb) {
                if (sb >= blocks) break;
                uint32_t B[NT][4];
#pragma unroll
                for (int x = 0; x < NT; ++x)
                    ldsm4t(B[x], uk + 2 * (x * PL + (sb * 16 + ra) * LA + ab * 16 + ka));
                mma_terms<KT, NT, KT - 1>(hi, lo, A[sb], B);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    Z[2 * ab + y][i] = fmaf(Z[2 * ab + y][i], carry, hi[y][i] + lo[y][i]);
        }
    }
    if (O) {
        // tokens beyond the sequence, in the tile's segment
        TO *o = static_cast<TO *>(p.o) + (b * p.length * p.heads + h) * p.dv + e0;
        const int64_t from = max(n, first), to = min(p.length, first + ca.seg_len);
        for (int64_t t = from + w; t < to; t += warps)
            for (int e = lane; e < ew; e += 32)
                Storage<TO>::store(o + t * p.heads * p.dv + e, 0.0f);
        // the segment with the last token (the first one, of an empty sequence)
        if (!p.sT || !(n > first ? n <= first + ca.seg_len : n == 0 && seg == 0)) return;
    }
    float *dst = O ? p.sT + sbase : seg_state;
#pragma unroll
    for (int j = 0; j < AP / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = er + (i >> 1) * 8, a = j * 8 + c2 + (i & 1);
            if (e < ew && a < p.dk) dst[O ? caller(e, a) : own(e, a)] = Z[j][i];
        }
}

template <typename T>
size_t chunk_smem(int AP, int warps, bool outputs) {
    const int NT = kTerms<T>, bufs = NT == 1 ? 2 : 1;
    return (size_t)kC * 2 * (NT * bufs * ((outputs ? 2 : 1) * (AP + 8) + warps * 16 + 8) +
                             (outputs ? kInner<T> * (kC + 8) : 0));
}
inline int chunk_warps(int dv) {
    const int w = (dv + 15) / 16;
    return w < 8 ? w : 8;
}

// Calls f with the padded key width.
template <class F>
fno_status_t with_width(int dk, F &&f) {
    if (dk <= 64) return f(std::integral_constant<int, 64>());
    return f(std::integral_constant<int, 128>());
}

// Token by token beyond 128 key columns, whose state does not fit the registers.
// p.segments > 1: the segments' local states, their prefix, then all segments
// side by side.
template <typename T, typename TO, bool REV>
fno_status_t scan(const fno_linattn_s &p, const ScanArgs &a, float *states, float scale_p,
                  cudaStream_t s) {
    if (a.dk > kChunkWidth) {
        const dim3 grid((unsigned)(p.batch * a.heads), (unsigned)ceil_div(a.dv, 8));
        k_linattn_scan<T, TO, REV><<<grid, 256, 0, s>>>(a);
        return launched();
    }
    const ChunkArgs ca{a, states, p.segments, p.seg_len, scale_p};
    const int warps = chunk_warps(a.dv);
    const int64_t bh = p.batch * a.heads;
    const dim3 grid((unsigned)(bh * p.segments), (unsigned)ceil_div(a.dv, warps * 16));
    return with_width(a.dk, [&](auto ap) {
        constexpr int AP = decltype(ap)::value;
        const auto run = [&](auto kernel, bool outputs) {
            const size_t smem = chunk_smem<T>(AP, warps, outputs);
            if (raise_smem_limit(kernel, smem) != cudaSuccess) return FNO_ERR_CUDA;
            kernel<<<grid, warps * 32, smem, s>>>(ca);
            return launched();
        };
        if (p.segments > 1) {
            fno_status_t st = run(k_linattn_chunk<T, T, AP, REV, false, 3>, false);
            if (st != FNO_OK) return st;
            st = segment_states(p, a, states, s);
            if (st != FNO_OK) return st;
        }
        return run(k_linattn_chunk<T, TO, AP, REV, true, 3>, true);
    });
}

template <typename T>
fno_status_t scan_of(const fno_linattn_s &p, const ScanArgs &a, bool rev, bool wide_out,
                     float *states, float scale_p, cudaStream_t s) {
    if (!rev) return scan<T, T, false>(p, a, states, scale_p, s);
    if (wide_out) return scan<T, float, true>(p, a, states, scale_p, s);
    return scan<T, T, true>(p, a, states, scale_p, s);
}

template <typename T> fno_status_t chunk_occupancy_of(const fno_linattn_s &p, int *ctas) {
    return with_width(p.dk, [&](auto ap) {
        constexpr int AP = decltype(ap)::value;
        const int warps = chunk_warps(p.dv);
        const size_t smem = chunk_smem<T>(AP, warps, true);
        const auto kernel = k_linattn_chunk<T, T, AP, false, true, 3>;
        if (raise_smem_limit(kernel, smem) == cudaSuccess &&
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kernel, warps * 32, smem) ==
                cudaSuccess && *ctas > 0)
            return FNO_OK;
        cudaGetLastError();
        return FNO_ERR_CUDA;
    });
}

}  // namespace linattn
}  // namespace fno
