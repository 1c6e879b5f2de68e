// fno_linear_grad.cu -- weight and bias gradient of a 1x1 linear from the
// 8-bit checkpoint of its input:
//   dw[o,i] = sum_{b,p} dy[b,o,p] code[b,i,p] scale[b,i,p/128],  db[o] = sum dy.
//
// The points are split over the grid; each CTA sums its share and a second
// kernel adds the shares in a fixed order.
#include "fno_ops_internal.h"
#include "fno_tc.cuh"

using namespace fno;
using namespace fno::ops;
using namespace fno::tcu;

struct fno_linear_grad_s {
    int64_t batch, points;
    int cin, cout;
    fno_dtype_t dtype;
    int sms;
    int *dev_err;
    int splits;              // shares of the (sample, group of 128 points) items
    size_t workspace;
};

namespace {

constexpr int kThreads = 512;
constexpr int kRows = kThreads / 16;              // rows that the threads load at a time
constexpr int kM = 128;                          // inputs of a tile: the tensor cores' rows
constexpr uint32_t kChunkA = kM * 128;           // 64 points of the codes: 128 rows x 128 bytes
// float32 dy as a sum of three bfloat16 terms (24 bits); 16-bit dy as it is
template <typename T> constexpr int kTerms = std::is_same<T, float>::value ? 3 : 1;
// outputs of a tile: two stages of operands within an SM's shared memory
template <typename T> constexpr int kMaxN = std::is_same<T, float>::value ? 64 : 128;
template <typename T> using Operand =
    typename std::conditional<std::is_same<T, __half>::value, __half, __nv_bfloat16>::type;

// Eight consecutive elements as they come from memory.  Where every row starts
// on 16 bytes (VEC: a point count that is a multiple of 8) they are one or two
// vector loads.  Elsewhere 8- and 16-bit elements come as the 4-byte words that
// hold them and are shifted into place when they are used, float32 one by one.
// Every load is a predicated instruction without a branch, so that a thread's
// loads are all in flight together (with the choice made at each load, the
// branches kept them apart: 611 us in place of 110 for 8 x 40 -> 60 x 64^3).
template <typename T, bool VEC>
struct Raw8 {
    static constexpr int kWords = 8 * (int)sizeof(T) / 4 + (VEC || sizeof(T) == 4 ? 0 : 1);
    uint32_t w[kWords];
    // `n` elements from `at` on are wanted.  Every word that is read has a wanted byte,
    // so that none reaches more than 3 bytes past them.
    __device__ __forceinline__ void load(const T *at, int n) {
        if constexpr (VEC) {
            constexpr int B = 8 * (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = 0;
            if (n > 0) {
                if constexpr (B == 8) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(at);
                    w[0] = u.x;
                    w[1] = u.y;
                } else {
#pragma unroll
                    for (int i = 0; i < B / 16; ++i) {
                        const uint4 u = reinterpret_cast<const uint4 *>(at)[i];
                        w[4 * i] = u.x;
                        w[4 * i + 1] = u.y;
                        w[4 * i + 2] = u.z;
                        w[4 * i + 3] = u.w;
                    }
                }
            }
        } else {
            const uint32_t *p =
                reinterpret_cast<const uint32_t *>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t(3));
            const int end =
                n > 0 ? n * (int)sizeof(T) + (int)(reinterpret_cast<uintptr_t>(at) & 3) : 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                w[i] = 0;
                if (i * 4 < end) w[i] = p[i];
            }
        }
    }
    // the same without a byte past the n elements (at the tensor's end)
    __device__ __forceinline__ void load_exact(const T *at, int n) {
        const unsigned char *from = reinterpret_cast<const unsigned char *>(at),
                            *to = from + n * sizeof(T),
                            *p = reinterpret_cast<const unsigned char *>(
                                reinterpret_cast<uintptr_t>(at) & ~uintptr_t(3));
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (p + 4 * i + j >= from && p + 4 * i + j < to)
                    w[i] |= (uint32_t)p[4 * i + j] << (8 * j);
        }
    }
    // the elements, those from n on 0; `shift`: 8 (address mod 4)
    __device__ __forceinline__ Pack<T, 8> get(int n, int shift) const {
        Pack<T, 8> r;
        if constexpr (VEC || sizeof(T) == 4) {
            memcpy(&r, w, sizeof(r));
        } else {
            uint32_t y[kWords - 1];
#pragma unroll
            for (int i = 0; i < kWords - 1; ++i) y[i] = __funnelshift_r(w[i], w[i + 1], shift);
            if (n < 8) {
                constexpr int E = 4 / (int)sizeof(T), B = 8 * (int)sizeof(T);
#pragma unroll
                for (int i = 0; i < kWords - 1; ++i) {
                    const int keep = n - i * E;            // elements of this word
                    y[i] = keep <= 0 ? 0u : keep >= E ? y[i] : y[i] & ((1u << (keep * B)) - 1u);
                }
            }
            memcpy(&r, y, sizeof(r));
        }
        return r;
    }
};

// two floats as the next bfloat16 term; they keep what it leaves.  A term but the last
// is the largest bfloat16 at most, so that an infinity leaves itself (and no
// inf - inf) and is the last term.
__device__ __forceinline__ uint32_t take_term(float &x, float &y, bool last) {
    uint32_t u;
    if (last) asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(u) : "f"(x), "f"(y));
    else asm("cvt.rn.satfinite.bf16x2.f32 %0, %2, %1;" : "=r"(u) : "f"(x), "f"(y));
    x -= __uint_as_float(u << 16);
    y -= __uint_as_float(u & 0xffff0000u);
    return u;
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float x, float y) {
    uint32_t u;
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(x, y);
        memcpy(&u, &h, 4);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        memcpy(&u, &h, 4);
    }
    return u;
}

// Partial gradients of a tile of 128 inputs x N outputs (N = 16 .. 128) over
// this CTA's blocks of 128 points: for each block
//   D[i][o] = sum_p code[i][p] dy[o][p]
// is one chain of kind::f16 tcgen05.mma (M = 128 inputs, K = 128 points; the
// codes are integers below 128 and exact in 16 bits, so every product is exact)
// into one of two tensor-memory accumulators, and each thread adds scale[i] D
// to its registers: a block of points is a group of the checkpoint, and with
// the inputs on the lanes its scale is one number a thread.
//
// The codes and dy pass through registers on their way to the swizzled operand
// tiles (the codes become 16-bit numbers, float32 dy three terms; rows of any
// length and alignment need it too), the next block's loads in flight over the
// conversion, the MMAs and the drain of this one.
//
// The tensor cores add up the 128 products of a block, which costs a digit of the
// float32 sums: 2.2e-7 relative for 8 x 40 -> 60 x 64^3.
//
// Measured: 16 x 64 -> 64 x 128^2 float32 34 us with the sum of the shares (84 MB,
// 2.5 TB/s; 264 us on the SIMT cores), 8 x 40 -> 60 x 64^3 bfloat16 137 us (338 MB,
// 2.5 TB/s; 1911 us).  A block of 128 points costs 2700 cycles, 660 of them the
// issue of its MMAs and 1200 of its loads; with more channels the same cycles
// move more (128 -> 128: 3.9 TB/s).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 1)
k_linear_grad_part(const T *__restrict__ dy, const int8_t *__restrict__ codes,
                   const float *__restrict__ scales, float *__restrict__ part, int64_t batch,
                   int64_t points, int cin, int cout, int64_t groups, int *err) {
    using TO = Operand<T>;
    constexpr int NT = kTerms<T>;
    constexpr int RA = kM / kRows, RB = kMaxN<T> / kRows;   // rows of a thread: codes, dy
    constexpr int NC = kMaxN<T> / 4;                     // accumulators of a thread
    constexpr uint32_t kCols = 2 * kMaxN<T>;             // two of D
    extern __shared__ char smem_raw[];
    char *base = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                          ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bar[2];
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int i0 = blockIdx.x * kM, o0 = blockIdx.y * kMaxN<T>;
    const int mi = min(kM, cin - i0), no = min(kMaxN<T>, cout - o0), N = (no + 15) / 16 * 16;
    const uint32_t chunk_b = N * 128, tile_a = 2 * kChunkA, stage = tile_a + NT * 2 * chunk_b;
    if (tid == 0) {
        for (int k = 0; k < 2; ++k)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(tc_smem_addr(&bar[k])));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (w == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(tc_smem_addr(&s_tmem)), "r"(kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // rows past the channels are never written: zero, once
    for (uint32_t e = tid; e < 2 * stage / 16; e += kThreads)
        reinterpret_cast<uint4 *>(base)[e] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    // a row of ones below the codes gives the sum of dy; a full tile of inputs
    // has no row for it, and the threads add up what they load
    const bool ones = mi < kM;
    if (ones && tid < kGroup)
        for (int k = 0; k < 2; ++k)
            *reinterpret_cast<TO *>(base + k * stage + (tid >> 6) * kChunkA +
                                    sw_off16(mi, tid & 63)) = TO(1.0f);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0), sb = tc_smem_addr(base);
    const int64_t items = batch * groups;
    const int r0 = tid >> 4, c8 = (tid & 15) * 8;        // rows r0 + 32 k, points c8 .. c8 + 7
    const int row_i = i0 + (w & 3) * 32 + lane;          // this thread's accumulator row
    const int hn = (N / 4 + 15) / 16 * 16;               // and columns c0 .. c0 + hn - 1
    const int c0 = (w >> 2) * hn;
    // two blocks' loads are in flight while a third is worked on
    struct Next {
        Raw8<int8_t, VEC> q[RA];
        Raw8<T, VEC> y[RB];
        int n, sh_q, sh_y;                               // (32 rows apart: the same shift)
        float scale;
    } next[2] = {};
    float sc = 0.0f, acc[NC] = {}, bias[RB] = {};
    // the loads run over this CTA's blocks in order: (b, g) is the next one
    // (and where its rows start, kept up with it)
    int64_t it = blockIdx.z, b = it / groups, g = it - b * groups;
    const int64_t row_step = (int64_t)kRows * points;
    const int8_t *q_row, *q_at;
    const T *y_row, *y_at;
    const float *s_row;
    const auto sample = [&]() {
        q_row = codes + (b * cin + i0 + r0) * points + c8;
        y_row = dy + (b * cout + o0 + r0) * points + c8;
        s_row = scales + (b * cin + row_i) * groups;
    };
    sample();
    q_at = q_row + g * kGroup;
    y_at = y_row + g * kGroup;
    const auto load = [&](Next &x) {
        if (it >= items) return;
        x.n = (int)max((int64_t)0, min((int64_t)8, points - g * kGroup - c8));
        if (!VEC) {
            x.sh_q = (int)(reinterpret_cast<uintptr_t>(q_at) & 3) * 8;
            x.sh_y = (int)(reinterpret_cast<uintptr_t>(y_at) & 3) * 8;
        }
        // words reach up to 3 bytes past the wanted elements: there are as many in
        // the tensor when 4 blocks follow, each of an element a row at least
        if (VEC || it + 4 < items) {
#pragma unroll
            for (int k = 0; k < RA; ++k) {
                if (kRows * k >= mi) break;
                x.q[k].load(q_at + k * row_step, r0 + kRows * k < mi ? x.n : 0);
            }
#pragma unroll
            for (int k = 0; k < RB; ++k) {
                if (kRows * k >= no) break;
                x.y[k].load(y_at + k * row_step, r0 + kRows * k < no ? x.n : 0);
            }
        } else {                                         // near the tensors' ends
#pragma unroll
            for (int k = 0; k < RA; ++k)
                x.q[k].load_exact(q_at + k * row_step, r0 + kRows * k < mi ? x.n : 0);
#pragma unroll
            for (int k = 0; k < RB; ++k)
                x.y[k].load_exact(y_at + k * row_step, r0 + kRows * k < no ? x.n : 0);
        }
        x.scale = row_i < i0 + mi ? s_row[g] : 1.0f;
        it += gridDim.z;
        g += gridDim.z;
        if (g < groups) {
            q_at += (int)gridDim.z * kGroup;
            y_at += (int)gridDim.z * kGroup;
        } else {
            do {
                g -= groups;
                ++b;
            } while (g >= groups);
            sample();
            q_at = q_row + g * kGroup;
            y_at = y_row + g * kGroup;
        }
    };
    const auto drain = [&](int n, float s) {             // D of block n, times the scales
        mbar_wait(&bar[n & 1], (uint32_t)(n >> 1), err);
        tc_after_sync();
        const uint32_t at = tmem + (n & 1) * kMaxN<T> + c0 + ((uint32_t)(w & 3) << 21);
#pragma unroll
        for (int k = 0; k < NC; k += 16) {
            if (k >= hn || c0 + k >= N) break;
            float d[16];
            tmem_ld16(at + k, d);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[k + j] = fmaf(s, d[j], acc[k + j]);
        }
        tc_before_sync();
    };
    int n = 0;
    const auto block = [&](Next &x) {
        // the stage was read by the MMAs of block n - 2, drained one block ago
        char *st = base + (n & 1) * stage;
#pragma unroll
        for (int k = 0; k < RA; ++k) {
            const int r = r0 + kRows * k;
            if (r >= mi) break;
            uint2 q;
            uint4 u;
            float f[8];
            const Pack<int8_t, 8> qk = x.q[k].get(x.n, x.sh_q);
            memcpy(&q, &qk, 8);
            code_values4(q.x, f);
            code_values4(q.y, f + 4);
            u.x = pack2<TO>(f[0], f[1]);
            u.y = pack2<TO>(f[2], f[3]);
            u.z = pack2<TO>(f[4], f[5]);
            u.w = pack2<TO>(f[6], f[7]);
            *reinterpret_cast<uint4 *>(st + (c8 >> 6) * kChunkA + sw_off16(r, c8 & 63)) = u;
        }
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            const int r = r0 + kRows * k;
            if (r >= no) break;
            char *dst = st + tile_a + (c8 >> 6) * chunk_b + sw_off16(r, c8 & 63);
            const Pack<T, 8> yk = x.y[k].get(x.n, x.sh_y);
            float f[8];
            if (NT > 1 || !ones)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = Storage<T>::load(&yk.v[j]);
            if (!ones)
                bias[k] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            if constexpr (NT == 1) {
                *reinterpret_cast<Pack<T, 8> *>(dst) = yk;
            } else {
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    uint4 u;
                    u.x = take_term(f[0], f[1], x + 1 == NT);
                    u.y = take_term(f[2], f[3], x + 1 == NT);
                    u.z = take_term(f[4], f[5], x + 1 == NT);
                    u.w = take_term(f[6], f[7], x + 1 == NT);
                    *reinterpret_cast<uint4 *>(dst + x * 2 * chunk_b) = u;
                }
            }
        }
        const float s_prev = sc;
        sc = x.scale;
        load(x);
        fence_async_smem();
        __syncthreads();
        if (w == 0 && elect_one()) {
            tc_after_sync();
            const uint32_t a = sb + (n & 1) * stage, d = tmem + (n & 1) * kMaxN<T>;
            const uint32_t id = idesc_f16(N, !std::is_same<TO, __half>::value);
#pragma unroll
            for (int x = NT - 1; x >= 0; --x)            // the small terms first
#pragma unroll
                for (int k = 0; k < kGroup / 16; ++k)
                    mma_f16(d, desc_sw128(a + (k >> 2) * kChunkA + (k & 3) * 32),
                            desc_sw128(a + tile_a + (2 * x + (k >> 2)) * chunk_b + (k & 3) * 32),
                            id, x < NT - 1 || k > 0);
            mma_commit(&bar[n & 1]);
        }
        if (n > 0) drain(n - 1, s_prev);
        ++n;
    };
    const int blocks = (int)((items - blockIdx.z + gridDim.z - 1) / gridDim.z);
    load(next[0]);
    load(next[1]);
    while (n < blocks) {
        block(next[0]);
        if (n < blocks) block(next[1]);
    }
    if (n > 0) drain(n - 1, sc);
    float *out = part + (int64_t)blockIdx.z * cout * (cin + 1);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int o = o0 + c0 + k;
        if (k >= hn || c0 + k >= no) break;
        if (row_i < i0 + mi) out[(int64_t)o * (cin + 1) + row_i] = acc[k];
        else if (ones && i0 == 0 && row_i == mi) out[(int64_t)o * (cin + 1) + cin] = acc[k];
    }
    if (!ones && i0 == 0)
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            float b = bias[k];
#pragma unroll
            for (int m = 8; m; m >>= 1) b += __shfl_xor_sync(0xffffffffu, b, m);
            const int r = r0 + kRows * k;
            if ((tid & 15) == 0 && r < no) out[(int64_t)(o0 + r) * (cin + 1) + cin] = b;
        }
    __syncthreads();
    if (w == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kCols));
}

// The shares of 32 elements added by 8 warps, then across the warps in order.
__global__ void __launch_bounds__(256)
k_linear_grad_sum(const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ db,
                  int cin, int cout, int splits) {
    __shared__ float sm[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t n = (int64_t)cout * (cin + 1);
    const int64_t e = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (e < n)
#pragma unroll 8
        for (int k = w; k < splits; k += 8) s += part[k * n + e];
    sm[w][lane] = s;
    __syncthreads();
    if (w || e >= n) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sm[k][lane];
    const int o = (int)(e / (cin + 1)), i = (int)(e % (cin + 1));
    if (i < cin) dw[(int64_t)o * cin + i] = s;
    else if (db) db[o] = s;
}

int tile_outputs(fno_dtype_t dtype) {
    return with_storage(dtype, [](auto t) { return kMaxN<decltype(t)>; });
}

template <typename T>
size_t part_smem(int cout) {
    const int n = ((cout < kMaxN<T> ? cout : kMaxN<T>) + 15) / 16 * 16;
    return 2 * (2 * (size_t)kChunkA + kTerms<T> * 2 * (size_t)n * 128) + 1024;
}

}  // namespace

extern "C" {

fno_status_t fno_linear_grad_plan(fno_linear_grad_t *out, int64_t batch, int32_t cin,
                                  int32_t cout, int64_t points, fno_dtype_t dtype) {
    if (!out) return FNO_ERR_INVALID_ARG;
    *out = nullptr;
    if (batch < 1 || points < 1 || cin < 1 || cout < 1 || !valid_dtype(dtype))
        return FNO_ERR_INVALID_ARG;
    if (cin > 4096 || cout > 4096 ||
        (double)batch * (cin > cout ? cin : cout) * (double)points > kMaxElems)
        return FNO_ERR_UNSUPPORTED;
    fno_linear_grad_s *p = new (std::nothrow) fno_linear_grad_s();
    if (!p) return FNO_ERR_OUT_OF_MEMORY;
    p->batch = batch;
    p->points = points;
    p->cin = cin;
    p->cout = cout;
    p->dtype = dtype;
    fno_status_t st = make_error_word(&p->dev_err);
    if (st == FNO_OK) st = device_sms(&p->sms);
    if (st != FNO_OK) {
        fno_linear_grad_destroy(p);
        return st;
    }
    // one CTA an SM, over the tiles and the shares of the points
    const int64_t tiles = ceil_div(cin, kM) * ceil_div(cout, tile_outputs(dtype));
    const int64_t items = batch * ceil_div(points, kGroup);
    int64_t s = p->sms / tiles;
    s = s < 1 ? 1 : s < items ? s : items;
    p->splits = (int)s;
    p->workspace = (size_t)p->splits * cout * (cin + 1) * 4;
    *out = p;
    return FNO_OK;
}

fno_status_t fno_linear_grad_workspace_size(fno_linear_grad_t p, size_t *bytes) {
    if (!p || !bytes) return FNO_ERR_INVALID_ARG;
    *bytes = p->workspace;
    return FNO_OK;
}

fno_status_t fno_linear_grad(fno_linear_grad_t p, const void *dy, const int8_t *codes,
                             const float *scales, float *dw, float *db, void *workspace,
                             fno_stream_t stream) {
    if (!p || !dy || !codes || !scales || !dw || !workspace) return FNO_ERR_INVALID_ARG;
    const int64_t groups = ceil_div(p->points, kGroup);
    const size_t xn = (size_t)p->batch * p->cin * p->points;
    fno_status_t st = check_operands(
        {{dy, (size_t)p->batch * p->cout * p->points * elem_bytes(p->dtype), false},
         {codes, xn, false}, {scales, (size_t)p->batch * p->cin * groups * 4, false},
         {dw, (size_t)p->cout * p->cin * 4, true}, {db, (size_t)p->cout * 4, true},
         {workspace, p->workspace, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    float *part = static_cast<float *>(workspace);
    const dim3 grid((unsigned)ceil_div(p->cin, kM),
                    (unsigned)ceil_div(p->cout, tile_outputs(p->dtype)),
                    (unsigned)p->splits);
    st = with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        const size_t smem = part_smem<T>(p->cout);
        const auto run = [&](auto kernel) {
            if (raise_smem_limit(kernel, smem) != cudaSuccess) return FNO_ERR_CUDA;
            kernel<<<grid, kThreads, smem, s>>>(static_cast<const T *>(dy), codes, scales, part,
                                                p->batch, p->points, p->cin, p->cout, groups,
                                                p->dev_err);
            return launched();
        };
        return p->points % 8 == 0 ? run(k_linear_grad_part<T, true>)
                                  : run(k_linear_grad_part<T, false>);
    });
    if (st != FNO_OK) return st;
    const int64_t n = (int64_t)p->cout * (p->cin + 1);
    k_linear_grad_sum<<<(unsigned)ceil_div(n, 32), 256, 0, s>>>(part, dw, db, p->cin,
                                                                     p->cout, p->splits);
    return launched();
}

fno_status_t fno_linear_grad_get_device_error(fno_linear_grad_t p, fno_stream_t stream) {
    return p ? read_error_word(p->dev_err, stream) : FNO_ERR_INVALID_ARG;
}

fno_status_t fno_linear_grad_destroy(fno_linear_grad_t p) {
    if (!p) return FNO_OK;
    cudaError_t e = p->dev_err ? cudaFree(p->dev_err) : cudaSuccess;
    delete p;
    return e == cudaSuccess ? FNO_OK : FNO_ERR_CUDA;
}

}  // extern "C"
