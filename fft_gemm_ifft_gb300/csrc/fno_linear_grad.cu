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

constexpr int kThreads = 256;
constexpr int kM = 128;                          // inputs of a tile: the tensor cores' rows
constexpr uint32_t kChunkA = kM * 128;           // 64 points of the codes: 128 rows x 128 bytes
// float32 dy as a sum of three bfloat16 terms (24 bits); 16-bit dy as it is
template <typename T> constexpr int kTerms = std::is_same<T, float>::value ? 3 : 1;
// outputs of a tile: two stages of operands within an SM's shared memory
template <typename T> constexpr int kMaxN = std::is_same<T, float>::value ? 64 : 128;
template <typename T> using Operand =
    typename std::conditional<std::is_same<T, __half>::value, __half, __nv_bfloat16>::type;

// Eight elements from `at` on, of which `n` are wanted (the others read as 0),
// by 16-byte loads where the address allows; elsewhere by the 4-byte words that
// hold them, shifted into place.  `end`: the tensor's end, past which nothing is
// read.
template <typename T>
__device__ __forceinline__ Pack<T, 8> load8(const T *at, int n, const T *end) {
    Pack<T, 8> r = {};
    constexpr int B = 8 * (int)sizeof(T), A = B < 16 ? B : 16;
    const uintptr_t u = reinterpret_cast<uintptr_t>(at);
    if (n <= 0) return r;
    if (u % A == 0 && n >= 8) return *reinterpret_cast<const Pack<T, 8> *>(at);
    if (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) r.v[i] = at[i];
        return r;
    }
    constexpr int W = B / 4;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(u & ~uintptr_t(3));
    const int sh = (int)(u & 3) * 8;
    if (n >= 8 && reinterpret_cast<const char *>(w + W + 1) <= reinterpret_cast<const char *>(end)) {
        uint32_t x[W + 1], y[W];
#pragma unroll
        for (int i = 0; i <= W; ++i) x[i] = w[i];
#pragma unroll
        for (int i = 0; i < W; ++i) y[i] = __funnelshift_r(x[i], x[i + 1], sh);
        memcpy(&r, y, sizeof(y));
        return r;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) r.v[i] = at[i];
    return r;
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
template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
k_linear_grad_part(const T *__restrict__ dy, const int8_t *__restrict__ codes,
                   const float *__restrict__ scales, float *__restrict__ part, int64_t batch,
                   int64_t points, int cin, int cout, int64_t groups, int *err) {
    using TO = Operand<T>;
    constexpr int NT = kTerms<T>;
    constexpr int RA = kM / 16, RB = kMaxN<T> / 16;         // rows of a thread: codes, dy
    extern __shared__ char smem_raw[];
    char *base = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                          ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bar[2];
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
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
                     ::"r"(tc_smem_addr(&s_tmem)), "r"(2u * kMaxN<T>));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // rows past the channels are never written: zero, once
    for (uint32_t e = tid; e < 2 * stage / 16; e += kThreads)
        reinterpret_cast<uint4 *>(base)[e] = make_uint4(0, 0, 0, 0);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = s_tmem, sb = tc_smem_addr(base);
    const int64_t items = batch * groups;
    const int r0 = tid >> 4, c8 = (tid & 15) * 8;        // rows r0 + 16 k, points c8 .. c8 + 7
    const int row_i = i0 + (w & 3) * 32 + lane;          // this thread's accumulator row
    const int hn = (N / 2 + 15) / 16 * 16;               // and columns half .. half + hn - 1
    const int half = (w >> 2) * hn;
    Pack<int8_t, 8> qa[RA];
    Pack<T, 8> yb[RB];
    float sc_next = 0.0f, sc = 0.0f, acc[kMaxN<T> / 2] = {}, bias[RB] = {};
    const auto load = [&](int64_t it) {
        const int64_t b = it / groups, g = it - b * groups, p = g * kGroup + c8;
        const int n = (int)min((int64_t)8, points - p);
#pragma unroll
        for (int k = 0; k < RA; ++k)
            if (r0 + 16 * k < mi)
                qa[k] = load8(codes + (b * cin + i0 + r0 + 16 * k) * points + p, n,
                              codes + batch * cin * points);
#pragma unroll
        for (int k = 0; k < RB; ++k)
            if (r0 + 16 * k < no)
                yb[k] = load8(dy + (b * cout + o0 + r0 + 16 * k) * points + p, n,
                              dy + batch * cout * points);
        sc_next = row_i < cin ? scales[(b * cin + row_i) * groups + g] : 0.0f;
    };
    const auto drain = [&](int n, float s) {             // D of block n, times the scales
        mbar_wait(&bar[n & 1], (uint32_t)(n >> 1), err);
        tc_after_sync();
        const uint32_t at = tmem + (n & 1) * kMaxN<T> + half + ((uint32_t)(w & 3) << 21);
#pragma unroll
        for (int k = 0; k < kMaxN<T> / 2; k += 16) {
            if (k >= hn || half + k >= N) break;
            float d[16];
            tmem_ld16(at + k, d);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[k + j] = fmaf(s, d[j], acc[k + j]);
        }
        tc_before_sync();
    };
    int n = 0;
    if (blockIdx.z < items) load(blockIdx.z);
    for (int64_t it = blockIdx.z; it < items; it += gridDim.z, ++n) {
        // the stage was read by the MMAs of block n - 2, drained one block ago
        char *st = base + (n & 1) * stage;
#pragma unroll
        for (int k = 0; k < RA; ++k) {
            const int r = r0 + 16 * k;
            if (r >= mi) break;
            uint2 q;
            uint4 u;
            float f[8];
            memcpy(&q, &qa[k], 8);
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
            const int r = r0 + 16 * k;
            if (r >= no) break;
            char *dst = st + tile_a + (c8 >> 6) * chunk_b + sw_off16(r, c8 & 63);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = Storage<T>::load(&yb[k].v[j]);
            bias[k] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            if constexpr (NT == 1) {
                *reinterpret_cast<Pack<T, 8> *>(dst) = yb[k];
            } else {
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    uint4 u;
                    u.x = take_term(f[0], f[1]);
                    u.y = take_term(f[2], f[3]);
                    u.z = take_term(f[4], f[5]);
                    u.w = take_term(f[6], f[7]);
                    *reinterpret_cast<uint4 *>(dst + x * 2 * chunk_b) = u;
                }
            }
        }
        const float s_prev = sc;
        sc = sc_next;
        if (it + gridDim.z < items) load(it + gridDim.z);
        fence_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_after_sync();
            const uint32_t a = sb + (n & 1) * stage, d = tmem + (n & 1) * kMaxN<T>;
            const uint32_t id = idesc_f16(N, !std::is_same<TO, __half>::value);
            for (int x = NT - 1; x >= 0; --x)            // the small terms first
                for (int k = 0; k < kGroup / 16; ++k)
                    mma_f16(d, desc_sw128(a + (k >> 2) * kChunkA + (k & 3) * 32),
                            desc_sw128(a + tile_a + (2 * x + (k >> 2)) * chunk_b + (k & 3) * 32),
                            id, x < NT - 1 || k > 0);
            mma_commit(&bar[n & 1]);
        }
        if (n > 0) drain(n - 1, s_prev);
    }
    if (n > 0) drain(n - 1, sc);
    float *out = part + (int64_t)blockIdx.z * cout * (cin + 1);
#pragma unroll
    for (int k = 0; k < kMaxN<T> / 2; ++k) {
        const int o = o0 + half + k;
        if (k < hn && half + k < no && row_i < cin) out[(int64_t)o * (cin + 1) + row_i] = acc[k];
    }
    if (i0 == 0)
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            float b = bias[k];
#pragma unroll
            for (int m = 8; m; m >>= 1) b += __shfl_xor_sync(0xffffffffu, b, m);
            const int r = r0 + 16 * k;
            if ((tid & 15) == 0 && r < no) out[(int64_t)(o0 + r) * (cin + 1) + cin] = b;
        }
    __syncthreads();
    if (w == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(2u * kMaxN<T>));
}

// The shares of 32 elements added by 8 warps, then across the warps in order.
__global__ void __launch_bounds__(kThreads)
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
        if (raise_smem_limit(k_linear_grad_part<T>, smem) != cudaSuccess) return FNO_ERR_CUDA;
        k_linear_grad_part<T><<<grid, kThreads, smem, s>>>(
            static_cast<const T *>(dy), codes, scales, part, p->batch, p->points, p->cin, p->cout,
            groups, p->dev_err);
        return launched();
    });
    if (st != FNO_OK) return st;
    const int64_t n = (int64_t)p->cout * (p->cin + 1);
    k_linear_grad_sum<<<(unsigned)ceil_div(n, 32), kThreads, 0, s>>>(part, dw, db, p->cin,
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
