// fno_linear_grad.cu -- weight and bias gradient of a 1x1 linear from the
// 8-bit checkpoint of its input:
//   dw[o,i] = sum_{b,p} dy[b,o,p] code[b,i,p] scale[b,i,p/128],  db[o] = sum dy.
//
// The points are split over the grid; each CTA sums its share and a second
// kernel adds the shares in a fixed order.
#include "fno_ops_internal.h"

using namespace fno;
using namespace fno::ops;

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

constexpr int kTile = 32;    // outputs x inputs of a CTA

// CTA (i tile, o tile, share): 32 x 32 gradients, 256 threads, 4 each.
template <typename T>
__global__ void __launch_bounds__(256)
k_linear_grad_part(const T *__restrict__ dy, const int8_t *__restrict__ codes,
                   const float *__restrict__ scales, float *__restrict__ part,
                   int64_t batch, int64_t points, int cin, int cout, int64_t groups) {
    __shared__ float sy[kTile][kGroup + 1], sx[kTile][kGroup + 1];
    const int i0 = blockIdx.x * kTile, o0 = blockIdx.y * kTile;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    float acc[4] = {}, bias[4] = {};
    const int64_t items = batch * groups;
    for (int64_t it = blockIdx.z; it < items; it += gridDim.z) {
        const int64_t b = it / groups, g = it - b * groups, p0 = g * kGroup;
        const int n = (int)min((int64_t)kGroup, points - p0);
        for (int e = threadIdx.x; e < kTile * kGroup; e += 256) {
            const int r = e / kGroup, c = e % kGroup;
            sy[r][c] = c < n && o0 + r < cout
                           ? Storage<T>::load(dy + (b * cout + o0 + r) * points + p0 + c) : 0.0f;
            const int64_t row = b * cin + i0 + r;
            sx[r][c] = c < n && i0 + r < cin
                           ? (float)codes[row * points + p0 + c] * scales[row * groups + g] : 0.0f;
        }
        __syncthreads();
        for (int c = 0; c < n; ++c) {
            const float xv = sx[tx][c];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[j] = fmaf(sy[ty + 8 * j][c], xv, acc[j]);
                bias[j] += sy[ty + 8 * j][c];
            }
        }
        __syncthreads();
    }
    float *out = part + (int64_t)blockIdx.z * cout * (cin + 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int o = o0 + ty + 8 * j, i = i0 + tx;
        if (o >= cout) continue;
        if (i < cin) out[(int64_t)o * (cin + 1) + i] = acc[j];
        if (i == 0) out[(int64_t)o * (cin + 1) + cin] = bias[j];
    }
}

__global__ void k_linear_grad_sum(const float *__restrict__ part, float *__restrict__ dw,
                                  float *__restrict__ db, int cin, int cout, int splits) {
    const int64_t n = (int64_t)cout * (cin + 1);
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= n) return;
    float s = 0.0f;
    for (int k = 0; k < splits; ++k) s += part[k * n + e];
    const int o = (int)(e / (cin + 1)), i = (int)(e % (cin + 1));
    if (i < cin) dw[(int64_t)o * cin + i] = s;
    else if (db) db[o] = s;
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
    const int64_t tiles = ceil_div(cin, kTile) * ceil_div(cout, kTile);
    const int64_t items = batch * ceil_div(points, kGroup);
    int64_t s = ceil_div(4 * p->sms, tiles);
    p->splits = (int)(s < items ? s : items);
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
    const dim3 grid((unsigned)ceil_div(p->cin, kTile), (unsigned)ceil_div(p->cout, kTile),
                    (unsigned)p->splits);
    with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        k_linear_grad_part<T><<<grid, 256, 0, s>>>(static_cast<const T *>(dy), codes, scales,
                                                   part, p->batch, p->points, p->cin, p->cout,
                                                   groups);
    });
    st = launched();
    if (st != FNO_OK) return st;
    const int64_t n = (int64_t)p->cout * (p->cin + 1);
    k_linear_grad_sum<<<(unsigned)ceil_div(n, 128), 128, 0, s>>>(part, dw, db, p->cin, p->cout,
                                                                 p->splits);
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
