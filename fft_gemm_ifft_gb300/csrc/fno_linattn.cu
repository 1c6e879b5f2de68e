// fno_linattn.cu -- linear attention with a decay for each head:
//   S_t = e^{log_decay} S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t.
//
// The gradients are scans of the same form: with g = scale dL/do,
//   dq_t = S_t g_t                               (forward scan of k v^T)
//   dk_t = R_t v_t,  dv_t = R_t^T k_t,  R_t = q_t g_t^T + e^{log_decay} R_{t+1}
// and dL/dS_0 = e^{log_decay} R_1, R starting from dL/dS_T.
#include <cmath>

#include "fno_ops_internal.h"

using namespace fno;
using namespace fno::ops;

struct fno_linattn_s {
    int64_t batch, length;
    int heads, kv_heads, dk, dv;
    fno_dtype_t dtype;
    uint32_t flags;
    int sms;
    int *dev_err;
    size_t workspace;
    size_t group_off[2];     // backward with shared heads: dk, dv of every query head
};

namespace {

constexpr int kMaxWidth = 256;

// One scan of the recurrence  Z = gamma Z + kw k_t v_t^T,  o_t = qw q_t Z + ...
// over one (sequence, query head, slice of 8 value columns): a warp per value
// column, the lanes over the key rows.  REV walks the tokens backwards and
// decays after the token instead of before it.
struct ScanArgs {
    const void *q, *k, *v;
    const float *log_decay;
    const int32_t *lengths;
    const float *s0;
    void *o;
    float *sT;
    int64_t length;
    int heads, gq, gk, gv;         // query heads; head sharing of q, k and v (query heads per row)
    int dk, dv;
    float scale_o, scale_k;        // of the output, of each k v^T added to the state
    bool s_transposed;             // s0 and sT are stored (dv, dk)
};

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

template <typename T, typename TO, bool REV>
fno_status_t scan(const ScanArgs &a, int64_t batch, cudaStream_t s) {
    const dim3 grid((unsigned)(batch * a.heads), (unsigned)ceil_div(a.dv, 8));
    k_linattn_scan<T, TO, REV><<<grid, 256, 0, s>>>(a);
    return launched();
}

// sum of the `g` query heads' float32 gradients of each shared head
template <typename T>
__global__ void k_linattn_group_sum(const float *__restrict__ in, T *__restrict__ out, int64_t n,
                                    int g, int d) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        const int64_t row = i / d;
        float s = 0.0f;
        for (int j = 0; j < g; ++j) s += in[(row * g + j) * d + (i - row * d)];
        Storage<T>::store(out + i, s);
    }
}

// One token: a CTA per (row, head, slice of value columns), the key rows over
// the warps.
template <typename T>
__global__ void __launch_bounds__(256)
k_linattn_step(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
               const float *__restrict__ log_decay, float scale, const int32_t *__restrict__ slots,
               int64_t num_slots, const float *state, float *new_state, T *__restrict__ o,
               int heads, int group, int dk, int dv) {
    __shared__ float sum[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.x % heads, e = blockIdx.y * 32 + lane;
    const int64_t b = blockIdx.x / heads;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    const bool live = slot >= 0 && slot < num_slots;
    float s = 0.0f;
    if (live && e < dv) {
        const float gm1 = expm1f(log_decay[h]);
        const int64_t base = (slot * heads + h) * (int64_t)dk * dv + e;
        const int64_t kv = b * (heads / group) + h / group;
        const float ve = Storage<T>::load(v + kv * dv + e);
        for (int d = w; d < dk; d += 8) {
            const float z0 = state[base + (int64_t)d * dv];
            const float z = fmaf(Storage<T>::load(k + kv * dk + d), ve, fmaf(z0, gm1, z0));
            new_state[base + (int64_t)d * dv] = z;
            s = fmaf(Storage<T>::load(q + (b * heads + h) * dk + d), z, s);
        }
    }
    sum[w][lane] = s;
    __syncthreads();
    if (w == 0 && e < dv) {
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t += sum[j][lane];
        Storage<T>::store(o + (b * heads + h) * dv + e, scale * t);
    }
}

struct Sizes {
    size_t q, k, v, o, s;    // bytes
};
Sizes sizes(const fno_linattn_s &p, int64_t length) {
    const size_t e = elem_bytes(p.dtype), n = (size_t)p.batch * length;
    return {n * p.heads * p.dk * e, n * p.kv_heads * p.dk * e, n * p.kv_heads * p.dv * e,
            n * p.heads * p.dv * e, (size_t)p.batch * p.heads * p.dk * p.dv * 4};
}

}  // namespace

extern "C" {

fno_status_t fno_linattn_plan(fno_linattn_t *out, int64_t batch, int64_t length, int32_t heads,
                              int32_t kv_heads, int32_t dk, int32_t dv, fno_dtype_t dtype,
                              uint32_t flags) {
    if (!out) return FNO_ERR_INVALID_ARG;
    *out = nullptr;
    if (batch < 1 || length < 1 || heads < 1 || kv_heads < 1 || heads % kv_heads || dk < 1 ||
        dv < 1 || !valid_dtype(dtype) || (flags & ~FNO_LINATTN_BACKWARD))
        return FNO_ERR_INVALID_ARG;
    if (dk > kMaxWidth || dv > kMaxWidth || (double)batch * heads > 2147483647.0 ||
        (double)batch * (double)length * heads * (dk > dv ? dk : dv) > kMaxElems)
        return FNO_ERR_UNSUPPORTED;
    fno_linattn_s *p = new (std::nothrow) fno_linattn_s();
    if (!p) return FNO_ERR_OUT_OF_MEMORY;
    p->batch = batch;
    p->length = length;
    p->heads = heads;
    p->kv_heads = kv_heads;
    p->dk = dk;
    p->dv = dv;
    p->dtype = dtype;
    p->flags = flags;
    fno_status_t st = make_error_word(&p->dev_err);
    if (st == FNO_OK) st = device_sms(&p->sms);
    if (st != FNO_OK) {
        fno_linattn_destroy(p);
        return st;
    }
    if ((flags & FNO_LINATTN_BACKWARD) && heads != kv_heads) {
        const size_t n = (size_t)batch * length * heads;
        p->group_off[1] = (n * dk * 4 + 255) & ~size_t(255);
        p->workspace = p->group_off[1] + n * dv * 4;
    }
    *out = p;
    return FNO_OK;
}

fno_status_t fno_linattn_workspace_size(fno_linattn_t p, size_t *bytes) {
    if (!p || !bytes) return FNO_ERR_INVALID_ARG;
    *bytes = p->workspace;
    return FNO_OK;
}

fno_status_t fno_linattn_forward(fno_linattn_t p, const void *q, const void *k, const void *v,
                                 const float *log_decay, float scale, const int32_t *lengths,
                                 const float *s0, void *o, float *sT, void *workspace,
                                 fno_stream_t stream) {
    if (!p || !q || !k || !v || !log_decay || !o || (p->workspace && !workspace))
        return FNO_ERR_INVALID_ARG;
    const Sizes n = sizes(*p, p->length);
    fno_status_t st = check_operands(
        {{q, n.q, false}, {k, n.k, false}, {v, n.v, false},
         {log_decay, (size_t)p->heads * 4, false}, {lengths, (size_t)p->batch * 4, false},
         {s0, n.s, false}, {o, n.o, true}, {sT, n.s, true, s0},
         {workspace, p->workspace, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    const int g = p->heads / p->kv_heads;
    ScanArgs a{q, k, v, log_decay, lengths, s0, o, sT, p->length, p->heads, 1, g, g,
               p->dk, p->dv, scale, 1.0f, false};
    return with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        return scan<T, T, false>(a, p->batch, reinterpret_cast<cudaStream_t>(stream));
    });
}

fno_status_t fno_linattn_backward(fno_linattn_t p, const void *q, const void *k, const void *v,
                                  const float *log_decay, float scale, const int32_t *lengths,
                                  const float *s0, const void *go, const float *gsT, void *dq,
                                  void *dk, void *dv, float *ds0, void *workspace,
                                  fno_stream_t stream) {
    if (!p || !(p->flags & FNO_LINATTN_BACKWARD) || !q || !k || !v || !log_decay || !go || !dq ||
        !dk || !dv || (p->workspace && !workspace))
        return FNO_ERR_INVALID_ARG;
    const Sizes n = sizes(*p, p->length);
    fno_status_t st = check_operands(
        {{q, n.q, false}, {k, n.k, false}, {v, n.v, false},
         {log_decay, (size_t)p->heads * 4, false}, {lengths, (size_t)p->batch * 4, false},
         {s0, n.s, false}, {go, n.o, false}, {gsT, n.s, false}, {dq, n.q, true}, {dk, n.k, true},
         {dv, n.v, true}, {ds0, n.s, true, gsT}, {workspace, p->workspace, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int g = p->heads / p->kv_heads;
    float *gk = static_cast<float *>(workspace);
    float *gv = reinterpret_cast<float *>(static_cast<char *>(workspace) + p->group_off[1]);
    // dq: queries go, keys v, values k, the state transposed
    const ScanArgs aq{go, v, k, log_decay, lengths, s0, dq, nullptr, p->length, p->heads, 1, g, g,
                      p->dv, p->dk, scale, 1.0f, true};
    // dk: queries v, keys go, values q;  dv: queries k, keys q, values go
    const ScanArgs ak{v, go, q, log_decay, lengths, gsT, g > 1 ? (void *)gk : dk, nullptr,
                      p->length, p->heads, g, 1, 1, p->dv, p->dk, 1.0f, scale, true};
    const ScanArgs av{k, q, go, log_decay, lengths, gsT, g > 1 ? (void *)gv : dv, ds0,
                      p->length, p->heads, g, 1, 1, p->dk, p->dv, 1.0f, scale, false};
    return with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        fno_status_t r = scan<T, T, false>(aq, p->batch, s);
        if (r != FNO_OK) return r;
        if (g == 1) {
            r = scan<T, T, true>(ak, p->batch, s);
            return r == FNO_OK ? scan<T, T, true>(av, p->batch, s) : r;
        }
        r = scan<T, float, true>(ak, p->batch, s);
        if (r == FNO_OK) r = scan<T, float, true>(av, p->batch, s);
        if (r != FNO_OK) return r;
        const int64_t rows = p->batch * p->length * p->kv_heads;
        k_linattn_group_sum<T><<<p->sms * 4, 256, 0, s>>>(gk, static_cast<T *>(dk), rows * p->dk,
                                                          g, p->dk);
        k_linattn_group_sum<T><<<p->sms * 4, 256, 0, s>>>(gv, static_cast<T *>(dv), rows * p->dv,
                                                          g, p->dv);
        return launched();
    });
}

fno_status_t fno_linattn_step(fno_linattn_t p, const void *q, const void *k, const void *v,
                              const float *log_decay, float scale, const int32_t *slots,
                              int64_t num_slots, const float *state, float *new_state, void *o,
                              fno_stream_t stream) {
    if (!p || !q || !k || !v || !log_decay || !state || !new_state || !o || num_slots < 1 ||
        (!slots && num_slots < p->batch))
        return FNO_ERR_INVALID_ARG;
    const Sizes n = sizes(*p, 1);
    if ((double)num_slots * p->heads * p->dk * p->dv > kMaxElems) return FNO_ERR_UNSUPPORTED;
    const size_t sb = (size_t)num_slots * p->heads * p->dk * p->dv * 4;
    fno_status_t st = check_operands(
        {{q, n.q, false}, {k, n.k, false}, {v, n.v, false},
         {log_decay, (size_t)p->heads * 4, false}, {slots, (size_t)p->batch * 4, false},
         {state, sb, false}, {new_state, sb, true, state}, {o, n.o, true}});
    if (st != FNO_OK) return st;
    if (inject("launch")) return FNO_ERR_CUDA;
    const dim3 grid((unsigned)(p->batch * p->heads), (unsigned)ceil_div(p->dv, 32));
    with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        k_linattn_step<T><<<grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
            static_cast<const T *>(q), static_cast<const T *>(k), static_cast<const T *>(v),
            log_decay, scale, slots, num_slots, state, new_state, static_cast<T *>(o), p->heads,
            p->heads / p->kv_heads, p->dk, p->dv);
    });
    return launched();
}

fno_status_t fno_linattn_get_device_error(fno_linattn_t p, fno_stream_t stream) {
    return p ? read_error_word(p->dev_err, stream) : FNO_ERR_INVALID_ARG;
}

fno_status_t fno_linattn_destroy(fno_linattn_t p) {
    if (!p) return FNO_OK;
    cudaError_t e = p->dev_err ? cudaFree(p->dev_err) : cudaSuccess;
    delete p;
    return e == cudaSuccess ? FNO_OK : FNO_ERR_CUDA;
}

}  // extern "C"
