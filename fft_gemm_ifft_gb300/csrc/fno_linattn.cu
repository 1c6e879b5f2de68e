// fno_linattn.cu -- linear attention with a decay for each head:
//   S_t = e^{log_decay} S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t.
//
// The gradients are scans of the same form: with g = scale dL/do,
//   dq_t = S_t g_t                               (forward scan of k v^T)
//   dk_t = R_t v_t,  dv_t = R_t^T k_t,  R_t = q_t g_t^T + e^{log_decay} R_{t+1}
// and dL/dS_0 = e^{log_decay} R_1, R starting from dL/dS_T.
#include "fno_linattn.h"

using namespace fno;
using namespace fno::ops;
using namespace fno::linattn;

namespace fno {
namespace linattn {
// instantiated in fno_linattn_{f32,f16,bf16}.cu
#define FNO_LINATTN_EXTERN(T)                                                                  \
    extern template fno_status_t scan_of<T>(const fno_linattn_s &, const ScanArgs &, bool,     \
                                            bool, float *, float, cudaStream_t);               \
    extern template fno_status_t chunk_occupancy_of<T>(const fno_linattn_s &, int *);
FNO_LINATTN_EXTERN(float)
FNO_LINATTN_EXTERN(__half)
FNO_LINATTN_EXTERN(__nv_bfloat16)
}  // namespace linattn
}  // namespace fno

namespace {

// local states -> the states in front of the segments, in place: a CTA for 256
// elements of one (sequence, head), the segments' local values loaded eight at a
// time ahead of the chain.
__global__ void __launch_bounds__(256)
k_linattn_prefix(ScanArgs p, float *__restrict__ states, int segments, int64_t seg_len) {
    const int size = p.dk * p.dv, at = blockIdx.y * 256 + threadIdx.x;
    const int64_t bh = blockIdx.x;
    if (at >= size) return;
    int64_t n = p.length;
    if (p.lengths) n = max((int64_t)0, min((int64_t)p.lengths[bh / p.heads], n));
    const float ld = p.log_decay[bh % p.heads];
    const float whole = expf(ld * (float)seg_len);
    float z = 0.0f;
    if (p.s0)
        z = p.s0[bh * size + (p.s_transposed ? at : (at % p.dk) * p.dv + at / p.dk)];
    float *s = states + bh * segments * size + at;
    for (int k0 = 0; k0 < segments; k0 += 8) {
        float local[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            local[k] = k0 + k + 1 < segments ? s[(int64_t)(k0 + k) * size] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k0 + k >= segments) break;
            s[(int64_t)(k0 + k) * size] = z;
            const int64_t len = min(seg_len, n - (k0 + k) * seg_len);
            if (len > 0) z = fmaf(z, len == seg_len ? whole : expf(ld * (float)len), local[k]);
        }
    }
}

fno_status_t scan(const fno_linattn_s &p, const ScanArgs &a, bool rev, bool wide_out,
                  float *states, float scale_p, cudaStream_t s) {
    if (tc_applies(p)) return tc_scan(p, a, rev, wide_out, states, scale_p, s);
    return with_storage(p.dtype, [&](auto t) {
        return scan_of<decltype(t)>(p, a, rev, wide_out, states, scale_p, s);
    });
}

// sum of the `g` query heads' float32 gradients of each shared head; V elements
// a thread (4 where the width allows)
template <typename T, int V>
__global__ void __launch_bounds__(256)
k_linattn_group_sum(const float *__restrict__ in, T *__restrict__ out, int64_t n, int g, int d) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (i >= n) return;
    const int64_t row = n <= 0xffffffffll ? (int64_t)((uint32_t)i / (uint32_t)d) : i / d;
    const float *at = in + row * (g - 1) * d + i;        // (row g) d + (i - row d)
    Pack<float, V> s = *reinterpret_cast<const Pack<float, V> *>(at);
#pragma unroll 4
    for (int j = 1; j < g; ++j) {
        const Pack<float, V> x = *reinterpret_cast<const Pack<float, V> *>(at + (int64_t)j * d);
#pragma unroll
        for (int k = 0; k < V; ++k) s.v[k] += x.v[k];
    }
    Pack<T, V> r;
#pragma unroll
    for (int k = 0; k < V; ++k) Storage<T>::store(&r.v[k], s.v[k]);
    *reinterpret_cast<Pack<T, V> *>(out + i) = r;
}
template <typename T>
void group_sum(const float *in, T *out, int64_t n, int g, int d, cudaStream_t s) {
    if (d % 4 == 0)
        k_linattn_group_sum<T, 4><<<(unsigned)ceil_div(n, 1024), 256, 0, s>>>(in, out, n, g, d);
    else
        k_linattn_group_sum<T, 1><<<(unsigned)ceil_div(n, 256), 256, 0, s>>>(in, out, n, g, d);
}

// One token: a CTA per (row, head).  V value columns a thread (4 where the width
// allows), the key rows over the threads that are left; eight rows' loads are in
// flight at a time, for the state read and written once is all that it costs: 64 of
// 96 slots, 16 heads, 64 x 64: 34 MB in 9.4 us, most of it latency; 128 x 128: 26 us,
// 5.2 TB/s.
constexpr int kStepThreads = 128;

template <typename T, int V>
__global__ void __launch_bounds__(kStepThreads)
k_linattn_step(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
               const float *__restrict__ log_decay, float scale, const int32_t *__restrict__ slots,
               int64_t num_slots, const float *state, float *new_state, T *__restrict__ o,
               int heads, int group, int dk, int dv) {
    __shared__ float sum[kStepThreads * V], sq[kMaxWidth], sk[kMaxWidth];
    const int h = blockIdx.x % heads;
    const int64_t b = blockIdx.x / heads;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    const bool live = slot >= 0 && slot < num_slots;
    const int64_t kv = b * (heads / group) + h / group;
    for (int d = threadIdx.x; d < dk; d += kStepThreads) {
        sq[d] = Storage<T>::load(q + (b * heads + h) * dk + d);
        sk[d] = Storage<T>::load(k + kv * dk + d);
    }
    __syncthreads();
    const float gm1 = expm1f(log_decay[h]);
    // columns in rounds of the threads (dv up to 256), rows over what is left
    const int lanes = (dv + V - 1) / V, across = lanes < kStepThreads ? lanes : kStepThreads;
    const int down = kStepThreads / across, mine = threadIdx.x % across, part = threadIdx.x / across;
    for (int round = 0; round < dv; round += across * V) {          // (every thread's)
        const int e0 = round + mine * V;
        Pack<float, V> s = {};
        if (live && part < down && e0 < dv) {
            const int64_t base = (slot * heads + h) * (int64_t)dk * dv + e0;
            Pack<float, V> ve;
#pragma unroll
            for (int i = 0; i < V; ++i) ve.v[i] = Storage<T>::load(v + kv * dv + e0 + i);
            for (int d0 = part; d0 < dk; d0 += 8 * down) {
                Pack<float, V> z[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (d0 + r * down < dk)
                        z[r] = *reinterpret_cast<const Pack<float, V> *>(
                            state + base + (int64_t)(d0 + r * down) * dv);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int d = d0 + r * down;
                    if (d >= dk) break;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        z[r].v[i] = fmaf(sk[d], ve.v[i], fmaf(z[r].v[i], gm1, z[r].v[i]));
                        s.v[i] = fmaf(sq[d], z[r].v[i], s.v[i]);
                    }
                    *reinterpret_cast<Pack<float, V> *>(new_state + base + (int64_t)d * dv) = z[r];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sum[threadIdx.x * V + i] = s.v[i];
        __syncthreads();
        if (part == 0 && e0 < dv) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float t = 0.0f;
                for (int r = 0; r < down; ++r) t += sum[(r * across + mine) * V + i];
                Storage<T>::store(o + (b * heads + h) * dv + e0 + i, scale * t);
            }
        }
        __syncthreads();
    }
}

}  // namespace

namespace fno {
namespace linattn {

fno_status_t segment_states(const fno_linattn_s &p, const ScanArgs &a, float *states,
                            cudaStream_t s) {
    const dim3 grid((unsigned)(p.batch * a.heads), (unsigned)ceil_div(a.dk * a.dv, 256));
    k_linattn_prefix<<<grid, 256, 0, s>>>(a, states, p.segments, p.seg_len);
    return launched();
}

}  // namespace linattn
}  // namespace fno

namespace {

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
    // time is split when the heads alone leave SMs idle, into one wave of CTAs
    // and segments of 4 chunks at least (a segment costs a second pass over k
    // and v)
    int per_sm = 1;
    const bool tc = tc_applies(*p);
    const int step = tc ? 128 : kC;          // tokens of a chunk
    if (tc)
        per_sm = tc_ctas(*p);
    else if (dk <= kChunkWidth)
        st = with_storage(dtype,
                          [&](auto t) { return chunk_occupancy_of<decltype(t)>(*p, &per_sm); });
    if (st != FNO_OK) {
        fno_linattn_destroy(p);
        return st;
    }
    const int64_t ctas = batch * heads * ceil_div(dv, 128);
    int64_t segs = (int64_t)per_sm * p->sms / ctas;
    const int64_t most = ceil_div(length, 4 * step);
    segs = segs < 1 ? 1 : segs < most ? segs : most;
    p->seg_len = ceil_div(ceil_div(length, segs), step) * step;
    p->segments = (int)ceil_div(length, p->seg_len);
    size_t at = 0;
    if (p->segments > 1) at = (size_t)batch * heads * p->segments * dk * dv * 4;
    if ((flags & FNO_LINATTN_BACKWARD) && heads != kv_heads) {
        const size_t n = (size_t)batch * length * heads;
        p->group_off[0] = (at + 255) & ~size_t(255);
        p->group_off[1] = (p->group_off[0] + n * dk * 4 + 255) & ~size_t(255);
        at = p->group_off[1] + n * dv * 4;
    }
    p->workspace = at;
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
               p->dk, p->dv, scale, 1.0f, false, false, false, sT && sT == s0};
    return scan(*p, a, false, false, static_cast<float *>(workspace), 1.0f,
                reinterpret_cast<cudaStream_t>(stream));
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
    float *states = static_cast<float *>(workspace);
    float *gk = reinterpret_cast<float *>(static_cast<char *>(workspace) + p->group_off[0]);
    float *gv = reinterpret_cast<float *>(static_cast<char *>(workspace) + p->group_off[1]);
    const bool in_place = ds0 && ds0 == gsT;
    // dq: queries go, keys v, values k, the state transposed
    const ScanArgs aq{go, v, k, log_decay, lengths, s0, dq, nullptr, p->length, p->heads, 1, g, g,
                      p->dv, p->dk, scale, 1.0f, true, false, false, false};
    // dk: queries v, keys go, values q;  dv: queries k, keys q, values go
    const ScanArgs ak{v, go, q, log_decay, lengths, gsT, g > 1 ? (void *)gk : dk, nullptr,
                      p->length, p->heads, g, 1, 1, p->dv, p->dk, 1.0f, scale, true, false,
                      ds0 != nullptr, in_place};
    const ScanArgs av{k, q, go, log_decay, lengths, gsT, g > 1 ? (void *)gv : dv, ds0,
                      p->length, p->heads, g, 1, 1, p->dk, p->dv, 1.0f, scale, false,
                      tc_applies(*p) && p->segments > 1, false, in_place};
    st = scan(*p, aq, false, false, states, 1.0f, s);
    if (st == FNO_OK) st = scan(*p, ak, true, g > 1, states, scale, s);
    if (st == FNO_OK) st = scan(*p, av, true, g > 1, states, scale, s);
    if (st != FNO_OK || g == 1) return st;
    return with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t rows = p->batch * p->length * p->kv_heads;
        group_sum(gk, static_cast<T *>(dk), rows * p->dk, g, p->dk, s);
        group_sum(gv, static_cast<T *>(dv), rows * p->dv, g, p->dv, s);
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
    with_storage(p->dtype, [&](auto t) {
        using T = decltype(t);
        const auto run = [&](auto kernel) {
            kernel<<<(unsigned)(p->batch * p->heads), kStepThreads, 0,
                     reinterpret_cast<cudaStream_t>(stream)>>>(
                static_cast<const T *>(q), static_cast<const T *>(k), static_cast<const T *>(v),
                log_decay, scale, slots, num_slots, state, new_state, static_cast<T *>(o),
                p->heads, p->heads / p->kv_heads, p->dk, p->dv);
        };
        if (p->dv % 4 == 0) run(k_linattn_step<T, 4>);
        else run(k_linattn_step<T, 1>);
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
