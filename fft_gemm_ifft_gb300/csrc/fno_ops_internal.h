// fno_ops_internal.h -- shared host and device helpers of the operators
// declared in fno_ops.h (not installed).
#pragma once

#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <new>
#include <type_traits>

#include "fno_internal.cuh"
#include "fno_ops.h"

namespace fno {
namespace ops {

constexpr double kMaxElems = 274877906944.0;    // 2^38: a byte each would fill the GPU
constexpr int kGroup = FNO_ACT8_GROUP;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool valid_dtype(fno_dtype_t t) { return t == FNO_F32 || t == FNO_F16 || t == FNO_BF16; }
inline size_t elem_bytes(fno_dtype_t t) { return t == FNO_F32 ? 4 : 2; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Host-side fault injection of the failure-path tests (as in the spectral
// calls): FNO_FAULT_INJECT names the site at which the library behaves as if
// the CUDA call there had failed.
inline bool inject(const char *site) {
    const char *v = std::getenv("FNO_FAULT_INJECT");
    return v && std::strcmp(v, site) == 0;
}

// An operand of a call: its bytes, whether the call writes it, and an input
// that it may coincide with exactly (an in-place update; no second input may lie
// there).
struct Operand {
    const void *p;
    size_t bytes;
    bool out;
    const void *same = nullptr;
};

// MISALIGNED / ALIASING checks over a call's operands (NULL ones are absent).
inline fno_status_t check_operands(std::initializer_list<Operand> all) {
    for (const Operand &a : all)
        if (!aligned16(a.p)) return FNO_ERR_MISALIGNED;
    for (const Operand &a : all) {
        if (!a.out || !a.p) continue;
        bool in_place = false;
        for (const Operand &b : all) {
            if (&a == &b || !b.p) continue;
            if (b.p == a.p && a.same == b.p && !b.out && !in_place) {
                in_place = true;
                continue;
            }
            const char *pa = static_cast<const char *>(a.p), *pb = static_cast<const char *>(b.p);
            if (pa < pb + b.bytes && pb < pa + a.bytes) return FNO_ERR_ALIASING;
        }
    }
    return FNO_OK;
}

// The status of the launches since the last check; clears the CUDA error.
inline fno_status_t launched() {
    return cudaGetLastError() == cudaSuccess ? FNO_OK : FNO_ERR_CUDA;
}

// The number of SMs of the current device.
inline fno_status_t device_sms(int *sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return FNO_ERR_CUDA;
    }
    return FNO_OK;
}

// Plan-owned device error word (as the spectral plans': first error wins).
inline fno_status_t make_error_word(int **word) {
    if (inject("plan_alloc")) return FNO_ERR_OUT_OF_MEMORY;
    if (cudaMalloc(word, 256) != cudaSuccess) {
        cudaGetLastError();
        *word = nullptr;
        return FNO_ERR_OUT_OF_MEMORY;
    }
    if (cudaMemset(*word, 0, 256) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        cudaFree(*word);
        *word = nullptr;
        return FNO_ERR_CUDA;
    }
    return FNO_OK;
}
inline fno_status_t read_error_word(int *word, fno_stream_t stream) {
    int v = 0;
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess ||
        cudaMemcpy(&v, word, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemset(word, 0, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return FNO_ERR_CUDA;
    }
    return v == kDevTimeout ? FNO_ERR_DEVICE_TIMEOUT : v == kDevBounds ? FNO_ERR_DEVICE_BOUNDS
                                                                       : FNO_OK;
}

// Elements of one 16-byte load, and a run of N elements moved as one (in
// 16-byte pieces at most: operands are no better aligned).
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);
template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Pack { T v[N]; };

// The 8-bit code of a group's elements: scale = m / 127, code = rint(x (127 / m)),
// with IEEE division and multiplication so that the codes are those of the
// written formula.  `mbits` = the largest |x| of the group as its bit pattern
// (unsigned order: NaN above infinity above every finite value).
struct Group8 {
    float scale, inv;
};
__device__ __forceinline__ Group8 group8(uint32_t mbits) {
    const float m = __uint_as_float(mbits);
    const bool keep = !(m < 1e-30f);
    return {keep ? __fdiv_rn(m, 127.0f) : 0.0f, keep ? __fdiv_rn(127.0f, m) : 0.0f};
}
__device__ __forceinline__ int code8(float x, float inv) {
    return __float2int_rn(__fmul_rn(x, inv));
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Pairs of floats in one instruction (each half rounded to nearest).
__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
        "add.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
        "mul.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 x, y, z, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
        "mov.b64 z, {%6, %7};\nfma.rn.f32x2 w, x, y, z;\nmov.b64 {%0, %1}, w;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, f2(-1.0f), a); }

// Exponential and reciprocal of the multi-function unit; subnormal results are 0.
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// (off by 2^-22.7 at most and by 2e-8 to 5e-8 on average, measured over [-20, 0])
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Asks for p's line to be in L2 when it is loaded.
__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Two neighbouring elements as they lie in memory.
template <typename T> struct Pair { uint32_t bits; };
template <> struct Pair<float> { float2 v; };

template <typename T>
__device__ __forceinline__ float2 to_float2(const Pair<T> &p) {
    return Storage<T>::load2(reinterpret_cast<const T *>(&p));
}
// (`wide`: pairs lie on their size; zero where nothing is left)
template <typename T>
__device__ __forceinline__ Pair<T> load_pair(const T *p, bool wide, int left) {
    Pair<T> r;
    if constexpr (sizeof(T) == 4) {
        r.v = make_float2(0.0f, 0.0f);
        if (wide) {
            if (left > 0) r.v = *reinterpret_cast<const float2 *>(p);
        } else {
            if (left > 0) r.v.x = p[0];
            if (left > 1) r.v.y = p[1];
        }
    } else {
        r.bits = 0;
        if (wide) {
            if (left > 0) r.bits = *reinterpret_cast<const uint32_t *>(p);
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
            if (left > 0) r.bits = h[0];
            if (left > 1) r.bits |= (uint32_t)h[1] << 16;
        }
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void store_pair(T *p, float2 v, bool wide, int left) {
    if (wide) {
        Pack<T, 2> o;
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            *reinterpret_cast<__nv_bfloat162 *>(&o) = __floats2bfloat162_rn(v.x, v.y);
        else if constexpr (std::is_same<T, __half>::value)
            *reinterpret_cast<__half2 *>(&o) = __floats2half2_rn(v.x, v.y);
        else o.v[0] = v.x, o.v[1] = v.y;
        if (left > 0) *reinterpret_cast<Pack<T, 2> *>(p) = o;
    } else {
        if (left > 0) Storage<T>::store(p, v.x);
        if (left > 1) Storage<T>::store(p + 1, v.y);
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// One lane of a warp, chosen where control flow is uniform: the MMAs' operands then
// stay in uniform registers (issued under a thread index they cost 90 cycles each).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(e));
    return e != 0;
}
// The values of four codes: the biased byte under the exponent of 2^23, less
// 2^23 + 128 (two instructions a code at full rate; a conversion runs at a
// quarter of it or less).
__device__ __forceinline__ void code_values4(uint32_t w, float *f) {
    w ^= 0x80808080u;
    f[0] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)) - 8388736.0f;
    f[1] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441)) - 8388736.0f;
    f[2] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442)) - 8388736.0f;
    f[3] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443)) - 8388736.0f;
}

}  // namespace ops
}  // namespace fno
