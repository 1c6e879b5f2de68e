// fno_linattn_tc.cu -- the linear attention's scans on the 5th generation tensor
// cores, key and value widths that are multiples of 8: up to 128 for bfloat16, 64
// for float32 and fp16.
//
// The same chunked form as fno_linattn_chunk.h, with chunks of 128 tokens, one
// tcgen05 tile: with Z the state in front of the chunk and g_i = gamma^i,
//   S = Q K^T,  P = S * [i >= j] g_{i-j}            (tensor memory, in place)
//   O = diag(g_{i+1}) Q Z + P V
//   Z <- g_m Z + W^T K (transposed),  W_j = g_{m-1-j} v_j, as KT bfloat16 terms
// All five operands lie in shared memory in one layout, rows of 64 elements
// under the 128-byte swizzle: Q and K are read along their rows for S and Q Z,
// and V, W and K across them (the tokens being summed over) for the others.  P
// is the left operand straight from tensor memory.  A CTA walks one segment of
// one (sequence, head); two halves of 256 threads share the work on a chunk:
//   half 0  half a token row a thread: weights from S to P, the output's rows
//   half 1  W from V, then half a value column of Z^T a thread: the float32
//           state stays in registers, its bfloat16 copy goes to shared memory
// and one thread of each issues the MMAs that its half feeds.
//
// Numbers as in fno_linattn_chunk.h: float32 and fp16 operands are three and two
// bfloat16 terms, a plane each.  For bfloat16, P and the state's copy have two terms
// (16 bits, under the output's own 8; with one term each, the outputs' relative error
// was 2.35e-3 where their own rounding gives 1.66e-3, and this pass took 72 us).  The
// two of the state's copy share one place: the second is written when Q Z has read the
// first.  The state is summed and carried in float32; W, what a chunk adds to it, has
// two terms, or three where a float32 state is the result.
//
// Measured: 2 x 8192 tokens, 16 heads, 128 wide, bfloat16 (4 segments a head): 92 us
// a pass over q, k, v with outputs, 45 us for the segments' states.  A chunk takes
// 10 900 cycles; an M = 128 MMA costs about 100 whatever its N, and a chunk has 56 of
// them: 8 for S, 16 each for Q Z, P V and W^T K.
// What is left is the order S, P, P V, output within a chunk: its operands fill
// shared memory, so that the next chunk's loads start when this one's are read.
#include "fno_linattn.h"
#include "fno_tc.cuh"

namespace fno {
namespace linattn {

using namespace ops;
using namespace tcu;

namespace {

constexpr int kT = 128;                          // tokens of a chunk
constexpr uint32_t kPanel = kT * 128;            // 128 tokens x 64 elements

// Up to so many segments each adds up its earlier ones' local states itself (its
// prologue reads them all at once); more are joined by a kernel in between, which
// reads each once but costs its launch and a trip through memory.  That kernel also
// joins the segments of a call whose final state replaces the initial one: every
// segment's prologue would read s0, which the last segment's CTA may have written.
constexpr int kFold = 8;

struct TcArgs {
    ScanArgs s;
    float *states;             // [b, h, segment][e][a]: local, then initial states
    int segments;
    int64_t seg_len;
    float scale_p;
    int *err;
    __host__ __device__ bool joined() const {
        return segments > kFold || (segments > 1 && s.joined);
    }
};

// operand read across its rows: 64-element panels `panel` bytes apart, groups of
// 8 rows 1024 bytes apart
__device__ __forceinline__ uint64_t desc_across(uint32_t addr, uint32_t panel) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(panel >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
constexpr uint32_t kAcrossA = 1u << 15, kAcrossB = 1u << 16;     // instruction descriptor bits
// D += A (tensor memory) B
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_st16u(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,"
                 "%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                   "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
                   "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
// all 32 columns of a thread's lane, one wait
__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}
__device__ __forceinline__ float2 bf16_pair(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// the next bfloat16 term of a pair, which keeps what it leaves (unless it is the last)
__device__ __forceinline__ uint32_t take_term(float2 &v, bool rest) {
    const uint32_t u = pack_bf16(v.x, v.y);
    if (rest) v = sub2(v, bf16_pair(u));
    return u;
}
__device__ __forceinline__ void half_sync(int which) {       // the 256 threads of a half
    asm volatile("bar.sync %0, 256;" ::"r"(1 + which) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}

// An output row on its way out: 16 bytes more than it has, against bank conflicts.
template <typename TO, int D> constexpr uint32_t kStageRow = D * sizeof(TO) + 16;
template <typename T> constexpr int kTerms = std::is_same<T, float>::value ? 3
                                             : std::is_same<T, __half>::value ? 2 : 1;
// bytes of W, whose place also takes the output tile
template <typename TO, int D, bool O, int KT>
constexpr uint32_t w_bytes() {
    const uint32_t w = KT * (D / 64) * kPanel, stage = (kT * kStageRow<TO, D> + 1023) / 1024 * 1024;
    return O && stage > w ? stage : w;
}
// bytes of the operands (K, V and Q, or K and V, twice where they fit): W first, so that what an MMA of 128 rows reads past a
// 64-row panel of it lies within them
template <typename T, typename TO, int D, bool O, int KT>
constexpr uint32_t operand_bytes() {
    return w_bytes<TO, D, O, KT>() +
           kTerms<T> * (D / 64) * (kPanel * (O ? 3 : kTerms<T> == 1 ? 4 : 2) + (O ? D * 128 : 0));
}

// O: outputs (else only the segment's local state); KT: terms of W.
template <typename T, typename TO, int D, bool REV, bool O, int KT>
__global__ void __launch_bounds__(O ? 512 : 256, D == 64 && O && kTerms<T> == 1 ? 2 : 1)
k_linattn_tc(TcArgs ca) {
    constexpr int NT = kTerms<T>, NP = D / 64, DH = D / 2, NB = NT > 1 ? 1 : D == 64 && O ? 2 : 4;
    static_assert(NT == 1 || D == 64, "the terms of 128 columns do not fit");
    constexpr uint32_t kPlane = NP * kPanel, kOp = NT * kPlane, kZPlane = NP * D * 128;
    constexpr bool TWICE = !O && NT == 1;                  // two of K and V
    constexpr uint32_t kKV = 2 * kOp;
    constexpr uint32_t kW = 0, kK = w_bytes<TO, D, O, KT>(), kV = kK + kOp, kQ = kV + kOp,
                       kZ = kQ + kOp;
    // terms of P and of the state's copy
    constexpr int PT = NT == 1 ? 2 : NT;
    // tensor memory: S / P, the output, W^T K.  bfloat16: each half of S gives its 64
    // columns to both terms of P, and Q Z is made where the output goes, and scaled
    // there before P V is added.  Others: P's terms past the first lie behind S, and
    // Q Z has columns of its own
    constexpr uint32_t cS = 0, cP = 128, cO = NT > 1 ? 256 : 128, cQZ = NT > 1 ? 320 : cO,
                       cD = !O ? 0 : NT > 1 ? 384 : cO + D;
    constexpr uint32_t kCols = !O ? D : D == 128 || NT > 1 ? 512 : 256;
    const auto p_at = [](int t, int c) -> uint32_t {       // term t of P from token c on
        return NT == 1 ? cS + (c & 64) + t * 32 + (c & 63) / 2
                       : (t ? cP + 64 * (t - 1) : cS) + c / 2;
    };
    extern __shared__ char smem_raw[];
    char *base = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                          ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bar_s, bar_o, bar_d, bar_z, bar_z2;
    __shared__ uint32_t s_tmem;
    __shared__ float pw[kT + 2];
    __shared__ float up[O ? 2 * kT : 1];           // scale_p gamma^(i - kT), 0 for i < kT
    __shared__ float4 down[8];                     // gamma^31 .. gamma^0
    const ScanArgs &p = ca.s;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int half = O ? warp >> 3 : 1, t8 = tid & 255, row = tid & 127, sub = t8 >> 7;
    const int seg = blockIdx.x % ca.segments;
    if (!O && seg == ca.segments - 1) return;      // no segment starts from its state
    const int64_t bh = blockIdx.x / ca.segments;
    const int h = (int)(bh % p.heads);
    const int64_t b = bh / p.heads;
    int64_t n = p.length;
    if (p.lengths) n = max((int64_t)0, min((int64_t)p.lengths[b], n));
    const int64_t first = seg * ca.seg_len, last = min(n, first + ca.seg_len);
    const int nq = p.heads / p.gq, nk = p.heads / p.gk, nv = p.heads / p.gv;
    if (tid == 0) {
        for (uint64_t *x : {&bar_s, &bar_o, &bar_d, &bar_z, &bar_z2})
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(tc_smem_addr(x)));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(tc_smem_addr(&s_tmem)), "r"(kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    {
        const float ld = p.log_decay[h];
        for (int i = tid; i < kT + 2; i += blockDim.x) pw[i] = i ? expf(ld * (float)i) : 1.0f;
        if (O && tid < 2 * kT)
            up[tid] = tid < kT ? 0.0f : ca.scale_p * (tid > kT ? expf(ld * (tid - kT)) : 1.0f);
        if (tid < 32) reinterpret_cast<float *>(down)[tid] = tid < 31 ? expf(ld * (31 - tid)) : 1.0f;
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t sb = tc_smem_addr(base), tmem = __shfl_sync(0xffffffffu, s_tmem, 0), lanes = (uint32_t)(warp & 3) << 21;

    // A tensor's rows of a chunk, zeros past the sequence and the width: thread t8
    // of a half takes the 16-byte piece `pc` of the rows r0, r0 + RS, ...
    constexpr int RS = 256 / (D / 8);
    const int r0 = t8 / (D / 8), pc = t8 % (D / 8);
    const uint32_t piece = (pc >> 3) * kPanel + sw_off16(r0, (pc & 7) * 8);
    struct Source {
        const T *at;               // this thread's piece of its first row of the next chunk
        int64_t row, chunk;        // steps, in elements
        bool have;                 // the piece lies within the width
    };
    const auto source = [&](const void *x, int heads, int shared, int w) {
        const int64_t stride = (int64_t)heads * w, t = first + r0;
        const T *at = static_cast<const T *>(x) + (b * p.length * heads + h / shared) * w +
                      (REV ? n - 1 - t : t) * stride + pc * 8;
        return Source{at, (REV ? -RS : RS) * stride, (REV ? -kT : kT) * stride, pc * 8 < w};
    };
    // One-term rows are copied asynchronously.  Rows of more terms come into
    // registers (`fetch`), early, and are split into their planes (`put`) when the
    // last chunk's are no longer read.
    struct Rows {
        Pack<T, 8> x[NT == 1 ? 1 : kT / RS];
    };
    const auto fetch = [&](uint32_t dst, Source &x, int64_t t0, Rows &to) {
        const int m = (int)min((int64_t)kT, last - t0) - r0;
        const T *at = x.at;
#pragma unroll
        for (int i = 0; i < kT / RS; ++i, at += x.row) {
            const bool have = x.have && i * RS < m;
            if constexpr (NT == 1) {
                cp_async16_or_zero(sb + dst + piece + i * RS * 128, have ? at : p.q, have);
            } else {
                to.x[i] = Pack<T, 8>{};
                if (have) to.x[i] = *reinterpret_cast<const Pack<T, 8> *>(at);
            }
        }
        x.at += x.chunk;
    };
    const auto put = [&](uint32_t dst, const Rows &from) {
        if constexpr (NT > 1) {
#pragma unroll
            for (int i = 0; i < kT / RS; ++i) {
                float2 f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[j] = make_float2(Storage<T>::load(&from.x[i].v[2 * j]),
                                       Storage<T>::load(&from.x[i].v[2 * j + 1]));
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    uint32_t y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = take_term(f[j], t + 1 < NT);
                    *reinterpret_cast<uint4 *>(base + dst + t * kPlane + piece + i * RS * 128) =
                        make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
    };
    Source q = source(p.q, nq, p.gq, p.dk), k = source(p.k, nk, p.gk, p.dk),
           v = source(p.v, nv, p.gv, p.dv);
    Rows rq, rk, rv;
    if (first < last) {
        if (O && half == 0) {
            fetch(kQ, q, first, rq);
            put(kQ, rq);
        }
        if (half == 1) {
            fetch(kK, k, first, rk);
            fetch(kV, v, first, rv);
            put(kK, rk);
            put(kV, rv);
        }
    }
    // all threads, once a chunk: the operands are there
    const auto meet = [&]() {
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        tc_before_sync();
        asm volatile("bar.sync 0, %0;" ::"n"(O ? 512 : 256) : "memory");
        tc_after_sync();
    };
    const bool has_state = O && (ca.segments > 1 || p.s0);
    // Q Z over the terms of Z that lie in shared memory (bfloat16: one at a time), added
    // to what is there or not
    const auto mma_qz = [&](bool add) {
        const uint32_t id = idesc_f16(D, true);
#pragma unroll
        for (int sum = NT - 1; sum >= 0; --sum)            // the small products first
#pragma unroll
            for (int x = 0; x <= sum; ++x)
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    mma_f16(tmem + cQZ,
                            desc_sw128(sb + kQ + x * kPlane + (i >> 2) * kPanel + (i & 3) * 32),
                            desc_sw128(sb + kZ + (sum - x) * kZPlane + (i >> 2) * (D * 128) +
                                       (i & 3) * 32), id, add);
                    add = true;
                }
    };
    if (half == 1) {
        // the state: row `row` of Z^T, half of its columns a thread
        const int64_t sbase = bh * (int64_t)p.dk * p.dv;
        const int64_t size = (int64_t)p.dk * p.dv;
        float *seg_state = ca.states + (bh * ca.segments + seg) * size + (int64_t)row * p.dk;
        const bool mine = row < D, stored = mine && row < p.dv;
        const int a0 = sub * DH;
        const auto caller = [&](int a) {
            return sbase + (p.s_transposed ? (int64_t)row * p.dk + a : (int64_t)a * p.dv + row);
        };
        float z[DH];
        const bool ready = ca.joined();                    // seg_state is the initial state
#pragma unroll
        for (int a = 0; a < DH; ++a) {
            z[a] = 0.0f;
            if (stored && has_state && a0 + a < p.dk) {
                if (ready) z[a] = seg_state[a0 + a];
                else if (p.s0) z[a] = p.s0[caller(a0 + a)];
            }
        }
        if (O && stored && p.states_t) {                   // another scan's, transposed
            const float *at = ca.states + (bh * ca.segments + (ready ? seg : 0)) * size +
                              (int64_t)a0 * p.dv + row;
            const float whole = expf(p.log_decay[h] * (float)ca.seg_len);
            for (int j = ready ? seg : 0; j < (ready ? seg + 1 : seg); ++j, at += size)
#pragma unroll
                for (int a = 0; a < DH; ++a)
                    if (a0 + a < p.dk) {
                        const float x = at[(int64_t)a * p.dv];
                        z[a] = ready ? x : fmaf(z[a], whole, x);
                    }
        } else if (O && !ready && stored) {                // the earlier segments' local states
            const float whole = expf(p.log_decay[h] * (float)ca.seg_len);
            const float *at = seg_state - seg * size + a0;
            for (int j = 0; j < seg; ++j, at += size)
#pragma unroll
                for (int a = 0; a < DH; a += 4)            // (dk is a multiple of 8)
                    if (a0 + a < p.dk) {
                        const float4 x = *reinterpret_cast<const float4 *>(at + a);
                        z[a] = fmaf(z[a], whole, x.x);
                        z[a + 1] = fmaf(z[a + 1], whole, x.y);
                        z[a + 2] = fmaf(z[a + 2], whole, x.z);
                        z[a + 3] = fmaf(z[a + 3], whole, x.w);
                    }
        }
        // its bfloat16 terms, the right operands of Q Z: all of them, or for bfloat16
        // the first, whose place the second takes when it has been read
        const auto publish = [&](bool second) {
#pragma unroll
            for (int c = 0; c < DH / 8; ++c) {
                float2 f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = make_float2(z[8 * c + 2 * j], z[8 * c + 2 * j + 1]);
                const int at = a0 / 8 + c;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    uint32_t y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[j] = take_term(f[j], t + 1 < PT);
                        if (NT == 1 && second) y[j] = take_term(f[j], false);
                    }
                    *reinterpret_cast<uint4 *>(base + kZ + t * kZPlane + (at >> 3) * (D * 128) +
                                               sw_off16(row, (at & 7) * 8)) =
                        make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        };
        if (mine && has_state) publish(false);
        int chunk = 0;
        uint32_t carried = 0;                              // chunks with a state in front
        for (int64_t t0 = first; t0 < last; t0 += kT, ++chunk) {
            const int m = (int)min((int64_t)kT, last - t0);
            const bool more = t0 + kT < last;
            meet();
            // (one term without outputs: there is room for the next chunk's K and V)
            const uint32_t at_kv = TWICE ? (chunk & 1) * kKV : 0;
            if (TWICE && more) {
                fetch(kK + (kKV - at_kv), k, t0 + kT, rk);
                fetch(kV + (kKV - at_kv), v, t0 + kT, rv);
            }
            // W: half of a token row a thread, NB pieces read before the first of their
            // terms is written
            const float2 f = f2(pw[max(0, m - 1 - row + REV)] * p.scale_k);
#pragma unroll
            for (int i0 = 0; i0 < DH / 8; i0 += NB) {
                uint4 u[NB][NT];
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const int c = a0 / 8 + i0 + i;
                        u[i][t] = *reinterpret_cast<uint4 *>(base + kV + at_kv + t * kPlane +
                                                             (c >> 3) * kPanel +
                                                             sw_off16(row, (c & 7) * 8));
                    }
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int c = a0 / 8 + i0 + i;
                    char *at = base + kW + (c >> 3) * kPanel + sw_off16(row, (c & 7) * 8);
                    float2 x[4] = {};
#pragma unroll
                    for (int t = NT - 1; t >= 0; --t) {
                        const uint32_t w[4] = {u[i][t].x, u[i][t].y, u[i][t].z, u[i][t].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[j] = t == NT - 1 ? bf16_pair(w[j]) : add2(x[j], bf16_pair(w[j]));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], f);
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        uint32_t y[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] = take_term(x[j], t + 1 < KT);
                        *reinterpret_cast<uint4 *>(at + t * kPlane) =
                            make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            const bool state2 = O && NT == 1 && (has_state || chunk > 0);
            if (state2) {
                mbar_wait(&bar_z, carried++, ca.err);
                tc_after_sync();
                if (mine) publish(true);
            }
            fence_async_smem();
            half_sync(1);
            if (warp == (O ? 8 : 0) && elect_one()) {
                if (state2) {
                    tc_after_sync();
                    mma_qz(true);
                    mma_commit(&bar_z2);
                }
                const uint32_t id = idesc_f16(D, true) | kAcrossA | kAcrossB;
                bool add = false;
#pragma unroll
                for (int sum = KT - 1; sum >= 0; --sum)    // the small products first
#pragma unroll
                    for (int t = 0; t <= sum; ++t) {
                        if (sum - t >= NT) continue;
#pragma unroll
                        for (int i = 0; i < kT / 16; ++i) {
                            mma_f16(tmem + cD,
                                    desc_across(sb + kW + t * kPlane + i * 2048, kPanel),
                                    desc_across(sb + kK + at_kv + (sum - t) * kPlane + i * 2048,
                                                kPanel), id, add);
                            add = true;
                        }
                    }
                mma_commit(&bar_d);
            }
            if (NT > 1 && more) {                          // on their way over the MMAs
                fetch(kK, k, t0 + kT, rk);
                fetch(kV, v, t0 + kT, rv);
            }
            mbar_wait(&bar_d, chunk, ca.err);
            if (O) mbar_wait(&bar_s, chunk, ca.err);
            tc_after_sync();
            if (!TWICE) {
                if (NT == 1 && more) fetch(kK, k, t0 + kT, rk);
                if (more) put(kK, rk);
                if (O) mbar_wait(&bar_o, chunk, ca.err);   // V and the state's copy were read
                if (NT == 1 && more) fetch(kV, v, t0 + kT, rv);
                if (more) put(kV, rv);
                tc_after_sync();
            }
            const float carry = pw[m];
            if ((warp & 3) * 32 < D)                       // (a warp's rows exist together)
#pragma unroll
                for (int c = 0; c < DH; c += 16) {
                    float x[16];
                    tmem_ld16(tmem + cD + a0 + c + lanes, x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) z[c + j] = fmaf(z[c + j], carry, x[j]);
                }
            if (O && more && mine) publish(false);
        }
        const bool ends = n > first ? n <= first + ca.seg_len : n == 0 && seg == 0;
        if (stored && (!O || (p.sT && ends))) {
#pragma unroll
            for (int a = 0; a < DH; ++a)
                if (a0 + a < p.dk) {
                    if (O) p.sT[caller(a0 + a)] = z[a];
                    else seg_state[a0 + a] = z[a];
                }
        }
    }
    if (O && half == 0) {
        const int diag = (warp & 3) * 32, a0 = sub * DH;
        const float fz = pw[row + !REV];
        bool zero = !has_state;
        int chunk = 0;
        uint32_t carried = 0;
        for (int64_t t0 = first; t0 < last; t0 += kT, ++chunk) {
            const int m = (int)min((int64_t)kT, last - t0);
            meet();
            if (warp == 0 && elect_one()) {
                const uint32_t id = idesc_f16(kT, true);
                bool add = false;
#pragma unroll
                for (int sum = NT - 1; sum >= 0; --sum)
#pragma unroll
                    for (int x = 0; x <= sum; ++x)
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint32_t at = (i >> 2) * kPanel + (i & 3) * 32;
                            mma_f16(tmem + cS, desc_sw128(sb + kQ + x * kPlane + at),
                                    desc_sw128(sb + kK + (sum - x) * kPlane + at), id, add);
                            add = true;
                        }
                mma_commit(&bar_s);
                if (!zero) mma_qz(false);
                if (NT == 1 && !zero) mma_commit(&bar_z);  // (others complete with P V)
            }
            mbar_wait(&bar_s, chunk, ca.err);
            tc_after_sync();
            // row `row` of P, the 32 columns of S at 32 sub, then at 64 + 32 sub.  P takes
            // the place of the S that it is read from (the first 64 columns, then, for
            // bfloat16, the others): all threads read those before any writes
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = (2 * i + sub) * 32;
                uint32_t y[16];
                float x[32];
                if (c > diag) {                            // above the diagonal
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = 0.0f;
                } else {
                    tmem_ld32(tmem + cS + c + lanes, x);
                    if (c == diag) {
                        // (the factor read whatever the condition: read under it, each
                        // element is a branch, 5000 cycles a block)
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            x[j] *= up[row - (c + j) + kT];
                            x[j] = row < c + j ? 0.0f : x[j];
                        }
                    } else {                               // gamma^(row - c - 31) gamma^(31 - j)
                        const float2 f = f2(up[row - c - 31 + kT]);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 g = down[j / 4];
                            const float2 lo = mul2(make_float2(x[j], x[j + 1]),
                                                   mul2(f, make_float2(g.x, g.y)));
                            const float2 hi = mul2(make_float2(x[j + 2], x[j + 3]),
                                                   mul2(f, make_float2(g.z, g.w)));
                            x[j] = lo.x;
                            x[j + 1] = lo.y;
                            x[j + 2] = hi.x;
                            x[j + 3] = hi.y;
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < PT; ++t) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float2 v = make_float2(x[2 * j], x[2 * j + 1]);
                        y[j] = take_term(v, t + 1 < PT);
                        x[2 * j] = v.x;
                        x[2 * j + 1] = v.y;
                    }
                    if (t == 0 && (NT == 1 || i == 0)) half_sync(0);
                    tmem_st16u(tmem + p_at(t, c) + lanes, y);
                }
            }
            if (NT == 1 && !zero) {                        // diag(g) Q Z, both terms of Z
                mbar_wait(&bar_z2, carried++, ca.err);
                tc_after_sync();
#pragma unroll
                for (int c = 0; c < DH; c += 16) {
                    float x[16];
                    tmem_ld16(tmem + cO + a0 + c + lanes, x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] *= fz;
                    tmem_st16(tmem + cO + a0 + c + lanes, x);
                }
            }
            tmem_st_wait();
            tc_before_sync();
            half_sync(0);
            if (warp == 0 && elect_one()) {
                tc_after_sync();
                const uint32_t id = idesc_f16(D, true) | kAcrossB;
                bool add = NT == 1 && !zero;
#pragma unroll
                for (int sum = PT - 1; sum >= 0; --sum)
#pragma unroll
                    for (int t = 0; t <= sum; ++t)
#pragma unroll
                        for (int i = 0; i < kT / 16; ++i) {
                            if (sum - t >= NT) continue;
                            mma_f16_ts(tmem + cO, tmem + p_at(t, i * 16),
                                       desc_across(sb + kV + (sum - t) * kPlane + i * 2048, kPanel),
                                       id, add);
                            add = true;
                        }
                mma_commit(&bar_o);
            }
            if (NT > 1 && t0 + kT < last) fetch(kQ, q, t0 + kT, rq);
            mbar_wait(&bar_o, chunk, ca.err);
            mbar_wait(&bar_d, chunk, ca.err);
            tc_after_sync();
            if (NT == 1 && t0 + kT < last) fetch(kQ, q, t0 + kT, rq);
            if (t0 + kT < last) put(kQ, rq);
            // the tile by way of W's place (W was read): a thread's own 16-byte stores
            // would each touch 32 rows
            char *stage = base + row * kStageRow<TO, D>;
#pragma unroll
            for (int c = 0; c < DH; c += 16) {
                float x[16];
                tmem_ld16(tmem + cO + a0 + c + lanes, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= p.scale_o;
                if (NT > 1 && !zero) {
                    float y2[16];
                    tmem_ld16(tmem + cQZ + a0 + c + lanes, y2);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = fmaf(y2[j], fz * p.scale_o, x[j]);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 8) {
                    Pack<TO, 8> u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) Storage<TO>::store(&u.v[i], x[j + i]);
                    *reinterpret_cast<Pack<TO, 8> *>(stage + (a0 + c + j) * sizeof(TO)) = u;
                }
            }
            half_sync(0);
            // ... and out by 16-byte pieces, a row's side by side
            constexpr int E = 16 / (int)sizeof(TO), PR = D / E, RO = 256 / PR;
            const int ro = t8 / PR, co = t8 % PR * E;
            const int64_t t = REV ? n - 1 - (t0 + ro) : t0 + ro;
            const int64_t hop = (int64_t)p.heads * p.dv * (REV ? -RO : RO);
            TO *o = static_cast<TO *>(p.o) + ((b * p.length + t) * p.heads + h) * p.dv + co;
            const char *from = base + ro * kStageRow<TO, D> + co * sizeof(TO);
            const int rows = co < p.dv ? m - ro : 0;
#pragma unroll
            for (int i = 0; i < kT / RO; ++i, o += hop)
                if (i * RO < rows)
                    *reinterpret_cast<uint4 *>(o) =
                        *reinterpret_cast<const uint4 *>(from + i * RO * kStageRow<TO, D>);
            zero = false;
        }
    }
    if (O) {
        // zeros past the sequence, in this segment's rows
        TO *o = static_cast<TO *>(p.o) + (b * p.length * p.heads + h) * p.dv;
        const int64_t from = max(n, first), to = min(p.length, first + ca.seg_len);
        const Pack<TO, 8> none = {};
        for (int64_t t = from + r0 + (half ? RS : 0); t < to; t += 2 * RS)
            if (pc * 8 < p.dv)
                *reinterpret_cast<Pack<TO, 8> *>(o + t * p.heads * p.dv + pc * 8) = none;
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kCols));
}

template <typename T, typename TO, int D, bool REV, int KT>
fno_status_t run(const fno_linattn_s &p, const TcArgs &ca, cudaStream_t s) {
    const int64_t bh = p.batch * ca.s.heads;
    const auto go = [&](auto kernel, int threads, size_t smem) {
        smem += 1024;
        if (raise_smem_limit(kernel, smem) != cudaSuccess) return FNO_ERR_CUDA;
        kernel<<<(unsigned)(bh * ca.segments), threads, smem, s>>>(ca);
        return launched();
    };
    if (ca.segments > 1 && !ca.s.states_t) {
        fno_status_t st = go(k_linattn_tc<T, T, D, REV, false, KT>, 256,
                             operand_bytes<T, T, D, false, KT>());
        if (st == FNO_OK && ca.joined()) st = segment_states(p, ca.s, ca.states, s);
        if (st != FNO_OK) return st;
    }
    return go(k_linattn_tc<T, TO, D, REV, true, KT>, 512, operand_bytes<T, TO, D, true, KT>());
}

template <typename T, int D, int KT>
fno_status_t directions(const fno_linattn_s &p, const TcArgs &ca, bool rev, bool wide_out,
                        cudaStream_t s) {
    if (!rev) return run<T, T, D, false, KT>(p, ca, s);
    if (wide_out) return run<T, float, D, true, KT>(p, ca, s);
    return run<T, T, D, true, KT>(p, ca, s);
}

}  // namespace

// Rows of whole 16-byte pieces; bfloat16 up to 128 columns, float32 and fp16, whose
// terms take three and two times the room, up to 64.
bool tc_applies(const fno_linattn_s &p) {
    const int most = p.dtype == FNO_BF16 ? 128 : 64;
    return p.dk <= most && p.dv <= most && p.dk % 8 == 0 && p.dv % 8 == 0;
}

// CTAs an SM holds (tensor memory and shared memory): two of the 64-wide bfloat16
int tc_ctas(const fno_linattn_s &p) {
    return p.dtype == FNO_BF16 && p.dk <= 64 && p.dv <= 64 ? 2 : 1;
}

fno_status_t tc_scan(const fno_linattn_s &p, const ScanArgs &a, bool rev, bool wide_out,
                     float *states, float scale_p, cudaStream_t s) {
    const TcArgs ca{a, states, p.segments, p.seg_len, scale_p, p.dev_err};
    if (p.dtype == FNO_F32) return directions<float, 64, 3>(p, ca, rev, wide_out, s);
    if (p.dtype == FNO_F16) return directions<__half, 64, 3>(p, ca, rev, wide_out, s);
    const bool exact = a.sT || a.exact;
    if (a.dk <= 64 && a.dv <= 64)
        return exact ? directions<__nv_bfloat16, 64, 3>(p, ca, rev, wide_out, s)
                     : directions<__nv_bfloat16, 64, 2>(p, ca, rev, wide_out, s);
    return exact ? directions<__nv_bfloat16, 128, 3>(p, ca, rev, wide_out, s)
                 : directions<__nv_bfloat16, 128, 2>(p, ca, rev, wide_out, s);
}

}  // namespace linattn
}  // namespace fno
