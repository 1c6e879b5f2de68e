// fno_linattn.h -- what the linear attention's translation units share.
#pragma once

#include "fno_ops_internal.h"

struct fno_linattn_s {
    int64_t batch, length;
    int heads, kv_heads, dk, dv;
    fno_dtype_t dtype;
    uint32_t flags;
    int sms;
    int *dev_err;
    size_t workspace;
    size_t group_off[2];     // backward with shared heads: dk, dv of every query head
    int segments;            // parts of the time axis that run side by side
    int64_t seg_len;
};

namespace fno {
namespace linattn {

constexpr int kMaxWidth = 256;
constexpr int kChunkWidth = 128;     // widest key of the chunked kernel
constexpr int kC = 64;               // tokens of a chunk

// A scan's operands: queries, keys and values of the scan (which the gradients
// take from other tensors than the forward).
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
    // tcgen05 scans: the segments' states are those that the scan before left, of
    // the same sums with keys and values exchanged; the states are wanted to
    // float32's digits although this scan returns none
    bool states_t, exact;
    // tcgen05 scans: s0 may be written by this call (it is sT), so that only a launch
    // before the outputs' reads it
    bool joined;
};

// One scan: in chunks up to 128 key columns, token by token beyond.  rev: from the
// last token; wide_out: the output is float32 whatever the storage type; scale_p:
// of the products of queries and keys.
template <typename T>
fno_status_t scan_of(const fno_linattn_s &p, const ScanArgs &a, bool rev, bool wide_out,
                     float *states, float scale_p, cudaStream_t s);
// The states in front of the segments from their local ones, in place (and from
// a.s0).
fno_status_t segment_states(const fno_linattn_s &p, const ScanArgs &a, float *states,
                            cudaStream_t s);
// The bfloat16 scans on tcgen05: whether a plan's widths allow them, the CTAs an
// SM holds, and the scan.
bool tc_applies(const fno_linattn_s &p);
int tc_ctas(const fno_linattn_s &p);
fno_status_t tc_scan(const fno_linattn_s &p, const ScanArgs &a, bool rev, bool wide_out,
                     float *states, float scale_p, cudaStream_t s);
// CTAs of the chunked kernel that an SM holds.
template <typename T> fno_status_t chunk_occupancy_of(const fno_linattn_s &p, int *ctas);

}  // namespace linattn
}  // namespace fno
