// fno_linattn_bf16.cu -- the linear attention's scans for bf16 storage.
#include "fno_linattn_chunk.h"

namespace fno {
namespace linattn {
template fno_status_t scan_of<__nv_bfloat16>(const fno_linattn_s &, const ScanArgs &, bool, bool, float *,
                                   float, cudaStream_t);
template fno_status_t chunk_occupancy_of<__nv_bfloat16>(const fno_linattn_s &, int *);
}  // namespace linattn
}  // namespace fno
