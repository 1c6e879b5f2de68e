// fno_linattn_f16.cu -- the linear attention's scans for f16 storage.
#include "fno_linattn_chunk.h"

namespace fno {
namespace linattn {
template fno_status_t scan_of<__half>(const fno_linattn_s &, const ScanArgs &, bool, bool, float *,
                                   float, cudaStream_t);
template fno_status_t chunk_occupancy_of<__half>(const fno_linattn_s &, int *);
}  // namespace linattn
}  // namespace fno
