// fno_scan_bwd_bf16.cu -- the selective scan's gradients for this storage type.
#include "fno_scan_bwd.h"

namespace fno {
namespace scan {
template fno_status_t backward_of<__nv_bfloat16>(const fno_scan_s &, Args, cudaStream_t);
}  // namespace scan
}  // namespace fno
