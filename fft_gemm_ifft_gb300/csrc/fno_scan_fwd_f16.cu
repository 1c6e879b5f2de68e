// fno_scan_fwd_f16.cu -- the selective scan forward for this storage type.
#include "fno_scan_fwd.h"

namespace fno {
namespace scan {
template fno_status_t forward_of<__half>(const fno_scan_s &, Args, cudaStream_t);
}  // namespace scan
}  // namespace fno
