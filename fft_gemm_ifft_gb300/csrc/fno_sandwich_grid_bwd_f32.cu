// fno_sandwich_grid_bwd_f32.cu -- the channels-first backward for f32 storage.
#include "fno_sandwich_grid_bwd.h"

namespace fno {
namespace sandwich {
template fno_status_t grid_backward_of<float>(const fno_sandwich_s &, const Args &, cudaStream_t);
template fno_status_t grid_shares_of<float>(const fno_sandwich_s &, int *);
}  // namespace sandwich
}  // namespace fno
