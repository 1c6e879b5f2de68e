// fno_sandwich_grid_bwd.cu -- which backward kernel a channels-first field takes.
#include "fno_sandwich_grid_bwd.h"

namespace fno {
namespace sandwich {

// instantiated in fno_sandwich_grid_bwd_{f32,f16,bf16}.cu
extern template fno_status_t grid_backward_of<float>(const fno_sandwich_s &, const Args &,
                                                     cudaStream_t);
extern template fno_status_t grid_backward_of<__half>(const fno_sandwich_s &, const Args &,
                                                      cudaStream_t);
extern template fno_status_t grid_backward_of<__nv_bfloat16>(const fno_sandwich_s &, const Args &,
                                                             cudaStream_t);
extern template fno_status_t grid_shares_of<float>(const fno_sandwich_s &, int *);
extern template fno_status_t grid_shares_of<__half>(const fno_sandwich_s &, int *);
extern template fno_status_t grid_shares_of<__nv_bfloat16>(const fno_sandwich_s &, int *);

// Staged tiles while the channels fit 16 warps of up to four parts (512
// channels), two stages where two CTAs of them fit an SM; else tiles that are
// read again for each round.
Way grid_backward_way(const fno_sandwich_desc_t &d) {
    const int c = d.channels;
    int parts = 1;           // of a warp
    while (parts <= 4 && c > kTileC * 16 * parts) parts *= 2;
    if (parts <= 4) {
        const int warps = (int)ceil_div(c, kTileC * parts);
        const int stage = tile_stage(c, d.points, kTileP / parts, (int)elem_bytes(d.dtype),
                                     false, true, true, true, d.gate == FNO_GATE_FULL);
        const int most = (kSmemPerSm / 2 - 1024 - tile_rest(c, warps)) / stage;
        return Way{kStaged, parts, kTileC, warps, most >= 2 ? 2 : 1};
    }
    if (c <= kWideC) return Way{kWide, d.points % 2 == 0 ? 2 : 1, 0, kWideWarps, 0};
    return Way{kAny, 0, 0, 0, 0};
}

fno_status_t grid_shares(const fno_sandwich_s &p, int *ctas, int64_t *most) {
    *most = p.d.batch / p.segs *
            ceil_div(p.d.points, p.bwd.kind == kWide ? 32 * p.bwd.vec : kTileP / p.bwd.vec);
    return with_storage(p.d.dtype,
                        [&](auto t) { return grid_shares_of<decltype(t)>(p, ctas); });
}

fno_status_t grid_backward(const fno_sandwich_s &p, const Args &a, cudaStream_t s) {
    return with_storage(p.d.dtype,
                        [&](auto t) { return grid_backward_of<decltype(t)>(p, a, s); });
}

}  // namespace sandwich
}  // namespace fno
