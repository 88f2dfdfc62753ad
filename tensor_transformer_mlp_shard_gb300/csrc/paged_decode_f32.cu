// Decode attention over an fp32 cache: the kernels by padded width and queries of a group.
#include "paged_decode.cuh"

namespace tpmlp {
namespace attn {

template <int DP>
static tp_status launch_width(DecodePlan &p, int *grid, cudaStream_t st) {
    if constexpr (DP <= 128)
        if (p.nh > 8) return launch_core<Tf32Core<DP, 2>>(p, grid, st);
    return p.nh == 1   ? launch_core<FloatCore<DP, 1>>(p, grid, st)
           : p.nh == 2 ? launch_core<FloatCore<DP, 2>>(p, grid, st)
           : p.nh <= kFloatQueries ? launch_core<FloatCore<DP, 4>>(p, grid, st)
                       : launch_core<Tf32Core<DP, 1>>(p, grid, st);
}

tp_status launch_decode_f32(DecodePlan &p, int *grid, cudaStream_t st) {
    return p.D <= 64    ? launch_width<64>(p, grid, st)
           : p.D <= 96  ? launch_width<96>(p, grid, st)
           : p.D <= 128 ? launch_width<128>(p, grid, st)
           : p.D <= 192 ? launch_width<192>(p, grid, st)
                        : launch_width<256>(p, grid, st);
}

}  // namespace attn
}  // namespace tpmlp
