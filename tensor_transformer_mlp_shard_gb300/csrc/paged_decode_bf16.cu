// Decode attention over a bf16 cache: the kernels by padded width and queries of a group.
#include "paged_decode.cuh"

namespace tpmlp {
namespace attn {

tp_status launch_decode_bf16(DecodePlan &p, int *grid, cudaStream_t st) {
    constexpr int kKind = CACHE_BF16;
    if (p.D <= 64)
        return p.nh <= 8 ? launch_core<TensorCore<kKind, 64, 1>>(p, grid, st) : launch_core<TensorCore<kKind, 64, 2>>(p, grid, st);
    if (p.D <= 128)
        return p.nh <= 8 ? launch_core<TensorCore<kKind, 128, 1>>(p, grid, st) : launch_core<TensorCore<kKind, 128, 2>>(p, grid, st);
    if (p.D <= 192)
        return p.nh <= 8 ? launch_core<TensorCore<kKind, 192, 1>>(p, grid, st) : launch_core<TensorCore<kKind, 192, 2>>(p, grid, st);
    return p.nh <= 8 ? launch_core<TensorCore<kKind, 256, 1>>(p, grid, st) : launch_core<TensorCore<kKind, 256, 2>>(p, grid, st);
}

}  // namespace attn
}  // namespace tpmlp
