// The block norm's backward kernels, bf16 with an fp32 stream.
#include "block_norm_bwd.cuh"

namespace tpmlp {
namespace bn {

Kernel bwd_kernel_mixed(const tp_block_norm_desc &d, const Shape &s) {
    return s.common ? of_types<__nv_bfloat16, float, true>(d, s) : of_types<__nv_bfloat16, float, false>(d, s);
}

}  // namespace bn
}  // namespace tpmlp
