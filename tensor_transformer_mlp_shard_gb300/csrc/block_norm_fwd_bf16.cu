// The block norm's forward kernels, all in bf16.
#include "block_norm_fwd.cuh"

namespace tpmlp {
namespace bn {

Kernel fwd_kernel_bf16(const tp_block_norm_desc &d, const Shape &s) {
    return s.common ? of_types<__nv_bfloat16, __nv_bfloat16, true>(d, s) : of_types<__nv_bfloat16, __nv_bfloat16, false>(d, s);
}

}  // namespace bn
}  // namespace tpmlp
