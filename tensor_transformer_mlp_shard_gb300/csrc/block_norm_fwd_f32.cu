// The block norm's forward kernels, all in fp32.
#include "block_norm_fwd.cuh"

namespace tpmlp {
namespace bn {

Kernel fwd_kernel_f32(const tp_block_norm_desc &d, const Shape &s) {
    return s.common ? of_types<float, float, true>(d, s) : of_types<float, float, false>(d, s);
}

}  // namespace bn
}  // namespace tpmlp
