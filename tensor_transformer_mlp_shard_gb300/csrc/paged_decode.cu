// Decode attention over a paged cache: the choice of kernels, the workspace and
// the join of rows that several blocks read.
#include "paged_decode.cuh"

namespace tpmlp {
namespace attn {

// How a key head's queries are cut into groups, each of which reads the keys:
// up to 16 to the columns of the matrix instructions.  Above 128 elements a head
// codes and fp32 take up to 8: with 16 the outputs leave a lane no registers for
// the conversions (100 rows of 128 heads x 256 over 8: 8-bit 30 us in two passes,
// 41 in one; bf16 42 and 41, and with 64 rows of up to 8000 positions 646 and 400,
// although 16 queries of 256 elements spill some 530 bytes a thread, of 192 some 260).
static void cut_queries(int dtype, int D, int per, int *groups, int *nh) {
    const int most = dtype == TP_DT_BF16 || D <= 128 ? 16 : 8;
    *groups = (per + most - 1) / most;
    *nh = (per + *groups - 1) / *groups;
}

static size_t partial_bytes(int nh, int D) {
    return (static_cast<size_t>(kMostBlocks) * 2 * part_floats(nh, D) * sizeof(float) + 255) / 256 * 256;
}

size_t decode_workspace_bytes(const tp_paged_desc &d) {
    int groups, nh;
    cut_queries(d.dtype, d.head_dim, d.heads / d.kv_heads, &groups, &nh);
    return partial_bytes(nh, d.head_dim) + kMostBlocks * sizeof(int4);
}

template <typename Act>
static tp_status launch_join(DecodePlan &p, int grid, cudaStream_t st) {
    const long long segments = static_cast<long long>(p.at.n) * p.row_heads;
    const int entries = p.by_segment ? static_cast<int>(segments) : grid;
    // parts of a segment: with more than 8, 16 warps take them
    const bool many = segments * 8 < grid;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(entries, many ? p.nh : (p.nh + 3) / 4);
    cfg.blockDim = dim3(many ? 512 : 128);
    // a few blocks leave room for the next kernel's beside them
    p.join_early = static_cast<int>(cfg.gridDim.x * cfg.gridDim.y) <= num_sms();
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_on() ? 1 : 0;
    launch_begin("paged_decode_join", st);
    cudaError_t e = cudaLaunchKernelEx(&cfg, many ? join_kernel<Act, 16> : join_kernel<Act, 1>, p);
    launch_end("paged_decode_join", st);
    return cuda_check(e, "paged_decode_join");
}

tp_status launch_decode(DecodePlan &p, int dtype, void *workspace, cudaStream_t st) {
    cut_queries(dtype, p.D, p.per, &p.groups, &p.nh);
    p.row_heads *= p.groups;
    p.by_hk = Divisor(p.hk);
    p.by_groups = Divisor(p.groups);
    p.partial = static_cast<float *>(workspace);
    p.joins = reinterpret_cast<int4 *>(static_cast<char *>(workspace) + partial_bytes(p.nh, p.D));
    int grid = 0;
    tp_status s = dtype == TP_DT_F32   ? launch_decode_f32(p, &grid, st)
                  : dtype == TP_DT_FP8 ? launch_decode_fp8(p, &grid, st)
                                       : launch_decode_bf16(p, &grid, st);
    if (s != TP_OK || grid == 0) return s;
    return dtype == TP_DT_F32 ? launch_join<float>(p, grid, st) : launch_join<__nv_bfloat16>(p, grid, st);
}

}  // namespace attn
}  // namespace tpmlp
