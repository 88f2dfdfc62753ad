// The block norm: the residual stream between one block and the next.
//   p = P(f)              post-norm of the block's output (none, RMS, LayerNorm)
//   y = a x + c g p       residual scale a, block scale c, gate g (none, per
//                         channel, per token, per element)
//   n = N(y)              the next block's pre-norm, of y as it is stored
// and the gradients of x, f, g and the norms' parameters from dy and dn.  With
//   fh = (f - mean) rstd, yh = (y - mean) rstd   (the forward's statistics),
//   h = dn wn,  D = dy + rstd (h - [mean(h)] - yh mean(h yh))
//   dx = a D,   dp = c g D,   hp = dp wp,
//   df = rstd (hp - [mean(hp)] - fh mean(hp fh))
// (the bracketed means belong to LayerNorm alone) and the sums over tokens
//   P1 = sum_m e fh, P0 = sum_m e, N1 = sum_m dn yh, N0 = sum_m dn, where e is
//   D times the token's or element's gate,
// from which dwp = c g P1, dbp = c g P0, dg = c (wp P1 + bp P0) (channel
// gate), dwn = N1 and dbn = N0 (g: the channel gate, else 1).
// Everything is one pass over the rows; sums, statistics and products are fp32.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <mutex>
#include <new>

#include "block_norm.cuh"

#define TRY(x)                        \
    do {                              \
        tp_status _s = (x);           \
        if (_s != TP_OK) return _s;   \
    } while (0)

namespace tpmlp {
namespace bn {

// ---------------------------------------------------------------------------
// Parameter gradients from the partial rows, which are still in L2: 16 columns a
// block, so that there are blocks for all SMs, and 64 threads down the rows of
// a column quadruple, the rows in a fixed order.  304 rows of two sums over 4096
// columns: 4 to 5 us after the backward, whose end its start overlaps.
// ---------------------------------------------------------------------------
constexpr int kFinalCols = 16;
struct FinalPlan {
    const float *partials;
    int chunks, H, use[4], zero_centered;
    float c;
    const void *post_w, *post_b, *gate;  // gate: the channel gate, or null
    float *dpost_w, *dpost_b, *dpre_w, *dpre_b, *dgate;
};

template <typename A>
__global__ void __launch_bounds__(256) param_grad_kernel(const __grid_constant__ FinalPlan p) {
    __shared__ float part[4][64][kFinalCols + 1];
    const int quad = threadIdx.x & 3, r = threadIdx.x >> 2;
    const int c0 = blockIdx.x * kFinalCols + quad * 4;  // H is a multiple of 8: a quadruple is whole or absent
    float4 s[4];
    const float *in[4];
    int slot = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        s[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        in[q] = p.partials + static_cast<long long>(slot) * p.chunks * p.H + c0;
        slot += p.use[q];
    }
    wait_for_stream();
    let_next_start();
    if (c0 < p.H)
#pragma unroll 2
        for (int i = r; i < p.chunks; i += 64)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (p.use[q]) {
                    const float4 v = *reinterpret_cast<const float4 *>(in[q] + static_cast<long long>(i) * p.H);
                    s[q].x += v.x; s[q].y += v.y; s[q].z += v.z; s[q].w += v.w;
                }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        part[q][r][quad * 4] = s[q].x;
        part[q][r][quad * 4 + 1] = s[q].y;
        part[q][r][quad * 4 + 2] = s[q].z;
        part[q][r][quad * 4 + 3] = s[q].w;
    }
    __syncthreads();
    // 16 lanes a column: 4 rows each, then over the lanes
    const int own = threadIdx.x >> 4, part_of = threadIdx.x & 15, col = blockIdx.x * kFinalCols + own;
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[q] += part[q][part_of * 4 + i][own];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v[q] += __shfl_xor_sync(0xffffffffu, v[q], o);
    }
    if (part_of || col >= p.H) return;
    const float g = p.gate ? load1<A>(p.gate, col) : 1.0f;
    if (p.dpost_w) p.dpost_w[col] = p.c * g * v[0];
    if (p.dpost_b) p.dpost_b[col] = p.c * g * v[1];
    if (p.dgate) {
        float t = v[0];
        if (p.post_w) t *= load1<A>(p.post_w, col) + (p.zero_centered ? 1.0f : 0.0f);
        if (p.post_b) t = fmaf(load1<A>(p.post_b, col), v[1], t);
        p.dgate[col] = p.c * t;
    }
    if (p.dpre_w) p.dpre_w[col] = v[2];
    if (p.dpre_b) p.dpre_b[col] = v[3];
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// How a row is taken, from its width and the bytes an element has in a stage
// (those that the kernel reads).
//   Up to 512 columns: by a warp, 8 or 16 elements a lane.
//   Wider, forward: by a block, 16 elements a thread (8192 x 4096 bf16 with two
//   LayerNorms: 56 us, 64 us with 8), above 8192 columns 32 (2048 x 16384 with
//   one RMS norm: 46 us, 86 us by a cluster).
//   Wider, backward: by a block, 8 elements a thread while its threads suffice
//   (its column sums take as many registers again: 8192 x 4096 with two
//   LayerNorms 78 us, 90 us with 16; fp32 126 us, 196 us with 16), else 16.
//   Where a block's threads or its shared memory do not hold a row: by a
//   cluster of 2 or 4 blocks.  Its barriers cost dear (8192 x 4096 bf16 forward:
//   84 us with 2 blocks, 48 us with one), so it is the last resort: above 8192
//   columns in the backward, and wherever two rows of all arrays exceed an SM's
//   shared memory.  In the backward that is fp32 from 6616 columns (5192 with an
//   element gate) and an fp32 stream with an element gate from 7632; in the
//   forward fp32 from 13224 (8472 with an element gate) and an fp32 stream with an
//   element gate from 13224.
static Shape shape_of(int H, int bytes, bool bwd) {
    Shape s = {};
    s.cluster = 1;
    s.E = H <= 256 ? 8 : 16;
    s.threads = 32 * kWarps;
    s.team = H <= 512 && kStages * s.threads * s.E * bytes <= kSmemMost ? kWarp : kBlock;
    if (s.team != kWarp) {
        const int most = bwd ? 16 : 32;  // elements a thread
        while (H > s.cluster * kMaxThreads * most || kStages * bytes * ((H + s.cluster - 1) / s.cluster + 32 * most) > kSmemMost)
            s.cluster *= 2;
        if (s.cluster > 1) s.team = kCluster;
        const int cols = (H + s.cluster - 1) / s.cluster;
        s.E = bwd && s.team == kBlock && cols <= kMaxThreads * 8 ? 8 : cols <= kMaxThreads * 16 ? 16 : 32;
        s.threads = ((cols + s.E - 1) / s.E + 31) / 32 * 32;
    }
    s.smem = kStages * s.threads * s.E * bytes;
    if (s.team == kWarp && s.smem < kWarps * s.E * 32 * 4) s.smem = kWarps * s.E * 32 * 4;  // the warps' sums at the end
    return s;
}

// A kernel and how many of its blocks an SM holds; the handle keeps the last
// device's, so that a call does not ask the runtime again.
struct Launch {
    Kernel k = nullptr;
    Shape s;
    int per_sm = 0, device = -1;
};
static std::mutex g_launch_mutex;

static tp_status prepare(Launch &kept, const tp_block_norm_desc &d, bool bwd, bool has_dy, int bytes, Launch &l) {
    int dev = 0;
    TRY(cuda_check(cudaGetDevice(&dev), "cudaGetDevice"));
    std::lock_guard<std::mutex> lock(g_launch_mutex);
    l = kept;
    if (l.device == dev) return TP_OK;
    l.s = shape_of(d.H, bytes, bwd);
    l.s.common = !d.seq_parallel && d.has_block && d.pre != TP_NORM_NONE && d.gate <= TP_GATE_CHANNEL &&
                 (!bwd || has_dy);
    l.k = d.dtype == TP_DT_F32  ? (bwd ? bwd_kernel_f32(d, l.s) : fwd_kernel_f32(d, l.s))
          : d.residual_f32      ? (bwd ? bwd_kernel_mixed(d, l.s) : fwd_kernel_mixed(d, l.s))
                                : (bwd ? bwd_kernel_bf16(d, l.s) : fwd_kernel_bf16(d, l.s));
    // the most any configuration takes: the attribute is the kernel's, and another handle's may need more
    TRY(cuda_check(cudaFuncSetAttribute(l.k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost), "block norm"));
    TRY(cuda_check(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&l.per_sm, l.k, l.s.threads, l.s.smem), "block norm"));
    if (l.per_sm < 1) return set_error(TP_ERR_CUDA, "block norm: no block fits an SM");
    l.device = dev;
    kept = l;
    return TP_OK;
}

static tp_status run(const Launch &l, Plan &p, int most, const char *name, cudaStream_t st, int *workers) {
    const Shape &s = l.s;
    const int rows = s.team == kWarp ? kWarps : 1;
    int blocks = l.per_sm * num_sms() / s.cluster;
    if (blocks > (p.M + rows - 1) / rows) blocks = (p.M + rows - 1) / rows;
    if (most && blocks > most) blocks = most;
    if (blocks < 1) blocks = 1;
    p.cluster = s.cluster;
    *workers = blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks * s.cluster);
    cfg.blockDim = dim3(s.threads);
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (pdl_on()) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (s.cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = s.cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    launch_begin(name, st);
    cudaError_t e = cudaLaunchKernelEx(&cfg, l.k, p);
    launch_end(name, st);
    return cuda_check(e, name);
}

}  // namespace bn
}  // namespace tpmlp

using namespace tpmlp;

struct tp_block_norm {
    tp_block_norm_desc d;
    int M, nx, rows_split;
    int use[4];
    bn::Launch fwd, bwd, bwd_alone;  // bwd_alone: without dY
};

static tp_status bn_pointer(const void *p, const char *name, int i, int n, unsigned align = 16) {
    char at[16] = "";
    if (n > 1) snprintf(at, sizeof(at), "[%d]", i);
    if (!p) return set_error(TP_ERR_ARG, "%s%s is NULL", name, at);
    if (reinterpret_cast<uintptr_t>(p) & (align - 1))
        return set_error(TP_ERR_ARG, "%s%s is not %u-byte aligned", name, at, align);
    return TP_OK;
}

// copies an array of n pointers into a plan after checking them
template <typename P>
static tp_status bn_array(P *const *in, int n, const char *name, P **out, unsigned align = 16) {
    if (!in) return set_error(TP_ERR_ARG, "%s: pointer array is NULL", name);
    for (int i = 0; i < n; ++i) {
        TRY(bn_pointer(in[i], name, i, n, align));
        out[i] = in[i];
    }
    return TP_OK;
}

static tp_status bn_validate(const tp_block_norm_desc *d) {
    if (!d) return set_error(TP_ERR_ARG, "descriptor is NULL");
    if (d->dtype != TP_DT_F32 && d->dtype != TP_DT_BF16)
        return set_error(TP_ERR_ARG, "bad dtype %d (the block norm takes TP_DT_F32 and TP_DT_BF16)", d->dtype);
    const int flags[4] = {d->residual_f32, d->seq_parallel, d->has_block, d->zero_centered};
    for (int f : flags)
        if (f != 0 && f != 1) return set_error(TP_ERR_ARG, "boolean flags must be 0 or 1");
    if (d->post < TP_NORM_NONE || d->post > TP_NORM_LAYER) return set_error(TP_ERR_ARG, "bad post norm %d", d->post);
    if (d->pre < TP_NORM_NONE || d->pre > TP_NORM_LAYER) return set_error(TP_ERR_ARG, "bad pre norm %d", d->pre);
    if (d->gate < TP_GATE_NONE || d->gate > TP_GATE_ELEMENT) return set_error(TP_ERR_ARG, "bad gate %d", d->gate);
    if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return set_error(TP_ERR_ARG, "eps must be positive and finite");
    if (!std::isfinite(d->residual_scale) || !std::isfinite(d->block_scale))
        return set_error(TP_ERR_ARG, "residual_scale and block_scale must be finite");
    if (!d->has_block) {
        if (d->pre == TP_NORM_NONE) return set_error(TP_ERR_ARG, "without a block there has to be a pre-norm");
        if (d->post != TP_NORM_NONE || d->gate != TP_GATE_NONE || d->residual_scale != 1.0f || d->block_scale != 1.0f)
            return set_error(TP_ERR_ARG, "post norm, gate and scales belong to a block (has_block = 1)");
    }
    if (d->T < 1 || d->T > TP_MAX_SHARDS)
        return set_error(TP_ERR_SHAPE, "T=%d outside 1..%d", d->T, TP_MAX_SHARDS);
    if (d->S < 0 || d->B < 0) return set_error(TP_ERR_SHAPE, "negative S or B");
    const long long M = static_cast<long long>(d->S) * d->B;
    if (M > (1ll << 24)) return set_error(TP_ERR_SHAPE, "M = S*B = %lld exceeds 2^24 tokens", M);
    if (d->H < 8 || d->H % 8) return set_error(TP_ERR_SHAPE, "H=%d must be a positive multiple of 8", d->H);
    if (d->H > bn::kMaxH) return set_error(TP_ERR_UNSUPPORTED, "H=%d above the kernels' row capacity %d", d->H, bn::kMaxH);
    if (d->seq_parallel && d->S % d->T)
        return set_error(TP_ERR_SHAPE, "sequence parallel needs S %% T == 0 (S=%d, T=%d)", d->S, d->T);
    return TP_OK;
}

static bn::Plan bn_plan(const tp_block_norm *h) {
    bn::Plan p = {};
    const tp_block_norm_desc &d = h->d;
    p.M = h->M;
    p.H = d.H;
    p.rows_split = h->rows_split;
    p.post = d.post;
    p.pre = d.pre;
    p.gate = d.gate;
    p.zero_centered = d.zero_centered;
    p.has_block = d.has_block;
    p.eps = d.eps;
    p.a = d.residual_scale;
    p.c = d.block_scale;
    for (int i = 0; i < 4; ++i) p.use[i] = h->use[i];
    return p;
}

// a token gate is read value by value: its shards need no more than a value's alignment
static unsigned bn_gate_align(const tp_block_norm *h) {
    return h->d.gate != TP_GATE_TOKEN ? 16 : h->d.dtype == TP_DT_F32 ? 4 : 2;
}

static tp_status bn_gate(const tp_block_norm *h, const void *const *gate, bn::Plan &p) {
    if (h->d.gate == TP_GATE_NONE) return TP_OK;
    return bn_array(gate, h->d.gate == TP_GATE_CHANNEL ? 1 : h->nx, "gate", p.g, bn_gate_align(h));
}

extern "C" {

tp_status tp_block_norm_create(const tp_block_norm_desc *desc, tp_block_norm **out) {
    if (!out) return set_error(TP_ERR_ARG, "out is NULL");
    *out = nullptr;
    TRY(bn_validate(desc));
    tp_block_norm *h = new (std::nothrow) tp_block_norm;
    if (!h) return set_error(TP_ERR_ARG, "out of host memory");
    h->d = *desc;
    h->M = desc->S * desc->B;
    h->nx = desc->seq_parallel ? desc->T : 1;
    h->rows_split = desc->seq_parallel ? h->M / desc->T : 0;
    h->use[0] = desc->post != TP_NORM_NONE || desc->gate == TP_GATE_CHANNEL;
    h->use[1] = desc->post == TP_NORM_LAYER;
    h->use[2] = desc->pre != TP_NORM_NONE;
    h->use[3] = desc->pre == TP_NORM_LAYER;
    *out = h;
    return TP_OK;
}

void tp_block_norm_destroy(tp_block_norm *h) { delete h; }

size_t tp_block_norm_workspace_bytes(const tp_block_norm *h) {
    if (!h) return 0;
    const int sums = h->use[0] + h->use[1] + h->use[2] + h->use[3];
    const int most = bn::max_chunks(h->d.H), chunks = h->M < most ? h->M : most;
    return sizeof(float) * sums * chunks * static_cast<size_t>(h->d.H);
}

tp_status tp_block_norm_fwd(tp_block_norm *h, const void *const *X, const void *const *F, const void *const *gate,
                            const void *post_w, const void *post_b, const void *pre_w, const void *pre_b,
                            void *const *Y, void *const *N, float *stats, void *stream) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    const tp_block_norm_desc &d = h->d;
    bn::Plan p = bn_plan(h);
    if (h->M == 0) return TP_OK;
    TRY(bn_array(X, h->nx, "X", p.x));
    if (d.has_block) {
        TRY(bn_array(F, h->nx, "F", p.f));
        TRY(bn_array(Y, h->nx, "Y", p.y));
        TRY(bn_gate(h, gate, p));
    }
    if (d.post != TP_NORM_NONE) TRY(bn_pointer(p.post_w = post_w, "post_w", 0, 1));
    if (d.post == TP_NORM_LAYER) TRY(bn_pointer(p.post_b = post_b, "post_b", 0, 1));
    if (d.pre != TP_NORM_NONE) {
        TRY(bn_pointer(p.pre_w = pre_w, "pre_w", 0, 1));
        TRY(bn_array(N, h->nx, "N", p.n));
    }
    if (d.pre == TP_NORM_LAYER) TRY(bn_pointer(p.pre_b = pre_b, "pre_b", 0, 1));
    if (stats) TRY(bn_pointer(p.stats = reinterpret_cast<float4 *>(stats), "stats", 0, 1));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int ea = d.dtype == TP_DT_F32 ? 4 : 2, er = d.residual_f32 ? 4 : ea;
    bn::Launch l;
    TRY(bn::prepare(h->fwd, d, false, false, er + (d.has_block ? ea : 0) + (d.gate == TP_GATE_ELEMENT ? ea : 0), l));
    int workers;
    return bn::run(l, p, 0, "block_norm_fwd", st, &workers);
}

tp_status tp_block_norm_bwd(tp_block_norm *h, const void *const *dY, const void *const *dN, const void *const *Y,
                            const void *const *F, const void *const *gate, const void *post_w, const void *post_b,
                            const void *pre_w, const float *stats, void *const *dX, void *const *dF,
                            void *const *dgate, float *dpost_w, float *dpost_b, float *dpre_w, float *dpre_b,
                            void *workspace, size_t workspace_bytes, void *stream) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    const tp_block_norm_desc &d = h->d;
    bn::Plan p = bn_plan(h);
    bn::FinalPlan fin = {};
    if (d.pre != TP_NORM_NONE) {
        TRY(bn_pointer(p.pre_w = pre_w, "pre_w", 0, 1));
        TRY(bn_pointer(fin.dpre_w = dpre_w, "dpre_w", 0, 1));
    }
    if (d.pre == TP_NORM_LAYER) TRY(bn_pointer(fin.dpre_b = dpre_b, "dpre_b", 0, 1));
    if (d.post != TP_NORM_NONE) {
        TRY(bn_pointer(p.post_w = post_w, "post_w", 0, 1));
        TRY(bn_pointer(fin.dpost_w = dpost_w, "dpost_w", 0, 1));
    }
    if (d.post == TP_NORM_LAYER) {
        TRY(bn_pointer(p.post_b = post_b, "post_b", 0, 1));
        TRY(bn_pointer(fin.dpost_b = dpost_b, "dpost_b", 0, 1));
    }
    if (d.gate == TP_GATE_CHANNEL) {
        TRY(bn_gate(h, gate, p));
        void *dg[1];
        TRY(bn_array(dgate, 1, "dgate", dg));
        fin.dgate = static_cast<float *>(dg[0]);
    }
    if (h->M > 0) {
        if (dY || d.pre == TP_NORM_NONE) TRY(bn_array(dY, h->nx, "dY", p.dy));
        TRY(bn_array(dX, h->nx, "dX", p.dx));
        if (d.pre != TP_NORM_NONE) {
            TRY(bn_array(dN, h->nx, "dN", p.dn));
            TRY(bn_array(Y, h->nx, "Y", p.y_in));
        }
        if (d.has_block) {
            if (d.post != TP_NORM_NONE || d.gate != TP_GATE_NONE) TRY(bn_array(F, h->nx, "F", p.f));
            TRY(bn_array(dF, h->nx, "dF", p.df));
        }
        if (d.gate == TP_GATE_TOKEN || d.gate == TP_GATE_ELEMENT) {
            TRY(bn_gate(h, gate, p));
            TRY(bn_array(dgate, h->nx, "dgate", p.dg, bn_gate_align(h)));
        }
        TRY(bn_pointer(p.stats_in = reinterpret_cast<const float4 *>(stats), "stats", 0, 1));
    }
    const size_t need = tp_block_norm_workspace_bytes(h);
    if (need) {
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
            return set_error(TP_ERR_ARG, "workspace is NULL or not 256-byte aligned");
        if (workspace_bytes < need)
            return set_error(TP_ERR_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.partials = static_cast<float *>(workspace);
    int grid = 0;
    if (h->M > 0) {
        const int ea = d.dtype == TP_DT_F32 ? 4 : 2, er = d.residual_f32 ? 4 : ea;
        p.need_f = d.has_block && (d.post != TP_NORM_NONE || d.gate != TP_GATE_NONE);
        const bool pre = d.pre != TP_NORM_NONE;
        bn::Launch l;
        TRY(bn::prepare(dY ? h->bwd : h->bwd_alone, d, true, dY != nullptr,
                        er + (pre ? er + ea : 0) + (p.need_f ? ea : 0) + (d.gate == TP_GATE_ELEMENT ? ea : 0), l));
        TRY(bn::run(l, p, bn::max_chunks(d.H), "block_norm_bwd", st, &grid));
    }
    if (!h->use[0] && !h->use[2]) return TP_OK;
    fin.partials = p.partials;
    fin.chunks = grid;
    fin.H = d.H;
    for (int i = 0; i < 4; ++i) fin.use[i] = h->use[i];
    fin.zero_centered = d.zero_centered;
    fin.c = d.block_scale;
    fin.post_w = p.post_w;
    fin.post_b = p.post_b;
    fin.gate = d.gate == TP_GATE_CHANNEL ? p.g[0] : nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((d.H + bn::kFinalCols - 1) / bn::kFinalCols);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_on() && grid ? 1 : 0;
    launch_begin("block_norm_param_grads", st);
    cudaError_t e = d.dtype == TP_DT_F32 ? cudaLaunchKernelEx(&cfg, bn::param_grad_kernel<float>, fin)
                                         : cudaLaunchKernelEx(&cfg, bn::param_grad_kernel<__nv_bfloat16>, fin);
    launch_end("block_norm_param_grads", st);
    return cuda_check(e, "block_norm_param_grads");
}

}  // extern "C"
