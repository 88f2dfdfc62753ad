// The forward kernels of the block norm (see block_norm.cu for the mathematics);
// each pair of types is compiled in a unit of its own (block_norm_fwd_*.cu).
#pragma once

#include "block_norm.cuh"

namespace tpmlp {
namespace bn {

// ---------------------------------------------------------------------------
// Forward.  A: type of f, g, n and the weights; R: type of x and y; E elements
// a thread, in vectors of V; LP, LN: the post- and the pre-norm is a LayerNorm.
// COMMON: there are a block and a pre-norm, no token or element gate and no
// token shards.
//
// A row is read once, lives in registers through both norms, and is written
// once, so HBM bounds the kernel: 8192 x 4096 bf16 (RMS, channel gate, RMS)
// takes 44 us, 6.2 TB/s of its 268 MB, 0.92 of a plain copy's rate; 16384 x
// 6144 with a LayerNorm, in 8 token shards, 142 us (5.7 TB/s, 0.85).  What is
// left is the launch and the chain of a row's two or three reductions (shuffles,
// a barrier, shuffles) with two blocks an SM to hide it: more and smaller
// blocks (80 registers) measured slower (46 and 171 us), as did short runs of
// rows dealt out by the hardware (54 and 175 us with 8 rows a block), whose
// blocks all start with the weights' loads.  Paired fp32 arithmetic is a
// quarter fewer instructions than single.
// ---------------------------------------------------------------------------
template <typename A, typename R, int E, Team TEAM, bool LP, bool LN, bool COMMON>
__global__ void __launch_bounds__(TEAM == kWarp ? 32 * kWarps : kMaxThreads) fwd_kernel(const __grid_constant__ Plan p) {
    constexpr bool WARP = TEAM == kWarp;
    constexpr int V = sizeof(R) == 2 ? 8 : 4, K = E / V, P = V / 2;
    __shared__ float red[2][3][kSlots];
    extern __shared__ __align__(16) uint8_t stages[];
    Reduce r = make_reduce<TEAM>(red, p);
    const Columns<K, V> c = make_columns<K, V, TEAM>(p, r);
    const int worker = WARP ? blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x / r.cluster;
    const int workers = WARP ? gridDim.x * kWarps : gridDim.x / r.cluster;
    const bool has_block = COMMON || p.has_block, has_pre = COMMON || p.pre != TP_NORM_NONE;
    const bool gate_rows = !COMMON && p.gate == TP_GATE_ELEMENT, token = !COMMON && p.gate == TP_GATE_TOKEN;
    const bool first = (WARP ? threadIdx.x & 31 : threadIdx.x) == 0 && r.rank == 0;
    const float inv_h = 1.0f / p.H, plus = p.zero_centered ? 1.0f : 0.0f;
    const uint32_t stage_bytes =
        blockDim.x * E * static_cast<uint32_t>(sizeof(R) + (has_block ? sizeof(A) : 0) + (gate_rows ? sizeof(A) : 0));
    const uint32_t base = smem_at(stages);
    Cursor next(p, worker, workers);
    auto fetch = [&](int slot) {
        if (next.row < p.M) {
            const int js = COMMON ? 0 : next.shard;
            const long long e = static_cast<long long>(next.local) * p.H;
            uint32_t at = base + slot * stage_bytes;
            at = stage<R>(at, static_cast<const R *>(p.x[js]) + e, c);
            if (has_block) at = stage<A>(at, static_cast<const A *>(p.f[js]) + e, c);
            if (gate_rows) stage<A>(at, static_cast<const A *>(p.g[js]) + e, c);
            next.advance(p);
        }
        copies_commit();
    };
    if (c.ragged) clear_stages(stages, kStages * stage_bytes);
    wait_for_stream();
    fetch(0);
    constexpr bool KEEP = E <= 16;  // 32 elements a thread leave no registers for them
    Factors<A, K, V, KEEP> pw, nw;       // the post-norm's, gate and block scale in it, and the pre-norm's
    Factors<A, K, V, KEEP && LP> pb;
    Factors<A, K, V, KEEP && LN> nb;
    pw.keep(p, c, p.post_w, plus, 1.0f, true);
    nw.keep(p, c, p.pre_w, plus, 1.0f, false);
    if (LP) pb.keep(p, c, p.post_b, 0.0f, 0.0f, true);
    if (LN) nb.keep(p, c, p.pre_b, 0.0f, 0.0f, false);
    int slot = 0;
    for (Cursor at_row(p, worker, workers); at_row.row < p.M; at_row.advance(p)) {
        fetch(slot ^ 1);  // into the slot of the row before
        const int js = COMMON ? 0 : at_row.shard;
        const long long e = static_cast<long long>(at_row.local) * p.H;
        const float gm = token ? load1<A>(p.g[js], at_row.local) : 1.0f;
        copies_wait();
        const uint8_t *at = stages + slot * stage_bytes;
        slot ^= 1;
        float2 y[K][P];
        staged<R>(at, c, y);
        float4 st = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
        if (has_block) {
            float2 f[K][P];
            staged<A>(at, c, f);
            if (p.post != TP_NORM_NONE) centre_row<TEAM, LP, V, K>(f, c, p.post, inv_h, p.eps, r, st.x, st.y);
            // y = a x + g (P(f) scaled): the row's factors first, then the channel's
            const float2 row_scale = both(LP ? st.y : st.y * gm);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float2 w[P], b[P];
                pw.get(p, c, k, p.post_w, plus, 1.0f, true, w);
                if (LP) pb.get(p, c, k, p.post_b, 0.0f, 0.0f, true, b);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    f[k][j] = __fmul2_rn(f[k][j], row_scale);
                    if (LP) f[k][j] = __fmul2_rn(__ffma2_rn(f[k][j], w[j], b[j]), both(gm));
                    y[k][j] = __fmul2_rn(y[k][j], both(p.a));
                }
                if (gate_rows) {
                    float2 g[P];
                    load<A, V>(at, (k * c.lanes + threadIdx.x) * V, g);
#pragma unroll
                    for (int j = 0; j < P; ++j) f[k][j] = __fmul2_rn(f[k][j], g[j]);
                }
#pragma unroll
                for (int j = 0; j < P; ++j)
                    y[k][j] = LP ? __fadd2_rn(f[k][j], y[k][j]) : __ffma2_rn(f[k][j], w[j], y[k][j]);
                const typename Pack<R, V>::Raw out = Pack<R, V>::pack(y[k]);
                if (c.on[k]) *reinterpret_cast<typename Pack<R, V>::Raw *>(static_cast<R *>(p.y[js]) + e + c.at(k)) = out;
                Pack<R, V>::unpack(out, y[k]);  // the pre-norm is of y as it is stored
            }
        }
        if (has_pre) {
            centre_row<TEAM, LN, V, K>(y, c, p.pre, inv_h, p.eps, r, st.z, st.w);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float2 w[P], b[P];
                nw.get(p, c, k, p.pre_w, plus, 1.0f, false, w);
                if (LN) nb.get(p, c, k, p.pre_b, 0.0f, 0.0f, false, b);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    y[k][j] = __fmul2_rn(y[k][j], both(st.w));
                    y[k][j] = LN ? __ffma2_rn(y[k][j], w[j], b[j]) : __fmul2_rn(y[k][j], w[j]);
                }
                if (c.on[k]) store<A, V>(static_cast<A *>(p.n[js]) + e, c.at(k), y[k]);
            }
        }
        if (p.stats && first) p.stats[at_row.row] = st;
    }
    let_next_start();
    if (TEAM == kCluster) cluster_sync();  // no block leaves while another may write into it
}

template <typename A, typename R, bool LP, bool LN, bool COMMON>
static Kernel pick(const Shape &s) {
    if (s.team == kWarp) return s.E == 8 ? fwd_kernel<A, R, 8, kWarp, LP, LN, COMMON> : fwd_kernel<A, R, 16, kWarp, LP, LN, COMMON>;
    // types whose widest row fits a block have no cluster
    if constexpr (kStages * (sizeof(R) + (COMMON ? 1 : 2) * sizeof(A)) * (kMaxH + 32 * 32) > kSmemMost)
        if (s.team == kCluster) return fwd_kernel<A, R, 16, kCluster, LP, LN, COMMON>;
    return s.E == 32 ? fwd_kernel<A, R, 32, kBlock, LP, LN, COMMON> : fwd_kernel<A, R, 16, kBlock, LP, LN, COMMON>;
}
template <typename A, typename R, bool COMMON>
static Kernel of_types(const tp_block_norm_desc &d, const Shape &s) {
    const bool lp = d.post == TP_NORM_LAYER, ln = d.pre == TP_NORM_LAYER;
    return lp ? (ln ? pick<A, R, true, true, COMMON>(s) : pick<A, R, true, false, COMMON>(s))
              : (ln ? pick<A, R, false, true, COMMON>(s) : pick<A, R, false, false, COMMON>(s));
}

}  // namespace bn
}  // namespace tpmlp
