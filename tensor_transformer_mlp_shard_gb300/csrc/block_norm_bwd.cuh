// The backward kernels of the block norm (see block_norm.cu for the mathematics);
// each pair of types is compiled in a unit of its own (block_norm_bwd_*.cu).
#pragma once

#include "block_norm.cuh"

namespace tpmlp {
namespace bn {

// ---------------------------------------------------------------------------
// Gradients of x, f and of a token or element gate, row by row, and this
// worker's share of the column sums in registers.  LP, LN: the post- and the
// pre-norm is a LayerNorm.  COMMON: there are dy, a pre-norm and a block, no
// token or element gate and no token shards; without the branches and the
// pointer lookups for the rest a row takes a fifth fewer instructions.
//
// Bound by HBM as the forward is: dy, y, dn and f are read once and dx and df
// written once.  8192 x 4096 bf16 (RMS, channel gate, RMS) takes 67 us in this
// kernel and 74 us with the parameter gradients, 5.4 TB/s of 403 MB (0.81 of a
// plain copy's rate); 4096 x 8192 with an fp32 stream and a LayerNorm 98 and
// 102 us (5.9 TB/s, 0.88).  Two blocks of 64 registers an SM, where both norms
// are RMS: one block of 73 took 118 us, its two barriers a row idle the SM.
// The column sums stay in registers over all rows of a worker: 304 rows of
// partial sums for 4096 columns and more, 10 MB that do not leave L2.
// ---------------------------------------------------------------------------
template <typename A, typename R, int E, Team TEAM, bool LP, bool LN, bool COMMON>
__global__ void __launch_bounds__(TEAM == kWarp ? 32 * kWarps : kMaxThreads,
                                  COMMON && E == 8 && TEAM == kBlock && !LP && !LN ? 2 : 1) bwd_kernel(const __grid_constant__ Plan p) {
    constexpr bool WARP = TEAM == kWarp;
    constexpr int V = sizeof(R) == 2 ? 8 : 4, K = E / V, P = V / 2;
    __shared__ float red[2][3][kSlots];
    extern __shared__ __align__(16) uint8_t stages[];
    Reduce r = make_reduce<TEAM>(red, p);
    const Columns<K, V> c = make_columns<K, V, TEAM>(p, r);
    const int worker = WARP ? blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x / r.cluster;
    const int workers = WARP ? gridDim.x * kWarps : gridDim.x / r.cluster;
    const bool has_pre = COMMON || p.pre != TP_NORM_NONE, has_dy = COMMON || p.dy[0] != nullptr;
    const bool has_block = COMMON || p.has_block, need_f = p.need_f;
    const bool gate_rows = !COMMON && p.gate == TP_GATE_ELEMENT, token = !COMMON && p.gate == TP_GATE_TOKEN;
    const bool row_gate = gate_rows || token;
    const bool first = (WARP ? threadIdx.x & 31 : threadIdx.x) == 0 && r.rank == 0;
    const float inv_h = 1.0f / p.H, plus = p.zero_centered ? 1.0f : 0.0f;
    const uint32_t row_bytes = blockDim.x * E *
                               static_cast<uint32_t>((has_dy ? sizeof(R) : 0) + (has_pre ? sizeof(R) + sizeof(A) : 0) +
                                                     (need_f ? sizeof(A) : 0) + (gate_rows ? sizeof(A) : 0));
    const uint32_t base = smem_at(stages);
    Cursor next(p, worker, workers);
    auto fetch = [&](int slot) {
        if (next.row < p.M) {
            const int js = COMMON ? 0 : next.shard;
            const long long e = static_cast<long long>(next.local) * p.H;
            uint32_t at = base + slot * row_bytes;
            if (has_dy) at = stage<R>(at, static_cast<const R *>(p.dy[js]) + e, c);
            if (has_pre) {
                at = stage<R>(at, static_cast<const R *>(p.y_in[js]) + e, c);
                at = stage<A>(at, static_cast<const A *>(p.dn[js]) + e, c);
            }
            if (need_f) at = stage<A>(at, static_cast<const A *>(p.f[js]) + e, c);
            if (gate_rows) stage<A>(at, static_cast<const A *>(p.g[js]) + e, c);
            next.advance(p);
        }
        copies_commit();
    };
    if (c.ragged) clear_stages(stages, kStages * row_bytes);
    wait_for_stream();
    fetch(0);
    // kept unless four column sums of 16 fill the registers (4096 x 8192 bf16 with two LayerNorms: 94 us, kept 117 us;
    // with one, 72 us, not kept 80 us, and with an fp32 stream 102 us, not kept 131 us)
    constexpr bool KEEP = E == 8 || !LP || !LN || sizeof(A) == 4;
    Factors<A, K, V, KEEP> gw, nw;  // the post-norm's weight, gate and block scale in it, and the pre-norm's
    gw.keep(p, c, p.post_w, plus, 1.0f, true);
    nw.keep(p, c, p.pre_w, plus, 1.0f, false);
    float2 p1[K][P], n1[K][P], p0[LP ? K : 1][P], n0[LN ? K : 1][P];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j) p1[k][j] = n1[k][j] = p0[LP ? k : 0][j] = n0[LN ? k : 0][j] = both(0.0f);
    int slot = 0;
    float4 st_next = worker < p.M ? p.stats_in[worker] : make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    for (Cursor at_row(p, worker, workers); at_row.row < p.M; at_row.advance(p)) {
        fetch(slot ^ 1);  // into the slot of the row before
        const int js = COMMON ? 0 : at_row.shard;
        const long long e = static_cast<long long>(at_row.local) * p.H;
        const float4 st = st_next;
        if (at_row.row + workers < p.M) st_next = p.stats_in[at_row.row + workers];
        const float gm = token ? load1<A>(p.g[js], at_row.local) : 1.0f;
        copies_wait();
        const uint8_t *at = stages + slot * row_bytes;
        slot ^= 1;
        float2 d[K][P];  // dy, then D
        auto read_dy = [&](const uint8_t *&from) {
            if (has_dy) {
                staged<R>(from, c, d);
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int j = 0; j < P; ++j) d[k][j] = both(0.0f);
            }
        };
        // Under a pre-LayerNorm dy stays staged until the row's sums are known: with it in
        // registers the branch for rows far from zero spills (4096 x 8192 bf16: 79 us, 72 so)
        const uint8_t *at_dy = at;
        if (LN) {
            if (has_dy) at += K * c.lanes * V * sizeof(R);
        } else {
            read_dy(at);
        }
        if (has_pre) {
            float2 yh[K][P], h[K][P];
            float m0, m1, none;
            float2 s0 = both(0.0f), s1 = both(0.0f);
            staged<R>(at, c, yh);
            const uint8_t *at_dn = at;
            staged<A>(at, c, h);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float2 w[P];
                nw.get(p, c, k, p.pre_w, plus, 1.0f, false, w);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (LN) yh[k][j] = __fadd2_rn(yh[k][j], both(-st.z));
                    yh[k][j] = __fmul2_rn(yh[k][j], both(st.w));
                    n1[k][j] = __ffma2_rn(h[k][j], yh[k][j], n1[k][j]);  // h is zero past the row
                    if (LN) n0[LN ? k : 0][j] = __fadd2_rn(n0[LN ? k : 0][j], h[k][j]);
                    h[k][j] = __fmul2_rn(h[k][j], w[j]);
                    if (LN) s0 = __fadd2_rn(s0, h[k][j]);
                    s1 = __ffma2_rn(h[k][j], yh[k][j], s1);
                }
            }
            m0 = s0.x + s0.y;
            m1 = s1.x + s1.y;
            if (LN)
                row_sum<TEAM, false>(m0, m1, none, r);
            else
                row_sum<TEAM>(m1, r);
            m0 *= -st.w * inv_h;
            m1 *= -st.w * inv_h;
            if (LN && far_from_zero(st.z, st.w)) {
                // yh - rest in the place of yh: in the sum, in D below (its part that
                // the columns share joins m0) and in the column sums
                const float rest = mean_left<TEAM, V, K>(yh, c, inv_h, r);
                m1 = fmaf(-rest, m0, m1);
                m0 = fmaf(-rest, m1, m0);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float2 dn[P];
                    load<A, V>(at_dn, (k * c.lanes + threadIdx.x) * V, dn);
#pragma unroll
                    for (int j = 0; j < P; ++j) n1[k][j] = __ffma2_rn(dn[j], both(-rest), n1[k][j]);
                }
            }
            if (LN) read_dy(at_dy);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (LN) d[k][j] = __fadd2_rn(d[k][j], both(m0));
                    d[k][j] = __ffma2_rn(h[k][j], both(st.w), __ffma2_rn(yh[k][j], both(m1), d[k][j]));
                }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c.on[k]) {
                float2 o[P];
#pragma unroll
                for (int j = 0; j < P; ++j) o[j] = __fmul2_rn(d[k][j], both(p.a));
                store<R, V>(static_cast<R *>(p.dx[js]) + e, c.at(k), o);
            }
        if (!has_block) continue;
        float2 fh[K][P];
        float m0, m1, dg;
        float2 s0 = both(0.0f), s1 = both(0.0f), s2 = both(0.0f);
        if (need_f) {
            staged<A>(at, c, fh);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (LP) fh[k][j] = __fadd2_rn(fh[k][j], both(-st.x));
                    fh[k][j] = __fmul2_rn(fh[k][j], both(st.y));  // no post-norm: 1
                }
            if (LP && far_from_zero(st.x, st.y)) {
                const float rest = mean_left<TEAM, V, K>(fh, c, inv_h, r);
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int j = 0; j < P; ++j) fh[k][j] = __fadd2_rn(fh[k][j], both(-rest));
            }
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) fh[k][j] = both(0.0f);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (row_gate && c.on[k]) {  // its gradient is D times p = fh w + b
                float2 pv[P], w[P];
#pragma unroll
                for (int j = 0; j < P; ++j) pv[j] = fh[k][j];
                if (p.post != TP_NORM_NONE) {
                    load<A, V>(p.post_w, c.at(k), w);
#pragma unroll
                    for (int j = 0; j < P; ++j) pv[j] = __fmul2_rn(pv[j], __fadd2_rn(w[j], both(plus)));
                    if (LP) {
                        load<A, V>(p.post_b, c.at(k), w);
#pragma unroll
                        for (int j = 0; j < P; ++j) pv[j] = __fadd2_rn(pv[j], w[j]);
                    }
                }
                if (gate_rows) {
                    load<A, V>(at, (k * c.lanes + threadIdx.x) * V, w);
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        pv[j] = __fmul2_rn(__fmul2_rn(d[k][j], pv[j]), both(p.c));
                        d[k][j] = __fmul2_rn(d[k][j], w[j]);
                    }
                    store<A, V>(static_cast<A *>(p.dg[js]) + e, c.at(k), pv);
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        s2 = __ffma2_rn(d[k][j], pv[j], s2);
                        d[k][j] = __fmul2_rn(d[k][j], both(gm));
                    }
                }
            }
            float2 w[P];
            gw.get(p, c, k, p.post_w, plus, 1.0f, true, w);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                p1[k][j] = __ffma2_rn(d[k][j], fh[k][j], p1[k][j]);
                if (LP) p0[LP ? k : 0][j] = __fadd2_rn(p0[LP ? k : 0][j], d[k][j]);
                d[k][j] = __fmul2_rn(d[k][j], w[j]);  // the gradient of fh
                if (LP) s0 = __fadd2_rn(s0, d[k][j]);
                s1 = __ffma2_rn(d[k][j], fh[k][j], s1);
            }
        }
        m0 = s0.x + s0.y;
        m1 = s1.x + s1.y;
        dg = s2.x + s2.y;
        float none;
        if (token)
            row_sum<TEAM, true>(m0, m1, dg, r);
        else if (LP)
            row_sum<TEAM, false>(m0, m1, none, r);
        else if (p.post != TP_NORM_NONE)
            row_sum<TEAM>(m1, r);
        if (token && first) store1<A>(p.dg[js], at_row.local, p.c * dg);
        m0 *= -st.y * inv_h;
        m1 *= -st.y * inv_h;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c.on[k]) {
                float2 o[P];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    o[j] = __fmul2_rn(d[k][j], both(st.y));
                    if (LP) o[j] = __fadd2_rn(o[j], both(m0));
                    // without a post-norm df has no part of f, whatever f holds
                    if (LP || p.post != TP_NORM_NONE) o[j] = __ffma2_rn(fh[k][j], both(m1), o[j]);
                }
                store<A, V>(static_cast<A *>(p.df[js]) + e, c.at(k), o);
            }
    }
    let_next_start();  // the parameter gradients' blocks, on the SMs that are done
    // one row of partial sums a worker (the warps of a block added in order)
    const int out_row = WARP ? blockIdx.x : worker, out_rows = WARP ? gridDim.x : workers;
    int used = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (!p.use[q]) continue;
        float *out = p.partials + (static_cast<long long>(used++) * out_rows + out_row) * p.H;
        float2 (*acc)[P] = q == 0 ? p1 : q == 1 ? p0 : q == 2 ? n1 : n0;
        const bool whole = q == 0 || q == 2 || (q == 1 ? LP : LN);
        if (WARP) {
            // the stages' memory serves again: every row has been read
            float *comb = reinterpret_cast<float *>(stages);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j)
                    *reinterpret_cast<float2 *>(comb + (threadIdx.x >> 5) * E * 32 + c.at(k) + 2 * j) = acc[whole ? k : 0][j];
            __syncthreads();
            for (int i = threadIdx.x; i < p.H; i += 32 * kWarps) {
                float s = 0.0f;
                for (int w = 0; w < kWarps; ++w) s += comb[w * E * 32 + i];
                out[i] = s;
            }
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c.on[k]) {
#pragma unroll
                    for (int j = 0; j < P; j += 2) {
                        const float2 u = acc[whole ? k : 0][j], v = acc[whole ? k : 0][j + 1];
                        *reinterpret_cast<float4 *>(out + c.at(k) + 2 * j) = make_float4(u.x, u.y, v.x, v.y);
                    }
                }
        }
    }
    if (TEAM == kCluster) cluster_sync();  // no block leaves while another may write into it
}

template <typename A, typename R, bool LP, bool LN, bool COMMON>
static Kernel pick(const Shape &s) {
    if (s.team == kWarp) return s.E == 8 ? bwd_kernel<A, R, 8, kWarp, LP, LN, COMMON> : bwd_kernel<A, R, 16, kWarp, LP, LN, COMMON>;
    if (s.team == kCluster) return bwd_kernel<A, R, 16, kCluster, LP, LN, COMMON>;
    return s.E == 8 ? bwd_kernel<A, R, 8, kBlock, LP, LN, COMMON> : bwd_kernel<A, R, 16, kBlock, LP, LN, COMMON>;
}
template <typename A, typename R, bool COMMON>
static Kernel of_types(const tp_block_norm_desc &d, const Shape &s) {
    const bool lp = d.post == TP_NORM_LAYER, ln = d.pre == TP_NORM_LAYER;
    return lp ? (ln ? pick<A, R, true, true, COMMON>(s) : pick<A, R, true, false, COMMON>(s))
              : (ln ? pick<A, R, false, true, COMMON>(s) : pick<A, R, false, false, COMMON>(s));
}

}  // namespace bn
}  // namespace tpmlp
