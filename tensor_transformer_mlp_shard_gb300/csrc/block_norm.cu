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
#include <new>

#include "device_common.cuh"
#include "internal.h"

namespace tpmlp {
namespace bn {

constexpr int kWarps = 8;           // warps of a block in the warp-per-row kernels
constexpr int kMaxThreads = 512;    // threads of a block in the block-per-row kernels
constexpr int kMaxH = 16384;        // kMaxThreads * 32 elements a thread
constexpr int kMaxChunks = 304;     // blocks of the backward, each writing one row of partial sums

struct Plan {
    int M, H, rows_split;
    int post, pre, gate, zero_centered, has_block;
    float eps, a, c;
    const void *x[kMaxShards], *f[kMaxShards], *g[kMaxShards];  // g: g[0] for a channel gate
    const void *y_in[kMaxShards], *dy[kMaxShards], *dn[kMaxShards];
    void *y[kMaxShards], *n[kMaxShards];
    void *dx[kMaxShards], *df[kMaxShards], *dg[kMaxShards];     // dg: token and element gates
    const void *post_w, *post_b, *pre_w, *pre_b;
    float4 *stats;                  // [M]: post mean, post rstd, pre mean, pre rstd
    const float4 *stats_in;
    float *partials;                // [sums][blocks][H]: the sums in use of P1, P0, N1, N0
    int use[4];
};

// ---------------------------------------------------------------------------
// vectors of V elements
// ---------------------------------------------------------------------------
template <typename T, int V>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
    using Raw = uint4;
    __device__ static void unpack(const Raw &w, float *v) {
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
        v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    }
    __device__ static Raw pack(const float *v) {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7]));
    }
};
template <>
struct Pack<__nv_bfloat16, 4> {
    using Raw = uint2;
    __device__ static void unpack(const Raw &w, float *v) {
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    }
    __device__ static Raw pack(const float *v) {
        return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
};
template <>
struct Pack<float, 4> {
    using Raw = float4;
    __device__ static void unpack(const Raw &w, float *v) { v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w; }
    __device__ static Raw pack(const float *v) { return make_float4(v[0], v[1], v[2], v[3]); }
};

template <typename T, int V>
__device__ __forceinline__ void load(const void *base, long long e, float *v) {
    Pack<T, V>::unpack(*reinterpret_cast<const typename Pack<T, V>::Raw *>(static_cast<const T *>(base) + e), v);
}
template <typename T, int V>
__device__ __forceinline__ void store(void *base, long long e, const float *v) {
    *reinterpret_cast<typename Pack<T, V>::Raw *>(static_cast<T *>(base) + e) = Pack<T, V>::pack(v);
}
// what v reads back as after a store in T
template <typename T, int V>
__device__ __forceinline__ void round_to(float *v) {
    if (sizeof(T) == 2) Pack<T, V>::unpack(Pack<T, V>::pack(v), v);
}
template <typename T>
__device__ __forceinline__ float load1(const void *base, long long e) {
    return static_cast<float>(static_cast<const T *>(base)[e]);
}
template <typename T>
__device__ __forceinline__ void store1(void *base, long long e, float v) {
    static_cast<T *>(base)[e] = static_cast<T>(v);
}

// shard of token `row` and its row there
__device__ __forceinline__ int shard_of(const Plan &p, int row, int &local) {
    const int j = p.rows_split ? row / p.rows_split : 0;
    local = row - j * p.rows_split;
    return j;
}

// Sums of N values over the threads of a row, for every one of them: a warp
// (WARP) or the block.  The block's form alternates between two buffers, so
// one barrier a call is enough: a buffer is written again only after the
// barrier of the call in between.
template <bool WARP, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[32][4], int &phase) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (WARP) return;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) red[phase][threadIdx.x >> 5][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = 0; w < warps; ++w) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += red[phase][w][i];
    }
    phase ^= 1;
}

// Mean and 1 / spread of a row, and the row less its mean in v.  LayerNorm takes
// its variance about the mean in a second pass over the registers, and that
// pass also sums what the fp32 mean left over: subtracting that too, a mean
// far above the spread costs no digits.
template <bool WARP, int V, int K>
__device__ __forceinline__ void centre_row(float (&v)[K][V], const bool (&on)[K], int kind, int H, float eps,
                                           float (*red)[32][4], int &phase, float &mean, float &rstd) {
    mean = 0.0f;
    float s[2] = {0.0f, 0.0f};
    if (kind == TP_NORM_LAYER) {
        float m[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) m[0] += v[k][j];  // elements past the row are zero
        row_sum<WARP>(m, red, phase);
        mean = m[0] / H;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on[k]) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[k][j] -= mean;
                    s[0] += v[k][j];
                    s[1] = fmaf(v[k][j], v[k][j], s[1]);
                }
            }
        row_sum<WARP>(s, red, phase);
        const float rest = s[0] / H;
        s[1] = fmaxf(s[1] - s[0] * rest, 0.0f);
        mean += rest;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) v[k][j] -= rest;
    } else {
        float q[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) q[0] = fmaf(v[k][j], v[k][j], q[0]);
        row_sum<WARP>(q, red, phase);
        s[1] = q[0];
    }
    rstd = 1.0f / sqrtf(s[1] / H + eps);
}

// w (1 + w when zero-centred) of the V channels from column c
template <typename A, int V>
__device__ __forceinline__ void load_weight(const void *w, int c, int zero_centered, float *v) {
    load<A, V>(w, c, v);
    if (zero_centered) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += 1.0f;
    }
}

// ---------------------------------------------------------------------------
// Forward.  A: type of f, g, n and the weights; R: type of x and y; E elements
// a thread, in vectors of V.
// ---------------------------------------------------------------------------
template <typename A, typename R, int E, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : kMaxThreads) fwd_kernel(const __grid_constant__ Plan p) {
    constexpr int V = sizeof(R) == 2 ? 8 : 4, K = E / V;
    __shared__ float red[2][32][4];
    int phase = 0;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int stride = WARP ? gridDim.x * kWarps : gridDim.x;
    bool on[K];
#pragma unroll
    for (int k = 0; k < K; ++k) on[k] = (t + k * nt) * V < p.H;
    for (int row = WARP ? blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x; row < p.M; row += stride) {
        int lr;
        const int js = shard_of(p, row, lr);
        const long long base = static_cast<long long>(lr) * p.H;
        float y[K][V], f[K][V];
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) y[k][j] = f[k][j] = 0.0f;
            if (on[k]) {
                load<R, V>(p.x[js], base + (t + k * nt) * V, y[k]);
                if (p.has_block) load<A, V>(p.f[js], base + (t + k * nt) * V, f[k]);
            }
        }
        float4 st = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
        if (p.has_block) {
            if (p.post != TP_NORM_NONE)
                centre_row<WARP, V, K>(f, on, p.post, p.H, p.eps, red, phase, st.x, st.y);
            const float gm = p.gate == TP_GATE_TOKEN ? p.c * load1<A>(p.g[js], lr) : p.c;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (on[k]) {
                    const int c = (t + k * nt) * V;
                    float w[V];
                    if (p.post != TP_NORM_NONE) {
                        load_weight<A, V>(p.post_w, c, p.zero_centered, w);
#pragma unroll
                        for (int j = 0; j < V; ++j) f[k][j] *= st.y * w[j];
                        if (p.post == TP_NORM_LAYER) {
                            load<A, V>(p.post_b, c, w);
#pragma unroll
                            for (int j = 0; j < V; ++j) f[k][j] += w[j];
                        }
                    }
                    if (p.gate == TP_GATE_CHANNEL || p.gate == TP_GATE_ELEMENT) {
                        load<A, V>(p.gate == TP_GATE_CHANNEL ? p.g[0] : p.g[js],
                                   p.gate == TP_GATE_CHANNEL ? c : base + c, w);
#pragma unroll
                        for (int j = 0; j < V; ++j) f[k][j] *= w[j];
                    }
#pragma unroll
                    for (int j = 0; j < V; ++j) y[k][j] = fmaf(p.a, y[k][j], gm * f[k][j]);
                    store<R, V>(p.y[js], base + c, y[k]);
                    round_to<R, V>(y[k]);
                }
        }
        if (p.pre != TP_NORM_NONE) {
            centre_row<WARP, V, K>(y, on, p.pre, p.H, p.eps, red, phase, st.z, st.w);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (on[k]) {
                    const int c = (t + k * nt) * V;
                    float w[V], o[V];
                    load_weight<A, V>(p.pre_w, c, p.zero_centered, w);
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] = y[k][j] * st.w * w[j];
                    if (p.pre == TP_NORM_LAYER) {
                        load<A, V>(p.pre_b, c, w);
#pragma unroll
                        for (int j = 0; j < V; ++j) o[j] += w[j];
                    }
                    store<A, V>(p.n[js], base + c, o);
                }
        }
        if (p.stats && t == 0) p.stats[row] = st;
    }
}

// ---------------------------------------------------------------------------
// Backward: gradients of x, f and of a token or element gate, row by row, and
// this block's share of the column sums in registers.
// ---------------------------------------------------------------------------
template <typename A, typename R, int E, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : kMaxThreads) bwd_kernel(const __grid_constant__ Plan p) {
    constexpr int V = sizeof(R) == 2 ? 8 : 4, K = E / V;
    __shared__ float red[2][32][4];
    int phase = 0;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int stride = WARP ? gridDim.x * kWarps : gridDim.x;
    const float inv_h = 1.0f / p.H;
    bool on[K];
    float acc[4][K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        on[k] = (t + k * nt) * V < p.H;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[0][k][j] = acc[1][k][j] = acc[2][k][j] = acc[3][k][j] = 0.0f;
    }
    const bool row_gate = p.gate == TP_GATE_TOKEN || p.gate == TP_GATE_ELEMENT;
    for (int row = WARP ? blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x; row < p.M; row += stride) {
        int lr;
        const int js = shard_of(p, row, lr);
        const long long base = static_cast<long long>(lr) * p.H;
        const float4 st = p.stats_in[row];
        float d[K][V];  // dy, then D
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) d[k][j] = 0.0f;
            if (on[k] && p.dy[js]) load<R, V>(p.dy[js], base + (t + k * nt) * V, d[k]);
        }
        if (p.pre != TP_NORM_NONE) {
            float yh[K][V], h[K][V], s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < V; ++j) yh[k][j] = h[k][j] = 0.0f;
                if (on[k]) {
                    const int c = (t + k * nt) * V;
                    float w[V];
                    load<R, V>(p.y_in[js], base + c, yh[k]);
                    load<A, V>(p.dn[js], base + c, h[k]);
                    load_weight<A, V>(p.pre_w, c, p.zero_centered, w);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        yh[k][j] = (yh[k][j] - st.z) * st.w;
                        acc[2][k][j] = fmaf(h[k][j], yh[k][j], acc[2][k][j]);
                        acc[3][k][j] += h[k][j];
                        h[k][j] *= w[j];
                        s[0] += h[k][j];
                        s[1] = fmaf(h[k][j], yh[k][j], s[1]);
                    }
                }
            }
            row_sum<WARP>(s, red, phase);
            const float m0 = p.pre == TP_NORM_LAYER ? s[0] * inv_h : 0.0f, m1 = s[1] * inv_h;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) d[k][j] += st.w * (h[k][j] - m0 - yh[k][j] * m1);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on[k]) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = p.a * d[k][j];
                store<R, V>(p.dx[js], base + (t + k * nt) * V, o);
            }
        if (!p.has_block) continue;
        const float gm = p.gate == TP_GATE_TOKEN ? load1<A>(p.g[js], lr) : 1.0f;
        const bool need_f = p.post != TP_NORM_NONE || p.gate != TP_GATE_NONE;
        float fh[K][V], s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) fh[k][j] = 0.0f;
            if (on[k]) {
                const int c = (t + k * nt) * V;
                float w[V], pv[V];
                if (need_f) load<A, V>(p.f[js], base + c, fh[k]);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    fh[k][j] = (fh[k][j] - st.x) * st.y;  // no post-norm: mean 0, rstd 1
                    w[j] = 1.0f;
                    pv[j] = fh[k][j];
                }
                if (p.post != TP_NORM_NONE) {
                    load_weight<A, V>(p.post_w, c, p.zero_centered, w);
                    if (row_gate) {
#pragma unroll
                        for (int j = 0; j < V; ++j) pv[j] = fh[k][j] * w[j];
                        if (p.post == TP_NORM_LAYER) {
                            float b[V];
                            load<A, V>(p.post_b, c, b);
#pragma unroll
                            for (int j = 0; j < V; ++j) pv[j] += b[j];
                        }
                    }
                }
                if (p.gate == TP_GATE_ELEMENT) {
                    float g[V], o[V];
                    load<A, V>(p.g[js], base + c, g);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        o[j] = p.c * d[k][j] * pv[j];
                        d[k][j] *= g[j];
                    }
                    store<A, V>(p.dg[js], base + c, o);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        s[2] = fmaf(d[k][j], pv[j], s[2]);  // the token gate's gradient
                        d[k][j] *= gm;
                    }
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    acc[0][k][j] = fmaf(d[k][j], fh[k][j], acc[0][k][j]);
                    acc[1][k][j] += d[k][j];
                }
                if (p.gate == TP_GATE_CHANNEL) {
                    float g[V];
                    load<A, V>(p.g[0], c, g);
#pragma unroll
                    for (int j = 0; j < V; ++j) d[k][j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    d[k][j] *= p.c * w[j];  // the gradient of fh
                    s[0] += d[k][j];
                    s[1] = fmaf(d[k][j], fh[k][j], s[1]);
                }
            }
        }
        float m0 = 0.0f, m1 = 0.0f;
        if (p.post != TP_NORM_NONE || p.gate == TP_GATE_TOKEN) {
            row_sum<WARP>(s, red, phase);
            if (p.post == TP_NORM_LAYER) m0 = s[0] * inv_h;
            if (p.post != TP_NORM_NONE) m1 = s[1] * inv_h;
            if (p.gate == TP_GATE_TOKEN && t == 0) store1<A>(p.dg[js], lr, p.c * s[2]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on[k]) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = st.y * (d[k][j] - m0 - fh[k][j] * m1);
                store<A, V>(p.df[js], base + (t + k * nt) * V, o);
            }
    }
    // one row of partial sums a block (the warps of a block added in order)
    __shared__ float comb[WARP ? kWarps * E * 32 : 1];
    int slot = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (!p.use[q]) continue;
        float *out = p.partials + (static_cast<long long>(slot++) * gridDim.x + blockIdx.x) * p.H;
        if (WARP) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    comb[(threadIdx.x >> 5) * E * 32 + (t + k * 32) * V + j] = acc[q][k][j];
            __syncthreads();
            for (int c = threadIdx.x; c < p.H; c += 32 * kWarps) {
                float s = 0.0f;
                for (int w = 0; w < kWarps; ++w) s += comb[w * E * 32 + c];
                out[c] = s;
            }
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (on[k]) {
#pragma unroll
                    for (int j = 0; j < V; j += 4)
                        *reinterpret_cast<float4 *>(out + (t + k * nt) * V + j) =
                            make_float4(acc[q][k][j], acc[q][k][j + 1], acc[q][k][j + 2], acc[q][k][j + 3]);
                }
        }
    }
}

// ---------------------------------------------------------------------------
// Parameter gradients from the partial rows: 32 columns a block, 8 threads a
// column, the rows in a fixed order.
// ---------------------------------------------------------------------------
struct FinalPlan {
    const float *partials;
    int chunks, H, use[4], zero_centered;
    float c;
    const void *post_w, *post_b, *gate;  // gate: the channel gate, or null
    float *dpost_w, *dpost_b, *dpre_w, *dpre_b, *dgate;
};

template <typename A>
__global__ void __launch_bounds__(256) param_grad_kernel(const __grid_constant__ FinalPlan p) {
    __shared__ float part[4][8][32];
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    int slot = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float s = 0.0f;
        if (p.use[q]) {
            const float *in = p.partials + static_cast<long long>(slot++) * p.chunks * p.H + col;
            if (col < p.H)
                for (int i = r; i < p.chunks; i += 8) s += in[static_cast<long long>(i) * p.H];
        }
        part[q][r][lane] = s;
    }
    __syncthreads();
    if (r || col >= p.H) return;
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[q] += part[q][i][lane];
    }
    const float g = p.gate ? load1<A>(p.gate, col) : 1.0f;
    if (p.dpost_w) p.dpost_w[col] = p.c * g * v[0];
    if (p.dpost_b) p.dpost_b[col] = p.c * g * v[1];
    if (p.dgate) {
        float s = v[0];
        if (p.post_w) s *= load1<A>(p.post_w, col) + (p.zero_centered ? 1.0f : 0.0f);
        if (p.post_b) s = fmaf(load1<A>(p.post_b, col), v[1], s);
        p.dgate[col] = p.c * s;
    }
    if (p.dpre_w) p.dpre_w[col] = v[2];
    if (p.dpre_b) p.dpre_b[col] = v[3];
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// Elements a thread (8, 16, 32) and whether a warp takes a row: rows of up to
// 1024 columns go to a warp each, wider ones to a block.
struct Shape {
    bool warp;
    int E, threads;
};
static Shape shape_of(int H) {
    Shape s;
    s.warp = H <= 1024;
    const int most = s.warp ? 32 : kMaxThreads;
    s.E = H <= most * 8 ? 8 : H <= most * 16 ? 16 : 32;
    s.threads = s.warp ? 32 * kWarps : ((H + s.E - 1) / s.E + 31) / 32 * 32;
    return s;
}

using Kernel = void (*)(Plan);
template <typename A, typename R, bool BWD>
static Kernel pick(const Shape &s) {
    if (BWD) {
        if (s.warp) return s.E == 8 ? bwd_kernel<A, R, 8, true> : s.E == 16 ? bwd_kernel<A, R, 16, true> : bwd_kernel<A, R, 32, true>;
        return s.E == 8 ? bwd_kernel<A, R, 8, false> : s.E == 16 ? bwd_kernel<A, R, 16, false> : bwd_kernel<A, R, 32, false>;
    }
    if (s.warp) return s.E == 8 ? fwd_kernel<A, R, 8, true> : s.E == 16 ? fwd_kernel<A, R, 16, true> : fwd_kernel<A, R, 32, true>;
    return s.E == 8 ? fwd_kernel<A, R, 8, false> : s.E == 16 ? fwd_kernel<A, R, 16, false> : fwd_kernel<A, R, 32, false>;
}

static Kernel kernel_for(const tp_block_norm_desc &d, bool bwd, const Shape &s) {
    using bf = __nv_bfloat16;
    if (d.dtype == TP_DT_F32) return bwd ? pick<float, float, true>(s) : pick<float, float, false>(s);
    if (d.residual_f32) return bwd ? pick<bf, float, true>(s) : pick<bf, float, false>(s);
    return bwd ? pick<bf, bf, true>(s) : pick<bf, bf, false>(s);
}

static int grid_for(Kernel k, const Shape &s, int M, int cap) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, s.threads, 0) != cudaSuccess || per_sm < 1) per_sm = 1;
    const int rows = s.warp ? kWarps : 1;
    int g = per_sm * num_sms();
    if (g > (M + rows - 1) / rows) g = (M + rows - 1) / rows;
    if (cap && g > cap) g = cap;
    return g;
}

}  // namespace bn
}  // namespace tpmlp

using namespace tpmlp;

struct tp_block_norm {
    tp_block_norm_desc d;
    int M, nx, rows_split;
    int use[4];
};

#define TRY(x)                        \
    do {                              \
        tp_status _s = (x);           \
        if (_s != TP_OK) return _s;   \
    } while (0)

static tp_status bn_pointer(const void *p, const char *name, int i, int n) {
    char at[16] = "";
    if (n > 1) snprintf(at, sizeof(at), "[%d]", i);
    if (!p) return set_error(TP_ERR_ARG, "%s%s is NULL", name, at);
    if (reinterpret_cast<uintptr_t>(p) & 15u) return set_error(TP_ERR_ARG, "%s%s is not 16-byte aligned", name, at);
    return TP_OK;
}

// copies an array of n pointers into a plan after checking them
template <typename P>
static tp_status bn_array(P *const *in, int n, const char *name, P **out) {
    if (!in) return set_error(TP_ERR_ARG, "%s: pointer array is NULL", name);
    for (int i = 0; i < n; ++i) {
        TRY(bn_pointer(in[i], name, i, n));
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

static tp_status bn_gate(const tp_block_norm *h, const void *const *gate, bn::Plan &p) {
    if (h->d.gate == TP_GATE_NONE) return TP_OK;
    return bn_array(gate, h->d.gate == TP_GATE_CHANNEL ? 1 : h->nx, "gate", p.g);
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
    const int chunks = h->M < bn::kMaxChunks ? h->M : bn::kMaxChunks;
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
    const bn::Shape s = bn::shape_of(d.H);
    const bn::Kernel k = bn::kernel_for(d, false, s);
    const int grid = bn::grid_for(k, s, h->M, 0);
    launch_begin("block_norm_fwd", st);
    k<<<grid, s.threads, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    launch_end("block_norm_fwd", st);
    return cuda_check(e, "block_norm_fwd");
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
            TRY(bn_array(dgate, h->nx, "dgate", p.dg));
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
        const bn::Shape s = bn::shape_of(d.H);
        const bn::Kernel k = bn::kernel_for(d, true, s);
        grid = bn::grid_for(k, s, h->M, bn::kMaxChunks);
        launch_begin("block_norm_bwd", st);
        k<<<grid, s.threads, 0, st>>>(p);
        cudaError_t e = cudaGetLastError();
        launch_end("block_norm_bwd", st);
        TRY(cuda_check(e, "block_norm_bwd"));
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
    launch_begin("block_norm_param_grads", st);
    if (d.dtype == TP_DT_F32)
        bn::param_grad_kernel<float><<<(d.H + 31) / 32, 256, 0, st>>>(fin);
    else
        bn::param_grad_kernel<__nv_bfloat16><<<(d.H + 31) / 32, 256, 0, st>>>(fin);
    cudaError_t e = cudaGetLastError();
    launch_end("block_norm_param_grads", st);
    return cuda_check(e, "block_norm_param_grads");
}

}  // extern "C"
