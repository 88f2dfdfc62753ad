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

#include "device_common.cuh"
#include "internal.h"

#define TRY(x)                        \
    do {                              \
        tp_status _s = (x);           \
        if (_s != TP_OK) return _s;   \
    } while (0)

namespace tpmlp {
namespace bn {

constexpr int kWarps = 8;           // warps of a block in the warp-per-row kernels
constexpr int kMaxThreads = 512;    // threads of a block in the block-per-row kernels
constexpr int kMaxCluster = 4;      // blocks that share a row
constexpr int kMaxH = 16384;
constexpr int kMaxChunks = 304;     // workers of the backward, each writing one row of partial sums

struct Plan {
    int M, H, rows_split;
    int post, pre, gate, zero_centered, has_block;
    int cluster, depth, need_f;     // blocks to a row, rows staged, f is read
    float eps, a, c;
    const void *x[kMaxShards], *f[kMaxShards], *g[kMaxShards];  // g: g[0] for a channel gate
    const void *y_in[kMaxShards], *dy[kMaxShards], *dn[kMaxShards];
    void *y[kMaxShards], *n[kMaxShards];
    void *dx[kMaxShards], *df[kMaxShards], *dg[kMaxShards];     // dg: token and element gates
    const void *post_w, *post_b, *pre_w, *pre_b;
    float4 *stats;                  // [M]: post mean, post rstd, pre mean, pre rstd
    const float4 *stats_in;
    float *partials;                // [sums][workers][H]: the sums in use of P1, P0, N1, N0
    int use[4];
};

// ---------------------------------------------------------------------------
// vectors of V elements, as V / 2 pairs
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 bf16_pair(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

template <typename T, int V>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
    using Raw = uint4;
    __device__ static void unpack(const Raw &w, float2 *v) {
        v[0] = bf16_pair(w.x); v[1] = bf16_pair(w.y); v[2] = bf16_pair(w.z); v[3] = bf16_pair(w.w);
    }
    __device__ static Raw pack(const float2 *v) {
        return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                          pack_bf16x2(v[3].x, v[3].y));
    }
};
template <>
struct Pack<__nv_bfloat16, 4> {
    using Raw = uint2;
    __device__ static void unpack(const Raw &w, float2 *v) { v[0] = bf16_pair(w.x); v[1] = bf16_pair(w.y); }
    __device__ static Raw pack(const float2 *v) {
        return make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
    }
};
template <>
struct Pack<float, 4> {
    using Raw = float4;
    __device__ static void unpack(const Raw &w, float2 *v) { v[0] = make_float2(w.x, w.y); v[1] = make_float2(w.z, w.w); }
    __device__ static Raw pack(const float2 *v) { return make_float4(v[0].x, v[0].y, v[1].x, v[1].y); }
};

template <typename T, int V>
__device__ __forceinline__ void load(const void *base, long long e, float2 *v) {
    Pack<T, V>::unpack(*reinterpret_cast<const typename Pack<T, V>::Raw *>(static_cast<const T *>(base) + e), v);
}
template <typename T, int V>
__device__ __forceinline__ void store(void *base, long long e, const float2 *v) {
    *reinterpret_cast<typename Pack<T, V>::Raw *>(static_cast<T *>(base) + e) = Pack<T, V>::pack(v);
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

// ---------------------------------------------------------------------------
// Staging.  A worker's next rows are on their way into shared memory while it
// works on one: a thread copies (cp.async) the very vectors that it will read
// itself, so its own wait is all the synchronisation, and the bytes in flight
// do not depend on registers or on how many blocks fit an SM.  A stage holds
// the arrays one after another, each [K][threads] vectors.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_at(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

template <typename T, int V>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if (V * sizeof(T) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups have landed
__device__ __forceinline__ void copies_wait(int n) {
    if (n >= 3)
        asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (n == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 1;" ::: "memory");
}
constexpr int kMaxDepth = 4;

// a thread's columns: vector k starts at column first + k * step
template <int K, int V>
struct Columns {
    int first, step, lanes;  // lanes: threads of the block (the stride of staged vectors)
    bool on[K], ragged;      // ragged: the row ends within this block's (or warp's) columns
    __device__ __forceinline__ int at(int k) const { return first + k * step; }
};

template <typename T, int K, int V>
__device__ __forceinline__ uint32_t stage(uint32_t at, const void *row, const Columns<K, V> &c) {
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (c.on[k])
            copy_async<T, V>(at + (k * c.lanes + threadIdx.x) * (V * sizeof(T)), static_cast<const T *>(row) + c.at(k));
    return at + K * c.lanes * static_cast<uint32_t>(V * sizeof(T));
}
// the staged vectors of one array; `at` moves to the next array
template <typename T, int K, int V>
__device__ __forceinline__ void staged(const uint8_t *&at, const Columns<K, V> &c, float2 (&v)[K][V / 2]) {
#pragma unroll
    for (int k = 0; k < K; ++k) load<T, V>(at, static_cast<int>(k * c.lanes + threadIdx.x) * V, v[k]);
    at += K * c.lanes * V * sizeof(T);
}
// Vectors past the row's end are never copied.  Where a block has such, its
// stages are cleared once, so that they read as zero and the arithmetic on
// them needs no condition.
__device__ __forceinline__ void clear_stages(uint8_t *stages, uint32_t bytes) {
    for (uint32_t i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16)
        *reinterpret_cast<uint4 *>(stages + i) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Sums over a row, for every thread of it: a warp, a block, or a cluster.
// ---------------------------------------------------------------------------
// TEAM: kWarp, kBlock or kCluster.
enum Team { kWarp = 0, kBlock = 1, kCluster = 2 };
struct Reduce {
    float (*red)[3][16 * kMaxCluster];  // [2][value][block of the cluster x warp]
    int phase, cluster, rank;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
template <Team TEAM>
__device__ __forceinline__ void put(Reduce &r, int value, int warp, float v) {
    float *mine = &r.red[r.phase][value][r.rank * 16 + warp];
    if (TEAM == kBlock) {
        *mine = v;
        return;
    }
    for (int b = 0; b < r.cluster; ++b) {
        uint32_t there;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_at(mine)), "r"(b));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
    }
}

// Two values: after the first exchange a half of the warp carries one, the
// other half the other, so they take 5 shuffles and not 10.  A third value (C)
// takes its own.  Buffers alternate, so one barrier a call is enough: a buffer
// is written again only after the barrier of the call in between.
template <Team TEAM>
__device__ __forceinline__ void team_sync() {
    if (TEAM == kCluster)
        cluster_sync();
    else
        __syncthreads();
}
template <Team TEAM, bool C>
__device__ __forceinline__ void row_sum(float &a, float &b, float &c, Reduce &r) {
    const int lane = threadIdx.x & 31;
    const bool low = lane < 16;
    float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (C) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    if (TEAM != kWarp) {
        if ((lane & 15) == 0) put<TEAM>(r, lane >> 4, threadIdx.x >> 5, v);
        if (C && lane == 0) put<TEAM>(r, 2, threadIdx.x >> 5, c);
        team_sync<TEAM>();
        const float *in = r.red[r.phase][lane >> 4] + (lane & 15), *in_c = r.red[r.phase][2] + (lane & 15);
        v = in[0];
        if (C) c = in_c[0];
        if (TEAM == kCluster)
            for (int k = 1; k < r.cluster; ++k) {
                v += in[k * 16];
                if (C) c += in_c[k * 16];
            }
        r.phase ^= 1;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            v += __shfl_xor_sync(0xffffffffu, v, o);
            if (C) c += __shfl_xor_sync(0xffffffffu, c, o);
        }
    }
    a = __shfl_sync(0xffffffffu, v, 0);
    b = __shfl_sync(0xffffffffu, v, 16);
}
template <Team TEAM>
__device__ __forceinline__ void row_sum(float &a, Reduce &r) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (TEAM == kWarp) return;
    if (lane == 0) put<TEAM>(r, 0, threadIdx.x >> 5, a);
    team_sync<TEAM>();
    const float *in = r.red[r.phase][0] + (lane & 15);
    a = in[0];
    if (TEAM == kCluster)
        for (int k = 1; k < r.cluster; ++k) a += in[k * 16];
    r.phase ^= 1;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
}

template <Team TEAM>
__device__ __forceinline__ Reduce make_reduce(float (*red)[3][16 * kMaxCluster], const Plan &p) {
    Reduce r = {red, 0, TEAM == kCluster ? p.cluster : 1, 0};
    if (TEAM == kWarp) return r;
    // warps that a block does not have add nothing
    for (int i = threadIdx.x; i < 2 * 3 * 16 * kMaxCluster; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;
    if (TEAM == kCluster) r.rank = cluster_rank();
    team_sync<TEAM>();  // and no block writes into one that has not begun
    return r;
}

template <int K, int V, Team TEAM>
__device__ __forceinline__ Columns<K, V> make_columns(const Plan &p, const Reduce &r) {
    constexpr bool WARP = TEAM == kWarp;
    Columns<K, V> c;
    const int lanes = WARP ? 32 : blockDim.x;
    c.lanes = blockDim.x;
    c.first = r.rank * lanes * K * V + (WARP ? threadIdx.x & 31 : threadIdx.x) * V;
    c.step = lanes * V;
    c.ragged = (r.rank + 1) * lanes * K * V > p.H;
#pragma unroll
    for (int k = 0; k < K; ++k) c.on[k] = c.at(k) < p.H;
    return c;
}

// Mean and 1 / spread of a row, and the row less its mean in v.  LayerNorm takes
// its variance about the mean in a second pass over the registers, and that
// pass also sums what the fp32 mean left over: subtracting that too, a mean
// far above the spread costs no digits.
template <Team TEAM, bool LN, int V, int K>
__device__ __forceinline__ void centre_row(float2 (&v)[K][V / 2], const Columns<K, V> &c, int kind, float inv_h,
                                           float eps, Reduce &r, float &mean, float &rstd) {
    mean = 0.0f;
    float2 s = both(0.0f), q = both(0.0f);
    if (LN && kind == TP_NORM_LAYER) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V / 2; ++j) s = __fadd2_rn(s, v[k][j]);
        mean = s.x + s.y;
        row_sum<TEAM>(mean, r);
        mean *= inv_h;
        s = both(0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float2 less = both(c.on[k] ? -mean : 0.0f);  // past the row's end zeros stay zeros
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                v[k][j] = __fadd2_rn(v[k][j], less);
                s = __fadd2_rn(s, v[k][j]);
                q = __ffma2_rn(v[k][j], v[k][j], q);
            }
        }
        float a = s.x + s.y, b = q.x + q.y, none;
        row_sum<TEAM, false>(a, b, none, r);
        const float rest = a * inv_h;
        mean += rest;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V / 2; ++j) v[k][j] = __fadd2_rn(v[k][j], both(-rest));
        rstd = rsqrtf(fmaxf(b - a * rest, 0.0f) * inv_h + eps);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V / 2; ++j) q = __ffma2_rn(v[k][j], v[k][j], q);
        float b = q.x + q.y;
        row_sum<TEAM>(b, r);
        rstd = rsqrtf(b * inv_h + eps);
    }
}

// v = w (1 + w when zero-centred) of a thread's columns, `none` without a weight;
// zero past the row's end, where what it multiplies may be anything finite
template <typename A, int K, int V>
__device__ __forceinline__ void load_weight(const void *w, const Columns<K, V> &c, float plus, float none,
                                            float2 (&v)[K][V / 2]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[k][j] = both(c.on[k] ? none : 0.0f);
        if (w && c.on[k]) {
            load<A, V>(w, c.at(k), v[k]);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) v[k][j] = __fadd2_rn(v[k][j], both(plus));
        }
    }
}
// v *= c times the channel gate (c alone without one)
template <typename A, int K, int V>
__device__ __forceinline__ void times_gate(const Plan &p, const Columns<K, V> &c, float2 (&v)[K][V / 2]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float2 g[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) g[j] = both(1.0f);
        if (p.gate == TP_GATE_CHANNEL && c.on[k]) load<A, V>(p.g[0], c.at(k), g);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[k][j] = __fmul2_rn(__fmul2_rn(v[k][j], g[j]), both(p.c));
    }
}

// ---------------------------------------------------------------------------
// Forward.  A: type of f, g, n and the weights; R: type of x and y; E elements
// a thread, in vectors of V; LN: one of the norms is a LayerNorm.
// ---------------------------------------------------------------------------
template <typename A, typename R, int E, Team TEAM, bool LN>
__global__ void __launch_bounds__(TEAM == kWarp ? 32 * kWarps : kMaxThreads) fwd_kernel(const __grid_constant__ Plan p) {
    constexpr bool WARP = TEAM == kWarp;
    constexpr int V = sizeof(R) == 2 ? 8 : 4, K = E / V, P = V / 2;
    __shared__ float red[2][3][16 * kMaxCluster];
    extern __shared__ __align__(16) uint8_t stages[];
    Reduce r = make_reduce<TEAM>(red, p);
    const Columns<K, V> c = make_columns<K, V, TEAM>(p, r);
    const int worker = WARP ? blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x / r.cluster;
    const int workers = WARP ? gridDim.x * kWarps : gridDim.x / r.cluster;
    const bool gate_rows = p.gate == TP_GATE_ELEMENT, first = (WARP ? threadIdx.x & 31 : threadIdx.x) == 0 && r.rank == 0;
    const float inv_h = 1.0f / p.H, plus = p.zero_centered ? 1.0f : 0.0f;
    const uint32_t stage_bytes =
        blockDim.x * E * static_cast<uint32_t>(sizeof(R) + (p.has_block ? sizeof(A) : 0) + (gate_rows ? sizeof(A) : 0));
    const uint32_t base = smem_at(stages);
    auto fetch = [&](int row, int slot) {
        if (row < p.M) {
            int lr;
            const int js = shard_of(p, row, lr);
            const long long e = static_cast<long long>(lr) * p.H;
            uint32_t at = base + slot * stage_bytes;
            at = stage<R>(at, static_cast<const R *>(p.x[js]) + e, c);
            if (p.has_block) at = stage<A>(at, static_cast<const A *>(p.f[js]) + e, c);
            if (gate_rows) stage<A>(at, static_cast<const A *>(p.g[js]) + e, c);
        }
        copies_commit();
    };
    if (c.ragged) clear_stages(stages, p.depth * stage_bytes);
    for (int i = 0; i < p.depth - 1; ++i) fetch(worker + i * workers, i);
    // weights of this thread's columns, the gate and the block's scale in the post-norm's
    float2 pw[K][P], nw[K][P], pb[LN ? K : 1][P], nb[LN ? K : 1][P];
    load_weight<A>(p.post_w, c, plus, 1.0f, pw);
    times_gate<A>(p, c, pw);
    load_weight<A>(p.pre_w, c, plus, 1.0f, nw);
    if constexpr (LN) {
        load_weight<A>(p.post_b, c, 0.0f, 0.0f, pb);
        times_gate<A>(p, c, pb);
        load_weight<A>(p.pre_b, c, 0.0f, 0.0f, nb);
    }
    int slot = 0;
    for (int row = worker; row < p.M; row += workers) {
        fetch(row + (p.depth - 1) * workers, slot == 0 ? p.depth - 1 : slot - 1);  // the slot of the row before
        int lr;
        const int js = shard_of(p, row, lr);
        const long long e = static_cast<long long>(lr) * p.H;
        const float gm = p.gate == TP_GATE_TOKEN ? load1<A>(p.g[js], lr) : 1.0f;
        copies_wait(p.depth - 1);
        const uint8_t *at = stages + slot * stage_bytes;
        slot = slot + 1 == p.depth ? 0 : slot + 1;
        float2 y[K][P];
        staged<R>(at, c, y);
        float4 st = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
        if (p.has_block) {
            float2 f[K][P];
            staged<A>(at, c, f);
            if (p.post != TP_NORM_NONE) centre_row<TEAM, LN, V, K>(f, c, p.post, inv_h, p.eps, r, st.x, st.y);
            // y = a x + g (P(f) scaled): the row's factors first, then the channel's
            const float2 row_scale = both(LN ? st.y : st.y * gm);
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    f[k][j] = __fmul2_rn(f[k][j], row_scale);
                    if (LN) f[k][j] = __fmul2_rn(__ffma2_rn(f[k][j], pw[k][j], pb[LN ? k : 0][j]), both(gm));
                    y[k][j] = __fmul2_rn(y[k][j], both(p.a));
                }
                if (gate_rows) {
                    float2 g[P];
                    load<A, V>(at, static_cast<int>(k * c.lanes + threadIdx.x) * V, g);
#pragma unroll
                    for (int j = 0; j < P; ++j) f[k][j] = __fmul2_rn(f[k][j], g[j]);
                }
#pragma unroll
                for (int j = 0; j < P; ++j)
                    y[k][j] = LN ? __fadd2_rn(f[k][j], y[k][j]) : __ffma2_rn(f[k][j], pw[k][j], y[k][j]);
                const typename Pack<R, V>::Raw out = Pack<R, V>::pack(y[k]);
                if (c.on[k]) *reinterpret_cast<typename Pack<R, V>::Raw *>(static_cast<R *>(p.y[js]) + e + c.at(k)) = out;
                Pack<R, V>::unpack(out, y[k]);  // the pre-norm is of y as it is stored
            }
        }
        if (p.pre != TP_NORM_NONE) {
            centre_row<TEAM, LN, V, K>(y, c, p.pre, inv_h, p.eps, r, st.z, st.w);
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    y[k][j] = __fmul2_rn(y[k][j], both(st.w));
                    y[k][j] = LN ? __ffma2_rn(y[k][j], nw[k][j], nb[LN ? k : 0][j]) : __fmul2_rn(y[k][j], nw[k][j]);
                }
                if (c.on[k]) store<A, V>(p.n[js], e + c.at(k), y[k]);
            }
        }
        if (p.stats && first) p.stats[row] = st;
    }
    if (TEAM == kCluster) cluster_sync();  // no block leaves while another may write into it
}

// ---------------------------------------------------------------------------
// Backward: gradients of x, f and of a token or element gate, row by row, and
// this worker's share of the column sums in registers.
// ---------------------------------------------------------------------------
template <typename A, typename R, int E, Team TEAM, bool LN>
__global__ void __launch_bounds__(TEAM == kWarp ? 32 * kWarps : kMaxThreads) bwd_kernel(const __grid_constant__ Plan p) {
    constexpr bool WARP = TEAM == kWarp;
    constexpr int V = sizeof(R) == 2 ? 8 : 4, K = E / V, P = V / 2, L = LN ? K : 1;
    __shared__ float red[2][3][16 * kMaxCluster];
    extern __shared__ __align__(16) uint8_t stages[];
    Reduce r = make_reduce<TEAM>(red, p);
    const Columns<K, V> c = make_columns<K, V, TEAM>(p, r);
    const int worker = WARP ? blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x / r.cluster;
    const int workers = WARP ? gridDim.x * kWarps : gridDim.x / r.cluster;
    const bool has_pre = p.pre != TP_NORM_NONE, has_dy = p.dy[0] != nullptr, gate_rows = p.gate == TP_GATE_ELEMENT;
    const bool row_gate = gate_rows || p.gate == TP_GATE_TOKEN;
    const bool first = (WARP ? threadIdx.x & 31 : threadIdx.x) == 0 && r.rank == 0;
    const float inv_h = 1.0f / p.H, plus = p.zero_centered ? 1.0f : 0.0f;
    const uint32_t stage_bytes = blockDim.x * E *
                                 static_cast<uint32_t>((has_dy ? sizeof(R) : 0) + (has_pre ? sizeof(R) + sizeof(A) : 0) +
                                                       (p.need_f ? sizeof(A) : 0) + (gate_rows ? sizeof(A) : 0));
    const uint32_t base = smem_at(stages);
    auto fetch = [&](int row, int slot) {
        if (row < p.M) {
            int lr;
            const int js = shard_of(p, row, lr);
            const long long e = static_cast<long long>(lr) * p.H;
            uint32_t at = base + slot * stage_bytes;
            if (has_dy) at = stage<R>(at, static_cast<const R *>(p.dy[js]) + e, c);
            if (has_pre) {
                at = stage<R>(at, static_cast<const R *>(p.y_in[js]) + e, c);
                at = stage<A>(at, static_cast<const A *>(p.dn[js]) + e, c);
            }
            if (p.need_f) at = stage<A>(at, static_cast<const A *>(p.f[js]) + e, c);
            if (gate_rows) stage<A>(at, static_cast<const A *>(p.g[js]) + e, c);
        }
        copies_commit();
    };
    if (c.ragged) clear_stages(stages, p.depth * stage_bytes);
    for (int i = 0; i < p.depth - 1; ++i) fetch(worker + i * workers, i);
    float2 gw[K][P], nw[K][P];  // c times the channel gate times the post-norm's weight; the pre-norm's weight
    load_weight<A>(p.post_w, c, plus, 1.0f, gw);
    times_gate<A>(p, c, gw);
    load_weight<A>(p.pre_w, c, plus, 1.0f, nw);
    float2 p1[K][P], n1[K][P], p0[L][P], n0[L][P];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j) p1[k][j] = n1[k][j] = p0[LN ? k : 0][j] = n0[LN ? k : 0][j] = both(0.0f);
    int slot = 0;
    float4 st_next = worker < p.M ? p.stats_in[worker] : make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    for (int row = worker; row < p.M; row += workers) {
        fetch(row + (p.depth - 1) * workers, slot == 0 ? p.depth - 1 : slot - 1);  // the slot of the row before
        int lr;
        const int js = shard_of(p, row, lr);
        const long long e = static_cast<long long>(lr) * p.H;
        const float4 st = st_next;
        if (row + workers < p.M) st_next = p.stats_in[row + workers];
        const float gm = p.gate == TP_GATE_TOKEN ? load1<A>(p.g[js], lr) : 1.0f;
        copies_wait(p.depth - 1);
        const uint8_t *at = stages + slot * stage_bytes;
        slot = slot + 1 == p.depth ? 0 : slot + 1;
        float2 d[K][P];  // dy, then D
        if (has_dy) {
            staged<R>(at, c, d);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) d[k][j] = both(0.0f);
        }
        if (has_pre) {
            float2 yh[K][P], h[K][P], s0 = both(0.0f), s1 = both(0.0f);
            staged<R>(at, c, yh);
            staged<A>(at, c, h);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (LN) yh[k][j] = __fadd2_rn(yh[k][j], both(-st.z));
                    yh[k][j] = __fmul2_rn(yh[k][j], both(st.w));
                    n1[k][j] = __ffma2_rn(h[k][j], yh[k][j], n1[k][j]);  // h is zero past the row
                    if (LN) n0[LN ? k : 0][j] = __fadd2_rn(n0[LN ? k : 0][j], h[k][j]);
                    h[k][j] = __fmul2_rn(h[k][j], nw[k][j]);
                    if (LN) s0 = __fadd2_rn(s0, h[k][j]);
                    s1 = __ffma2_rn(h[k][j], yh[k][j], s1);
                }
            float m0 = s0.x + s0.y, m1 = s1.x + s1.y, none;
            if (LN)
                row_sum<TEAM, false>(m0, m1, none, r);
            else
                row_sum<TEAM>(m1, r);
            m0 = LN && p.pre == TP_NORM_LAYER ? -st.w * m0 * inv_h : 0.0f;
            m1 *= -st.w * inv_h;
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
                store<R, V>(p.dx[js], e + c.at(k), o);
            }
        if (!p.has_block) continue;
        float2 fh[K][P], s0 = both(0.0f), s1 = both(0.0f), s2 = both(0.0f);
        if (p.need_f) {
            staged<A>(at, c, fh);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (LN) fh[k][j] = __fadd2_rn(fh[k][j], both(-st.x));  // no post-norm: mean 0, 1 / spread 1
                    fh[k][j] = __fmul2_rn(fh[k][j], both(st.y));
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
                        if (p.post == TP_NORM_LAYER) {
                            load<A, V>(p.post_b, c.at(k), w);
#pragma unroll
                            for (int j = 0; j < P; ++j) pv[j] = __fadd2_rn(pv[j], w[j]);
                        }
                    }
                    if (gate_rows) {
                        load<A, V>(at, static_cast<int>(k * c.lanes + threadIdx.x) * V, w);
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            pv[j] = __fmul2_rn(__fmul2_rn(d[k][j], pv[j]), both(p.c));
                            d[k][j] = __fmul2_rn(d[k][j], w[j]);
                        }
                        store<A, V>(p.dg[js], e + c.at(k), pv);
                    } else {
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            s2 = __ffma2_rn(d[k][j], pv[j], s2);
                            d[k][j] = __fmul2_rn(d[k][j], both(gm));
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    p1[k][j] = __ffma2_rn(d[k][j], fh[k][j], p1[k][j]);
                    if (LN) p0[LN ? k : 0][j] = __fadd2_rn(p0[LN ? k : 0][j], d[k][j]);
                    d[k][j] = __fmul2_rn(d[k][j], gw[k][j]);  // the gradient of fh
                    if (LN) s0 = __fadd2_rn(s0, d[k][j]);
                    s1 = __ffma2_rn(d[k][j], fh[k][j], s1);
                }
            }
        float m0 = s0.x + s0.y, m1 = s1.x + s1.y, dg = s2.x + s2.y;
        if (p.gate == TP_GATE_TOKEN) {
            row_sum<TEAM, true>(m0, m1, dg, r);
            if (first) store1<A>(p.dg[js], lr, p.c * dg);
        } else if (p.post != TP_NORM_NONE) {
            if (LN)
                row_sum<TEAM, false>(m0, m1, dg, r);
            else
                row_sum<TEAM>(m1, r);
        }
        m0 = LN && p.post == TP_NORM_LAYER ? -st.y * m0 * inv_h : 0.0f;
        m1 = p.post != TP_NORM_NONE ? -st.y * m1 * inv_h : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c.on[k]) {
                float2 o[P];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    o[j] = __ffma2_rn(fh[k][j], both(m1), both(m0));
                    o[j] = __ffma2_rn(d[k][j], both(st.y), o[j]);
                }
                store<A, V>(p.df[js], e + c.at(k), o);
            }
    }
    // the parameter gradients' blocks may take the SMs that are done; they wait for the whole grid
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // one row of partial sums a worker (the warps of a block added in order)
    const int out_row = WARP ? blockIdx.x : worker, out_rows = WARP ? gridDim.x : workers;
    int used = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (!p.use[q]) continue;
        float *out = p.partials + (static_cast<long long>(used++) * out_rows + out_row) * p.H;
        float2 (*acc)[P] = q == 0 ? p1 : q == 1 ? p0 : q == 2 ? n1 : n0;
        if (WARP) {
            // the stages' memory serves again: every row has been read
            float *comb = reinterpret_cast<float *>(stages);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j)
                    *reinterpret_cast<float2 *>(comb + (threadIdx.x >> 5) * E * 32 + c.at(k) + 2 * j) = acc[LN || !(q & 1) ? k : 0][j];
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
                        const float2 u = acc[LN || !(q & 1) ? k : 0][j], v = acc[LN || !(q & 1) ? k : 0][j + 1];
                        *reinterpret_cast<float4 *>(out + c.at(k) + 2 * j) = make_float4(u.x, u.y, v.x, v.y);
                    }
                }
        }
    }
    if (TEAM == kCluster) cluster_sync();  // no block leaves while another may write into it
}

// Parameter gradients from the partial rows: 32 columns a block, 32 threads a
// column quadruple, the rows in a fixed order.
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
    __shared__ float part[4][32][33];
    const int quad = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int c0 = blockIdx.x * 32 + quad * 4;  // H is a multiple of 8: a quadruple is whole or absent
    float4 s[4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int slot = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        s[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!p.use[q]) continue;
        const float *in = p.partials + static_cast<long long>(slot++) * p.chunks * p.H + c0;
        if (c0 < p.H)
#pragma unroll 5
            for (int i = r; i < p.chunks; i += 32) {
                const float4 v = *reinterpret_cast<const float4 *>(in + static_cast<long long>(i) * p.H);
                s[q].x += v.x; s[q].y += v.y; s[q].z += v.z; s[q].w += v.w;
            }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        part[q][r][quad * 4] = s[q].x;
        part[q][r][quad * 4 + 1] = s[q].y;
        part[q][r][quad * 4 + 2] = s[q].z;
        part[q][r][quad * 4 + 3] = s[q].w;
    }
    __syncthreads();
    // 8 lanes a column: 4 rows each, then over the lanes
    const int own = threadIdx.x >> 3, eighth = threadIdx.x & 7, col = blockIdx.x * 32 + own;
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[q] += part[q][eighth * 4 + i][own];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v[q] += __shfl_xor_sync(0xffffffffu, v[q], o);
    }
    if (eighth || col >= p.H) return;
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
// (those that the kernel reads): rows of up to 1024 columns by a warp with 8,
// 16 or 32 elements a lane, wider ones by a block with 8 or 16 elements a
// thread, and where a block's threads or its shared memory (two stages at
// least) do not hold a row, by a cluster of 2 or 4 blocks.
struct Shape {
    bool warp;
    int E, threads, cluster, depth;
    int smem;
};
// dynamic shared memory of a block when `blocks` of them share an SM's 228 KB
// (each also takes 1.5 KB of static buffers and 1 KB of the system's)
static int smem_share(int blocks) { return (blocks == 1 ? 225 : 228) * 1024 / blocks - 2560; }

static Shape shape_of(int H, int bytes, int blocks_per_sm) {
    Shape s;
    s.cluster = 1;
    s.E = H <= 256 ? 8 : H <= 512 ? 16 : 32;
    s.threads = 32 * kWarps;
    s.warp = H <= 1024 && 2 * s.threads * s.E * bytes <= smem_share(1);
    if (!s.warp) {
        while (H > s.cluster * kMaxThreads * 16 || 2 * bytes * ((H + s.cluster - 1) / s.cluster + 512) > smem_share(1))
            s.cluster *= 2;
        const int cols = (H + s.cluster - 1) / s.cluster;
        s.E = cols <= kMaxThreads * 8 ? 8 : 16;
        s.threads = ((cols + s.E - 1) / s.E + 31) / 32 * 32;
    }
    const int stage = s.threads * s.E * bytes;
    s.depth = smem_share(blocks_per_sm) / stage;
    s.depth = s.depth < 2 ? 2 : s.depth > kMaxDepth ? kMaxDepth : s.depth;
    s.smem = s.depth * stage;
    if (s.warp && s.smem < kWarps * s.E * 32 * 4) s.smem = kWarps * s.E * 32 * 4;  // the warps' sums at the end
    return s;
}

using Kernel = void (*)(Plan);
template <typename A, typename R, bool BWD, bool LN>
static Kernel pick(const Shape &s) {
    if (BWD) {
        if (s.warp) return s.E == 8 ? bwd_kernel<A, R, 8, kWarp, LN> : s.E == 16 ? bwd_kernel<A, R, 16, kWarp, LN> : bwd_kernel<A, R, 32, kWarp, LN>;
        if (s.cluster > 1) return s.E == 8 ? bwd_kernel<A, R, 8, kCluster, LN> : bwd_kernel<A, R, 16, kCluster, LN>;
        return s.E == 8 ? bwd_kernel<A, R, 8, kBlock, LN> : bwd_kernel<A, R, 16, kBlock, LN>;
    }
    if (s.warp) return s.E == 8 ? fwd_kernel<A, R, 8, kWarp, LN> : s.E == 16 ? fwd_kernel<A, R, 16, kWarp, LN> : fwd_kernel<A, R, 32, kWarp, LN>;
    if (s.cluster > 1) return s.E == 8 ? fwd_kernel<A, R, 8, kCluster, LN> : fwd_kernel<A, R, 16, kCluster, LN>;
    return s.E == 8 ? fwd_kernel<A, R, 8, kBlock, LN> : fwd_kernel<A, R, 16, kBlock, LN>;
}
template <bool BWD, bool LN>
static Kernel pick(const tp_block_norm_desc &d, const Shape &s) {
    using bf = __nv_bfloat16;
    if (d.dtype == TP_DT_F32) return pick<float, float, BWD, LN>(s);
    return d.residual_f32 ? pick<bf, float, BWD, LN>(s) : pick<bf, bf, BWD, LN>(s);
}

// A kernel and how many of its blocks an SM holds; the handle keeps the last
// device's, so that a call does not ask the runtime again.
struct Launch {
    Kernel k = nullptr;
    Shape s;
    int per_sm = 0, device = -1;
};
static std::mutex g_launch_mutex;

static tp_status prepare(Launch &kept, const tp_block_norm_desc &d, bool bwd, int bytes, Launch &l) {
    int dev = 0;
    TRY(cuda_check(cudaGetDevice(&dev), "cudaGetDevice"));
    std::lock_guard<std::mutex> lock(g_launch_mutex);
    l = kept;
    if (l.device == dev) return TP_OK;
    const bool ln = d.post == TP_NORM_LAYER || d.pre == TP_NORM_LAYER;
    // the deepest stages that still leave room for the blocks that registers allow
    int want = 1;
    for (;;) {
        l.s = shape_of(d.H, bytes, want);
        l.k = bwd ? (ln ? pick<true, true>(d, l.s) : pick<true, false>(d, l.s))
                  : (ln ? pick<false, true>(d, l.s) : pick<false, false>(d, l.s));
        TRY(cuda_check(cudaFuncSetAttribute(l.k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_share(1)), "block norm"));
        int by_registers = 0;
        TRY(cuda_check(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&by_registers, l.k, l.s.threads, 0), "block norm"));
        if (by_registers <= want || l.s.depth == 2) break;
        want = by_registers;
    }
    TRY(cuda_check(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&l.per_sm, l.k, l.s.threads, l.s.smem), "block norm"));
    if (l.per_sm < 1) return set_error(TP_ERR_CUDA, "block norm: no block fits an SM");
    l.device = dev;
    kept = l;
    return TP_OK;
}

static tp_status run(const Launch &l, Plan &p, int most, const char *name, cudaStream_t st, int *workers) {
    const Shape &s = l.s;
    const int rows = s.warp ? kWarps : 1;
    int blocks = l.per_sm * num_sms() / s.cluster;
    if (blocks > (p.M + rows - 1) / rows) blocks = (p.M + rows - 1) / rows;
    if (most && blocks > most) blocks = most;
    if (blocks < 1) blocks = 1;
    p.cluster = s.cluster;
    p.depth = s.depth;
    *workers = blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks * s.cluster);
    cfg.blockDim = dim3(s.threads);
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.cluster > 1 ? 1 : 0;
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
    bn::Launch fwd, bwd;
};

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
    const int ea = d.dtype == TP_DT_F32 ? 4 : 2, er = d.residual_f32 ? 4 : ea;
    bn::Launch l;
    TRY(bn::prepare(h->fwd, d, false, er + (d.has_block ? ea : 0) + (d.gate == TP_GATE_ELEMENT ? ea : 0), l));
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
        const int ea = d.dtype == TP_DT_F32 ? 4 : 2, er = d.residual_f32 ? 4 : ea;
        p.need_f = d.has_block && (d.post != TP_NORM_NONE || d.gate != TP_GATE_NONE);
        const bool pre = d.pre != TP_NORM_NONE;
        bn::Launch l;
        TRY(bn::prepare(h->bwd, d, true,
                        er + (pre ? er + ea : 0) + (p.need_f ? ea : 0) + (d.gate == TP_GATE_ELEMENT ? ea : 0), l));
        TRY(bn::run(l, p, bn::kMaxChunks, "block_norm_bwd", st, &grid));
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
    cfg.gridDim = dim3((d.H + 31) / 32);
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
