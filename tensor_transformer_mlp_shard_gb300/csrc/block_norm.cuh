// Device code shared by the block norm's forward and backward kernels (see
// block_norm.cu for the mathematics): vectors, staging, sums over a row.
#pragma once

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"

namespace tpmlp {
namespace bn {

constexpr int kWarps = 8;           // warps of a block in the warp-per-row kernels
constexpr int kMaxThreads = 512;    // threads of a block in the block-per-row kernels
constexpr int kMaxCluster = 4;      // blocks that share a row
constexpr int kSlots = 16 * kMaxCluster;  // partial sums of a row: one a warp
constexpr int kMaxH = 16384;
constexpr int kSmemMost = 225 * 1024 - 2560;  // dynamic shared memory; the static buffers and the system take the rest
// workers of the backward, each writing one row of partial sums: two blocks an
// SM for rows of 4096 columns and more, up to eight for narrower ones
constexpr int max_chunks(int H) { return H >= 4096 ? 304 : H <= 1024 ? 1216 : 304 * 4096 / H; }

struct Plan {
    int M, H, rows_split;
    int post, pre, gate, zero_centered, has_block;
    int cluster, need_f;            // blocks to a row; f is read
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

// (a row's start is the same for the whole block: a thread's own part of an
// address is 32 bits and the same in every row)
template <typename T, int V>
__device__ __forceinline__ void load(const void *base, uint32_t e, float2 *v) {
    Pack<T, V>::unpack(*reinterpret_cast<const typename Pack<T, V>::Raw *>(static_cast<const T *>(base) + e), v);
}
template <typename T, int V>
__device__ __forceinline__ void store(void *base, uint32_t e, const float2 *v) {
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

// A worker's rows: every `step`th, with the token shard that holds each and the
// row's place there (one division at the start, none a row).
struct Cursor {
    int row, step, shard, local;
    __device__ __forceinline__ Cursor(const Plan &p, int first, int s) : row(first), step(s) {
        shard = p.rows_split ? row / p.rows_split : 0;
        local = row - shard * p.rows_split;
    }
    __device__ __forceinline__ void advance(const Plan &p) {
        row += step;
        local += step;
        if (p.rows_split)
            while (local >= p.rows_split) {
                local -= p.rows_split;
                ++shard;
            }
    }
};

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
// all but the newest group have landed
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }
// Programmatic dependent launch: a kernel may start while the one before it in
// the stream ends, sets up what is its own, and waits before it touches memory.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
constexpr int kStages = 2;  // a row being worked on and the next (3 and 4 measured no faster)

// a thread's columns: vector k starts at column first + k * step
template <int K, int V>
struct Columns {
    uint32_t first, step, lanes;  // lanes: threads of the block (the stride of staged vectors)
    bool on[K], ragged;           // ragged: the row ends within this block's (or warp's) columns
    __device__ __forceinline__ uint32_t at(int k) const { return first + k * step; }
};

template <typename T, int K, int V>
__device__ __forceinline__ uint32_t stage(uint32_t at, const void *row, const Columns<K, V> &c) {
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (c.on[k])
            copy_async<T, V>(at + (k * c.lanes + threadIdx.x) * static_cast<uint32_t>(V * sizeof(T)), static_cast<const T *>(row) + c.at(k));
    return at + K * c.lanes * static_cast<uint32_t>(V * sizeof(T));
}
// the staged vectors of one array; `at` moves to the next array
template <typename T, int K, int V>
__device__ __forceinline__ void staged(const uint8_t *&at, const Columns<K, V> &c, float2 (&v)[K][V / 2]) {
#pragma unroll
    for (int k = 0; k < K; ++k) load<T, V>(at, (k * c.lanes + threadIdx.x) * V, v[k]);
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
    float (*red)[3][kSlots];  // [2][value][block of the cluster x warp]
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
__device__ __forceinline__ Reduce make_reduce(float (*red)[3][kSlots], const Plan &p) {
    Reduce r = {red, 0, TEAM == kCluster ? p.cluster : 1, 0};
    if (TEAM == kWarp) return r;
    // warps that a block does not have add nothing
    for (int i = threadIdx.x; i < 2 * 3 * kSlots; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;
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
    for (int k = 0; k < K; ++k) c.on[k] = c.at(k) < static_cast<uint32_t>(p.H);
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

// Mean of a normalised row, v = (x - mean) / spread, for every thread of it.
// The statistics hold the mean rounded to fp32, so it is not zero but up to 2^-24
// |mean| / spread, the same for all columns: a bias, which a sum over tokens
// does not average out.  Up to a mean of one spread that is within v's own
// rounding; the backward takes it off the rows whose mean is larger (one row's
// condition, the same for all threads that work on it).
__device__ __forceinline__ bool far_from_zero(float mean, float rstd) { return fabsf(mean) * rstd > 1.0f; }
template <Team TEAM, int V, int K>
__device__ __forceinline__ float mean_left(const float2 (&v)[K][V / 2], const Columns<K, V> &c, float inv_h, Reduce &r) {
    float2 s = both(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (c.on[k]) {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) s = __fadd2_rn(s, v[k][j]);
        }
    float rest = s.x + s.y;
    row_sum<TEAM>(rest, r);
    return rest * inv_h;
}

// A vector of per-channel factors of a thread's columns: zero past the row's
// end, where what it multiplies may be anything finite.  KEEP: read once and
// kept in registers; otherwise read again (from L1 or L2) at every row, where
// the registers are worth more.
//   weight: w (1 + w when zero-centred), `none` without one; gated: times the
//   channel gate and the block's scale.
template <typename A, int K, int V, bool KEEP>
struct Factors {
    float2 kept[KEEP ? K : 1][V / 2];
    __device__ __forceinline__ static void read(const Plan &p, const Columns<K, V> &c, int k, const void *w, float plus,
                                                float none, bool gated, float2 *v) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[j] = both(c.on[k] ? none : 0.0f);
        if (w && c.on[k]) {
            load<A, V>(w, c.at(k), v);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) v[j] = __fadd2_rn(v[j], both(plus));
        }
        if (!gated) return;
        if (p.gate == TP_GATE_CHANNEL && c.on[k]) {
            float2 g[V / 2];
            load<A, V>(p.g[0], c.at(k), g);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) v[j] = __fmul2_rn(v[j], g[j]);
        }
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[j] = __fmul2_rn(v[j], both(p.c));
    }
    __device__ __forceinline__ void keep(const Plan &p, const Columns<K, V> &c, const void *w, float plus, float none,
                                         bool gated) {
        if constexpr (KEEP) {
#pragma unroll
            for (int k = 0; k < K; ++k) read(p, c, k, w, plus, none, gated, kept[k]);
        }
    }
    __device__ __forceinline__ void get(const Plan &p, const Columns<K, V> &c, int k, const void *w, float plus,
                                        float none, bool gated, float2 *v) const {
        if constexpr (KEEP) {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) v[j] = kept[k][j];
        } else {
            read(p, c, k, w, plus, none, gated, v);
        }
    }
};

// Which kernel a row takes (chosen in block_norm.cu).
struct Shape {
    int team, E, threads, cluster, smem;
    bool common;  // what almost every call has; see the kernels
};
using Kernel = void (*)(Plan);
Kernel fwd_kernel_bf16(const tp_block_norm_desc &d, const Shape &s);
Kernel fwd_kernel_mixed(const tp_block_norm_desc &d, const Shape &s);
Kernel fwd_kernel_f32(const tp_block_norm_desc &d, const Shape &s);
Kernel bwd_kernel_bf16(const tp_block_norm_desc &d, const Shape &s);
Kernel bwd_kernel_mixed(const tp_block_norm_desc &d, const Shape &s);
Kernel bwd_kernel_f32(const tp_block_norm_desc &d, const Shape &s);

}  // namespace bn
}  // namespace tpmlp
