// What the kernels around the attention projections share: the shards' head
// layout, the position rotation, the paged cache's addressing.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "internal.h"

namespace tpmlp {
namespace attn {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxPairs = kMaxHeadDim / 2;
constexpr int kMaxRows = 1 << 20;  // rows of a call, and rows and columns of its table

__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// n / d for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1 (Granlund and Montgomery, 1994) the quotient
// is (n + hi(m n)) >> l; the sum fits 32 bits.
struct Divisor {
    uint32_t m = 1, l = 0, d = 1;
    Divisor() = default;
    explicit Divisor(uint32_t by) : d(by) {
        while ((1ull << l) < by) ++l;
        m = static_cast<uint32_t>((((1ull << l) - by) << 32) / by + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (n + __umulhi(n, m)) >> l; }
    __device__ __forceinline__ uint32_t divmod(uint32_t n, uint32_t &rest) const {
        const uint32_t q = div(n);
        rest = n - q * d;
        return q;
    }
};

// The paged cache's geometry and the rows' places in it.
struct Pages {
    const int32_t *positions, *sequences, *table;
    int n, table_rows, table_cols, pages, page_size;
    Divisor page;
    unsigned *index_word;  // takes `owner` when an index is out of range
    unsigned owner;
};

// 448 / amax, or 1 where that would not be a normal number
__device__ __forceinline__ float cache_scale(const float *amax, int head) {
    const float a = amax[head];
    return a >= 0x1p-100f && a <= 3.0e38f ? 448.0f / a : 1.0f;
}

__device__ __forceinline__ void bad_index(const Pages &p) { *reinterpret_cast<volatile unsigned *>(p.index_word) = p.owner; }

// The pairs' angles per position in turns, as fractions of 2^64: a position
// times one of them wraps to the exact angle within the turn, which a
// product in 32 bits (or 64, far out) loses.
struct Turns {
    uint64_t per_position[kMaxPairs];
    float a;  // attention factor
};

tp_status rope_validate(const tp_rope_desc *r, int head_dim);
void rope_turns(const tp_rope_desc &r, Turns *t);

// a cos and a sin of pair i at position p: the angle to 2^-33 of a turn, taken
// to the nearest quarter turn in integers so that the rest, at most an eighth,
// is fp32 to 2^-25 of itself
__device__ __forceinline__ float2 turn(const Turns &t, int i, int p) {
    const uint64_t phase = t.per_position[i] * static_cast<uint32_t>(p);
    const uint32_t hi = static_cast<uint32_t>((phase + 0x80000000ull) >> 32);
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    const int rest = static_cast<int>(hi - (quarter << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
    // quarter 0: (c, s)  1: (-s, c)  2: (-c, -s)  3: (s, -c)
    return make_float2((quarter == 1 || quarter == 2 ? -x : x) * t.a, (quarter & 2 ? -y : y) * t.a);
}

// Decode attention (paged_decode.cu).
struct DecodePlan {
    const void *q[kMaxShards], *k[kMaxShards], *v[kMaxShards];
    void *o[kMaxShards];
    Pages at;
    int hq, hk, per;       // query and key heads of a shard, query heads of a key head
    int groups, nh;        // groups that a key head's queries are cut into, queries of a group
    int row_heads;         // T * hk * groups
    Divisor by_hk, by_groups;
    int D, window;
    float scale_log2;      // scale * log2(e)
    const float *k_amax, *v_amax;
    float *partial;        // [blocks][2][nh * (D + 2)]
    int4 *joins;           // [blocks]
    int resident;          // blocks that run at once
    int join_early;        // the kernel after the join may start beside it
    int by_segment;        // joins are listed by (row, head) rather than by block
};
size_t decode_workspace_bytes(const tp_paged_desc &d);
tp_status launch_decode(DecodePlan &p, int dtype, void *workspace, cudaStream_t st);

}  // namespace attn
}  // namespace tpmlp
