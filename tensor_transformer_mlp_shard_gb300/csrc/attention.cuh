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
    float a, a_rest;  // attention factor, and what its rounding lost
};

tp_status rope_validate(const tp_rope_desc *r, int head_dim);
void rope_turns(const tp_rope_desc &r, Turns *t);

// a cos and a sin at position p of a pair's turn, rounded as if they had been exact
// (up to position 32768 but for one in 1000; one in 50 with 32 bits of the angle):
// keys in 8 bits should lie on the same side of a code's edge as the definition's.
// The angle is taken to the nearest quarter in integers; the rest x, an eighth of
// a turn at most, and the first two terms of either series are pairs of fp32
// numbers (Dekker's products and Knuth's sums), the later terms, Taylor's up to
// x^13, single ones.  About 60 operations a pair and token, against some 1500 of
// its heads.
__device__ __forceinline__ float2 turn(const Turns &t, uint64_t per_position, int p) {
    const uint64_t phase = per_position * static_cast<uint32_t>(p);
    const uint32_t hi = static_cast<uint32_t>((phase + 0x80000000ull) >> 32);
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    const int rest = static_cast<int>(hi - (quarter << 30));
    const float rough = static_cast<float>(rest);
    // in half turns, with what the 32 bits and the conversion lost
    const float r = rough * 0x1p-31f;
    const float r_rest = fmaf(static_cast<float>(static_cast<int>(static_cast<uint32_t>(phase))), 0x1p-63f, static_cast<float>(rest - static_cast<int>(rough)) * 0x1p-31f);
    constexpr float kPi = 0x1.921fb6p+1f, kPiRest = -0x1.777a5cp-24f;                // pi
    constexpr float kSixth = 0x1.555556p-3f, kSixthRest = -0x1.555556p-28f;          // 1 / 3!
    constexpr float k24th = 0x1.555556p-5f, k24thRest = -0x1.555556p-30f;            // 1 / 4!
    const float x = __fmul_rn(r, kPi), x_rest = fmaf(r, kPi, -x) + fmaf(r, kPiRest, r_rest * kPi);
    const float z = __fmul_rn(x, x), z_rest = fmaf(x + x, x_rest, fmaf(x, x, -z));
    // sin x = x - x^3 / 6 + x^5 p(z)
    float q = 1.0f / 6227020800.0f;
    q = fmaf(q, z, -1.0f / 39916800.0f);
    q = fmaf(q, z, 1.0f / 362880.0f);
    q = fmaf(q, z, -1.0f / 5040.0f);
    q = fmaf(q, z, 1.0f / 120.0f);
    const float u = __fmul_rn(z, x), u_rest = fmaf(z, x_rest, fmaf(z_rest, x, fmaf(z, x, -u)));
    const float v = __fmul_rn(u, kSixth), v_rest = fmaf(u, kSixthRest, fmaf(u_rest, kSixth, fmaf(u, kSixth, -v)));
    const float s0 = __fsub_rn(x, v), sb = __fsub_rn(s0, x);
    const float s1 = __fsub_rn(x, __fsub_rn(s0, sb)) - __fadd_rn(v, sb) + (fmaf(__fmul_rn(z, u), q, x_rest) - v_rest);
    // cos x = 1 - z / 2 + z^2 / 24 + z^3 p(z)
    q = 1.0f / 479001600.0f;
    q = fmaf(q, z, -1.0f / 3628800.0f);
    q = fmaf(q, z, 1.0f / 40320.0f);
    q = fmaf(q, z, -1.0f / 720.0f);
    const float w = __fmul_rn(z, z), w_rest = fmaf(z + z, z_rest, fmaf(z, z, -w));
    const float y = __fmul_rn(w, k24th), y_rest = fmaf(w, k24thRest, fmaf(w_rest, k24th, fmaf(w, k24th, -y)));
    const float h = __fmul_rn(0.5f, z), c = __fsub_rn(1.0f, h), c_rest = __fsub_rn(__fsub_rn(1.0f, c), h);
    const float c0 = __fadd_rn(c, y), cb = __fsub_rn(c0, c);
    const float c1 = __fsub_rn(c, __fsub_rn(c0, cb)) + __fsub_rn(y, cb) + (fmaf(__fmul_rn(w, z), q, y_rest) + fmaf(-0.5f, z_rest, c_rest));
    // times a, in one rounding each
    const float sa = __fmul_rn(s0, t.a), ca = __fmul_rn(c0, t.a);
    const float sn = sa + fmaf(s1, t.a, fmaf(s0, t.a_rest, fmaf(s0, t.a, -sa)));
    const float cs = ca + fmaf(c1, t.a, fmaf(c0, t.a_rest, fmaf(c0, t.a, -ca)));
    const float cosine = quarter & 1 ? sn : cs, sine = quarter & 1 ? cs : sn;
    // quarter 0: (c, s)  1: (-s, c)  2: (-c, -s)  3: (s, -c)
    return make_float2(quarter == 1 || quarter == 2 ? -cosine : cosine, quarter & 2 ? -sine : sine);
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
    int cluster;           // blocks of a segment, where each has some (0: dealt out)
    int join_early;        // the kernel after the join may start beside it
    int by_segment;        // joins are listed by (row, head) rather than by block
};
size_t decode_workspace_bytes(const tp_paged_desc &d);
tp_status launch_decode(DecodePlan &p, int dtype, void *workspace, cudaStream_t st);

}  // namespace attn
}  // namespace tpmlp
