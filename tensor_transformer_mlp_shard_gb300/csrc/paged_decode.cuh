// Decode attention over a paged cache: o = sum_j w_j v_j, w = softmax(scale q.k_j).
//
// Bound by HBM: each key and value is read once, for all queries of its head.
// The positions of all rows and key heads are one list of units (64 positions; of wide
// fp32 heads 32), in order of row, head, position; every block takes an equal stretch
// of it (as many blocks as are resident), so that uneven lengths load the SMs
// evenly and one long row is split over all of them.  Within a stretch, the
// units of one (row, head) are a segment; a segment that ends in another block
// leaves its running maximum, sum and unnormalised output in the workspace, at
// most two a block, and a second kernel joins them, in the blocks' order.
//
// Four warps share a unit, 16 or 8 positions (a core's kRows) each, and keep softmax
// states of their own until the segment ends: no barrier in the loop.  Each warp has a
// ring of stages in shared memory that it fills by asynchronous 16-byte copies,
// several steps ahead; what bounds the kernel is how many bytes are on their
// way.  From there its lanes read fragments of the matrix instructions as they
// lie: the contraction over the head's elements may take them in any order, so a
// lane reads 16 contiguous bytes and its elements stand for whichever the
// instruction calls k; the same holds for the rows of V^T, which only name
// output elements.  Positions are the 16 rows of K and of P^T, the queries of a
// head its 8 columns, so that one query wastes tensor work (which is cheap
// here) and no bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "attention.cuh"

namespace tpmlp {
namespace attn {

constexpr int kWarps = 4;
constexpr int kBlock = 32 * kWarps;
constexpr int kMostResident = 768;      // blocks that run at once
constexpr int kMostBlocks = 2 * kMostResident;  // of a launch, and so of the workspace
// A segment costs its block this many positions besides its own (its pages,
// queries and first keys have to arrive, its parts to be added): without it the
// blocks that have short rows end last (fp32 window case 37 us, with it 27).
constexpr int kSegmentPositions = 192;
// A row up to this long is read by one warp where there are more segments than
// blocks.
constexpr int kShortPositions = 128;
// Rows that may see no more than kBlockPositions a block of a cluster of up to
// kCluster, and whose clusters fit three quarters of the resident blocks, have a
// cluster each.  So have rows of more than kShortPositions and up to
// kBlockPositions, a block each, where that makes no more than twice the resident
// blocks: a table's columns say little about the rows, and blocks come and go more
// slowly than a resident block's warps take short ones (8-bit, 608 segments of 256
// elements, twice the resident: of up to 500 positions 28 us, 34 by the list, of up
// to 30 13 and 11; 2432 segments: 84 and 84 us, 49 and 19).  Four times, where
// a window is the bound, which most rows will fill (8-bit, 1072 segments of 235,
// 2.4 times the resident: 25 us, 30 by the list).
constexpr int kCluster = 8, kBlockPositions = 512;
// With so many units a resident block, one unit in kTailShare goes to half as many blocks more.
constexpr int kSpread = 32, kTailShare = 8;

// Queries of an fp32 key head that plain fp32 products take; more go to Tf32Core,
// whose splits cost the same for up to 8 (4 queries of 256 elements: 59 us, by
// tf32 71; 16 of 128: 140 us in four passes, by tf32 78).
constexpr int kFloatQueries = 4;

enum CacheKind : int { CACHE_BF16 = 0, CACHE_FP8 = 1, CACHE_F32 = 2 };

// A segment of a row: what the warps need to walk it.
struct Segment {
    const int32_t *pages;       // the row's table
    int head, t0, t1;           // key head of the shard; steps [t0, t1)
    int first, last;            // positions that the row sees
};

// A step: R positions, the step-th R of the sequence.  They lie in one page;
// `block` is their place in the cache in blocks of R rows of head_dim, kNone
// where the row sees none of them or the page is out of range.
constexpr uint32_t kNone = 0xffffffffu;
template <int R>
__device__ __forceinline__ uint32_t block_at(const DecodePlan &p, const Segment &s, int step) {
    if (step >= s.t1) return kNone;
    const int base = step * R;
    if (base > s.last || base + R - 1 < s.first) return kNone;
    uint32_t in_page;
    const int page = s.pages[p.at.page.divmod(base, in_page)];
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.at.pages)) {
        bad_index(p.at);
        return kNone;
    }
    return (static_cast<uint32_t>(page) * p.hk + s.head) * (p.at.page_size / R) + in_page / R;
}

// the positions [lo, hi) of a step that the row sees
struct Seen {
    int lo, hi;
};
template <int R>
__device__ __forceinline__ Seen seen_at(const Segment &s, int step) {
    const int base = step * R;
    return {max(s.first - base, 0), min(s.last - base, R - 1) + 1};
}

// `bytes` of 16 bytes, 0 or 16, the rest zero
__device__ __forceinline__ void copy16(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// R rows of ROW bytes (the padded width) in a stage, the eight 16-byte pieces of
// a 128-byte line exchanged so that the fragments' reads meet no bank twice:
// keys are read four pieces of 8 rows at a time, values one or two pieces of
// every other row.
template <int ROW>
__device__ __forceinline__ int swizzle_k(int row) {
    return ROW % 128 ? 0 : (row & 1) << 6;
}
__device__ __forceinline__ int swizzle_v(int row) { return ((row >> 1) & 3) << 5; }

// A step's keys and values on their way to a stage: eight lanes copy a line of a row
// (four, half a line, where rows are not whole lines).  What lies behind the head's width, and rows
// that are not seen, become zero.
template <class Core, bool WHOLE>
__device__ __forceinline__ void fetch_rows(int row_bytes, const char *k, const char *v, const Seen &s, uint32_t to) {
    constexpr int R = Core::kRows, ROW = Core::kRowBytes, kLine = ROW % 128 ? 64 : 128, kLanes = kLine / 16, kStep = 32 / kLanes;
    const int lane = threadIdx.x & 31, row0 = lane / kLanes, at = 16 * (lane % kLanes);
    const int off = row0 * row_bytes + at;
    const uint32_t lane_to = to + row0 * ROW + at;
#pragma unroll
    for (int i = 0; i < R / kStep; ++i) {
        const int row = i * kStep + row0;
        const bool in = WHOLE || (row >= s.lo && row < s.hi);
#pragma unroll
        for (int j = 0; j < ROW / kLine; ++j) {
            const int bytes = in && j * kLine + at < row_bytes ? 16 : 0;
            const uint32_t d = lane_to + i * kStep * ROW + j * kLine;
            const int from = off + i * kStep * row_bytes + j * kLine;
            copy16(d ^ Core::swizzle_keys(row), k + from, bytes);
            copy16((d + R * ROW) ^ Core::swizzle_values(row), v + from, bytes);
        }
    }
}
template <class Core>
__device__ __forceinline__ void fetch(const DecodePlan &p, const void *k, const void *v, const Seen &s, uint32_t block, uint32_t to) {
    const int row_bytes = p.D * static_cast<int>(sizeof(typename Core::Cache));
    const uint64_t at = static_cast<uint64_t>(block) * (Core::kRows * row_bytes);
    const char *kp = static_cast<const char *>(k) + at, *vp = static_cast<const char *>(v) + at;
    if (s.lo == 0 && s.hi == Core::kRows)
        fetch_rows<Core, true>(row_bytes, kp, vp, s, to);
    else
        fetch_rows<Core, false>(row_bytes, kp, vp, s, to);
}

// 2^x to 2^-22 of itself, zero below 2^-126
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 8x8 matrix of 16-bit elements, a row to four lanes, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int KIND>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (KIND == CACHE_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// four E4M3 codes as two pairs of fp16 numbers, exactly (NaN stays NaN)
__device__ __forceinline__ void halves_of_codes(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
}

// ---------------------------------------------------------------------------
// 16-bit products: bf16 caches as they are, E4M3 codes as fp16
// ---------------------------------------------------------------------------
// Lane l = 4g + t.  Score tile: C[position][query], position g or g + 8, queries
// 2t, 2t + 1 of each 8.  Output tile: C[element][query], elements 2i and 2i + 1
// of the VD that the lane holds of every value row, the same two queries.
template <int KIND, int DP, int NT>
struct TensorCore {
    static constexpr bool k8 = KIND == CACHE_FP8;
    using Cache = typename std::conditional<k8, uint8_t, __nv_bfloat16>::type;
    using Act = __nv_bfloat16;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kTileElems = DP;
    static constexpr int kRows = 16, kRowBytes = DP * static_cast<int>(sizeof(Cache));
    // about 192 KB of stages an SM; 16 queries over codes take more registers, so fewer blocks.
    // Rows of 384 bytes: two blocks of two stages rather than one of four, whose warps were too
    // few (152 rows of up to 1000 positions, 8 key heads of 144 elements: 71 us, 88 with one)
    static constexpr bool kFewer = k8 && NT == 2;
    static constexpr int kStages = kRowBytes == 64 ? (kFewer ? 8 : 6) : kRowBytes == 128 ? (kFewer ? 6 : 4) : kRowBytes == 384 ? 2 : kRowBytes % 256 ? 4 : 3;
    static constexpr int kBlocksPerSm = (kRowBytes == 384 ? 2 : kRowBytes == 64 ? 4 : kRowBytes == 128 ? 3 : kRowBytes <= 256 ? 2 : 1) - kFewer;
    __device__ __forceinline__ static int swizzle_keys(int row) { return swizzle_k<kRowBytes>(row); }
    __device__ __forceinline__ static int swizzle_values(int row) { return swizzle_v(row); }
    static constexpr int KC = k8 ? DP / 64 : DP / 32;       // 16-byte loads of a lane's key row
    static constexpr int VD = k8 && DP % 128 == 0 ? 16 : 8; // elements of a lane's value load
    static constexpr int VB = DP / (8 * VD);
    static constexpr int VW = VD * (k8 ? 1 : 2) / 4;        // 32-bit words of one

    uint32_t q[NT][DP / 16][2];
    float sc[NT][2];     // score to log2 units, of the lane's queries
    float m[NT][2], l[NT][2];
    float acc[VB][VD / 2][NT][4];
    int g, t;

    // the group's nq queries, from the row of its first, on their way
    __device__ __forceinline__ void fetch_queries(const DecodePlan &p, const Act *qrow, int nq, uint32_t) {
        const int lane = threadIdx.x & 31;
        g = lane >> 2;
        t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = 8 * n + g;
            const Act *src = qrow + h * p.D;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                // bf16: lane's 8 elements 32c + 8t; codes: its 16 elements 64(c/2) + 16t, 8 at a time
                const int e = k8 ? 64 * (c / 2) + 16 * t + 8 * (c % 2) : 32 * c + 8 * t;
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (h < nq && e < p.D) w = *reinterpret_cast<const uint4 *>(src + e);
                q[n][2 * c][0] = w.x;
                q[n][2 * c][1] = w.y;
                q[n][2 * c + 1][0] = w.z;
                q[n][2 * c + 1][1] = w.w;
            }
        }
    }

    // the queries are there: nothing seen yet
    __device__ __forceinline__ void begin(const DecodePlan &p, int kv_head, const float *) {
        float kscale = 1.0f;
        if (k8) kscale = 1.0f / cache_scale(p.k_amax, kv_head);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float unit = p.scale_log2;
            if constexpr (k8) {
                // fp16 holds a bf16 number's bits but not its range: the query times a power of two
                // that brings its largest element to [2^14, 2^15); what falls below fp16's smallest
                // is 2^-38 of that
                float top = 0.0f;
#pragma unroll
                for (int c = 0; c < DP / 16; ++c)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        top = fmaxf(top, fmaxf(fabsf(bf16_lo(q[n][c][r])), fabsf(bf16_hi(q[n][c][r]))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // exponent of the power of two, within what two normal factors can make
                int e = 0;
                if (top > 0.0f && top <= 3.4e38f) e = min(max(14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), -113), 126);
                const float up = __int_as_float((e + 127) << 23);
#pragma unroll
                for (int c = 0; c < DP / 16; ++c)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const __half2 x = __floats2half2_rn(bf16_lo(q[n][c][r]) * up, bf16_hi(q[n][c][r]) * up);
                        q[n][c][r] = *reinterpret_cast<const uint32_t *>(&x);
                    }
                // the lanes hold query g here, queries 2t and 2t + 1 in the scores
                unit = unit * kscale;
                const int e0 = __shfl_sync(0xffffffffu, e, 8 * t), e1 = __shfl_sync(0xffffffffu, e, 8 * t + 4);
                // finite, so that a score of zero stays zero
                sc[n][0] = fminf(fmaxf(unit * __int_as_float((127 - e0) << 23), -3.0e38f), 3.0e38f);
                sc[n][1] = fminf(fmaxf(unit * __int_as_float((127 - e1) << 23), -3.0e38f), 3.0e38f);
            } else {
                sc[n][0] = sc[n][1] = unit;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                m[n][r] = -INFINITY;
                l[n][r] = 0.0f;
            }
        }
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
            for (int i = 0; i < VD / 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[b][i][n][r] = 0.0f;
    }

    float s[NT][4];

    __device__ __forceinline__ void scores(const char *k, const Seen &st) {
        float c2[NT][2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) c2[n][x][r] = 0.0f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            uint32_t kr[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 x = *reinterpret_cast<const uint4 *>(
                    k + (((g + 8 * r) * kRowBytes + 64 * c + 16 * t) ^ swizzle_k<kRowBytes>(g)));
                kr[r][0] = x.x;
                kr[r][1] = x.y;
                kr[r][2] = x.z;
                kr[r][3] = x.w;
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {  // word pairs of the load
                if constexpr (k8) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t a0, a1, a2, a3;
                        halves_of_codes(kr[0][2 * w + u], a0, a2);
                        halves_of_codes(kr[1][2 * w + u], a1, a3);
                        const int k = 4 * c + 2 * w + u;
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816<KIND>(c2[n][u], a0, a1, a2, a3, q[n][k][0], q[n][k][1]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816<KIND>(c2[n][w], kr[0][2 * w], kr[1][2 * w], kr[0][2 * w + 1], kr[1][2 * w + 1],
                                       q[n][2 * c + w][0], q[n][2 * c + w][1]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[n][r] = (c2[n][0][r] + c2[n][1][r]) * sc[n][r & 1];
        if (st.lo > 0 || st.hi < 16) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = r < 2 ? g : g + 8;
                    if (row < st.lo || row >= st.hi) s[n][r] = -INFINITY;
                }
        }
    }

    // The weights as the sum of two 16-bit numbers: one bf16 would be off by as much
    // as the output's own rounding.  The second product is free for bf16 caches,
    // bound by memory, and costs 2% with codes (8-bit batch 132 us with one fp16, 135
    // us with two).  Two bf16 hold a weight to 2^-17 of itself.  Two fp16 hold it to
    // 2^-22, but not finer than 2^-25, where their steps end; and small weights may
    // be all that an output is made of, where the value at the dominant position is
    // zero.  So with codes the weights are 2^kUp at the reference m, and m follows the
    // steps' largest down as well as up: a step whose largest weight is below
    // 2^(kUp - kDrop) has m lowered to it, and its weights are held to 2^-22 of that one.
    // Softmaxes without a dominant position hardly get there (scores of standard
    // deviation 3.6: one step of 16 in 2000), and pay for the look (8-bit batch 142 us,
    // 139 without; each row with such a position 144 us).
    static constexpr float kUp = k8 ? 15.0f : 0.0f, kDrop = 18.0f;
    // The sum of weights stays below 2^kMostSum when the reference falls, and so the
    // outputs finite: weights below 2^-70 of the largest are held to fewer digits, below
    // 2^-88 to none.
    static constexpr int kMostSum = 64;
    // In a step that moves the reference down, or up by kRise, positions that are alone at
    // the top (none from kSmall to kLarge) go first, and those below kSmall in another pass.
    static constexpr float kRise = 14.0f, kSmall = 0x1p-8f, kLarge = 0x1p6f;
    static constexpr int kPasses = 6;  // at most: the last takes all that is left
    uint32_t ph[NT][2], pl[NT][2];

    // scores to weights; codes: whether the reference has far to go, up (it has been) or down
    __device__ __forceinline__ bool softmax() {
        float top[NT][2];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = fmaxf(s[n][r], s[n][r + 2]);
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                top[n][r] = x;
                if constexpr (k8)
                    move |= !(fabsf(x - m[n][r] - (kUp - 0.5f * kDrop)) <= 0.5f * kDrop);  // 2^-3 to 2^15
                else
                    move |= x > m[n][r];
            }
        bool far = false, up = false;
        if (__any_sync(0xffffffffu, move)) {
            if constexpr (k8) {
                bool rise = false, fall = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        // rounded up, so that no weight is above 2^kUp, to a whole number, so that what is
                        // there is scaled without error however often the reference goes up and down
                        top[n][r] = ceilf(__fadd_ru(top[n][r], -kUp));
                        rise |= top[n][r] > m[n][r] + kRise;
                        fall |= top[n][r] < m[n][r] - kDrop;
                    }
                up = __any_sync(0xffffffffu, rise);
                far = __any_sync(0xffffffffu, fall);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float now = fmaxf(m[n][r], top[n][r]);
                    const float f = now == -INFINITY ? 1.0f : exp2_fast(m[n][r] - now);
                    m[n][r] = now;
                    l[n][r] *= f;
                    scale_outputs(n, r, f);
                }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float top_of = m[n][r & 1] == -INFINITY ? 0.0f : m[n][r & 1];
                s[n][r] = exp2_fast(s[n][r] - top_of);
            }
        if (up && !far) {  // a row's first step, as a rule: nothing to do but beside a dominant position
            bool small = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) small |= s[n][r] > 0.0f && s[n][r] < kSmall;
            far = __any_sync(0xffffffffu, small);
        }
        return far;
    }

    __device__ __forceinline__ void scale_outputs(int n, int r, float f) {
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
            for (int i = 0; i < VD / 2; ++i) {
                acc[b][i][n][r] *= f;
                acc[b][i][n][r + 2] *= f;
            }
    }

    // four weights of the lane into the sums and, as pairs of 16-bit numbers, transposed
    __device__ __forceinline__ void take(int n, const float (&w)[4]) {
        l[n][0] += w[0] + w[2];
        l[n][1] += w[1] + w[3];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if constexpr (k8) {
                const __half2 x = __floats2half2_rn(w[2 * r], w[2 * r + 1]);
                const __half2 y = __floats2half2_rn(w[2 * r] - __low2float(x), w[2 * r + 1] - __high2float(x));
                ph[n][r] = transpose8(*reinterpret_cast<const uint32_t *>(&x));
                pl[n][r] = transpose8(*reinterpret_cast<const uint32_t *>(&y));
            } else {
                const uint32_t hi = pack_bf16x2(w[2 * r], w[2 * r + 1]);
                ph[n][r] = transpose8(hi);
                pl[n][r] = transpose8(pack_bf16x2(w[2 * r] - bf16_lo(hi), w[2 * r + 1] - bf16_hi(hi)));
            }
        }
    }

    // Lowers the reference to the weights that are left where they are small, and takes
    // them, or the uppermost where these are alone.  Returns whether any are left: a
    // query's largest never is.  No lane goes a way of its own.
    __device__ __forceinline__ bool take_lowered(int pass) {
        bool left = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float w[4], x[2];
            int exponent[2];
            bool small = false;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                x[c] = fmaxf(s[n][c], s[n][c + 2]);
#pragma unroll
                for (int o = 4; o < 32; o *= 2) x[c] = fmaxf(x[c], __shfl_xor_sync(0xffffffffu, x[c], o));
                exponent[c] = x[c] > 0.0f ? static_cast<int>(__float_as_uint(x[c]) >> 23) - 127 : 0;
                small |= exponent[c] < static_cast<int>(kUp - kDrop);
            }
            if (__any_sync(0xffffffffu, small)) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float all = l[n][c];
#pragma unroll
                    for (int o = 4; o < 32; o *= 2) all += __shfl_xor_sync(0xffffffffu, all, o);
                    const int sum = static_cast<int>(__float_as_uint(all) >> 23) - 126;  // all < 2^sum; NaN: above kMostSum
                    const int by = exponent[c] < static_cast<int>(kUp - kDrop) ? max(min(14 - exponent[c], kMostSum - sum), 0) : 0;
                    const float now = __fadd_ru(m[n][c], -static_cast<float>(by));
                    const float f = by > 0 ? exp2_fast(m[n][c] - now) : 1.0f;
                    m[n][c] = now;
                    l[n][c] *= f;
                    scale_outputs(n, c, f);
                    s[n][c] *= f;
                    s[n][c + 2] *= f;
                    x[c] *= f;
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bool among = (s[n][c] >= kSmall && s[n][c] < kLarge) || (s[n][c + 2] >= kSmall && s[n][c + 2] < kLarge);
                const uint32_t lanes = __ballot_sync(0xffffffffu, among) & (0x11111111u << t);
                const bool alone = x[c] >= kLarge && lanes == 0u && pass < kPasses - 1;
#pragma unroll
                for (int r = c; r < 4; r += 2) {
                    const bool later = alone && s[n][r] < kSmall;  // NaN is taken
                    w[r] = later ? 0.0f : s[n][r];
                    s[n][r] = later ? s[n][r] : 0.0f;
                    left |= s[n][r] > 0.0f;
                }
            }
            take(n, w);
        }
        return __any_sync(0xffffffffu, left);
    }

    __device__ __forceinline__ void values(const char *v) {
#pragma unroll
        for (int b = 0; b < VB; ++b) {
            uint32_t vr[4][VW];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 2 * t + (r & 1) + 8 * (r >> 1);  // swizzled as row 2t is
                const char *at = v + ((row * kRowBytes + 32 * VW * b + 4 * VW * g) ^ (t << 5));
                if constexpr (VW == 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(at);
                    vr[r][0] = x.x;
                    vr[r][1] = x.y;
                    vr[r][2] = x.z;
                    vr[r][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(at);
                    vr[r][0] = x.x;
                    vr[r][1] = x.y;
                }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                // the same element of two neighbouring positions to one register
#pragma unroll
                for (int u = 0; u < (k8 ? 2 : 1); ++u) {
                    uint32_t a0, a1, a2, a3;
                    if constexpr (k8) {
                        const uint32_t x = __byte_perm(vr[0][w], vr[1][w], u ? 0x7362 : 0x5140);
                        const uint32_t y = __byte_perm(vr[2][w], vr[3][w], u ? 0x7362 : 0x5140);
                        halves_of_codes(x, a0, a1);
                        halves_of_codes(y, a2, a3);
                    } else {
                        a0 = __byte_perm(vr[0][w], vr[1][w], 0x5410);
                        a1 = __byte_perm(vr[0][w], vr[1][w], 0x7632);
                        a2 = __byte_perm(vr[2][w], vr[3][w], 0x5410);
                        a3 = __byte_perm(vr[2][w], vr[3][w], 0x7632);
                    }
                    const int i = k8 ? 2 * w + u : w;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816<KIND>(acc[b][i][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
                        mma16816<KIND>(acc[b][i][n], a0, a1, a2, a3, pl[n][0], pl[n][1]);
                    }
                }
            }
        }
    }

    // one step, its stage in shared memory
    __device__ __forceinline__ void step(const DecodePlan &, const char *stage, const Seen &seen) {
        scores(stage, seen);
        const bool far = softmax();
        const char *v = stage + kRows * kRowBytes;
        if (k8 && far) {
            bool left;
            int pass = 0;
            do {
                left = take_lowered(pass++);
                __syncwarp();
                values(v);
            } while (left);
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) take(n, s[n]);
            values(v);
        }
    }

    // the warp's state to shared memory: out [kHeads][DP], top and sum [kHeads]
    __device__ __forceinline__ void finish(const DecodePlan &p, float *out, float *top, float *sum) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = l[n][r];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                const int h = 8 * n + 2 * t + r;
                if (g == 0) {
                    top[h] = m[n][r];
                    sum[h] = x;
                }
#pragma unroll
                for (int b = 0; b < VB; ++b)
#pragma unroll
                    for (int i = 0; i < VD / 2; i += 2)
                        *reinterpret_cast<float4 *>(out + h * DP + 8 * VD * b + VD * g + 2 * i) =
                            make_float4(acc[b][i][n][r], acc[b][i][n][r + 2], acc[b][i + 1][n][r], acc[b][i + 1][n][r + 2]);
            }
    }
};

// ---------------------------------------------------------------------------
// fp32 products
// ---------------------------------------------------------------------------
// Eight lanes share a position, DP / 8 elements each; the four groups of lanes
// keep softmax states of their own.  Queries lie in shared memory, a copy for each
// warp.
template <int DP, int NH>
struct FloatCore {
    using Cache = float;
    using Act = float;
    static constexpr int kHeads = NH;
    static constexpr int kTileElems = DP;
    static constexpr int kRows = DP <= 64 ? 16 : 8, kRowBytes = DP * 4;
    // 192 elements: as for bf16 (24 heads over 8, 76 rows of up to 500: 53 us, 63 by one block)
    static constexpr int kStages = DP == 96 ? 4 : DP == 192 ? 2 : 3;
    static constexpr int kBlocksPerSm = DP <= 192 ? 2 : 1;
    static constexpr int J = DP / 32;        // 16-byte pieces of a row that a lane has
    static constexpr int I = kRows / 4;      // positions of a lane
    __device__ __forceinline__ static int swizzle_keys(int) { return 0; }
    __device__ __forceinline__ static int swizzle_values(int) { return 0; }

    const float *q;   // [NH][DP]
    float m[NH], l[NH];
    float acc[NH][J][4];
    int tg, sub;

    // the group's nq queries to the warp's place in shared memory, on their way
    __device__ __forceinline__ void fetch_queries(const DecodePlan &p, const Act *qrow, int nq, uint32_t to) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = lane; i < NH * DP / 4; i += 32) {
            const int h = i / (DP / 4), e = 4 * (i % (DP / 4));
            copy16(to + 16 * i, qrow + (h < nq && e < p.D ? h * p.D + e : 0), h < nq && e < p.D ? 16 : 0);
        }
    }

    __device__ __forceinline__ void begin(const DecodePlan &, int, const float *warp_q) {
        const int lane = threadIdx.x & 31;
        tg = lane >> 3;
        sub = lane & 7;
        q = warp_q;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[h][j][r] = 0.0f;
        }
    }

    __device__ __forceinline__ void step(const DecodePlan &p, const char *stage, const Seen &seen) {
        const float *k = reinterpret_cast<const float *>(stage) + tg * DP + 4 * sub, *v = k + kRows * DP;
        float s[I][NH];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int i = 0; i < I; ++i) s[i][h] = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float4 x[I];
#pragma unroll
            for (int i = 0; i < I; ++i) x[i] = *reinterpret_cast<const float4 *>(k + 4 * i * DP + 32 * j);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float4 y = *reinterpret_cast<const float4 *>(q + h * DP + 32 * j + 4 * sub);
#pragma unroll
                for (int i = 0; i < I; ++i)
                    s[i][h] = fmaf(y.x, x[i].x, fmaf(y.y, x[i].y, fmaf(y.z, x[i].z, fmaf(y.w, x[i].w, s[i][h]))));
            }
        }
        bool rise = false;
        float top[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            top[h] = m[h];
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float x = s[i][h];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                const int row = 4 * i + tg;
                s[i][h] = row >= seen.lo && row < seen.hi ? x * p.scale_log2 : -INFINITY;
                top[h] = fmaxf(top[h], s[i][h]);
            }
            rise |= top[h] > m[h];
        }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float by = top[h] == -INFINITY ? 1.0f : exp2_fast(m[h] - top[h]);
                m[h] = top[h];
                l[h] *= by;
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[h][j][r] *= by;
            }
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const float top_of = m[h] == -INFINITY ? 0.0f : m[h];
#pragma unroll
            for (int i = 0; i < I; ++i) {
                s[i][h] = exp2_fast(s[i][h] - top_of);
                l[h] += s[i][h];
            }
        }
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float4 x = *reinterpret_cast<const float4 *>(v + 4 * i * DP + 32 * j);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    acc[h][j][0] = fmaf(s[i][h], x.x, acc[h][j][0]);
                    acc[h][j][1] = fmaf(s[i][h], x.y, acc[h][j][1]);
                    acc[h][j][2] = fmaf(s[i][h], x.z, acc[h][j][2]);
                    acc[h][j][3] = fmaf(s[i][h], x.w, acc[h][j][3]);
                }
            }
    }

    __device__ __forceinline__ void finish(const DecodePlan &p, float *out, float *top, float *sum) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float now = m[h];
            now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 8));
            now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 16));
            const float f = m[h] == -INFINITY ? 0.0f : exp2_fast(m[h] - now);
            float x = l[h] * f;
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            if ((threadIdx.x & 31) == 0) {
                top[h] = now;
                sum[h] = x;
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float r[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    r[k] = acc[h][j][k] * f;
                    r[k] += __shfl_xor_sync(0xffffffffu, r[k], 8);
                    r[k] += __shfl_xor_sync(0xffffffffu, r[k], 16);
                }
                if (tg == 0) *reinterpret_cast<float4 *>(out + h * DP + 32 * j + 4 * sub) = make_float4(r[0], r[1], r[2], r[3]);
            }
        }
    }
};

// ---------------------------------------------------------------------------
// fp32 products by tf32: more than four queries of an fp32 cache
// ---------------------------------------------------------------------------
// Keys, queries and weights are split into the nearest tf32 and the rest, at most
// 2^-11 of them and of either sign, whose own tf32 part is taken (to 2^-23 of the
// number); values into the tf32 they are cut to and the rest, at most 2^-10 (to 2^-21),
// so that the largest ones stay finite.  x y = hi hi + hi lo + lo hi misses lo lo
// and what the rests miss, in fp32 sums: 2^-21 of a key's product, 2^-19.8 of a value's.
// (With all cut lo lo would have the product's sign and reach 2^-20 in the scores; with
// a look for the largest numbers at every one 40 heads of 256 over 8, 16 rows of up to
// 4000, take 192 us, now 146.)  Fragments as in TensorCore, with 4-byte elements: a
// lane's 16 bytes of a key are two contractions of 8, and the rows of V^T the
// elements 2i and 2i + 1 of its four.  Queries lie in shared memory.  Sums of hi hi are
// kept apart in the scores.  A step with a score that is not finite has its scores
// by plain products: the rest of an infinity is NaN, NaN may be cut to an infinity, and
// the largest numbers rounded to one.
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void split_cut(float x, uint32_t &hi, uint32_t &lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
// NaN comes out in lo at least, a number of 2^128 - 2^116 or more as an infinity and its opposite
__device__ __forceinline__ void split_nearest(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

template <int DP, int NT>
struct Tf32Core {
    using Cache = float;
    using Act = float;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kTileElems = DP;
    // two blocks an SM where their stages and queries fit beside each other (64 heads of 72
    // elements over 8, 64 rows of up to 4000: 110 us, 150 by one block)
    static constexpr int kBlocksPerSm = DP == 64 || (DP <= 128 && NT == 1) ? 2 : 1;
    static constexpr int kRows = DP <= 96 || (DP == 128 && NT == 2) ? 16 : 8, kRowBytes = DP * 4, H = kRows / 8;
    static constexpr int kStages = DP % 96 ? 3 : 4 / kBlocksPerSm;
    // keys are read four pieces of 8 rows at a time, values two of four rows
    __device__ __forceinline__ static int swizzle_keys(int row) { return (row & 1) << 6; }
    __device__ __forceinline__ static int swizzle_values(int row) { return (row & 3) << 5; }

    const char *q;  // [kHeads][DP], its 16-byte pieces exchanged as a key's
    float m[NT][2], l[NT][2];
    float acc[DP / 32][2][NT][4];
    int g, t;

    __device__ __forceinline__ void fetch_queries(const DecodePlan &p, const Act *qrow, int nq, uint32_t to) {
        const int lane = threadIdx.x & 31;
#pragma unroll 4
        for (int i = lane; i < kHeads * DP / 4; i += 32) {
            const int h = i / (DP / 4), e = 4 * (i % (DP / 4));
            const bool in = h < nq && e < p.D;
            copy16(to + ((16 * i) ^ swizzle_keys(h)), qrow + (in ? h * p.D + e : 0), in ? 16 : 0);
        }
    }

    __device__ __forceinline__ void begin(const DecodePlan &, int, const float *warp_q) {
        const int lane = threadIdx.x & 31;
        g = lane >> 2;
        t = lane & 3;
        q = reinterpret_cast<const char *>(warp_q);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                m[n][r] = -INFINITY;
                l[n][r] = 0.0f;
            }
#pragma unroll
        for (int b = 0; b < DP / 32; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[b][i][n][r] = 0.0f;
    }

    // The lane's scores by fp32 products, where tf32 left one that is not finite.
    __device__ __forceinline__ void plain_scores(const char *stage, float (&s)[NT][2 * H]) const {
#pragma unroll 1
        for (int i = 0; i < NT * 2 * H; ++i) {
            const int n = i / (2 * H), r = i - n * 2 * H, row = r < 2 ? g : g + 8, query = 8 * n + 2 * t + (r & 1);
            float x = 0.0f;
#pragma unroll 1
            for (int e = 0; e < 4 * DP; e += 16) {
                const float4 k = *reinterpret_cast<const float4 *>(stage + ((row * kRowBytes + e) ^ swizzle_keys(row)));
                const float4 y = *reinterpret_cast<const float4 *>(q + ((query * kRowBytes + e) ^ swizzle_keys(query)));
                x = fmaf(y.x, k.x, fmaf(y.y, k.y, fmaf(y.z, k.z, fmaf(y.w, k.w, x))));
            }
#pragma unroll
            for (int j = 0; j < NT * 2 * H; ++j)
                if (j == i) s[j / (2 * H)][j % (2 * H)] = x;
        }
    }

    __device__ __forceinline__ void step(const DecodePlan &p, const char *stage, const Seen &seen) {
        float big[NT][4] = {}, rest[NT][4] = {};
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            uint32_t hi[2][4] = {}, lo[2][4] = {};  // of the two contractions: rows g and g + 8, elements 2u and 2u + 1
#pragma unroll
            for (int r = 0; r < H; ++r) {
                const float4 x = *reinterpret_cast<const float4 *>(stage + (((g + 8 * r) * kRowBytes + 64 * c + 16 * t) ^ swizzle_keys(g)));
                split_nearest(x.x, hi[0][r], lo[0][r]);
                split_nearest(x.y, hi[0][r + 2], lo[0][r + 2]);
                split_nearest(x.z, hi[1][r], lo[1][r]);
                split_nearest(x.w, hi[1][r + 2], lo[1][r + 2]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 y = *reinterpret_cast<const float4 *>(q + (((8 * n + g) * kRowBytes + 64 * c + 16 * t) ^ swizzle_keys(g)));
                uint32_t qh[4], ql[4];
                split_nearest(y.x, qh[0], ql[0]);
                split_nearest(y.y, qh[1], ql[1]);
                split_nearest(y.z, qh[2], ql[2]);
                split_nearest(y.w, qh[3], ql[3]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mma1688(big[n], hi[u], qh[2 * u], qh[2 * u + 1]);
                    mma1688(rest[n], hi[u], ql[2 * u], ql[2 * u + 1]);
                    mma1688(rest[n], lo[u], qh[2 * u], qh[2 * u + 1]);
                }
            }
        }
        float s[NT][2 * H];
        bool odd = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2 * H; ++r) {
                s[n][r] = big[n][r] + rest[n][r];
                odd |= !(fabsf(s[n][r]) <= 3.4e38f);
            }
        if (__any_sync(0xffffffffu, odd)) plain_scores(stage, s);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2 * H; ++r) {
                const int row = r < 2 ? g : g + 8;
                s[n][r] = row >= seen.lo && row < seen.hi ? s[n][r] * p.scale_log2 : -INFINITY;
            }

        float top[NT][2];
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = H == 2 ? fmaxf(s[n][r], s[n][r + 2 * (H - 1)]) : s[n][r];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                top[n][r] = x;
                rise |= x > m[n][r];
            }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float now = fmaxf(m[n][r], top[n][r]);
                    const float f = now == -INFINITY ? 1.0f : exp2_fast(m[n][r] - now);
                    m[n][r] = now;
                    l[n][r] *= f;
#pragma unroll
                    for (int b = 0; b < DP / 32; ++b)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            acc[b][i][n][r] *= f;
                            acc[b][i][n][r + 2] *= f;
                        }
                }
        }
        // P^T as the second operand: positions t and t + 4 (of each 8) of query g, from the lanes that have them
        uint32_t ph[NT][H][2], pl[NT][H][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int r = 0; r < 2 * H; ++r) {
                const float top_of = m[n][r & 1] == -INFINITY ? 0.0f : m[n][r & 1];
                s[n][r] = exp2_fast(s[n][r] - top_of);
                l[n][r & 1] += s[n][r];
            }
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int from = 4 * (t + 4 * j) + g / 2;
                    const float even = __shfl_sync(0xffffffffu, s[n][2 * h], from), odd = __shfl_sync(0xffffffffu, s[n][2 * h + 1], from);
                    split_nearest(g & 1 ? odd : even, ph[n][h][j], pl[n][h][j]);
                }
        }
        const char *v = stage + kRows * kRowBytes;
#pragma unroll
        for (int b = 0; b < DP / 32; ++b)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                // positions t and t + 4 of the 8, the lane's four elements
                const float4 x = *reinterpret_cast<const float4 *>(v + (((t + 8 * h) * kRowBytes + 128 * b + 16 * g) ^ (t << 5)));
                const float4 y = *reinterpret_cast<const float4 *>(v + (((t + 4 + 8 * h) * kRowBytes + 128 * b + 16 * g) ^ (t << 5)));
                uint32_t hi[2][4], lo[2][4];
                split_cut(x.x, hi[0][0], lo[0][0]);
                split_cut(x.y, hi[0][1], lo[0][1]);
                split_cut(x.z, hi[1][0], lo[1][0]);
                split_cut(x.w, hi[1][1], lo[1][1]);
                split_cut(y.x, hi[0][2], lo[0][2]);
                split_cut(y.y, hi[0][3], lo[0][3]);
                split_cut(y.z, hi[1][2], lo[1][2]);
                split_cut(y.w, hi[1][3], lo[1][3]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma1688(acc[b][i][n], hi[i], ph[n][h][0], ph[n][h][1]);
                        mma1688(acc[b][i][n], hi[i], pl[n][h][0], pl[n][h][1]);
                        mma1688(acc[b][i][n], lo[i], ph[n][h][0], ph[n][h][1]);
                    }
            }
    }

    __device__ __forceinline__ void finish(const DecodePlan &, float *out, float *top, float *sum) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = l[n][r];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                const int h = 8 * n + 2 * t + r;
                if (g == 0) {
                    top[h] = m[n][r];
                    sum[h] = x;
                }
#pragma unroll
                for (int b = 0; b < DP / 32; ++b)
                    *reinterpret_cast<float4 *>(out + h * DP + 32 * b + 4 * g) =
                        make_float4(acc[b][0][n][r], acc[b][0][n][r + 2], acc[b][1][n][r], acc[b][1][n][r + 2]);
            }
    }
};

// ---------------------------------------------------------------------------
// the blocks' stretches
// ---------------------------------------------------------------------------
// Where a row's positions lie, and how many units a key head of it has (at
// least one, so that every row has an output).
struct Row {
    int first, last, t0, units;
};
template <int R>
__device__ __forceinline__ Row row_at(const DecodePlan &p, int r, bool *bad) {
    constexpr int kUnit = R * kWarps;
    Row x;
    const int pos = p.at.positions[r];
    const int seq = p.at.sequences ? p.at.sequences[r] : r;
    // a position in the table's columns: pos / page_size < table_cols
    const bool ok = pos < 0 || (static_cast<unsigned>(seq) < static_cast<unsigned>(p.at.table_rows) &&
                                static_cast<int>(p.at.page.div(max(pos, 0))) < p.at.table_cols);
    if (bad) *bad = !ok;
    x.last = ok ? max(pos, -1) : -1;
    x.first = p.window > 0 ? max(0, x.last - p.window + 1) : 0;
    x.t0 = x.first / kUnit;
    x.units = x.last < 0 ? 1 : x.last / kUnit - x.t0 + 1;
    return x;
}

template <typename Act>
__device__ __forceinline__ void store8(Act *to, const float *f) {
    if constexpr (sizeof(Act) == 2)
        *reinterpret_cast<uint4 *>(to) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    else {
        reinterpret_cast<float4 *>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// row-head index rh of a row -> shard, key head of the shard, first query
struct HeadAt {
    int shard, kv, query;
};
__device__ __forceinline__ HeadAt head_at(const DecodePlan &p, int rh) {
    HeadAt h;
    uint32_t group, kv;
    const uint32_t k = p.by_groups.divmod(rh, group);
    h.shard = p.by_hk.divmod(k, kv);
    h.kv = kv;
    h.query = kv * p.per + group * p.nh;
    return h;
}
// queries of a group: the last group of a head may have fewer
__device__ __forceinline__ int queries_of(const DecodePlan &p, int rh) {
    uint32_t group;
    p.by_groups.divmod(rh, group);
    return min(p.nh, p.per - static_cast<int>(group) * p.nh);
}

// A group's outputs [nh][D], maxima [nh] and sums [nh], in whole 16 bytes.
inline __host__ __device__ int part_floats(int nh, int D) { return (nh * (D + 2) + 3) & ~3; }

// An output is (sum of values / sum of weights) * value scale, in this order: with
// codes the weights' sum reaches 2^64 and the scale may be as small as 2^-109.

// Elements e.. of query h from the states of warps w0..w1 (their outputs `pitch`
// bytes apart): eight of the sum, its maximum, the sum of weights.
template <int NH, int DP>
__device__ __forceinline__ void add_warps(const char *outs, int pitch, const float *top, const float *sum, int h, int e, int w0, int w1,
                                          float (&f)[8], float &most, float &all) {
    most = -INFINITY;
    all = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    for (int j = w0; j < w1; ++j) most = fmaxf(most, top[j * NH + h]);
    for (int j = w0; j < w1; ++j) {
        const float t = top[j * NH + h], by = t == -INFINITY ? 0.0f : exp2_fast(t - most);
        all = fmaf(sum[j * NH + h], by, all);
        const float4 *o = reinterpret_cast<const float4 *>(outs + j * pitch) + (h * DP + e) / 4;
        const float4 a = o[0], b = o[1];
        f[0] = fmaf(a.x, by, f[0]); f[1] = fmaf(a.y, by, f[1]); f[2] = fmaf(a.z, by, f[2]); f[3] = fmaf(a.w, by, f[3]);
        f[4] = fmaf(b.x, by, f[4]); f[5] = fmaf(b.y, by, f[5]); f[6] = fmaf(b.z, by, f[6]); f[7] = fmaf(b.w, by, f[7]);
    }
}

// Registers a thread so that an SM holds so many blocks and has 8192 left: a block
// of the kernel before (the join of the call before, say) that is still there
// must not keep one of these out until another ends (8-bit batch: 166 to
// 173 us with one block late, 135 without).
constexpr int registers_of(int blocks) {
    return (65536 - 8192) / (blocks * kBlock) / 8 * 8 < 255 ? (65536 - 8192) / (blocks * kBlock) / 8 * 8 : 255;
}

// The blocks' shares of the cost.  SMs differ by up to a tenth in what memory
// gives them, so with enough to do, an eighth of the cost goes to blocks beyond
// the resident ones, which take it up as those end (batch 167 -> 164 us, long 300
// -> 295 us; equal shares for four times the resident blocks: 174 and 302 us).
struct Shares {
    long long total, main;  // main: of the resident blocks
    int resident, rest;
    __device__ __forceinline__ Shares(long long cost, int resident_blocks, int all) : total(cost) {
        resident = static_cast<int>(min(cost, static_cast<long long>(resident_blocks)));
        const bool spread = cost >= static_cast<long long>(resident_blocks) * kSpread;
        rest = spread ? all - resident_blocks : 0;
        main = spread ? cost - cost / kTailShare : cost;
    }
    __device__ __forceinline__ int blocks() const { return resident + rest; }
    // where block c's share begins
    __device__ __forceinline__ long long begin(int c) const {
        return c <= resident ? main * c / resident : main + (total - main) * (c - resident) / rest;
    }
    // the block whose share holds x
    __device__ __forceinline__ int owner(long long x) const {
        return static_cast<int>(x < main ? ((x + 1) * resident + main - 1) / main - 1
                                         : resident + ((x + 1 - main) * rest + (total - main) - 1) / (total - main) - 1);
    }
};

// A segment's part that a block, or one warp of it, takes.
struct Work {
    Segment s;
    int r, rh, u0, u1, units;  // row, head of the row; units [u0, u1) of `units`
    bool brief;                // one warp's
    bool valid;
};

// One warp's steps of a segment are every `by`-th from its first one.  They pass
// through its ring of S stages, of which the last kOut also take its output
// at the end; the first kEarly stages of the next segment are under way by then.
template <class Core>
struct Ring {
    static constexpr int R = Core::kRows, S = Core::kStages, kStage = 2 * R * Core::kRowBytes, kBytes = S * kStage;
    static constexpr int kOut = (Core::kHeads * Core::kTileElems * 4 + kStage - 1) / kStage;
    static constexpr int kEarly = S - kOut < S - 1 ? S - kOut : S - 1;
    static_assert(kEarly >= 1, "a stage for the next segment beside the output");

    // lane i's look-up of the i-th of 32 steps
    __device__ __forceinline__ static uint32_t look_up(const DecodePlan &p, const Segment &s, int first, int by) {
        return block_at<R>(p, s, first + by * (threadIdx.x & 31));
    }
    template <int FROM, int TO>
    __device__ __forceinline__ static void begin(const DecodePlan &p, const Segment &s, const void *k, const void *v, int first, int by,
                                                 uint32_t blocks, uint32_t to) {
#pragma unroll 1
        for (int i = FROM; i < TO; ++i) {
            const uint32_t block = __shfl_sync(0xffffffffu, blocks, i);
            if (block != kNone) fetch<Core>(p, k, v, seen_at<R>(s, first + by * i), block, to + i * kStage);
            copies_end();
        }
    }
    // begin<0, kEarly> has been called
    __device__ __forceinline__ static void walk(Core &core, const DecodePlan &p, const Segment &s, const void *k, const void *v, int first,
                                                int by, uint32_t blocks_now, char *ring) {
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
        begin<kEarly, S - 1>(p, s, k, v, first, by, blocks_now, to);
        int stage = 0, ahead = S - 1;
        for (int from = first; from < s.t1; from += 32 * by) {
            uint32_t blocks_next = kNone;
            if (from + 32 * by < s.t1) blocks_next = look_up(p, s, from + 32 * by, by);
            const int n = min(32, (s.t1 - from + by - 1) / by);
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                copies_wait<S - 2>();
                __syncwarp();  // every lane's copies of this step are there, and the step before has been read
                const uint32_t then = __shfl_sync(0xffffffffu, i + S - 1 < 32 ? blocks_now : blocks_next, (i + S - 1) & 31);
                if (then != kNone) fetch<Core>(p, k, v, seen_at<R>(s, from + by * (i + S - 1)), then, to + ahead * kStage);
                copies_end();
                if (__shfl_sync(0xffffffffu, blocks_now, i) != kNone)
                    core.step(p, ring + stage * kStage, seen_at<R>(s, from + by * i));
                stage = stage + 1 == S ? 0 : stage + 1;
                ahead = ahead + 1 == S ? 0 : ahead + 1;
            }
            blocks_now = blocks_next;
        }
        copies_wait<0>();
        __syncwarp();
    }
};

template <class Core>
__global__ void __maxnreg__(registers_of(Core::kBlocksPerSm)) decode_kernel(const __grid_constant__ DecodePlan p) {
    using Act = typename Core::Act;
    constexpr int DP = Core::kTileElems, NH = Core::kHeads, R = Core::kRows;
    using Stages = Ring<Core>;
    constexpr int kRing = Stages::kBytes, kOutAt = (Core::kStages - Stages::kOut) * Stages::kStage;
    constexpr int kSegmentCost = kSegmentPositions / (R * kWarps), kShort = kShortPositions / (R * kWarps);
    // with more segments than blocks, a short one is a single warp's
    const bool alone = !p.by_segment;
    auto is_short = [&](int units) { return alone && units <= kShort; };
    auto cost_of = [&](int units) { return is_short(units) ? units + 1 : units + kSegmentCost; };
    extern __shared__ __align__(128) char ring[];  // [kWarps][stages]
    __shared__ float top[kWarps * NH], sum[kWarps * NH];
    __shared__ __align__(16) float q_smem[sizeof(Act) == 4 ? kWarps * NH * DP : 4];
    __shared__ long long scan[kWarps], start_cost;
    __shared__ int start_row;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_for_stream();
    let_next_start();

    // cost of all rows, and the row that this block's stretch starts in
    const int each = (p.at.n + kBlock - 1) / kBlock, r0 = min(threadIdx.x * each, p.at.n), r1 = min(r0 + each, p.at.n);
    long long mine = 0;
    for (int r = r0; r < r1; ++r) {
        bool bad;
        mine += cost_of(row_at<R>(p, r, &bad).units);
        if (bad && blockIdx.x == 0) bad_index(p.at);
    }
    mine *= p.row_heads;
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) scan[warp] = before;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    before -= mine;
    const Shares shares(total, p.resident, gridDim.x);
    const int c = blockIdx.x;
    if (c >= shares.blocks()) {
        if (!p.by_segment && threadIdx.x == 0) p.joins[c] = make_int4(0, 0, 0, 0);
        return;
    }
    const long long from_cost = shares.begin(c), to_cost = shares.begin(c + 1);
    if (from_cost >= before && from_cost < before + mine) {
        long long x = before;
        int r = r0;
        for (;; ++r) {
            const long long n = static_cast<long long>(cost_of(row_at<R>(p, r, nullptr).units)) * p.row_heads;
            if (from_cost < x + n || r + 1 == r1) break;
            x += n;
        }
        start_row = r;
        start_cost = x;
    }
    __syncthreads();

    // the parts of the block's share that this warp has, one after another
    int r = start_row, turn = 0;
    Row row = row_at<R>(p, r, nullptr), after = row_at<R>(p, min(r + 1, p.at.n - 1), nullptr);
    int rh = min(static_cast<int>((from_cost - start_cost) / cost_of(row.units)), p.row_heads - 1);
    long long at_cost = start_cost + static_cast<long long>(rh) * cost_of(row.units);  // where the segment's cost begins
    auto take = [&]() {
        Work w;
        w.valid = false;
        while (at_cost < to_cost) {
            w.brief = is_short(row.units);
            // a segment's cost before its first unit belongs to whoever has that unit; a short segment, to
            // whoever has its beginning
            const long long first_unit = at_cost + (w.brief ? 0 : kSegmentCost);
            w.units = row.units;
            w.u0 = w.brief ? 0 : static_cast<int>(max(from_cost - first_unit, 0ll));
            w.u1 = w.brief ? row.units : static_cast<int>(min(to_cost - first_unit, static_cast<long long>(row.units)));
            w.valid = w.brief ? at_cost >= from_cost && (turn++ & (kWarps - 1)) == warp : w.u1 > w.u0;
            w.r = r;
            w.rh = rh;
            w.s.t0 = (row.t0 + w.u0) * kWarps;
            w.s.t1 = (row.t0 + w.u1) * kWarps;
            w.s.first = row.first;
            w.s.last = row.last;
            at_cost += cost_of(row.units);
            if (++rh == p.row_heads) {
                if (++r == p.at.n) at_cost = to_cost;
                rh = 0;
                row = after;
                after = row_at<R>(p, min(r + 1, p.at.n - 1), nullptr);
            }
            if (w.valid) break;
        }
        return w;
    };
    // what follows from a part's row and head
    auto place = [&](Work &w, HeadAt &at) {
        at = head_at(p, w.rh);
        w.s.head = at.kv;
        w.s.pages = p.at.table + static_cast<long long>(w.s.last < 0 ? 0 : p.at.sequences ? p.at.sequences[w.r] : w.r) * p.at.table_cols;
    };
    auto first_of = [&](const Work &w) { return w.s.t0 + (w.brief ? 0 : warp); };
    auto by_of = [&](const Work &w) { return w.brief ? 1 : kWarps; };
    char *mine_at = ring + warp * kRing;
    const uint32_t mine_to = static_cast<uint32_t>(__cvta_generic_to_shared(mine_at));
    float *mine_q = sizeof(Act) == 4 ? q_smem + warp * NH * DP : nullptr;
    const uint32_t mine_q_to = sizeof(Act) == 4 ? static_cast<uint32_t>(__cvta_generic_to_shared(mine_q)) : 0u;
    const int chunks = p.D / 8;

    Core core;
    auto start = [&](const Work &w, const HeadAt &at, uint32_t blocks) {
        core.fetch_queries(p, static_cast<const Act *>(p.q[at.shard]) + (static_cast<long long>(w.r) * p.hq + at.query) * p.D,
                           queries_of(p, w.rh), mine_q_to);
        Stages::template begin<0, Stages::kEarly>(p, w.s, p.k[at.shard], p.v[at.shard], first_of(w), by_of(w), blocks, mine_to);
    };
    bool listed = false;
    Work w = take();
    HeadAt at = {};
    uint32_t blocks = kNone;
    if (w.valid) {
        place(w, at);
        blocks = Stages::look_up(p, w.s, first_of(w), by_of(w));
        start(w, at, blocks);
    }
    while (w.valid) {
        core.begin(p, at.shard * p.hk + at.kv, mine_q);
        // the next part's pages are looked up meanwhile
        Work x = take();
        HeadAt x_at = {};
        uint32_t x_blocks = kNone;
        if (x.valid) {
            place(x, x_at);
            x_blocks = Stages::look_up(p, x.s, first_of(x), by_of(x));
        }
        Stages::walk(core, p, w.s, p.k[at.shard], p.v[at.shard], first_of(w), by_of(w), blocks, mine_at);
        // its first keys and values are on their way while this one's are added up
        if (x.valid) start(x, x_at, x_blocks);
        core.finish(p, reinterpret_cast<float *>(mine_at + kOutAt), top + warp * NH, sum + warp * NH);
        if (w.brief)
            __syncwarp();
        else
            __syncthreads();

        const int nq = queries_of(p, w.rh);
        const long long q_at = (static_cast<long long>(w.r) * p.hq + at.query) * p.D;
        const float vscale = p.v_amax ? 1.0f / cache_scale(p.v_amax, at.shard * p.hk + at.kv) : 1.0f;
        const bool whole = w.u0 == 0 && w.u1 == w.units;
        // slot 0: began in an earlier block; 1: ends in a later one
        float *part = p.partial + (static_cast<long long>(c) * 2 + (w.u0 == 0 ? 1 : 0)) * part_floats(p.nh, p.D);
        const int w0 = w.brief ? warp : 0, w1 = w.brief ? warp + 1 : kWarps;  // whose states make the segment's
        for (int i = w.brief ? lane : threadIdx.x; i < nq * chunks; i += w.brief ? 32 : kBlock) {
            const int h = i / chunks, e = (i - h * chunks) * 8;
            float most, all, f[8];
            add_warps<NH, DP>(ring + kOutAt, kRing, top, sum, h, e, w0, w1, f, most, all);
            if (whole) {
                const float by = 1.0f / all;
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = all == 0.0f ? 0.0f : f[j] * by * vscale;
                store8(static_cast<Act *>(p.o[at.shard]) + q_at + static_cast<long long>(h) * p.D + e, f);
            } else {
                store8(part + h * p.D + e, f);
                if (e == 0) {
                    part[p.nh * p.D + h] = most;
                    part[p.nh * (p.D + 1) + h] = all;
                }
            }
        }
        if (w.u0 == 0 && !w.brief && threadIdx.x == 0 && (p.by_segment || !whole)) {
            // up to the block that holds the segment's last unit: u1 lies where the share ends, unless that is c
            const int last = whole ? c : shares.owner(to_cost + (w.units - w.u1) - 1);
            p.joins[p.by_segment ? w.r * p.row_heads + w.rh : c] = make_int4(w.r, w.rh, c, last);
            listed = !whole;
        }
        // the outputs have been read: the next steps may take their stages
        if (w.brief)
            __syncwarp();
        else
            __syncthreads();
        w = x;
        at = x_at;
        blocks = x_blocks;
    }
    if (!p.by_segment && !listed && threadIdx.x == 0) p.joins[c] = make_int4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// few and short segments: a cluster for each
// ---------------------------------------------------------------------------
// The blocks of a cluster take equal parts of one segment and add them up through
// each other's shared memory: no second launch, no look at the other rows.  One
// sequence of 2000 positions, 8 key heads: 8.2 us a call, 11.1 by the list and its
// join (5.9 and 8.4 us in a captured graph).
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// the address of a block's own shared memory in block `rank` of its cluster
__device__ __forceinline__ uint32_t in_block(uint32_t at, uint32_t rank) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
    return to;
}
__device__ __forceinline__ float cluster_read(uint32_t at) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ float4 cluster_read4(uint32_t at) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at) : "memory");
    return x;
}

template <class Core>
__global__ void __maxnreg__(registers_of(Core::kBlocksPerSm)) cluster_kernel(const __grid_constant__ DecodePlan p) {
    using Act = typename Core::Act;
    using Stages = Ring<Core>;
    constexpr int DP = Core::kTileElems, NH = Core::kHeads, R = Core::kRows;
    constexpr int kRing = Stages::kBytes, kOutAt = (Core::kStages - Stages::kOut) * Stages::kStage;
    static_assert(NH * DP * 4 <= kOutAt, "the block's sum lies before its first warp's output");
    extern __shared__ __align__(128) char ring[];  // [kWarps][stages]; then the block's output [NH][DP]
    __shared__ float top[kWarps * NH], sum[kWarps * NH], tops[NH], sums[NH];
    __shared__ __align__(16) float q_smem[sizeof(Act) == 4 ? kWarps * NH * DP : 4];
    const int warp = threadIdx.x >> 5, rank = static_cast<int>(cluster_rank());
    const int size = p.cluster, segment = blockIdx.x / size, r = segment / p.row_heads, rh = segment - r * p.row_heads;
    wait_for_stream();
    let_next_start();
    bool bad;
    const Row row = row_at<R>(p, r, &bad);
    if (bad && rank == 0 && threadIdx.x == 0) bad_index(p.at);
    const HeadAt at = head_at(p, rh);
    const int nq = queries_of(p, rh), chunks = p.D / 8;
    Segment s;
    s.head = at.kv;
    s.t0 = (row.t0 + row.units * rank / size) * kWarps;
    s.t1 = (row.t0 + row.units * (rank + 1) / size) * kWarps;
    s.first = row.first;
    s.last = row.last;
    s.pages = p.at.table + static_cast<long long>(row.last < 0 ? 0 : p.at.sequences ? p.at.sequences[r] : r) * p.at.table_cols;
    const long long q_at = (static_cast<long long>(r) * p.hq + at.query) * p.D;
    char *mine_at = ring + warp * kRing;
    const uint32_t mine_to = static_cast<uint32_t>(__cvta_generic_to_shared(mine_at));
    float *mine_q = sizeof(Act) == 4 ? q_smem + warp * NH * DP : nullptr;

    Core core;
    const uint32_t blocks = Stages::look_up(p, s, s.t0 + warp, kWarps);
    core.fetch_queries(p, static_cast<const Act *>(p.q[at.shard]) + q_at, nq,
                       sizeof(Act) == 4 ? static_cast<uint32_t>(__cvta_generic_to_shared(mine_q)) : 0u);
    Stages::template begin<0, Stages::kEarly>(p, s, p.k[at.shard], p.v[at.shard], s.t0 + warp, kWarps, blocks, mine_to);
    core.begin(p, at.shard * p.hk + at.kv, mine_q);
    Stages::walk(core, p, s, p.k[at.shard], p.v[at.shard], s.t0 + warp, kWarps, blocks, mine_at);
    core.finish(p, reinterpret_cast<float *>(mine_at + kOutAt), top + warp * NH, sum + warp * NH);
    __syncthreads();
    // the block's sum, to where its first warp's stages were
    for (int i = threadIdx.x; i < nq * chunks; i += kBlock) {
        const int h = i / chunks, e = (i - h * chunks) * 8;
        float most, all, f[8];
        add_warps<NH, DP>(ring + kOutAt, kRing, top, sum, h, e, 0, kWarps, f, most, all);
        store8(reinterpret_cast<float *>(ring) + h * DP + e, f);
        if (e == 0) {
            tops[h] = most;
            sums[h] = all;
        }
    }
    cluster_meet();
    const float vscale = p.v_amax ? 1.0f / cache_scale(p.v_amax, at.shard * p.hk + at.kv) : 1.0f;
    const uint32_t out_to = static_cast<uint32_t>(__cvta_generic_to_shared(ring)), tops_to = static_cast<uint32_t>(__cvta_generic_to_shared(tops)),
                   sums_to = static_cast<uint32_t>(__cvta_generic_to_shared(sums));
    // four elements a thread, the blocks' in turn
    for (int i = rank * kBlock + threadIdx.x; i < nq * chunks * 2; i += size * kBlock) {
        const int h = i / (2 * chunks), e = (i - h * 2 * chunks) * 4;
        float most = -INFINITY, all = 0.0f, t[kCluster], l[kCluster];
        float4 x[kCluster], f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            t[c] = -INFINITY;
            l[c] = 0.0f;
            x[c] = f;
            if (c < size) {
                t[c] = cluster_read(in_block(tops_to + 4 * h, c));
                l[c] = cluster_read(in_block(sums_to + 4 * h, c));
                x[c] = cluster_read4(in_block(out_to + 4 * (h * DP + e), c));
            }
            most = fmaxf(most, t[c]);
        }
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const float by = t[c] == -INFINITY ? 0.0f : exp2_fast(t[c] - most);
            all = fmaf(l[c], by, all);
            f.x = fmaf(x[c].x, by, f.x); f.y = fmaf(x[c].y, by, f.y); f.z = fmaf(x[c].z, by, f.z); f.w = fmaf(x[c].w, by, f.w);
        }
        const float by = 1.0f / all;
        const float4 o = all == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                     : make_float4(f.x * by * vscale, f.y * by * vscale, f.z * by * vscale, f.w * by * vscale);
        Act *to = static_cast<Act *>(p.o[at.shard]) + q_at + static_cast<long long>(h) * p.D + e;
        if constexpr (sizeof(Act) == 2)
            *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        else
            *reinterpret_cast<float4 *>(to) = o;
    }
    cluster_meet();  // no block leaves while another reads its memory
}

// Joins the parts of the segments that several blocks read: W warps a query,
// each a part in turn, 4 elements a lane.
template <typename Act, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) join_kernel(const __grid_constant__ DecodePlan p) {
    constexpr int kQueries = W == 1 ? 4 : 1;  // queries of a block
    __shared__ float tops[W], sums[W];
    __shared__ __align__(16) float4 outs[W == 1 ? 1 : W][64];
    wait_for_stream();
    if (p.join_early) let_next_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y * kQueries + (W == 1 ? warp : 0);
    const int4 j = p.joins[blockIdx.x];
    if (j.z == j.w) return;  // one block has done it all (or there is none)
    const int nq = queries_of(p, j.y);
    if (h >= nq) return;
    const long long stride = part_floats(p.nh, p.D);
    // the part of block c: its second slot where the segment begins, else the first
    const float *base = p.partial + static_cast<long long>(j.z) * 2 * stride + stride;
    const int n = j.w - j.z + 1;
    auto part = [&](int i) { return i == 0 ? base : base + (2 * i - 1) * stride; };
    const int e0 = 4 * lane, e1 = 128 + 4 * lane;
    float most = -INFINITY, all = 0.0f;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
    for (int i0 = W == 1 ? 0 : warp; i0 < n; i0 += 4 * W) {
        // four parts at once, so that one wait serves them all
        float top[4], sum[4];
        float4 va[4], vb[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            top[u] = -INFINITY;
            sum[u] = 0.0f;
            va[u] = vb[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i0 + u * W < n) {
                const float *x = part(i0 + u * W);
                top[u] = x[p.nh * p.D + h];
                sum[u] = x[p.nh * (p.D + 1) + h];
                if (e0 < p.D) va[u] = *reinterpret_cast<const float4 *>(x + h * p.D + e0);
                if (e1 < p.D) vb[u] = *reinterpret_cast<const float4 *>(x + h * p.D + e1);
            }
        }
        const float now = fmaxf(most, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
        const float old = most == -INFINITY ? 0.0f : exp2_fast(most - now);
        most = now;
        all *= old;
        a.x *= old; a.y *= old; a.z *= old; a.w *= old;
        b.x *= old; b.y *= old; b.z *= old; b.w *= old;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float by = top[u] == -INFINITY ? 0.0f : exp2_fast(top[u] - now);
            all = fmaf(sum[u], by, all);
            a.x = fmaf(va[u].x, by, a.x); a.y = fmaf(va[u].y, by, a.y); a.z = fmaf(va[u].z, by, a.z); a.w = fmaf(va[u].w, by, a.w);
            b.x = fmaf(vb[u].x, by, b.x); b.y = fmaf(vb[u].y, by, b.y); b.z = fmaf(vb[u].z, by, b.z); b.w = fmaf(vb[u].w, by, b.w);
        }
    }
    if constexpr (W > 1) {
        if (lane == 0) {
            tops[warp] = most;
            sums[warp] = all;
        }
        outs[warp][lane] = a;
        outs[warp][32 + lane] = b;
        __syncthreads();
        if (threadIdx.x >= 64) return;
        most = -INFINITY;
        for (int w = 0; w < W; ++w) most = fmaxf(most, tops[w]);
        all = 0.0f;
        a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = 0; w < W; ++w) {
            const float by = tops[w] == -INFINITY ? 0.0f : exp2_fast(tops[w] - most);
            all = fmaf(sums[w], by, all);
            const float4 v = outs[w][threadIdx.x];
            a.x = fmaf(v.x, by, a.x); a.y = fmaf(v.y, by, a.y); a.z = fmaf(v.z, by, a.z); a.w = fmaf(v.w, by, a.w);
        }
    }
    const HeadAt at = head_at(p, j.y);
    const float vscale = p.v_amax ? 1.0f / cache_scale(p.v_amax, at.shard * p.hk + at.kv) : 1.0f;
    const float by = 1.0f / all;
    Act *o = static_cast<Act *>(p.o[at.shard]) + (static_cast<long long>(j.x) * p.hq + at.query + h) * p.D;
    auto put = [&](int e, const float4 &v) {
        if (e >= p.D) return;
        const float4 r = all == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                     : make_float4(v.x * by * vscale, v.y * by * vscale, v.z * by * vscale, v.w * by * vscale);
        if constexpr (sizeof(Act) == 2)
            *reinterpret_cast<uint2 *>(o + e) = make_uint2(pack_bf16x2(r.x, r.y), pack_bf16x2(r.z, r.w));
        else
            *reinterpret_cast<float4 *>(o + e) = r;
    };
    if constexpr (W == 1) {
        put(e0, a);
        put(e1, b);
    } else {
        put(4 * threadIdx.x, a);
    }
}

// Launches the kernels of a core: as many blocks as are resident (or as there is
// room for in the workspace), or the clusters; *grid is 0 where nothing is to join.
template <class Core>
tp_status launch_core(DecodePlan &p, int *grid, cudaStream_t st) {
    constexpr int kSmem = kWarps * Ring<Core>::kBytes;
    static int per_sm[64] = {};  // by device
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_check(e, "cudaGetDevice");
    if (dev < 0 || dev >= 64) return set_error(TP_ERR_UNSUPPORTED, "device ordinal %d above 63", dev);
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!per_sm[dev]) {
            int n = 0;
            e = cudaFuncSetAttribute(decode_kernel<Core>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(cluster_kernel<Core>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_kernel<Core>, kBlock, kSmem);
            if (e != cudaSuccess) return cuda_check(e, "paged_decode");
            if (n < 1) return set_error(TP_ERR_CUDA, "paged_decode: no block fits an SM");
            per_sm[dev] = n;
        }
        p.resident = std::min(per_sm[dev] * num_sms(), kMostResident);
    }
    const long long segments = static_cast<long long>(p.at.n) * p.row_heads;
    long long seen = static_cast<long long>(p.at.table_cols) * p.at.page_size;
    const bool windowed = p.window > 0 && p.window < seen;
    if (windowed) seen = p.window;
    p.cluster = seen > kShortPositions && seen <= kBlockPositions && segments <= (windowed ? 4 : 2) * p.resident ? 1 : 0;
    for (int size = 1; size <= kCluster; size *= 2)
        if (segments * size * 4 <= p.resident * 3 && seen <= size * kBlockPositions && (size == 1 || seen > (size - 1) * Core::kRows * kWarps))
            p.cluster = size;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (pdl_on()) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (p.cluster) {
        *grid = 0;
        cfg.gridDim = dim3(static_cast<unsigned>(segments) * p.cluster);
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = p.cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    } else {
        *grid = p.resident + p.resident / 2;
        cfg.gridDim = dim3(*grid);
        p.by_segment = segments <= *grid;
    }
    launch_begin("paged_decode", st);
    e = p.cluster ? cudaLaunchKernelEx(&cfg, cluster_kernel<Core>, p) : cudaLaunchKernelEx(&cfg, decode_kernel<Core>, p);
    launch_end("paged_decode", st);
    return cuda_check(e, "paged_decode");
}

// by the padded width (64, 128, 192, 256; fp32 also 96) and the queries of a group
tp_status launch_decode_bf16(DecodePlan &p, int *grid, cudaStream_t st);
tp_status launch_decode_fp8(DecodePlan &p, int *grid, cudaStream_t st);
tp_status launch_decode_f32(DecodePlan &p, int *grid, cudaStream_t st);

}  // namespace attn
}  // namespace tpmlp
