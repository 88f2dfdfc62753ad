// AdamW over a list of tensors, and the global gradient norm that clips it.
//   g' = s g            s: gradient scale, times the clip factor
//   m  = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//   w  = w - l d w - l / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// with l = lr * lr_scale and the weight decay d of the tensor.  One pass: every
// array is read once and written once, in fp32 arithmetic.
//
// States in 8 bits.  m and r = sqrt(v) are kept as e4m3 codes with one fp32
// scale for 256 consecutive elements, scale = max |x| / 448.  Storing the root
// halves the exponent range that v needs: codes span 2^-9 .. 448, so r reaches
// 2^-17.8 below its block's largest value.  Rounding is stochastic: m and v
// move by a fraction 1 - b of themselves a step, far less than the 1/16 that a
// 3-bit mantissa resolves, and round-to-nearest would leave them where they
// are; rounded up with a probability equal to the fraction of the step they
// keep their expectation.  The bits come from a hash of (seed, t, tensor,
// block, element), so a step is a function of its arguments.  A root above
// zero is never rounded to zero: a zero root under a momentum that is not
// zero would make the next step m / eps.
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "device_common.cuh"
#include "internal.h"

namespace tpmlp {
namespace adam {

constexpr int kThreads = 256;
constexpr int kBlock = 256;                     // elements that share a scale: a warp's, 8 a lane
constexpr int kChunk = kThreads / 32 * kBlock;  // elements a thread block takes at a time
constexpr int kNormChunk = 8 * 4 * kThreads;    // the gradient norm's chunk: 8 loads of 4 a thread in flight
constexpr int kNormBlocks = 3648;
constexpr uint32_t kMix1 = 0x9E3779B9u, kMix2 = 0xB504F333u;  // fractions of the golden ratio and of sqrt(2)

// The control block in device memory: what the gradient norm leaves for the step.
struct Ctl {
    float norm;          // of the scaled gradients
    float scale;         // gradient scale times clip factor
    int finite;          // 0: the step changes nothing
    int steps;           // steps taken, this one among them
    float inv_bc1;       // 1 / (1 - b1^t)
    float inv_root_bc2;  // 1 / sqrt(1 - b2^t)
    unsigned ticket;     // blocks of the norm that are done
    unsigned pad;
    double partial[kNormBlocks];
};
static_assert(sizeof(Ctl) <= TP_ADAMW_CTL_BYTES, "control block");

struct Entry {
    void *w, *p;        // fp32 weights; their bf16 copy, or null
    const void *g;
    void *m, *v;        // fp32, or e4m3 codes
    float *ms, *vs;     // scales of the codes
    long long n;
};

// Entries of the index over a table: a search of its few hundred chunk numbers
// from the middle is a chain of reads past the constant cache, this leaves a
// step or two of it.
constexpr int kCoarse = 64;

// Tensors of one launch, in the kernel's parameters: no copy to the device, no
// allocation, and a launch captured into a graph carries its own table.
template <int CAP>
struct Table {
    int count, base;    // tensors here, and the index of the first of them in the list
    int shift;          // chunk c lies in one of the tensors coarse[c >> shift] .. coarse[(c >> shift) + 1]
    unsigned short coarse[kCoarse + 1];
    int chunk0[CAP + 1];
    float lr_scale[CAP], decay[CAP];
    Entry t[CAP];
};

// The table's size is a launch's parameter bytes, at most 32764 with the rest: a
// short list takes the small one.
constexpr int kSmall = 40, kLarge = 420;

// The tables of a list's launches, made when the list or its gradients change.
template <int CAP>
struct Plans {
    Table<CAP> *step = nullptr, *norm = nullptr;
    int launches = 0;
};

struct Hyper {
    float lr, b1, b2, c1, c2, eps, scale, inv_bc1, inv_root_bc2;  // c: 1 - b, rounded once
    uint32_t seed, step;
    const Ctl *ctl;
};

// tensor that holds chunk c: the last whose first chunk is at most c
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP> &tab, int c) {
    int lo = tab.coarse[c >> tab.shift], hi = tab.coarse[(c >> tab.shift) + 1];
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.chunk0[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Elements are addressed as (a chunk's start, the same for the whole block; an
// offset of 32 bits within the chunk, a thread's own and the same in every
// chunk).  4 of them from e, as two pairs; unless FULL, those past n read as zero.
template <bool FULL>
__device__ __forceinline__ void load4(const float *p, uint32_t e, uint32_t n, float2 *v) {
    if (FULL || e + 4 <= n) {
        const float4 w = *reinterpret_cast<const float4 *>(p + e);
        v[0] = make_float2(w.x, w.y);
        v[1] = make_float2(w.z, w.w);
    } else {
        float t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = e + j < n ? p[e + j] : 0.0f;
        v[0] = make_float2(t[0], t[1]);
        v[1] = make_float2(t[2], t[3]);
    }
}
template <bool FULL>
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, uint32_t e, uint32_t n, float2 *v) {
    uint2 w = make_uint2(0u, 0u);
    if (FULL || e + 4 <= n) {
        w = *reinterpret_cast<const uint2 *>(p + e);
    } else {
        const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
        if (e < n) w.x = q[e];
        if (e + 1 < n) w.x |= static_cast<uint32_t>(q[e + 1]) << 16;
        if (e + 2 < n) w.y = q[e + 2];
    }
    v[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
    v[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
}
template <bool FULL>
__device__ __forceinline__ void store4(float *p, uint32_t e, uint32_t n, const float2 *v) {
    if (FULL || e + 4 <= n) {
        *reinterpret_cast<float4 *>(p + e) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    } else {
        if (e < n) p[e] = v[0].x;
        if (e + 1 < n) p[e + 1] = v[0].y;
        if (e + 2 < n) p[e + 2] = v[1].x;
    }
}
template <bool FULL>
__device__ __forceinline__ void store4(__nv_bfloat16 *p, uint32_t e, uint32_t n, const float2 *v) {
    const uint2 w = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
    if (FULL || e + 4 <= n) {
        *reinterpret_cast<uint2 *>(p + e) = w;
    } else {
        unsigned short *q = reinterpret_cast<unsigned short *>(p);
        if (e < n) q[e] = static_cast<unsigned short>(w.x);
        if (e + 1 < n) q[e + 1] = static_cast<unsigned short>(w.x >> 16);
        if (e + 2 < n) q[e + 2] = static_cast<unsigned short>(w.y);
    }
}

// e4m3 codes, 4 in a word
template <bool FULL>
__device__ __forceinline__ uint32_t load4_codes(const uint8_t *p, uint32_t e, uint32_t n) {
    if (FULL || e + 4 <= n) return *reinterpret_cast<const uint32_t *>(p + e);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (e + j < n) w |= static_cast<uint32_t>(p[e + j]) << (8 * j);
    return w;
}
template <bool FULL>
__device__ __forceinline__ void store4_codes(uint8_t *p, uint32_t e, uint32_t n, uint32_t w) {
    if (FULL || e + 4 <= n) {
        *reinterpret_cast<uint32_t *>(p + e) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (e + j < n) p[e + j] = static_cast<uint8_t>(w >> (8 * j));
    }
}
__device__ __forceinline__ void decode4(uint32_t w, float2 *v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t two;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<unsigned short>(w >> (16 * h))));
        v[h] = __half22float2(*reinterpret_cast<const __half2 *>(&two));
    }
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// 1 / x to one unit in the last place, for a normal x (eps is one, and a root
// is below 2^64); past 2^126 it is zero
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Square roots, rounded correctly for v from 2^-100 up: one Newton step from
// the approximate reciprocal root, its residual s^2 - v exact in a fused
// operation (Markstein, IBM J. Res. Dev. 34, 1990).  test_gpu_adamw_roots.py
// compares 2^17 of them with IEEE roots.  With sqrtf the profile counted ten
// branch instructions an element more.
constexpr float kRootMin = 7.8886091e-31f;  // 2^-100
__device__ __forceinline__ float2 roots(float2 v) {
    float2 y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(v.x));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(v.y));
    const float2 s = __fmul2_rn(v, y), rest = __ffma2_rn(s, s, make_float2(-v.x, -v.y));
    return __ffma2_rn(rest, __fmul2_rn(y, both(-0.5f)), s);
}
// Largest magnitude of three, NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// two products that no addition is fused with
__device__ __forceinline__ float2 mul(float a, float2 x) { return make_float2(__fmul_rn(a, x.x), __fmul_rn(a, x.y)); }

// 32 bits to 32 well-spread bits: xor-shifts and odd multipliers
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * kMix1;
    x = (x ^ (x >> 15)) * kMix2;
    return x ^ (x >> 16);
}

// The hash of element e of a block is mix(key ^ e kMix1), its low half the
// random bits of m and its high half those of the root.  The first xor-shift
// is linear: taken of the key and of e kMix1 apart, the element's part is the
// same for every block.  Both halves come out where round_e4m3 adds them, at
// bits 8..23.
__device__ __forceinline__ void random_bits(uint32_t shifted_key, uint32_t e_mix1, uint32_t &of_m, uint32_t &of_r) {
    uint32_t x = (shifted_key ^ e_mix1 ^ (e_mix1 >> 16)) * kMix1;
    x = (x ^ (x >> 15)) * kMix2;
    const uint32_t t = x >> 8;
    of_m = ((x << 8) ^ t) & 0x00FFFF00u;
    of_r = t & 0x00FFFF00u;
}

// |x|, 0 .. 448 but for rounding, scaled by 2^-120, to the bits of one of its
// two neighbouring e4m3 values in the top byte, the upper one with a
// probability of its nearness (16 random bits of it).  At that scale e4m3's
// smallest normal value, 2^-6, is fp32's, 2^-126, so the formats' subnormal
// values coincide too: a code's 7 bits are bits 20..26 of the fp32 value, and
// one integer addition rounds in both ranges.  448 plus the most random bits
// that there are, 0x7EFFFF00, stays below 0x7F000000 (the code of NaN), and so
// do the few units in the last place that 448 |x| / max |x| may exceed it by.
__device__ __forceinline__ uint32_t round_e4m3(float x, uint32_t bits) {
    return (__float_as_uint(x) << 4) + bits;  // the shift drops the sign
}
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Scale of a block from its lanes' largest magnitudes, and the factor that its
// values take before rounding, 2^-120 448 / t.  Below 2^-100 (where 448 / t
// nears the range of fp32) a block is kept as zero.  Above 2^12 the factor would
// leave that range: the values take 2^-64 first, and `large` says so.  `poison`
// marks a block that holds a NaN or an infinity (as integers the magnitudes'
// bits order NaN above all): its codes are then NaN.
struct Scale {
    float factor, scale;
    bool large;
    uint32_t poison;
};
__device__ __forceinline__ Scale block_scale(float lane_top) {
    const float t = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(lane_top) & 0x7FFFFFFFu));
    const bool zero = t < 7.888609e-31f;
    Scale s;
    s.large = t > 4096.0f;
    s.factor = zero ? 0.0f : __fmul_rn(__frcp_rn(t), 448.0f) * (s.large ? 1.38777878e-17f : 7.52316385e-37f);  // 2^-56, 2^-120
    s.scale = zero ? 0.0f : __fmul_rn(t, 1.0f / 448.0f);
    s.poison = t < __uint_as_float(0x7F800000u) ? 0u : 0x7F7F7F7Fu;
    return s;
}
__device__ __forceinline__ void scale_values(const Scale &s, float2 (&x)[2][2]) {
    if (s.large) {  // the whole warp
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) x[j][i] = __fmul2_rn(x[j][i], both(5.42101086e-20f));  // 2^-64
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) x[j][i] = __fmul2_rn(x[j][i], both(s.factor));
}

// ---------------------------------------------------------------------------
// The step.  A warp takes 256 consecutive elements (a block of the 8-bit
// states), 8 a lane in two runs of 4, so that every load and store of a warp
// is contiguous and a block's largest value is one warp reduction.
//
// Bound by HBM.  134M bf16 parameters with fp32 master copies and gradients:
// 30 bytes an element with 32-bit states, 580 us (6.9 TB/s), and 18 bytes with
// 8-bit states, 352 us (6.9 TB/s, above a plain copy's rate).  With 8 bits the
// arithmetic is nearly as long as the memory's time, and with bf16 gradients
// and fp32 parameters (14 bytes) it is longer: 349 us.  Hence the loads staged a
// chunk ahead, the rounding in two integer operations, one hash for both
// states, the roots without branches, the paired products and the extremes of
// three (558 us with none of them and even runs of chunks), and four blocks of 64
// registers.  bf16 parameters fit these; fp32 parameters spill 8 bytes (16 with
// bf16 gradients).
// ---------------------------------------------------------------------------
// What a lane reads of a block.
template <typename G, int BITS>
struct Values {
    float2 w[2][2], g[2][2], m[2][2], v[2][2];
    uint32_t mc[2], vc[2];
    float ms, vs;
};

// A chunk of a tensor: where its arrays start, and the elements that are left
// of the tensor from there on (at most a chunk's count).
template <typename G>
struct Chunk {
    float *w;
    __nv_bfloat16 *p;
    const G *g;
    void *m, *v;
    float *ms, *vs;
    uint32_t left;
};
template <typename G, int BITS>
__device__ __forceinline__ Chunk<G> chunk_of(const Entry &t, int index) {
    const long long e = static_cast<long long>(index) * kChunk, blk = static_cast<long long>(index) * (kChunk / kBlock);
    Chunk<G> k;
    k.w = static_cast<float *>(t.w) + e;
    k.p = static_cast<__nv_bfloat16 *>(t.p) + e;
    k.g = static_cast<const G *>(t.g) + e;
    k.m = static_cast<char *>(t.m) + e * (BITS / 8);
    k.v = static_cast<char *>(t.v) + e * (BITS / 8);
    k.ms = t.ms + blk;
    k.vs = t.vs + blk;
    const long long left = t.n - e;
    k.left = left < kChunk ? static_cast<uint32_t>(left) : kChunk;
    return k;
}

template <bool FULL, typename G, int BITS>
__device__ __forceinline__ void read_block(const Chunk<G> &t, uint32_t e0, Values<G, BITS> &x) {
    if (BITS == 8) {
        x.ms = t.ms[threadIdx.x >> 5];
        x.vs = t.vs[threadIdx.x >> 5];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t e = e0 + j * 128;
        load4<FULL>(static_cast<const float *>(t.w), e, t.left, x.w[j]);
        load4<FULL>(t.g, e, t.left, x.g[j]);
        if (BITS == 32) {
            load4<FULL>(static_cast<const float *>(t.m), e, t.left, x.m[j]);
            load4<FULL>(static_cast<const float *>(t.v), e, t.left, x.v[j]);
        } else {
            x.mc[j] = load4_codes<FULL>(static_cast<const uint8_t *>(t.m), e, t.left);
            x.vc[j] = load4_codes<FULL>(static_cast<const uint8_t *>(t.v), e, t.left);
        }
    }
}

// `staged`: where the weights are staged (8 bits, whole blocks), else null.
template <bool FULL, bool HALF, typename G, int BITS>
__device__ __forceinline__ void step_block(const Chunk<G> &t, uint32_t e0, Values<G, BITS> &x, const float *staged, uint32_t key,
                                           uint32_t e_mix1, const Hyper &hy, float scale, float decay,
                                           float rate, float inv_root_bc2) {
    const uint32_t n = t.left;
    float2 (&w)[2][2] = x.w, (&g)[2][2] = x.g, (&m)[2][2] = x.m, (&v)[2][2] = x.v;
    uint32_t (&mc)[2] = x.mc, (&vc)[2] = x.vc;
    float &ms = x.ms, &vs = x.vs;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (BITS == 8) {
            decode4(mc[j], m[j]);
            decode4(vc[j], v[j]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (BITS == 8) {
                m[j][i] = __fmul2_rn(m[j][i], both(ms));
                v[j][i] = __fmul2_rn(v[j][i], both(vs));
                v[j][i] = __fmul2_rn(v[j][i], v[j][i]);
            }
            // The states are those of separately rounded products and sums: contracted
            // into fused operations, which of them is fused would be part of the result.
            // The compiler does contract the paired forms, so products that are added
            // are single ones.
            const float2 gi = __fmul2_rn(g[j][i], both(scale)), cg = __fmul2_rn(both(hy.c2), gi);
            m[j][i] = __fadd2_rn(mul(hy.b1, m[j][i]), mul(hy.c1, gi));
            v[j][i] = __fadd2_rn(mul(hy.b2, v[j][i]), make_float2(__fmul_rn(cg.x, gi.x), __fmul_rn(cg.y, gi.y)));
        }
    }
    float2 root[2][2];
    float top_m = 0.0f, top_r = 0.0f;
    uint32_t some[2] = {0x01010101u, 0x01010101u};  // a byte for each element: its root is above zero
    if (BITS == 8) {
        float least = 3.4e38f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                root[j][i] = roots(v[j][i]);
                least = min3(least, v[j][i].x, v[j][i].y);
                top_m = max_abs3(top_m, m[j][i].x, m[j][i].y);
                top_r = max_abs3(top_r, root[j][i].x, root[j][i].y);
            }
        // outside what roots() takes (zeros above all), where it may have left a NaN
        if (!(least >= kRootMin && top_r < __uint_as_float(0x7F800000u))) {
            top_r = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                some[j] = 0u;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    root[j][i] = make_float2(sqrtf(v[j][i].x), sqrtf(v[j][i].y));
                    top_r = max_abs3(top_r, root[j][i].x, root[j][i].y);
                    some[j] |= (root[j][i].x > 0.0f ? 1u << (16 * i) : 0u) | (root[j][i].y > 0.0f ? 256u << (16 * i) : 0u);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t e = e0 + j * 128;
        if (BITS == 8 && FULL) load4<true>(staged, (j * kThreads + threadIdx.x) * 4, 0, w[j]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (BITS == 32) root[j][i] = make_float2(sqrtf(v[j][i].x), sqrtf(v[j][i].y));
            const float2 d = __ffma2_rn(root[j][i], both(inv_root_bc2), both(hy.eps));
            const float2 q = __fmul2_rn(m[j][i], both(-rate));
            w[j][i] = __ffma2_rn(q, make_float2(reciprocal(d.x), reciprocal(d.y)),
                                 __ffma2_rn(both(-decay), w[j][i], w[j][i]));
        }
        store4<FULL>(t.w, e, n, w[j]);
        if (HALF) store4<FULL>(t.p, e, n, w[j]);
        if (BITS == 32) {
            store4<FULL>(static_cast<float *>(t.m), e, n, m[j]);
            store4<FULL>(static_cast<float *>(t.v), e, n, v[j]);
        }
    }
    if (BITS == 32) return;
    const Scale sm = block_scale(top_m), sr = block_scale(top_r);
    const uint32_t shifted_key = key ^ (key >> 16);
    scale_values(sm, m);
    scale_values(sr, root);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t cm[4], cr[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t of_m, of_r;
            random_bits(shifted_key, e_mix1 + (j * 128 + 2 * i) * kMix1, of_m, of_r);
            cm[2 * i] = round_e4m3(m[j][i].x, of_m);
            cr[2 * i] = round_e4m3(root[j][i].x, of_r);
            random_bits(shifted_key, e_mix1 + (j * 128 + 2 * i + 1) * kMix1, of_m, of_r);
            cm[2 * i + 1] = round_e4m3(m[j][i].y, of_m);
            cr[2 * i + 1] = round_e4m3(root[j][i].y, of_r);
        }
        const uint32_t sign = top_bytes(__float_as_uint(m[j][0].x), __float_as_uint(m[j][0].y),
                                        __float_as_uint(m[j][1].x), __float_as_uint(m[j][1].y)) & 0x80808080u;
        mc[j] = top_bytes(cm[0], cm[1], cm[2], cm[3]) | sign | sm.poison;
        vc[j] = top_bytes(cr[0], cr[1], cr[2], cr[3]) | sr.poison;
        // bit 7 of each byte: whether it is zero; a root above zero keeps a code above zero
        const uint32_t none = ~(((vc[j] & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | vc[j]);
        vc[j] |= (none >> 7) & some[j];
        store4_codes<FULL>(static_cast<uint8_t *>(t.m), e0 + j * 128, n, mc[j]);
        store4_codes<FULL>(static_cast<uint8_t *>(t.v), e0 + j * 128, n, vc[j]);
    }
    ms = sm.scale;
    vs = sr.scale;
    if ((threadIdx.x & 31) == 0) {
        t.ms[threadIdx.x >> 5] = ms;
        t.vs[threadIdx.x >> 5] = vs;
    }
}

// A run of consecutive chunks for every thread block, and the tensor that the
// current one lies in.
template <int CAP>
struct Walk {
    int c, end, ti;
    __device__ __forceinline__ Walk(const Table<CAP> &tab) {
        const int chunks = tab.chunk0[tab.count];
        // even runs: the first `chunks % blocks` are one longer
        const int each = chunks / gridDim.x, more = chunks - each * gridDim.x;
        const int b = blockIdx.x;
        c = b * each + min(b, more);
        end = c + each + (b < more);
        ti = c < end ? tensor_of(tab, c) : 0;
    }
    __device__ __forceinline__ void next(const Table<CAP> &tab) {
        if (++c < end)
            while (tab.chunk0[ti + 1] <= c) ++ti;
    }
};

// The asynchronous copies of the 8-bit form: every lane stages its own values
// of the blocks ahead, and reads back only those, so a wait on its own copies
// is all the synchronisation there is.
constexpr int kStages = 2;
template <typename G>
constexpr int stage_bytes() { return kThreads * (2 * 16 + 2 * 4 * static_cast<int>(sizeof(G)) + 6 * 4); }

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <typename G>
__device__ __forceinline__ void stage_block(const Chunk<G> &t, uint32_t e, uint32_t at) {
    at += threadIdx.x * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        copy_async16(at + j * kThreads * 16, t.w + (e + j * 128));
        if (sizeof(G) == 4)
            copy_async16(at + (2 + j) * kThreads * 16, t.g + (e + j * 128));
        else
            copy_async8(at + 2 * kThreads * 16 + (j * kThreads - static_cast<int>(threadIdx.x)) * 8, t.g + (e + j * 128));
    }
    at += kThreads * (32 + 8 * sizeof(G)) - threadIdx.x * 12;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        copy_async4(at + j * kThreads * 4, static_cast<const uint8_t *>(t.m) + (e + j * 128));
        copy_async4(at + (2 + j) * kThreads * 4, static_cast<const uint8_t *>(t.v) + (e + j * 128));
    }
    copy_async4(at + 4 * kThreads * 4, t.ms + (threadIdx.x >> 5));  // every lane its own copy of the scales
    copy_async4(at + 5 * kThreads * 4, t.vs + (threadIdx.x >> 5));
}
template <typename G>
__device__ __forceinline__ void staged_block(const uint8_t *at, Values<G, 8> &x) {
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(at + kThreads * (32 + 8 * sizeof(G)));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        load4<true>(reinterpret_cast<const G *>(at + 2 * kThreads * 16), (j * kThreads + threadIdx.x) * 4, 0, x.g[j]);
        x.mc[j] = codes[j * kThreads + threadIdx.x];
        x.vc[j] = codes[(2 + j) * kThreads + threadIdx.x];
    }
    x.ms = __uint_as_float(codes[4 * kThreads + threadIdx.x]);
    x.vs = __uint_as_float(codes[5 * kThreads + threadIdx.x]);
}

template <int CAP, bool HALF, typename G, int BITS>
__global__ void __launch_bounds__(kThreads, 4) step_kernel(const __grid_constant__ Table<CAP> tab,
                                                           const __grid_constant__ Hyper hy) {
    extern __shared__ __align__(16) uint8_t stages[];
    float scale = hy.scale, inv_bc1 = hy.inv_bc1, inv_root_bc2 = hy.inv_root_bc2;
    uint32_t step = hy.step;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before, whose end this launch overlaps
    if (hy.ctl) {
        if (!hy.ctl->finite) return;
        scale = hy.ctl->scale;
        inv_bc1 = hy.ctl->inv_bc1;
        inv_root_bc2 = hy.ctl->inv_root_bc2;
        step = static_cast<uint32_t>(hy.ctl->steps);
    }
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t at_step = mix(hy.seed + kMix1 * step);
    const uint32_t e_mix1 = lane * 4 * kMix1;
    const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(stages));
    const uint32_t e0 = warp * kBlock + lane * 4;
    Walk<CAP> now(tab), ahead = now;
    // stages the next whole block of this warp; a group is committed in any case, so that the count of groups is that of chunks
    auto fetch = [&](int slot) {
        if (ahead.c < ahead.end) {
            const Chunk<G> t = chunk_of<G, BITS>(tab.t[ahead.ti], ahead.c - tab.chunk0[ahead.ti]);
            if ((warp + 1) * kBlock <= t.left) stage_block<G>(t, e0, smem + slot * stage_bytes<G>());
            ahead.next(tab);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (BITS == 8) {
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i);
    }
    int slot = 0, of = -1;
    uint32_t of_tensor = 0;
    float decay = 0.0f, rate = 0.0f;
    for (; now.c < now.end; now.next(tab)) {
        const int ti = now.ti, index = now.c - tab.chunk0[ti];
        const Chunk<G> t = chunk_of<G, BITS>(tab.t[ti], index);
        if (ti != of) {
            of = ti;
            const float lr = hy.lr * tab.lr_scale[ti];
            decay = lr * tab.decay[ti];
            rate = lr * inv_bc1;
            of_tensor = mix(at_step ^ (static_cast<uint32_t>(tab.base + ti) * kMix2 + 1u));
        }
        uint32_t key = 0;
        if (BITS == 8) key = mix(of_tensor + static_cast<uint32_t>(index * (kChunk / kBlock) + warp));
        Values<G, BITS> x;
        if (BITS == 8) {
            fetch(slot == 0 ? kStages - 1 : slot - 1);  // the slot read in the last round
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        }
        if ((warp + 1) * kBlock <= t.left) {
            if constexpr (BITS == 8)
                staged_block<G>(stages + slot * stage_bytes<G>(), x);
            else
                read_block<true, G, BITS>(t, e0, x);
            step_block<true, HALF, G, BITS>(t, e0, x, reinterpret_cast<const float *>(stages + slot * stage_bytes<G>()), key, e_mix1, hy, scale, decay, rate, inv_root_bc2);
        } else if (warp * kBlock < t.left) {
            read_block<false, G, BITS>(t, e0, x);
            step_block<false, HALF, G, BITS>(t, e0, x, nullptr, key, e_mix1, hy, scale, decay, rate, inv_root_bc2);
        }
        slot = slot + 1 == kStages ? 0 : slot + 1;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------
// The gradient norm.  Every block leaves one sum of squares; the block that
// finishes last adds them in their order, so the result does not depend on
// which it is.  Within a thread the squares (rounded to fp32) are added with
// the error of every addition kept beside the sum (Knuth's two-sum), 7
// additions an element, in pairs; fp64, which this machine has few units for,
// comes once at the end (one fp64 addition for 8 elements was the bound before:
// 157 us for 134M fp32 gradients; now 85 us, 6.3 TB/s, and 101 us right after
// a step, whose last writes still leave L2).  The norm is then the rounded norm
// of the rounded squares, whatever the order, and the clip factor that scales
// every gradient does not move with the list's grouping.
//
// That needs squares that fp32 holds.  A thread's sum tells: between 2^-90 and
// 2^90 none overflowed, and what underflowed was less than 2^-38 of it (a thread
// has at most 2^21 elements, and loses up to 2^-150 of each).  A thread whose sum
// lies outside reads its gradients again, scaled, and joins in fp64: any finite
// gradients have their norm.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __fadd2_rn(a, make_float2(-b.x, -b.y)); }

struct NormArgs {
    Ctl *ctl;
    float grad_scale, max_norm;
    float log_beta1, log_beta2;
    int first, last;  // of the launches over one list
};

// (s, rest) += the squares of g, or of k g
template <bool SCALED, int L>
__device__ __forceinline__ void add_squares(const float2 (&g)[L][2], float k, float2 &s, float2 &rest) {
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float x = SCALED ? __fmul_rn(g[j][i].x, k) : g[j][i].x, y = SCALED ? __fmul_rn(g[j][i].y, k) : g[j][i].y;
            const float2 q = make_float2(__fmul_rn(x, x), __fmul_rn(y, y));
            const float2 z = __fadd2_rn(s, q), d = sub2(z, s);
            rest = __fadd2_rn(rest, __fadd2_rn(sub2(s, sub2(z, d)), sub2(q, d)));
            s = z;
        }
}
constexpr float kSumMin = 8.077935669463161e-28f, kSumMax = 1.2379400392853803e+27f;  // 2^-90, 2^90
// A thread's sum where fp32 does not hold its squares, all its gradients read
// again (a NaN or an infinity among them: NaN).  Not inlined, for the registers.
template <int CAP, typename G>
__device__ __noinline__ double scaled_squares(const Table<CAP> &tab, bool large) {
    constexpr int L = kNormChunk / (4 * kThreads);
    float2 s = both(0.0f), rest = both(0.0f);
    for (Walk<CAP> now(tab); now.c < now.end; now.next(tab)) {
        const long long e0 = static_cast<long long>(now.c - tab.chunk0[now.ti]) * kNormChunk, left = tab.t[now.ti].n - e0;
        const G *in = static_cast<const G *>(tab.t[now.ti].g) + e0;
        const uint32_t n = left < kNormChunk ? static_cast<uint32_t>(left) : kNormChunk;
        float2 g[L][2];
#pragma unroll
        for (int j = 0; j < L; ++j) load4<false>(in, threadIdx.x * 4 + j * 4 * kThreads, n, g[j]);
        add_squares<true>(g, large ? 8.271806125530277e-25f : 1.2676506002282294e+30f, s, rest);  // 2^-80, 2^100
    }
    return (static_cast<double>(s.x) + s.y + rest.x + rest.y) * (large ? 1.461501637330903e+48 : 6.223015277861142e-61);  // 2^160, 2^-200
}

// (s, rest) += (a, b): the error of s + a joins the rests
__device__ __forceinline__ void add_pair(float &s, float &rest, float a, float b) {
    const float z = __fadd_rn(s, a), d = __fsub_rn(z, s);
    rest = rest + b + (__fsub_rn(s, __fsub_rn(z, d)) + __fsub_rn(a, d));
    s = z;
}

__device__ __forceinline__ double block_sum(double s, double *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    return s;
}

// (five blocks an SM for bf16, whose loads are half as large: 40M gradients in 97 tensors 4 us longer with four)
template <int CAP, typename G>
__global__ void __launch_bounds__(kThreads, sizeof(G) == 2 ? 5 : 4) norm_kernel(const __grid_constant__ Table<CAP> tab,
                                                                                const __grid_constant__ NormArgs a) {
    __shared__ double red[kThreads / 32];
    __shared__ int is_last;
    float2 s = both(0.0f), rest = both(0.0f);
    Walk<CAP> now(tab);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (; now.c < now.end; now.next(tab)) {
        const long long e0 = static_cast<long long>(now.c - tab.chunk0[now.ti]) * kNormChunk, left = tab.t[now.ti].n - e0;
        const G *in = static_cast<const G *>(tab.t[now.ti].g) + e0;
        const uint32_t e = threadIdx.x * 4, n = left < kNormChunk ? static_cast<uint32_t>(left) : kNormChunk;
        constexpr int L = kNormChunk / (4 * kThreads);
        float2 g[L][2];
        if (n == kNormChunk) {
#pragma unroll
            for (int j = 0; j < L; ++j) load4<true>(in, e + j * 4 * kThreads, n, g[j]);
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j) load4<false>(in, e + j * 4 * kThreads, n, g[j]);
        }
        add_squares<false>(g, 1.0f, s, rest);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    double beyond = 0.0;
    const float size = s.x + s.y;
    if (!(size >= kSumMin && size <= kSumMax)) {
        beyond = scaled_squares<CAP, G>(tab, !(size < kSumMin));
        s = rest = both(0.0f);
    }
    add_pair(s.x, rest.x, s.y, rest.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        add_pair(s.x, rest.x, __shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, rest.x, o));
    if (__any_sync(0xffffffffu, beyond != 0.0)) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) beyond += __shfl_xor_sync(0xffffffffu, beyond, o);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = static_cast<double>(s.x) + rest.x + beyond;
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) sum += red[w];
        if (!a.first) sum += a.ctl->partial[blockIdx.x];
        a.ctl->partial[blockIdx.x] = sum;
        is_last = 0;
        if (a.last) {
            __threadfence();
            is_last = atomicAdd(&a.ctl->ticket, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    sum = 0.0;
    for (int i = threadIdx.x; i < gridDim.x; i += kThreads) sum += __ldcg(&a.ctl->partial[i]);
    sum = block_sum(sum, red);
    if (threadIdx.x) return;
    const float norm = static_cast<float>(sqrt(sum) * a.grad_scale);
    // the states hold squares of scaled gradients: the clipped norm, which bounds these, has to have one
    const float most = fminf(norm, a.max_norm);
    const bool finite = norm <= 3.402823466e38f && most * most <= 3.402823466e38f;
    a.ctl->ticket = 0;
    a.ctl->norm = norm;
    a.ctl->finite = finite;
    a.ctl->scale = a.grad_scale * fminf(__frcp_rn(norm) * a.max_norm, 1.0f);
    if (finite) {
        const int t = ++a.ctl->steps;
        // 1 - b^t = -expm1(t log b), without fp64's slow powers and without cancellation
        a.ctl->inv_bc1 = -1.0f / expm1f(t * a.log_beta1);
        a.ctl->inv_root_bc2 = 1.0f / sqrtf(-expm1f(t * a.log_beta2));
    }
}

__global__ void ctl_init_kernel(Ctl *ctl, int steps) {
    if (threadIdx.x == 0) {
        ctl->norm = 0.0f;
        ctl->scale = 1.0f;
        ctl->finite = 0;
        ctl->steps = steps;
        ctl->inv_bc1 = ctl->inv_root_bc2 = 1.0f;
        ctl->ticket = 0;
    }
}

}  // namespace adam
}  // namespace tpmlp

using namespace tpmlp;

struct tp_adamw {
    tp_adamw_desc d;
    tp_adamw_tensor *t;
    long long norm_chunks;
    adam::Plans<adam::kSmall> few;   // the launches' tables: these for a short list,
    adam::Plans<adam::kLarge> many;  // these for a long one
};

#define TRY(x)                        \
    do {                              \
        tp_status _s = (x);           \
        if (_s != TP_OK) return _s;   \
    } while (0)

static tp_status aw_pointer(const void *p, const char *name, int i, unsigned align = 16) {
    if (!p) return set_error(TP_ERR_ARG, "%s[%d] is NULL", name, i);
    if (reinterpret_cast<uintptr_t>(p) & (align - 1))
        return set_error(TP_ERR_ARG, "%s[%d] is not %u-byte aligned", name, i, align);
    return TP_OK;
}

static tp_status aw_validate(const tp_adamw_desc *d, const tp_adamw_tensor *t) {
    if (!d) return set_error(TP_ERR_ARG, "descriptor is NULL");
    if (d->n_tensors < 1 || d->n_tensors > TP_ADAMW_MAX_TENSORS)
        return set_error(TP_ERR_SHAPE, "n_tensors=%d outside 1..%d", d->n_tensors, TP_ADAMW_MAX_TENSORS);
    if (d->param_dtype != TP_DT_F32 && d->param_dtype != TP_DT_BF16)
        return set_error(TP_ERR_ARG, "bad param_dtype %d", d->param_dtype);
    if (d->grad_dtype != TP_DT_F32 && d->grad_dtype != TP_DT_BF16)
        return set_error(TP_ERR_ARG, "bad grad_dtype %d", d->grad_dtype);
    if (d->state_bits != 8 && d->state_bits != 32)
        return set_error(TP_ERR_ARG, "state_bits=%d is neither 8 nor 32", d->state_bits);
    if (!(d->beta1 >= 0.0 && d->beta1 < 1.0) || !(d->beta2 >= 0.0 && d->beta2 < 1.0))
        return set_error(TP_ERR_ARG, "beta1 and beta2 must be in [0, 1)");
    if (!(d->eps >= 1.17549435e-38f) || !std::isfinite(d->eps))
        return set_error(TP_ERR_ARG, "eps must be a positive normal number");
    if (!t) return set_error(TP_ERR_ARG, "tensors is NULL");
    long long chunks = 0;
    for (int i = 0; i < d->n_tensors; ++i) {
        if (t[i].n < 0) return set_error(TP_ERR_SHAPE, "tensor %d: negative element count", i);
        if (t[i].n > (1ll << 38)) return set_error(TP_ERR_SHAPE, "tensor %d: more than 2^38 elements", i);
        chunks += (t[i].n + adam::kChunk - 1) / adam::kChunk;
        if (chunks >= (1ll << 30)) return set_error(TP_ERR_SHAPE, "more than 2^41 elements");
        if (!std::isfinite(t[i].lr_scale) || !std::isfinite(t[i].weight_decay))
            return set_error(TP_ERR_ARG, "tensor %d: lr_scale and weight_decay must be finite", i);
        if (t[i].n == 0) continue;
        TRY(aw_pointer(t[i].param, "param", i));
        if (d->param_dtype == TP_DT_BF16) TRY(aw_pointer(t[i].master, "master", i));
        TRY(aw_pointer(t[i].grad, "grad", i));
        TRY(aw_pointer(t[i].m, "m", i));
        TRY(aw_pointer(t[i].v, "v", i));
        if (d->state_bits == 8) {
            TRY(aw_pointer(t[i].m_scale, "m_scale", i, 4));
            TRY(aw_pointer(t[i].v_scale, "v_scale", i, 4));
        }
    }
    return TP_OK;
}

namespace tpmlp {
namespace adam {

// the table of tensors [i, i + CAP) of the list, or what it has of them
template <int CAP>
static void fill(const tp_adamw *h, int i, int chunk, Table<CAP> &tab) {
    tab.base = i;
    tab.count = 0;
    tab.chunk0[0] = 0;
    for (; i < h->d.n_tensors && tab.count < CAP; ++i) {
        const tp_adamw_tensor &s = h->t[i];
        Entry &e = tab.t[tab.count];
        const bool half = h->d.param_dtype == TP_DT_BF16;
        e.w = half ? static_cast<void *>(s.master) : s.param;
        e.p = half ? s.param : nullptr;
        e.g = s.grad;
        e.m = s.m;
        e.v = s.v;
        e.ms = s.m_scale;
        e.vs = s.v_scale;
        e.n = s.n;
        tab.lr_scale[tab.count] = s.lr_scale;
        tab.decay[tab.count] = s.weight_decay;
        tab.chunk0[tab.count + 1] = tab.chunk0[tab.count] + static_cast<int>((s.n + chunk - 1) / chunk);
        ++tab.count;
    }
    const int chunks = tab.chunk0[tab.count];
    for (tab.shift = 0; (chunks >> tab.shift) >= kCoarse; ++tab.shift) {
    }
    for (int k = 0, t = 0; k <= kCoarse; ++k) {
        const long long c = static_cast<long long>(k) << tab.shift;
        while (t + 1 < tab.count && tab.chunk0[t + 1] <= c) ++t;
        tab.coarse[k] = static_cast<unsigned short>(t);
    }
}

// Thread blocks for a number of chunks.  Even runs for just the resident blocks
// end unevenly (SMs were busy 0.9 of the time) and spread what is read and
// written at one time over the whole list; short runs are dealt out by the
// hardware, in order, as blocks finish.  134M elements in 8 bits: 494 us with
// one run a resident block, 417 with runs of 6 or 7 chunks, 364 with 2, 416
// with single ones, which stage nothing ahead.  The norm's blocks end with a
// reduction and an atomic, so its runs are longer (8 chunks and 2: 23 and 25 us
// for 24M elements in 300 tensors, the same for one large one).
constexpr int kRun = 2, kNormRun = 8;
static int blocks_for(int chunks, int run, int resident) {
    if (chunks <= resident) return chunks;
    const int runs = (chunks + run - 1) / run;
    return runs > resident ? runs : resident;
}

// A launch whose start may overlap the end of the kernel before it.
static cudaLaunchConfig_t launch_config(int grid, int smem, cudaStream_t st, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_on() ? 1 : 0;
    return cfg;
}

template <int CAP>
static tp_status step_launch(const Table<CAP> &tab, const tp_adamw_desc &d, const Hyper &hy, cudaStream_t st) {
    using bf = __nv_bfloat16;
    using K = void (*)(Table<CAP>, Hyper);
    K k;
    const bool half = d.param_dtype == TP_DT_BF16, gh = d.grad_dtype == TP_DT_BF16;
    if (d.state_bits == 32)
        k = half ? (gh ? step_kernel<CAP, true, bf, 32> : step_kernel<CAP, true, float, 32>)
                 : (gh ? step_kernel<CAP, false, bf, 32> : step_kernel<CAP, false, float, 32>);
    else
        k = half ? (gh ? step_kernel<CAP, true, bf, 8> : step_kernel<CAP, true, float, 8>)
                 : (gh ? step_kernel<CAP, false, bf, 8> : step_kernel<CAP, false, float, 8>);
    const int chunks = tab.chunk0[tab.count];
    if (!chunks) return TP_OK;
    const int grid = blocks_for(chunks, kRun, 4 * num_sms());
    const int smem = d.state_bits == 8 ? kStages * (gh ? stage_bytes<bf>() : stage_bytes<float>()) : 0;
    static_assert(kStages * stage_bytes<float>() <= 48 * 1024, "within what a launch may ask for without an attribute");
    launch_begin("adamw_step", st);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = launch_config(grid, smem, st, attr);
    void *args[] = {const_cast<Table<CAP> *>(&tab), const_cast<Hyper *>(&hy)};  // no copies of the table on the way
    cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(k), args);
    launch_end("adamw_step", st);
    return cuda_check(e, "adamw_step");
}

template <int CAP>
static tp_status norm_launch(const Table<CAP> &tab, const tp_adamw_desc &d, const NormArgs &a, int grid,
                             cudaStream_t st) {
    launch_begin("adamw_grad_norm", st);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = launch_config(grid, 0, st, attr);
    using K = void (*)(Table<CAP>, NormArgs);
    const K k = d.grad_dtype == TP_DT_BF16 ? norm_kernel<CAP, __nv_bfloat16> : norm_kernel<CAP, float>;
    void *args[] = {const_cast<Table<CAP> *>(&tab), const_cast<NormArgs *>(&a)};
    cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(k), args);
    launch_end("adamw_grad_norm", st);
    return cuda_check(e, "adamw_grad_norm");
}

static_assert(sizeof(Table<kLarge>) + sizeof(Hyper) <= 32764, "a launch's parameters");
static_assert(sizeof(Table<kLarge>) + sizeof(NormArgs) <= 32764, "a launch's parameters");

// (re)makes the tables of a handle; false without memory for them
template <int CAP>
static bool make_plans(tp_adamw *h, Plans<CAP> &p) {
    const int launches = (h->d.n_tensors + CAP - 1) / CAP;
    if (!p.step) p.step = new (std::nothrow) Table<CAP>[launches];
    if (!p.norm) p.norm = new (std::nothrow) Table<CAP>[launches];
    if (!p.step || !p.norm) return false;
    p.launches = launches;
    for (int k = 0; k < launches; ++k) {
        fill(h, k * CAP, kChunk, p.step[k]);
        fill(h, k * CAP, kNormChunk, p.norm[k]);
    }
    return true;
}
static bool make_plans(tp_adamw *h) {
    h->norm_chunks = 0;
    for (int i = 0; i < h->d.n_tensors; ++i) h->norm_chunks += (h->t[i].n + kNormChunk - 1) / kNormChunk;
    return h->d.n_tensors <= kSmall ? make_plans(h, h->few) : make_plans(h, h->many);
}

template <int CAP>
static tp_status step_all(const Plans<CAP> &p, const tp_adamw_desc &d, const Hyper &hy, cudaStream_t st) {
    for (int k = 0; k < p.launches; ++k) TRY(step_launch(p.step[k], d, hy, st));
    return TP_OK;
}

template <int CAP>
static tp_status norm_all(const Plans<CAP> &p, const tp_adamw *h, NormArgs a, cudaStream_t st) {
    int grid = blocks_for(static_cast<int>(h->norm_chunks), kNormRun, 4 * num_sms());
    grid = grid < 1 ? 1 : grid > kNormBlocks ? kNormBlocks : grid;
    for (int k = 0; k < p.launches; ++k) {
        a.first = k == 0;
        a.last = k == p.launches - 1;
        TRY(norm_launch(p.norm[k], h->d, a, grid, st));
    }
    return TP_OK;
}

}  // namespace adam
}  // namespace tpmlp

static tp_status aw_ctl(const void *ctl) {
    if (!ctl || (reinterpret_cast<uintptr_t>(ctl) & 255u))
        return set_error(TP_ERR_ARG, "ctl is NULL or not 256-byte aligned");
    return TP_OK;
}

extern "C" {

tp_status tp_adamw_create(const tp_adamw_desc *desc, const tp_adamw_tensor *tensors, tp_adamw **out) {
    if (!out) return set_error(TP_ERR_ARG, "out is NULL");
    *out = nullptr;
    TRY(aw_validate(desc, tensors));
    tp_adamw *h = new (std::nothrow) tp_adamw;
    tp_adamw_tensor *t = new (std::nothrow) tp_adamw_tensor[desc->n_tensors];
    if (!h || !t) {
        delete h;
        delete[] t;
        return set_error(TP_ERR_ARG, "out of host memory");
    }
    h->d = *desc;
    h->t = t;
    for (int i = 0; i < desc->n_tensors; ++i) t[i] = tensors[i];
    if (!adam::make_plans(h)) {
        tp_adamw_destroy(h);
        return set_error(TP_ERR_ARG, "out of host memory");
    }
    *out = h;
    return TP_OK;
}

void tp_adamw_destroy(tp_adamw *h) {
    if (!h) return;
    delete[] h->few.step;
    delete[] h->few.norm;
    delete[] h->many.step;
    delete[] h->many.norm;
    delete[] h->t;
    delete h;
}

tp_status tp_adamw_set_grads(tp_adamw *h, const void *const *grads) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    if (!grads) return set_error(TP_ERR_ARG, "grads is NULL");
    for (int i = 0; i < h->d.n_tensors; ++i)
        if (h->t[i].n) TRY(aw_pointer(grads[i], "grad", i));
    for (int i = 0; i < h->d.n_tensors; ++i) h->t[i].grad = grads[i];
    adam::make_plans(h);  // in the memory it has
    return TP_OK;
}

tp_status tp_adamw_ctl_init(void *ctl, int steps_done, void *stream) {
    TRY(aw_ctl(ctl));
    if (steps_done < 0) return set_error(TP_ERR_ARG, "steps_done=%d is negative", steps_done);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    launch_begin("adamw_ctl_init", st);
    adam::ctl_init_kernel<<<1, 32, 0, st>>>(static_cast<adam::Ctl *>(ctl), steps_done);
    cudaError_t e = cudaGetLastError();
    launch_end("adamw_ctl_init", st);
    return cuda_check(e, "adamw_ctl_init");
}

tp_status tp_adamw_grad_norm(tp_adamw *h, float grad_scale, float max_norm, void *ctl, void *stream) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    TRY(aw_ctl(ctl));
    if (!(grad_scale > 0.0f) || !std::isfinite(grad_scale))
        return set_error(TP_ERR_ARG, "grad_scale must be positive and finite");
    if (!(max_norm > 0.0f)) return set_error(TP_ERR_ARG, "max_norm must be positive (infinity: no clipping)");
    adam::NormArgs a = {};
    a.ctl = static_cast<adam::Ctl *>(ctl);
    a.grad_scale = grad_scale;
    a.max_norm = max_norm;
    a.log_beta1 = static_cast<float>(std::log(h->d.beta1));  // -infinity for 0: 1 - b^t is 1
    a.log_beta2 = static_cast<float>(std::log(h->d.beta2));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return h->few.launches ? adam::norm_all(h->few, h, a, st) : adam::norm_all(h->many, h, a, st);
}

tp_status tp_adamw_step(tp_adamw *h, float lr, float grad_scale, int step, const void *ctl, void *stream) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    if (!std::isfinite(lr)) return set_error(TP_ERR_ARG, "lr must be finite");
    adam::Hyper hy = {};
    hy.lr = lr;
    hy.b1 = static_cast<float>(h->d.beta1);
    hy.b2 = static_cast<float>(h->d.beta2);
    hy.c1 = static_cast<float>(1.0 - h->d.beta1);
    hy.c2 = static_cast<float>(1.0 - h->d.beta2);
    hy.eps = h->d.eps;
    hy.seed = h->d.seed;
    if (ctl) {
        TRY(aw_ctl(ctl));
        hy.ctl = static_cast<const adam::Ctl *>(ctl);
    } else {
        if (step < 1) return set_error(TP_ERR_ARG, "step=%d: steps count from 1", step);
        if (!std::isfinite(grad_scale)) return set_error(TP_ERR_ARG, "grad_scale must be finite");
        hy.scale = grad_scale;
        hy.step = static_cast<uint32_t>(step);
        hy.inv_bc1 = static_cast<float>(1.0 / (1.0 - std::pow(h->d.beta1, step)));
        hy.inv_root_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(h->d.beta2, step)));
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return h->few.launches ? adam::step_all(h->few, h->d, hy, st) : adam::step_all(h->many, h->d, hy, st);
}

}  // extern "C"
