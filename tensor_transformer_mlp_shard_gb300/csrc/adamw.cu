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
constexpr int kNormBlocks = 608;
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

// Tensors of one launch, in the kernel's parameters: no copy to the device, no
// allocation, and a launch captured into a graph carries its own table.
template <int CAP>
struct Table {
    int count, base;    // tensors here, and the index of the first of them in the list
    int chunk0[CAP + 1];
    float lr_scale[CAP], decay[CAP];
    Entry t[CAP];
};

struct Hyper {
    float lr, b1, b2, c1, c2, eps, scale, inv_bc1, inv_root_bc2;  // c: 1 - b, rounded once
    uint32_t seed, step;
    const Ctl *ctl;
};

// tensor that holds chunk c: the last whose first chunk is at most c
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP> &tab, int c) {
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.chunk0[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// 4 elements from e, those past n read as zero
__device__ __forceinline__ void load4(const float *p, long long e, long long n, float *v) {
    if (e + 4 <= n) {
        const float4 w = *reinterpret_cast<const float4 *>(p + e);
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = e + j < n ? p[e + j] : 0.0f;
    }
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, long long e, long long n, float *v) {
    if (e + 4 <= n) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p + e);
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = e + j < n ? __bfloat162float(p[e + j]) : 0.0f;
    }
}
__device__ __forceinline__ void store4(float *p, long long e, long long n, const float *v) {
    if (e + 4 <= n) {
        *reinterpret_cast<float4 *>(p + e) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e + j < n) p[e + j] = v[j];
    }
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, long long e, long long n, const float *v) {
    if (e + 4 <= n) {
        *reinterpret_cast<uint2 *>(p + e) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e + j < n) p[e + j] = __float2bfloat16_rn(v[j]);
    }
}

// e4m3 codes, 4 in a word
__device__ __forceinline__ uint32_t load4_codes(const uint8_t *p, long long e, long long n) {
    if (e + 4 <= n) return *reinterpret_cast<const uint32_t *>(p + e);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (e + j < n) w |= static_cast<uint32_t>(p[e + j]) << (8 * j);
    return w;
}
__device__ __forceinline__ void store4_codes(uint8_t *p, long long e, long long n, uint32_t w) {
    if (e + 4 <= n) {
        *reinterpret_cast<uint32_t *>(p + e) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e + j < n) p[e + j] = static_cast<uint8_t>(w >> (8 * j));
    }
}
__device__ __forceinline__ void decode4(uint32_t w, float *v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t two;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<unsigned short>(w >> (16 * h))));
        const __half2 x = *reinterpret_cast<const __half2 *>(&two);
        v[2 * h] = __low2float(x);
        v[2 * h + 1] = __high2float(x);
    }
}
__device__ __forceinline__ uint32_t encode4(const float *v) {
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
    return lo | (static_cast<uint32_t>(hi) << 16);
}

// 32 bits to 32 well-spread bits: xor-shifts and odd multipliers
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * kMix1;
    x = (x ^ (x >> 15)) * kMix2;
    return x ^ (x >> 16);
}

// x >= 0, at most 448 but for rounding, to a neighbouring e4m3 value, the
// upper one with a probability of its nearness (16 random bits of it).  Below
// 2^-6 the steps stop shrinking (2^-9): adding 2^-6 puts x where its 3 leading
// mantissa bits are those steps.
__device__ __forceinline__ float round_e4m3(float x, uint32_t bits) {
    const float lift = x < 0.015625f ? 0.015625f : 0.0f;
    const uint32_t u = (__float_as_uint(x + lift) + (bits << 4)) & 0xFFF00000u;
    return fminf(__uint_as_float(u) - lift, 448.0f);
}

// Codes and scale of a block's values, 8 a lane: element j * 128 + 4 lane + i.
template <bool ROOT>
__device__ __forceinline__ void quantise(const float (&x)[2][4], const uint32_t (&bits)[2][4], uint32_t (&codes)[2],
                                         float &scale) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[j][i]) & 0x7FFFFFFFu);
    // as integers the order is that of the magnitudes, with NaN above all
    const float t = __uint_as_float(__reduce_max_sync(0xffffffffu, top));
    // below 2^-100 (where 448 / t nears the range of fp32) a block is zero
    const float inv = t < 7.888609e-31f ? 0.0f : __fmul_rn(__frcp_rn(t), 448.0f);
    scale = t < 7.888609e-31f ? 0.0f : __fmul_rn(t, 1.0f / 448.0f);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = fabsf(x[j][i]) * inv;
            q[i] = round_e4m3(a, ROOT ? bits[j][i] >> 16 : bits[j][i] & 0xFFFFu);
            if (a != a) q[i] = a;  // fminf would drop a NaN
            if (ROOT) {
                if (x[j][i] > 0.0f && inv > 0.0f) q[i] = fmaxf(q[i], 0.001953125f);
            } else {
                q[i] = copysignf(q[i], x[j][i]);
            }
        }
        codes[j] = encode4(q);
    }
}

// ---------------------------------------------------------------------------
// The step.  A warp takes 256 consecutive elements (a block of the 8-bit
// states), 8 a lane in two runs of 4.
// ---------------------------------------------------------------------------
template <int CAP, bool HALF, typename G, int BITS>
__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Table<CAP> tab,
                                                        const __grid_constant__ Hyper hy) {
    float scale = hy.scale, inv_bc1 = hy.inv_bc1, inv_root_bc2 = hy.inv_root_bc2;
    uint32_t step = hy.step;
    if (hy.ctl) {
        if (!hy.ctl->finite) return;
        scale = hy.ctl->scale;
        inv_bc1 = hy.ctl->inv_bc1;
        inv_root_bc2 = hy.ctl->inv_root_bc2;
        step = static_cast<uint32_t>(hy.ctl->steps);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t at_step = mix(hy.seed + kMix1 * step);
    for (int c = blockIdx.x; c < tab.chunk0[tab.count]; c += gridDim.x) {
        const int ti = tensor_of(tab, c);
        const Entry &t = tab.t[ti];
        const long long n = t.n;
        const long long blk = static_cast<long long>(c - tab.chunk0[ti]) * (kThreads / 32) + warp;
        if (blk * kBlock >= n) continue;
        const float lr = hy.lr * tab.lr_scale[ti];
        const float decay = lr * tab.decay[ti], rate = lr * inv_bc1;
        float w[2][4], g[2][4], m[2][4], v[2][4];
        uint32_t mc[2], vc[2];
        float ms = 0.0f, vs = 0.0f;
        if (BITS == 8) {
            ms = t.ms[blk];
            vs = t.vs[blk];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const long long e = blk * kBlock + j * 128 + lane * 4;
            load4(static_cast<const float *>(t.w), e, n, w[j]);
            load4(static_cast<const G *>(t.g), e, n, g[j]);
            if (BITS == 32) {
                load4(static_cast<const float *>(t.m), e, n, m[j]);
                load4(static_cast<const float *>(t.v), e, n, v[j]);
            } else {
                mc[j] = load4_codes(static_cast<const uint8_t *>(t.m), e, n);
                vc[j] = load4_codes(static_cast<const uint8_t *>(t.v), e, n);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const long long e = blk * kBlock + j * 128 + lane * 4;
            if (BITS == 8) {
                decode4(mc[j], m[j]);
                decode4(vc[j], v[j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (BITS == 8) {
                    m[j][i] *= ms;
                    v[j][i] *= vs;
                    v[j][i] *= v[j][i];
                }
                // the states are those of separately rounded products and sums: contracted
                // into fused operations, which of them is fused would be part of the result
                const float gi = __fmul_rn(g[j][i], scale);
                m[j][i] = __fadd_rn(__fmul_rn(hy.b1, m[j][i]), __fmul_rn(hy.c1, gi));
                v[j][i] = __fadd_rn(__fmul_rn(hy.b2, v[j][i]), __fmul_rn(__fmul_rn(hy.c2, gi), gi));
                const float root = sqrtf(v[j][i]);
                w[j][i] -= decay * w[j][i] + rate * m[j][i] / fmaf(root, inv_root_bc2, hy.eps);
                if (BITS == 8) v[j][i] = root;
            }
            store4(static_cast<float *>(t.w), e, n, w[j]);
            if (HALF) store4(static_cast<__nv_bfloat16 *>(t.p), e, n, w[j]);
            if (BITS == 32) {
                store4(static_cast<float *>(t.m), e, n, m[j]);
                store4(static_cast<float *>(t.v), e, n, v[j]);
            }
        }
        if (BITS == 8) {
            const uint32_t key = mix(mix(at_step ^ (static_cast<uint32_t>(tab.base + ti) * kMix2 + 1u)) +
                                     static_cast<uint32_t>(blk));
            uint32_t bits[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) bits[j][i] = mix(key ^ ((j * 128 + lane * 4 + i) * kMix1));
            quantise<false>(m, bits, mc, ms);
            quantise<true>(v, bits, vc, vs);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const long long e = blk * kBlock + j * 128 + lane * 4;
                store4_codes(static_cast<uint8_t *>(t.m), e, n, mc[j]);
                store4_codes(static_cast<uint8_t *>(t.v), e, n, vc[j]);
            }
            if (lane == 0) {
                t.ms[blk] = ms;
                t.vs[blk] = vs;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The gradient norm.  Every block leaves one sum of squares; the block that
// finishes last adds them in their order, so the result does not depend on
// which it is.  Within a thread the squares (rounded to fp32) are added with
// the error of every addition kept beside the sum (Knuth's two-sum), 6
// additions an element; fp64 additions, which this machine has few units for,
// come once a chunk.  The norm is then the rounded norm of the rounded
// squares, whatever the order, and the clip factor that scales every gradient
// does not move with the list's grouping.
// ---------------------------------------------------------------------------
struct NormArgs {
    Ctl *ctl;
    float grad_scale, max_norm;
    double beta1, beta2;
    int first, last;  // of the launches over one list
};

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

template <int CAP, typename G>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table<CAP> tab,
                                                        const __grid_constant__ NormArgs a) {
    __shared__ double red[kThreads / 32];
    __shared__ int is_last;
    double sum = 0.0;
    for (int c = blockIdx.x; c < tab.chunk0[tab.count]; c += gridDim.x) {
        const int ti = tensor_of(tab, c);
        const long long n = tab.t[ti].n;
        const long long e = static_cast<long long>(c - tab.chunk0[ti]) * kChunk + threadIdx.x * 4;
        float s = 0.0f, rest = 0.0f;
#pragma unroll
        for (int j = 0; j < kChunk / (4 * kThreads); ++j) {
            float g[4];
            load4(static_cast<const G *>(tab.t[ti].g), e + j * 4 * kThreads, n, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float q = __fmul_rn(g[i], g[i]);
                const float z = __fadd_rn(s, q), a = __fsub_rn(z, s);
                rest += __fadd_rn(__fsub_rn(s, __fsub_rn(z, a)), __fsub_rn(q, a));
                s = z;
            }
        }
        sum += static_cast<double>(s) + static_cast<double>(rest);
    }
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) {
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
    const bool finite = norm <= 3.402823466e38f;
    a.ctl->ticket = 0;
    a.ctl->norm = norm;
    a.ctl->finite = finite;
    a.ctl->scale = a.grad_scale * fminf(__frcp_rn(norm) * a.max_norm, 1.0f);
    if (finite) {
        const int t = ++a.ctl->steps;
        a.ctl->inv_bc1 = static_cast<float>(1.0 / (1.0 - pow(a.beta1, t)));
        a.ctl->inv_root_bc2 = static_cast<float>(1.0 / sqrt(1.0 - pow(a.beta2, t)));
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
    if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return set_error(TP_ERR_ARG, "eps must be positive and finite");
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

// tensors [i, i + tab.count) of the list; returns the index after the last
template <int CAP>
static int fill(const tp_adamw *h, int i, Table<CAP> &tab) {
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
        tab.chunk0[tab.count + 1] = tab.chunk0[tab.count] + static_cast<int>((s.n + kChunk - 1) / kChunk);
        ++tab.count;
    }
    return i;
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
    const int chunks = tab.chunk0[tab.count], most = 8 * num_sms();
    if (!chunks) return TP_OK;
    launch_begin("adamw_step", st);
    k<<<chunks < most ? chunks : most, kThreads, 0, st>>>(tab, hy);
    cudaError_t e = cudaGetLastError();
    launch_end("adamw_step", st);
    return cuda_check(e, "adamw_step");
}

template <int CAP>
static tp_status norm_launch(const Table<CAP> &tab, const tp_adamw_desc &d, const NormArgs &a, int grid,
                             cudaStream_t st) {
    launch_begin("adamw_grad_norm", st);
    if (d.grad_dtype == TP_DT_BF16)
        norm_kernel<CAP, __nv_bfloat16><<<grid, kThreads, 0, st>>>(tab, a);
    else
        norm_kernel<CAP, float><<<grid, kThreads, 0, st>>>(tab, a);
    cudaError_t e = cudaGetLastError();
    launch_end("adamw_grad_norm", st);
    return cuda_check(e, "adamw_grad_norm");
}

template <int CAP>
static tp_status step_all(const tp_adamw *h, const Hyper &hy, cudaStream_t st) {
    Table<CAP> tab;
    for (int i = 0; i < h->d.n_tensors;) {
        i = fill(h, i, tab);
        TRY(step_launch(tab, h->d, hy, st));
    }
    return TP_OK;
}

template <int CAP>
static tp_status norm_all(const tp_adamw *h, NormArgs a, cudaStream_t st) {
    Table<CAP> tab;
    long long chunks = 0;
    for (int i = 0; i < h->d.n_tensors; ++i) chunks += (h->t[i].n + kChunk - 1) / kChunk;
    int grid = kNormBlocks < 4 * num_sms() ? kNormBlocks : 4 * num_sms();
    if (chunks < grid) grid = chunks > 0 ? static_cast<int>(chunks) : 1;
    for (int i = 0; i < h->d.n_tensors;) {
        a.first = i == 0;
        i = fill(h, i, tab);
        a.last = i == h->d.n_tensors;
        TRY(norm_launch(tab, h->d, a, grid, st));
    }
    return TP_OK;
}

// The table's size is a launch's parameter bytes: a short list takes the small one.
constexpr int kSmall = 40, kLarge = 360;

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
    *out = h;
    return TP_OK;
}

void tp_adamw_destroy(tp_adamw *h) {
    if (!h) return;
    delete[] h->t;
    delete h;
}

tp_status tp_adamw_set_grads(tp_adamw *h, const void *const *grads) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    if (!grads) return set_error(TP_ERR_ARG, "grads is NULL");
    for (int i = 0; i < h->d.n_tensors; ++i)
        if (h->t[i].n) TRY(aw_pointer(grads[i], "grad", i));
    for (int i = 0; i < h->d.n_tensors; ++i) h->t[i].grad = grads[i];
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
    a.beta1 = h->d.beta1;
    a.beta2 = h->d.beta2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return h->d.n_tensors <= adam::kSmall ? adam::norm_all<adam::kSmall>(h, a, st) : adam::norm_all<adam::kLarge>(h, a, st);
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
    return h->d.n_tensors <= adam::kSmall ? adam::step_all<adam::kSmall>(h, hy, st) : adam::step_all<adam::kLarge>(h, hy, st);
}

}  // extern "C"
