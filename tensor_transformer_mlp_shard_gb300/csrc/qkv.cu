// Rotary positions of the QKV shards, in training (tp_rotary_*) and on the way
// into a paged key-value cache (tp_paged_append).
//
// One kernel serves both: it reads the QKV tensor once, 16 bytes a load, turns
// the pairs of the queries and keys in fp32 and writes them once, to where the
// mode says (the same columns; or the query tensor and the cache's slots).  It
// is bound by HBM.  A block takes a few tokens: their cosines and sines, which
// all heads share, are computed once, by one thread a pair, while the first
// loads are on their way, and kept in shared memory; a table in memory would
// cost as many bytes as a head.  An item is two chunks of a head: with pairs
// (i, i + dim/2) a chunk and its partner, else one from either half of what is
// left.  A thread has one item of every token, so that where it lies is worked
// out once for all of the block's tokens, and copies it to a ring of its own in
// shared memory, three tokens ahead: the bytes on their way do not cost
// registers, and no thread waits for another (but where an odd half puts the
// partners across the chunks of other threads).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <mutex>
#include <new>
#include <type_traits>

#include "attention.cuh"

#define TRY(x)                        \
    do {                              \
        tp_status _s = (x);           \
        if (_s != TP_OK) return _s;   \
    } while (0)

namespace tpmlp {
namespace attn {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;   // tokens of a block
constexpr int kFlight = 3;     // of them that a thread copies ahead

// the most that a block asks for: 8 tokens of 128 pairs, twice, the ring of 256 threads
static_assert(sizeof(float) * 4 * kMaxTokens * kMaxPairs + kFlight * 2 * 16 * kThreads < 48 * 1024 - 512, "a kernel's shared memory unasked");

enum Mode : int { ROTATE = 0, APPEND = 1, APPEND8 = 2 };

struct QkvPlan {
    const void *x[kMaxShards];
    void *y[kMaxShards];                      // ROTATE: like x; APPEND: Q
    void *k[kMaxShards], *v[kMaxShards];      // APPEND: the cache
    Pages at;                                 // ROTATE: positions (or null), n and no table
    const float *k_amax, *v_amax;             // APPEND8
    Divisor batch;                            // ROTATE: position of token m without positions: m / B
    int hq, hk, per, grouped, columns;        // columns: heads of a row, hq + 2 hk
    int D, half, interleaved;                 // half: pairs of a head
    int pair_items;                           // items of a head whose chunks are partners
    int rest_items;                           // the others
    int in_place;
    int side, passes;                         // tokens of a block: `side` at a time, `passes` times
    int rounds, round_threads;                // of so many items of side tokens
    int round_items;                          // side * T * slots * items
    Divisor by_items, by_slots, by_shards, by_group;
    int turn_pitch;                           // of the cosines of a token in shared memory
    float sign;                               // -1: the transposed rotation
    Turns turns;
};

template <typename E, int VE>
struct Chunk {  // VE elements as they are stored
    static constexpr int kBytes = VE * sizeof(E);
    using Word = typename std::conditional<kBytes == 16, uint4, typename std::conditional<kBytes == 8, uint2, uint32_t>::type>::type;
    Word w;
    __device__ __forceinline__ void store(E *p) const { *reinterpret_cast<Word *>(p) = w; }
    __device__ __forceinline__ void unpack(float (&f)[VE]) const {
        const E *e = reinterpret_cast<const E *>(&w);
#pragma unroll
        for (int i = 0; i < VE; ++i) f[i] = static_cast<float>(e[i]);
    }
    __device__ __forceinline__ void pack(const float (&f)[VE]) {
        E *e = reinterpret_cast<E *>(&w);
#pragma unroll
        for (int i = 0; i < VE; ++i) e[i] = static_cast<E>(f[i]);
    }
};

// fp32 to codes in one rounding
template <int VE>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&f)[VE], float scale) {
    alignas(8) uint8_t c[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) c[i] = __nv_cvt_float_to_fp8(f[i] * scale, __NV_SATFINITE, __NV_E4M3);
    if constexpr (VE == 8)
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(c);
    else if constexpr (VE == 4)
        *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(c);
    else
        *reinterpret_cast<uint16_t *>(p) = *reinterpret_cast<const uint16_t *>(c);
}

enum Kind : int { QUERY = 0, KEY = 1, VALUE = 2 };

template <int BYTES>
__device__ __forceinline__ void copy_chunk(uint32_t to, const void *from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}

// Where a thread's item is.
struct Item {
    int token;        // of the side's; -1: none
    int shard, kind, head, column, a, b;  // a, b: the chunks' first elements (b = -1: none)
    int n;            // of the head's items
};

template <int VE>
__device__ __forceinline__ Item item_at(const QkvPlan &p, int i) {
    Item it;
    if (i >= p.round_items) {
        it.token = -1;
        return it;
    }
    uint32_t item, slot, shard;
    const uint32_t rest = p.by_items.divmod(i, item), row = p.by_slots.divmod(rest, slot);
    it.token = p.by_shards.divmod(row, shard);
    it.shard = shard;
    if (p.grouped) {
        uint32_t r;
        const int j = p.by_group.divmod(slot, r);  // a group: its queries, the key and, out of place, the value
        it.column = j * (p.per + 2) + r;
        it.kind = static_cast<int>(r) < p.per ? QUERY : static_cast<int>(r) == p.per ? KEY : VALUE;
        it.head = it.kind == QUERY ? j * p.per + r : j;
    } else {
        it.column = slot;
        const int s = slot;
        it.kind = s < p.hq ? QUERY : s < p.hq + p.hk ? KEY : VALUE;
        it.head = it.kind == QUERY ? s : it.kind == KEY ? s - p.hq : s - p.hq - p.hk;
    }
    const int n = it.n = item;
    if (n < p.pair_items) {
        it.a = n * VE;
        it.b = it.a + p.half;
    } else {
        // two halves of what is left, so that neighbouring threads read neighbouring chunks
        it.a = (p.pair_items + n) * VE;
        it.b = it.a + p.rest_items * VE;
        if (it.b >= (p.in_place ? 2 * p.half : p.D)) it.b = -1;
    }
    return it;
}

// N cosines or sines from shared memory
template <int N>
__device__ __forceinline__ void read_turns(float *to, const float *from) {
    if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(from);
        to[0] = v.x; to[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(from + i);
            to[i] = v.x; to[i + 1] = v.y; to[i + 2] = v.z; to[i + 3] = v.w;
        }
    }
}

// products and sums rounded one by one, as the definition in fp32 has them
__device__ __forceinline__ void turn_pair(float x, float y, float c, float s, float &to_x, float &to_y) {
    to_x = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    to_y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// the pairs (first + 2i, first + 2i + 1) of a chunk, those that turn
template <int VE>
__device__ __forceinline__ void turn_neighbours(float (&f)[VE], int first, int half, const float *cs, const float *sn) {
    if (first / 2 >= half) return;
    float c[VE / 2], s[VE / 2];
    read_turns<VE / 2>(c, cs + first / 2);
    read_turns<VE / 2>(s, sn + first / 2);
#pragma unroll
    for (int e = 0; e < VE; e += 2)
        if ((first + e) / 2 < half) {
            const float x = f[e], y = f[e + 1];
            turn_pair(x, y, c[e / 2], s[e / 2], f[e], f[e + 1]);
        }
}

// The 16 bytes of a head from element j0 on, wherever they begin, from the chunks
// of its items: `head` is the first item's place among a stage's chunks, of which
// the second halves lie `half_at` further.  What lies outside the chunks that
// turn is any of them.
template <typename E, int VE>
__device__ __forceinline__ void window(uint32_t (&to)[4], int j0, const QkvPlan &p, const uint4 *head, int half_at) {
    const int last = (2 * p.half - 1) / VE, c = j0 >= 0 ? j0 / VE : -1, by = j0 & (VE - 1);
    auto chunk = [&](int i) {
        i = min(max(i, 0), last);
        return i < p.rest_items ? head[i] : head[half_at + i - p.rest_items];
    };
    const uint4 x = chunk(c), y = chunk(c + 1);
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    constexpr int kWord = 4 / sizeof(E);  // elements of a word
    static_assert(VE == 4 * kWord, "chunks of 16 bytes");
    if (by & (2 * kWord)) {
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
    }
    if (by & kWord) {
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
    }
    if constexpr (kWord == 2) {
        if (by & 1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) to[k] = w[k];
}

// The elements of a chunk that turn, with partners from other chunks; cs and sn are
// by element, the sines with their signs.
template <typename E, int VE>
__device__ __forceinline__ void turn_apart(Chunk<E, VE> &chunk, float (&f)[VE], int first, const QkvPlan &p, const uint4 *head, int half_at,
                                           const float *cs, const float *sn) {
    if (first >= 2 * p.half) return;
    alignas(16) uint32_t partner[4];
    window<E, VE>(partner, first < p.half ? first + p.half : first - p.half, p, head, half_at);
    const E *x = reinterpret_cast<const E *>(partner);
    float g[VE], c[VE], s[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) g[e] = static_cast<float>(x[e]);
    if (first < p.half && first + VE > p.half) {  // both halves' elements: the later ones' partners are elsewhere
        window<E, VE>(partner, first - p.half, p, head, half_at);
#pragma unroll
        for (int e = 0; e < VE; ++e)
            if (first + e >= p.half) g[e] = static_cast<float>(x[e]);
    }
    read_turns<VE>(c, cs + first);
    read_turns<VE>(s, sn + first);
    E *own = reinterpret_cast<E *>(&chunk.w);
#pragma unroll
    for (int e = 0; e < VE; ++e)
        if (first + e < 2 * p.half) {
            f[e] = __fadd_rn(__fmul_rn(f[e], c[e]), __fmul_rn(g[e], s[e]));
            own[e] = static_cast<E>(f[e]);
        }
}

// APART: pairs (i, i + half) of an odd half, whose partners lie across the chunks:
// the block meets once a token, when all of its chunks are there.
template <typename E, int VE, int MODE, bool APART>
__global__ void __launch_bounds__(kThreads) qkv_kernel(const __grid_constant__ QkvPlan p) {
    constexpr int kBytes = Chunk<E, VE>::kBytes;
    using Word = typename Chunk<E, VE>::Word;
    // [tokens][pairs] cosines (APART: [elements]), as many sines, then [kFlight][2][threads] chunks
    extern __shared__ __align__(16) char smem[];
    __shared__ long long slot_of[kMaxTokens];  // APPEND: the slot's row of the cache, of key head 0
    __shared__ int active[kMaxTokens];
    const int tokens = p.side * p.passes, token0 = blockIdx.x * tokens, pitch = p.turn_pitch;
    float *cs = reinterpret_cast<float *>(smem), *sn = cs + tokens * pitch;
    Word *ring = reinterpret_cast<Word *>(sn + tokens * pitch) + threadIdx.x;
    const uint32_t ring_to = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const long long width = static_cast<long long>(p.columns) * p.D;
    bool turned = false;
    wait_for_stream();
    for (int round = blockIdx.y; round < p.rounds; round += gridDim.y) {
        const Item it = item_at<VE>(p, static_cast<int>(threadIdx.x) < p.round_threads ? round * p.round_threads + static_cast<int>(threadIdx.x) : p.round_items);
        const bool two = it.b >= 0;
        const E *x = nullptr;
        E *y = nullptr;  // ROTATE, queries
        void *cache = nullptr;
        long long y_step = 0;
        float scale = 1.0f;
        int count = 0;   // of the thread's tokens
        if (it.token >= 0) {
            const int m = token0 + it.token;
            count = m < p.at.n ? min(p.passes, (p.at.n - m + p.side - 1) / p.side) : 0;
            x = static_cast<const E *>(p.x[it.shard]) + it.column * p.D + m * width;
            if (MODE == ROTATE) {
                y = static_cast<E *>(p.y[it.shard]) + it.column * p.D;
                y_step = width;
            } else if (it.kind == QUERY) {
                y = static_cast<E *>(p.y[it.shard]) + it.head * p.D;
                y_step = static_cast<long long>(p.hq) * p.D;
            } else {
                cache = it.kind == KEY ? p.k[it.shard] : p.v[it.shard];
                if (MODE == APPEND8) scale = cache_scale(it.kind == KEY ? p.k_amax : p.v_amax, it.shard * p.hk + it.head);
            }
            if (y) y += m * y_step;
            y_step *= p.side;
        }
        const long long x_step = width * p.side;
        // the thread's chunks of its pass-th token to slot `to` of its ring
        auto copy = [&](int pass, int to) {
            if (pass < count) {
                const E *from = x + pass * x_step;
                const uint32_t at = ring_to + to * (2 * kBytes) * blockDim.x;
                copy_chunk<kBytes>(at, from + it.a);
                if (two) copy_chunk<kBytes>(at + kBytes * blockDim.x, from + it.b);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < (APART ? kFlight - 1 : kFlight); ++i) copy(i, i);
        if (!turned) {
            auto position = [&](int m) {
                return MODE == ROTATE && !p.at.positions ? static_cast<int>(p.batch.div(m)) : p.at.positions[m];
            };
            if (threadIdx.x < tokens && token0 + static_cast<int>(threadIdx.x) < p.at.n) {
                const int m = token0 + threadIdx.x, pos = position(m);
                int ok = pos >= 0;
                if (MODE != ROTATE && ok) {
                    const int seq = p.at.sequences ? p.at.sequences[m] : m;
                    uint32_t off;
                    const int col = p.at.page.divmod(pos, off);
                    ok = static_cast<unsigned>(seq) < static_cast<unsigned>(p.at.table_rows) && col < p.at.table_cols;
                    const int page = ok ? p.at.table[static_cast<long long>(seq) * p.at.table_cols + col] : -1;
                    ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.at.pages);
                    if (!ok && blockIdx.y == 0) bad_index(p.at);
                    // the heads of a page lie page_size rows apart
                    slot_of[threadIdx.x] = static_cast<long long>(page) * p.hk * p.at.page_size + off;
                }
                active[threadIdx.x] = ok;
            }
            // a thread keeps to one pair, whose turn a position is read once: the lanes' different ones come
            // one after another
            const int groups = max(1, static_cast<int>(blockDim.x) / max(1, p.half));
            for (int k = threadIdx.x; k < groups * p.half; k += blockDim.x) {
                const int pair = k % p.half;
                const uint64_t per_position = p.turns.per_position[pair];
                for (int t = k / p.half; t < tokens && token0 + t < p.at.n; t += groups) {
                    const float2 r = turn(p.turns, per_position, position(token0 + t));
                    const float s = r.y * p.sign;
                    cs[t * pitch + pair] = r.x;
                    sn[t * pitch + pair] = APART ? -s : s;
                    if (APART) {
                        cs[t * pitch + p.half + pair] = r.x;
                        sn[t * pitch + p.half + pair] = s;
                    }
                }
            }
            turned = true;
            __syncthreads();
        }
        int slot = 0;
        for (int pass = 0; pass < (APART ? p.passes : count); ++pass) {
            if constexpr (APART) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kFlight - 2) : "memory");
                __syncthreads();  // and the token before has been read
                copy(pass + kFlight - 1, slot == 0 ? kFlight - 1 : slot - 1);
            } else {
                asm volatile("cp.async.wait_group %0;" ::"n"(kFlight - 1) : "memory");
            }
            const bool here = !APART || pass < count;
            const Word *stage = ring + slot * 2 * blockDim.x;
            Chunk<E, VE> a, b;
            a.w = stage[0];
            if (two) b.w = stage[blockDim.x];
            const int t = pass * p.side + it.token;
            const bool on = here && active[t];
            if (on || (MODE == ROTATE && !p.in_place && here)) {  // otherwise padding stays as it was
                float fa[VE], fb[VE];
                a.unpack(fa);
                if (two) b.unpack(fb);
                if (it.kind != VALUE && on) {
                    const float *c_of = cs + t * pitch, *s_of = sn + t * pitch;
                    if constexpr (APART) {
                        const uint4 *head = stage - it.n;
                        turn_apart<E, VE>(a, fa, it.a, p, head, blockDim.x, c_of, s_of);
                        if (two) turn_apart<E, VE>(b, fb, it.b, p, head, blockDim.x, c_of, s_of);
                    } else if (p.interleaved) {
                        if constexpr (VE >= 4) {  // whole 16 bytes
                            turn_neighbours<VE>(fa, it.a, p.half, c_of, s_of);
                            a.pack(fa);
                            if (two) {
                                turn_neighbours<VE>(fb, it.b, p.half, c_of, s_of);
                                b.pack(fb);
                            }
                        }
                    } else if (it.a < p.half) {
                        float c[VE], s[VE];
                        read_turns<VE>(c, c_of + it.a);
                        read_turns<VE>(s, s_of + it.a);
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            const float f = fa[e], g = fb[e];
                            turn_pair(f, g, c[e], s[e], fa[e], fb[e]);
                        }
                        a.pack(fa);
                        b.pack(fb);
                    }
                }
                if (MODE == ROTATE || it.kind == QUERY) {
                    E *to = y + pass * y_step;
                    a.store(to + it.a);
                    if (two) b.store(to + it.b);
                } else {
                    const long long row = (slot_of[t] + static_cast<long long>(it.head) * p.at.page_size) * p.D;
                    if (MODE == APPEND) {
                        E *to = static_cast<E *>(cache) + row;
                        a.store(to + it.a);
                        if (two) b.store(to + it.b);
                    } else if constexpr (MODE == APPEND8) {
                        uint8_t *to = static_cast<uint8_t *>(cache) + row;
                        store_codes<VE>(to + it.a, fa, scale);
                        if (two) store_codes<VE>(to + it.b, fb, scale);
                    }
                }
            }
            if constexpr (!APART) copy(pass + kFlight, slot);
            slot = slot + 1 == kFlight ? 0 : slot + 1;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if constexpr (APART) __syncthreads();  // the next round's copies take the stages
    }
    // not earlier: blocks of this kernel between those of the next one leave an SM's
    // registers in pieces, and the next kernel's last block without a place
    let_next_start();
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
tp_status rope_validate(const tp_rope_desc *r, int head_dim) {
    if (r->dim < 0 || r->dim > head_dim || r->dim % 2)
        return set_error(TP_ERR_ARG, "rope.dim=%d is not an even number up to head_dim=%d", r->dim, head_dim);
    if (r->pairs != TP_ROPE_HALVES && r->pairs != TP_ROPE_INTERLEAVED) return set_error(TP_ERR_ARG, "bad rope.pairs %d", r->pairs);
    if (r->scaling < TP_ROPE_NONE || r->scaling > TP_ROPE_PARTS) return set_error(TP_ERR_ARG, "bad rope.scaling %d", r->scaling);
    if (!(r->base >= 1.0) || !std::isfinite(r->base)) return set_error(TP_ERR_ARG, "rope.base must be finite and at least 1");
    if (!(r->factor >= 1.0) || !std::isfinite(r->factor)) return set_error(TP_ERR_ARG, "rope.factor must be finite and at least 1");
    if (r->scaling == TP_ROPE_NONE && r->factor != 1.0) return set_error(TP_ERR_ARG, "rope.factor belongs to a scaling");
    if (!(r->attention_factor >= 0.0) || r->attention_factor > 1e6)
        return set_error(TP_ERR_ARG, "rope.attention_factor must be 0 (the default) or positive, up to 1e6");
    if (r->scaling == TP_ROPE_PARTS) {
        if (!(r->original > 0.0) || !std::isfinite(r->original)) return set_error(TP_ERR_ARG, "rope.original must be positive and finite");
        if (!(r->slow >= 0.0) || !(r->fast > r->slow) || !std::isfinite(r->fast))
            return set_error(TP_ERR_ARG, "rope.fast must be finite and above rope.slow >= 0");
    }
    return TP_OK;
}

// A number as the sum of two doubles, to about 2^-100: a position multiplies what
// 53 bits of a frequency lose by up to 2^31.  Sums after Knuth, products after Dekker
// with the machine's fma; every product goes through fma, so that no compiler
// takes it into a sum of its own.
struct Pair {
    double hi, lo;
};
static Pair pair_sum(double a, double b) {
    const double s = a + b, x = s - a;
    return {s, (a - (s - x)) + (b - x)};
}
static Pair operator*(Pair a, Pair b) {
    const double p = std::fma(a.hi, b.hi, 0.0), rest = std::fma(a.hi, b.hi, -p);
    return pair_sum(p, std::fma(a.hi, b.lo, std::fma(a.lo, b.hi, rest)));
}
static Pair operator+(Pair a, Pair b) {
    const Pair s = pair_sum(a.hi, b.hi);
    return pair_sum(s.hi, s.lo + (a.lo + b.lo));
}
static Pair inverse(Pair a) {
    const double x = 1.0 / a.hi;
    const Pair off = Pair{1.0, 0.0} + a * Pair{-x, 0.0};  // 1 - a x
    return pair_sum(x, std::fma(x, off.hi, 0.0));
}
static Pair power(Pair a, int n) {
    Pair y = {1.0, 0.0};
    for (; n > 0; n >>= 1, a = a * a)
        if (n & 1) y = y * a;
    return y;
}
// a^(-1/n): a double's root and one step of Newton's method, which squares its error
static Pair inverse_root(double a, int n) {
    const Pair x = {std::pow(a, -1.0 / n), 0.0};
    const Pair off = Pair{1.0, 0.0} + power(x, n) * Pair{-a, 0.0};  // 1 - a x^n
    return pair_sum(x.hi, std::fma(x.hi, off.hi / n, 0.0));
}

void rope_turns(const tp_rope_desc &r, Turns *t) {
    const Pair turn = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / 2 pi
    const int half = r.dim / 2;
    const Pair slower = inverse({r.factor, 0.0});
    // of neighbouring pairs; with NTK base^(-1/half) s^(-1/(half - 1))
    Pair ratio = {1.0, 0.0};
    if (half > 0) ratio = inverse_root(r.base, half);
    if (r.scaling == TP_ROPE_NTK && half > 1) ratio = ratio * inverse_root(r.factor, half - 1);
    for (int i = 0; i < half; ++i) {
        Pair f = power(ratio, i);
        if (r.scaling == TP_ROPE_LINEAR) f = f * slower;
        if (r.scaling == TP_ROPE_PARTS) {
            // k f + (1 - k) f / s
            Pair keep = {(r.original * (f.hi * turn.hi) - r.slow) / (r.fast - r.slow), 0.0};
            if (keep.hi > -1.0 && keep.hi < 2.0)
                keep = (f * turn * Pair{r.original, 0.0} + Pair{-r.slow, 0.0}) * inverse(pair_sum(r.fast, -r.slow));
            if (!(keep.hi > 0.0)) keep = {0.0, 0.0};
            if (keep.hi >= 1.0) keep = {1.0, 0.0};
            f = f * (keep + (Pair{1.0, 0.0} + keep * Pair{-1.0, 0.0}) * slower);
        }
        // to the nearest 2^-64 of a turn
        const Pair turns = f * turn;
        const double whole = std::floor(turns.hi * 0x1p64);
        t->per_position[i] = static_cast<uint64_t>(whole) + static_cast<uint64_t>(std::llrint((turns.hi * 0x1p64 - whole) + turns.lo * 0x1p64));
    }
    for (int i = half; i < kMaxPairs; ++i) t->per_position[i] = 0;
    double a = r.attention_factor;
    if (a == 0.0) a = r.scaling == TP_ROPE_PARTS ? 0.1 * std::log(r.factor) + 1.0 : 1.0;
    t->a = static_cast<float>(a);
    t->a_rest = static_cast<float>(a - t->a);
}

template <typename E, int MODE>
static auto kernel_of(int ve, bool apart) -> void (*)(QkvPlan) {
    constexpr int kMost = 16 / sizeof(E);
    if (apart) return qkv_kernel<E, kMost, MODE, true>;
    if constexpr (kMost == 8)
        if (ve == 8) return qkv_kernel<E, 8, MODE, false>;
    return ve == 4 ? qkv_kernel<E, 4, MODE, false> : qkv_kernel<E, 2, MODE, false>;
}

// Fills in what follows from the sizes and launches.  `T` shards, `in_place`:
// only what is rotated is touched.
static tp_status launch_qkv(QkvPlan &p, int T, int elem, int mode, const char *name, cudaStream_t st) {
    // 16 bytes a chunk; with pairs (i, i + half) both chunks have to begin on one: half
    // as many elements until the half holds a whole number of them, of an even half.
    // An odd one would leave single elements, and goes by whole chunks with the
    // partners across them (APART: bf16, 5160 tokens of 112 heads, 57 pairs 113 us,
    // by elements 205; a half of 28 131 us by chunks of 4, 149 across).
    const bool apart = !p.interleaved && p.half % 2;
    int ve = 16 / elem;
    if (!p.interleaved && !apart)
        while (p.half % ve) ve /= 2;
    if (p.interleaved && p.half == 0) p.interleaved = 0;
    const int chunks = p.D / ve, partners = p.interleaved || apart ? 0 : p.half / ve;
    p.pair_items = partners;
    const int rotated = p.interleaved || apart ? ((2 * p.half + ve - 1) / ve + 1) / 2 : partners;
    const int items = p.in_place ? rotated : partners + (chunks - 2 * partners + 1) / 2;
    p.rest_items = items - partners;
    const int group = p.per + (p.in_place ? 1 : 2);
    const int slots = p.grouped ? p.hk * group : p.hq + p.hk * (p.in_place ? 1 : 2);
    if (items == 0) return TP_OK;  // nothing turns, in place
    const int per_token = T * slots * items;
    // narrow tensors: several tokens side by side
    p.side = 1;
    while (p.side < 4 && 2 * p.side * per_token <= kThreads) p.side *= 2;
    p.round_items = p.side * per_token;
    // rounds of equally many items: of whole warps, or of whole heads where the items
    // of a head need each other's chunks
    const int unit = apart ? items : 32, most_items = kThreads / unit * unit;
    p.rounds = (p.round_items + most_items - 1) / most_items;
    p.round_threads = ((p.round_items + p.rounds - 1) / p.rounds + unit - 1) / unit * unit;
    const int threads = (p.round_threads + 31) / 32 * 32;
    p.by_items = Divisor(items);
    p.by_slots = Divisor(slots);
    p.by_shards = Divisor(T);
    p.by_group = Divisor(group);
    void (*k)(QkvPlan) = nullptr;
    if (elem == 4)
        k = mode == ROTATE ? kernel_of<float, ROTATE>(ve, apart) : kernel_of<float, APPEND>(ve, apart);
    else
        k = mode == ROTATE   ? kernel_of<__nv_bfloat16, ROTATE>(ve, apart)
            : mode == APPEND ? kernel_of<__nv_bfloat16, APPEND>(ve, apart)
                             : kernel_of<__nv_bfloat16, APPEND8>(ve, apart);
    // Tokens after one another, where there are enough blocks all the same: 4, and 8
    // with the lookups in the table before them (32768 tokens backward 118 us with 4,
    // 121 with 8; 8092 into the cache 38 us with 8, 40 with 4).
    const int most = mode == ROTATE ? 4 : 8;
    p.passes = 1;
    while (2 * p.passes * p.side <= most && p.at.n / (2 * p.passes * p.side) >= 4 * num_sms()) p.passes *= 2;
    p.turn_pitch = p.half > 0 ? ((apart ? 2 * p.half : p.half) + 7) / 8 * 8 : 8;
    const int ring = kFlight * 2 * ve * elem * threads, turns = sizeof(float) * 2 * p.side * p.turn_pitch;
    const int blocks = (p.at.n + p.side * p.passes - 1) / (p.side * p.passes);
    // few tokens: the rounds on blocks of their own
    const int across = std::min(p.rounds, std::max(1, 8 * num_sms() / blocks));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, across);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = ring + p.passes * turns;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_on() ? 1 : 0;
    launch_begin(name, st);
    cudaError_t e = cudaLaunchKernelEx(&cfg, k, p);
    launch_end(name, st);
    return cuda_check(e, name);
}

}  // namespace attn
}  // namespace tpmlp

using namespace tpmlp;
using attn::kMaxRows;

struct tp_rotary {
    tp_rotary_desc d;
    int M;
    attn::Turns turns;
};

struct tp_paged {
    tp_paged_desc d;
    int word;        // of g_tp_index
    unsigned owner;  // what is written there
    float scale;
    attn::Turns turns;
};

static tp_status at_pointer(const void *p, const char *name, int i, int n, unsigned align) {
    if (p && !(reinterpret_cast<uintptr_t>(p) & (align - 1))) return TP_OK;
    char at[16] = "";
    if (n > 1) snprintf(at, sizeof(at), "[%d]", i);
    if (!p) return set_error(TP_ERR_ARG, "%s%s is NULL", name, at);
    return set_error(TP_ERR_ARG, "%s%s is not %u-byte aligned", name, at, align);
}

// copies an array of n pointers into a plan after checking them
template <typename P>
static tp_status at_array(P *const *in, int n, const char *name, P **out) {
    if (!in) return set_error(TP_ERR_ARG, "%s: pointer array is NULL", name);
    for (int i = 0; i < n; ++i) {
        TRY(at_pointer(in[i], name, i, n, 16));
        out[i] = in[i];
    }
    return TP_OK;
}

static tp_status at_heads(int T, int heads, int kv_heads, int head_dim, int grouped) {
    if (grouped != 0 && grouped != 1) return set_error(TP_ERR_ARG, "grouped must be 0 or 1");
    if (T < 1 || T > TP_MAX_SHARDS) return set_error(TP_ERR_SHAPE, "T=%d outside 1..%d", T, TP_MAX_SHARDS);
    if (kv_heads < 1 || kv_heads % T) return set_error(TP_ERR_SHAPE, "kv_heads=%d must be a positive multiple of T=%d", kv_heads, T);
    if (heads < 1 || heads > 4096 || heads % kv_heads)
        return set_error(TP_ERR_SHAPE, "heads=%d must be a multiple of kv_heads=%d, up to 4096", heads, kv_heads);
    if (head_dim < 8 || head_dim % 8) return set_error(TP_ERR_SHAPE, "head_dim=%d must be a positive multiple of 8", head_dim);
    if (head_dim > attn::kMaxHeadDim)
        return set_error(TP_ERR_UNSUPPORTED, "head_dim=%d above the kernels' %d", head_dim, attn::kMaxHeadDim);
    return TP_OK;
}

static tp_status rotate(tp_rotary *h, const void *const *in, const char *in_name, const int32_t *positions,
                        void *const *out, const char *out_name, bool back, void *stream) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    const tp_rotary_desc &d = h->d;
    if (h->M == 0) return TP_OK;
    attn::QkvPlan p = {};
    TRY(at_array(in, d.T, in_name, p.x));
    TRY(at_array(out, d.T, out_name, p.y));
    int same = 0;
    for (int i = 0; i < d.T; ++i) same += p.x[i] == p.y[i];
    if (same != 0 && same != d.T)
        return set_error(TP_ERR_ARG, "%s and %s: either every shard in place or none", in_name, out_name);
    if (positions) TRY(at_pointer(positions, "positions", 0, 1, 4));
    p.at.positions = positions;
    p.at.n = h->M;
    p.batch = attn::Divisor(d.B);
    p.hq = d.heads / d.T;
    p.hk = d.kv_heads / d.T;
    p.per = d.heads / d.kv_heads;
    p.grouped = d.grouped;
    p.columns = p.hq + 2 * p.hk;
    p.D = d.head_dim;
    p.half = d.rope.dim / 2;
    p.interleaved = d.rope.pairs == TP_ROPE_INTERLEAVED;
    p.in_place = same != 0;
    p.sign = back ? -1.0f : 1.0f;
    p.turns = h->turns;
    return attn::launch_qkv(p, d.T, d.dtype == TP_DT_F32 ? 4 : 2, attn::ROTATE, back ? "rotary_bwd" : "rotary_fwd",
                            static_cast<cudaStream_t>(stream));
}

static tp_status at_rows(const tp_paged_desc &d, const int32_t *positions, const int32_t *sequences, int n,
                         const int32_t *table, int table_rows, int table_cols, const float *k_amax, const float *v_amax,
                         attn::Pages &at) {
    if (n > kMaxRows) return set_error(TP_ERR_SHAPE, "n=%d above %d rows", n, kMaxRows);
    if (table_rows < 1 || table_rows > kMaxRows || table_cols < 1 || table_cols > kMaxRows)
        return set_error(TP_ERR_SHAPE, "table of %d x %d outside 1..%d", table_rows, table_cols, kMaxRows);
    TRY(at_pointer(positions, "positions", 0, 1, 4));
    if (sequences)
        TRY(at_pointer(sequences, "sequences", 0, 1, 4));
    else if (n > table_rows)
        return set_error(TP_ERR_SHAPE, "n=%d rows without sequences, but a table of %d", n, table_rows);
    TRY(at_pointer(table, "table", 0, 1, 4));
    if (d.dtype == TP_DT_FP8) {
        TRY(at_pointer(k_amax, "k_amax", 0, 1, 4));
        TRY(at_pointer(v_amax, "v_amax", 0, 1, 4));
    }
    at.positions = positions;
    at.sequences = sequences;
    at.table = table;
    at.n = n;
    at.table_rows = table_rows;
    at.table_cols = table_cols;
    at.pages = d.pages;
    at.page_size = d.page_size;
    at.page = attn::Divisor(d.page_size);
    return TP_OK;
}

// Index words: a kernel that meets an index out of range writes its handle's
// number, which no other handle of the process has, so that what a handle
// before left in the word says nothing.
constexpr int kIndexWords = 1024;
__device__ unsigned g_tp_index[kIndexWords];
static std::mutex g_index_mu;
static bool g_index_used[kIndexWords];
static unsigned g_index_owners = 0;

static tp_status index_word(int word, unsigned **at) {
    static unsigned *base[64] = {};
    int dev = 0;
    TRY(cuda_check(cudaGetDevice(&dev), "cudaGetDevice"));
    if (dev < 0 || dev >= 64) return set_error(TP_ERR_UNSUPPORTED, "device ordinal %d above 63", dev);
    std::lock_guard<std::mutex> lock(g_index_mu);
    if (!base[dev]) {
        void *p = nullptr;
        TRY(cuda_check(cudaGetSymbolAddress(&p, g_tp_index), "cudaGetSymbolAddress(index)"));
        base[dev] = static_cast<unsigned *>(p);
    }
    *at = base[dev] + word;
    return TP_OK;
}

extern "C" {

tp_status tp_rotary_create(const tp_rotary_desc *desc, tp_rotary **out) {
    if (!out) return set_error(TP_ERR_ARG, "out is NULL");
    *out = nullptr;
    if (!desc) return set_error(TP_ERR_ARG, "descriptor is NULL");
    if (desc->dtype != TP_DT_F32 && desc->dtype != TP_DT_BF16)
        return set_error(TP_ERR_ARG, "bad dtype %d (the rotation takes TP_DT_F32 and TP_DT_BF16)", desc->dtype);
    TRY(at_heads(desc->T, desc->heads, desc->kv_heads, desc->head_dim, desc->grouped));
    TRY(attn::rope_validate(&desc->rope, desc->head_dim));
    if (desc->S < 0 || desc->B < 0) return set_error(TP_ERR_SHAPE, "negative S or B");
    const long long M = static_cast<long long>(desc->S) * desc->B;
    if (M > (1ll << 24)) return set_error(TP_ERR_SHAPE, "M = S*B = %lld exceeds 2^24 tokens", M);
    tp_rotary *h = new (std::nothrow) tp_rotary;
    if (!h) return set_error(TP_ERR_ARG, "out of host memory");
    h->d = *desc;
    h->M = static_cast<int>(M);
    attn::rope_turns(desc->rope, &h->turns);
    *out = h;
    return TP_OK;
}

void tp_rotary_destroy(tp_rotary *h) { delete h; }

tp_status tp_rotary_fwd(tp_rotary *h, const void *const *X, const int32_t *positions, void *const *Y, void *stream) {
    return rotate(h, X, "X", positions, Y, "Y", false, stream);
}

tp_status tp_rotary_bwd(tp_rotary *h, const void *const *dY, const int32_t *positions, void *const *dX, void *stream) {
    return rotate(h, dY, "dY", positions, dX, "dX", true, stream);
}

tp_status tp_paged_create(const tp_paged_desc *desc, tp_paged **out) {
    if (!out) return set_error(TP_ERR_ARG, "out is NULL");
    *out = nullptr;
    if (!desc) return set_error(TP_ERR_ARG, "descriptor is NULL");
    if (desc->dtype != TP_DT_F32 && desc->dtype != TP_DT_BF16 && desc->dtype != TP_DT_FP8)
        return set_error(TP_ERR_ARG, "bad dtype %d", desc->dtype);
    TRY(at_heads(desc->T, desc->heads, desc->kv_heads, desc->head_dim, desc->grouped));
    if (desc->dtype == TP_DT_FP8 && desc->head_dim % 16)
        return set_error(TP_ERR_SHAPE, "head_dim=%d must be a multiple of 16 with TP_DT_FP8", desc->head_dim);
    TRY(attn::rope_validate(&desc->rope, desc->head_dim));
    if (desc->page_size < 16 || desc->page_size % 16 || desc->page_size > kMaxRows)
        return set_error(TP_ERR_SHAPE, "page_size=%d must be a multiple of 16 in 16..%d", desc->page_size, kMaxRows);
    if (desc->pages < 1) return set_error(TP_ERR_SHAPE, "pages=%d must be positive", desc->pages);
    if (static_cast<long long>(desc->pages) * (desc->kv_heads / desc->T) * (desc->page_size / 8) >= 0xffffffffll)
        return set_error(TP_ERR_SHAPE, "pages=%d of %d positions and %d key heads: 2^35 rows of a cache or more", desc->pages,
                         desc->page_size, desc->kv_heads / desc->T);
    if (desc->window < 0) return set_error(TP_ERR_ARG, "window=%d is negative", desc->window);
    // the scores are taken to base 2
    if (!std::isfinite(static_cast<float>(static_cast<double>(desc->scale) * 1.4426950408889634)))
        return set_error(TP_ERR_ARG, "scale must be finite, and below 2^128 / log2(e)");
    tp_paged *h = new (std::nothrow) tp_paged;
    if (!h) return set_error(TP_ERR_ARG, "out of host memory");
    h->d = *desc;
    h->scale = desc->scale != 0.0f ? desc->scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(desc->head_dim)));
    attn::rope_turns(desc->rope, &h->turns);
    {
        std::lock_guard<std::mutex> lock(g_index_mu);
        h->word = 0;
        while (h->word < kIndexWords && g_index_used[h->word]) ++h->word;
        if (h->word < kIndexWords) {
            g_index_used[h->word] = true;
            if (++g_index_owners == 0) ++g_index_owners;
            h->owner = g_index_owners;
        }
    }
    if (h->word == kIndexWords) {
        delete h;
        return set_error(TP_ERR_UNSUPPORTED, "more than %d live handles (each owns an index word)", kIndexWords);
    }
    *out = h;
    return TP_OK;
}

void tp_paged_destroy(tp_paged *h) {
    if (!h) return;
    {
        std::lock_guard<std::mutex> lock(g_index_mu);
        g_index_used[h->word] = false;
    }
    delete h;
}

size_t tp_paged_workspace_bytes(const tp_paged *h) { return h ? attn::decode_workspace_bytes(h->d) : 0; }

tp_status tp_paged_sync_status(tp_paged *h, void *stream) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned *at = nullptr, v = 0;
    TRY(index_word(h->word, &at));
    TRY(cuda_check(cudaStreamSynchronize(st), "cudaStreamSynchronize"));
    TRY(cuda_check(cudaMemcpy(&v, at, sizeof(v), cudaMemcpyDeviceToHost), "cudaMemcpy(index)"));
    if (v != h->owner) return TP_OK;
    v = 0;
    TRY(cuda_check(cudaMemcpy(at, &v, sizeof(v), cudaMemcpyHostToDevice), "cudaMemcpy(index)"));
    return set_error(TP_ERR_INDEX, "a page, sequence or position was out of range");
}

tp_status tp_paged_append(tp_paged *h, const void *const *X, const int32_t *positions, const int32_t *sequences, int n,
                          const int32_t *table, int table_rows, int table_cols, const float *k_amax,
                          const float *v_amax, void *const *Q, void *const *K, void *const *V, void *stream) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    const tp_paged_desc &d = h->d;
    if (n < 0) return set_error(TP_ERR_SHAPE, "n=%d is negative", n);
    if (n == 0) return TP_OK;
    attn::QkvPlan p = {};
    TRY(at_rows(d, positions, sequences, n, table, table_rows, table_cols, k_amax, v_amax, p.at));
    TRY(at_array(X, d.T, "X", p.x));
    TRY(at_array(Q, d.T, "Q", p.y));
    TRY(at_array(K, d.T, "K", p.k));
    TRY(at_array(V, d.T, "V", p.v));
    TRY(index_word(h->word, &p.at.index_word));
    p.at.owner = h->owner;
    p.k_amax = d.dtype == TP_DT_FP8 ? k_amax : nullptr;
    p.v_amax = d.dtype == TP_DT_FP8 ? v_amax : nullptr;
    p.hq = d.heads / d.T;
    p.hk = d.kv_heads / d.T;
    p.per = d.heads / d.kv_heads;
    p.grouped = d.grouped;
    p.columns = p.hq + 2 * p.hk;
    p.D = d.head_dim;
    p.half = d.rope.dim / 2;
    p.interleaved = d.rope.pairs == TP_ROPE_INTERLEAVED;
    p.sign = 1.0f;
    p.turns = h->turns;
    return attn::launch_qkv(p, d.T, d.dtype == TP_DT_F32 ? 4 : 2, d.dtype == TP_DT_FP8 ? attn::APPEND8 : attn::APPEND,
                            "paged_append", static_cast<cudaStream_t>(stream));
}

tp_status tp_paged_decode(tp_paged *h, const void *const *Q, const int32_t *positions, const int32_t *sequences, int n,
                          const int32_t *table, int table_rows, int table_cols, const float *k_amax,
                          const float *v_amax, const void *const *K, const void *const *V, void *const *O,
                          void *workspace, size_t workspace_bytes, void *stream) {
    if (!h) return set_error(TP_ERR_ARG, "handle is NULL");
    const tp_paged_desc &d = h->d;
    if (n < 0) return set_error(TP_ERR_SHAPE, "n=%d is negative", n);
    if (n == 0) return TP_OK;
    attn::DecodePlan p = {};
    TRY(at_rows(d, positions, sequences, n, table, table_rows, table_cols, k_amax, v_amax, p.at));
    TRY(at_array(Q, d.T, "Q", p.q));
    TRY(at_array(K, d.T, "K", p.k));
    TRY(at_array(V, d.T, "V", p.v));
    TRY(at_array(O, d.T, "O", p.o));
    const size_t need = tp_paged_workspace_bytes(h);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return set_error(TP_ERR_ARG, "workspace is NULL or not 256-byte aligned");
    if (workspace_bytes < need)
        return set_error(TP_ERR_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    TRY(index_word(h->word, &p.at.index_word));
    p.at.owner = h->owner;
    p.k_amax = d.dtype == TP_DT_FP8 ? k_amax : nullptr;
    p.v_amax = d.dtype == TP_DT_FP8 ? v_amax : nullptr;
    p.hq = d.heads / d.T;
    p.hk = d.kv_heads / d.T;
    p.per = d.heads / d.kv_heads;
    p.D = d.head_dim;
    p.window = d.window;
    p.scale_log2 = static_cast<float>(static_cast<double>(h->scale) * 1.4426950408889634);
    p.row_heads = d.kv_heads;  // times the groups
    return attn::launch_decode(p, d.dtype, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
