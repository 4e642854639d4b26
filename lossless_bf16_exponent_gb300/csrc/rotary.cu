// rotary.cu -- rotary positions, alone (forward and gradient) and fused with
// the append of new keys and values to a paged cache.
//
// Pair i of a head turns by the angle position * f_i. The rates are 64-bit
// fixed-point turns, so the phase is one wrapping integer product: whole turns
// fall away exactly and no position is too large. Its upper 32 bits, as half
// turns in [-1, 1), go to sincospif, which needs no range reduction. (A product
// position * f_i in 32-bit floats is off by 4e-3 radians at position 131,072.)
//
// Bound: HBM. Each element is read and written once; a pair costs six
// multiply-adds. A CTA takes a few consecutive tokens (or, where tokens are
// few, a share of one token's heads): it computes their cosines and sines once
// into shared memory, then walks the tokens' rows front to back, so that the
// grid reads and writes a few compact streams. A thread moves two vectors at
// once: the two halves of V pairs (half layout), 2 V adjacent elements
// (interleaved) or 2 V elements that are only copied; two such items are
// loaded before the first is stored, the CTA's first ones before the angles are
// computed. V is the widest of 16 bytes, 8 bytes and one element that the
// rotary dimension, strides and addresses allow.
// Measured: 16,388 tokens of 72 heads of 128, BF16: 98 us, 6.2 TB/s, 91 % of the measured copy rate; 4,095 new
// tokens of 32 + 16 heads, half of each turned, to an E5M2 cache: 17 us (77 MB, floor 11).
#include <algorithm>
#include <type_traits>

#include "kv_internal.cuh"

namespace uzkv {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 2;         // items a thread loads before it stores the first
constexpr uint32_t kMaxTokens = 16;  // of a CTA

struct Params {
    Rows x, y, k, v;  // queries (or the tensor) and their result; new keys and values
    Cache cache;
    const int32_t* positions;
    const int32_t* counts;
    const uint64_t* turns;
    int64_t position_stride;
    uint32_t sequences, tokens, q_heads, kv_heads, head_dim, half;  // half: rotary_dim / 2
    uint32_t items;                 // of a head: pairs of vectors
    uint32_t group, splits, share;  // tokens of a CTA; CTAs of a token and heads of each
    uint32_t layout;
    float magnitude, sign;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// 16-bit elements stay packed in pairs until they are used.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// V elements of a row as they lie in memory.
template <typename T, int V>
struct Raw {
    static constexpr int kWords = (sizeof(T) * V + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const char* p) {
        if constexpr (sizeof(T) * V == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else if constexpr (sizeof(T) * V == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x, w[1] = x.y;
        } else if constexpr (sizeof(T) * V == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void get(float* x) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < V; e++) x[e] = __uint_as_float(w[e]);
        } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float2 v = unpack2<T>(w[e / 2]);
                x[e] = v.x;
                if (e + 1 < V) x[e + 1] = v.y;
            }
        }
    }
};

// V results to a row of D; bits are those of the operand where nothing turned and the types agree.
template <typename D, int V>
__device__ __forceinline__ void put(char* p, const float* x) {
    Vec<D, V> o;
#pragma unroll
    for (int e = 0; e < V; e++) o.e[e] = from_f32<D>(x[e]);
    *reinterpret_cast<Vec<D, V>*>(p) = o;
}

template <typename D, bool kHalf, typename T, int V>
__device__ __forceinline__ void store_pairs(char* row, uint32_t ea, uint32_t eb, bool has_b, const Raw<T, V>& a,
                                            const Raw<T, V>& b, bool turn, const float2* cs) {
    if (std::is_same<D, T>::value && !turn) {
        *reinterpret_cast<Vec<T, V>*>(row + ea * sizeof(T)) = *reinterpret_cast<const Vec<T, V>*>(a.w);
        if (has_b) *reinterpret_cast<Vec<T, V>*>(row + eb * sizeof(T)) = *reinterpret_cast<const Vec<T, V>*>(b.w);
        return;
    }
    float x[2 * V];
    a.get(x);
    b.get(x + V);
    if (turn) {
#pragma unroll
        for (int e = 0; e < V; e++) {
            const int i = kHalf ? e : 2 * e, j = kHalf ? V + e : 2 * e + 1;
            const float2 v = cs[e];
            const float p = x[i], q = x[j];
            x[i] = p * v.x - q * v.y;
            x[j] = q * v.x + p * v.y;
        }
    }
    put<D, V>(row + ea * sizeof(D), x);
    if (has_b) put<D, V>(row + eb * sizeof(D), x + V);
}

// Where a token's rows are.
struct Token {
    const char *x, *k, *v;
    char* y;
    Place place;
    int32_t position;
    bool live;
};

template <typename T, typename C, int V, bool kHalf, bool kAppend>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ Params p) {
    extern __shared__ float2 turned[];  // [group][half]: cosine and sine, magnitude and direction applied
    __shared__ Token tokens[kMaxTokens];
    const uint32_t tid = threadIdx.x;
    const uint32_t block = blockIdx.x / p.splits, split = blockIdx.x - block * p.splits;
    const uint64_t first = (uint64_t)block * p.group, all = (uint64_t)p.sequences * p.tokens;
    const uint32_t count = (uint32_t)min((uint64_t)p.group, all - first);
    const uint32_t heads_all = p.q_heads + (kAppend ? 2 * p.kv_heads : 0);
    const uint32_t head0 = split * p.share, heads = min(p.share, heads_all - head0);
    const uint32_t turning = p.half / V;  // items that turn; the rest copy
    const uint32_t per_token = heads * p.items, total = count * per_token;

    // An item's place: token of the CTA, head of the share, item of the head; a step of kThreads in that mixed radix.
    struct At {
        uint32_t token, head, item;
    };
    const uint32_t first_token = tid / per_token, in = tid - first_token * per_token;
    At at{first_token, in / p.items, in % p.items};
    const uint32_t step_token = kThreads / per_token, step_in = kThreads - step_token * per_token;
    const uint32_t step_head = step_in / p.items, step_item = step_in - step_head * p.items;
    auto next = [&](At& a) {
        a.item += step_item;
        a.head += step_head;
        a.token += step_token;
        if (a.item >= p.items) {
            a.item -= p.items;
            a.head++;
        }
        if (a.head >= heads) {
            a.head -= heads;
            a.token++;
        }
    };
    auto columns = [&](uint32_t item, uint32_t& ea, uint32_t& eb) {
        if (item >= turning) {
            ea = 2 * p.half + 2 * V * (item - turning);
            eb = ea + V;
        } else if (kHalf) {
            ea = item * V;
            eb = p.half + ea;
        } else {
            ea = 2 * V * item;
            eb = ea + V;
        }
    };
    if (tid < count) {
        const uint64_t n = first + tid;
        const uint32_t b = (uint32_t)(n / p.tokens), t = (uint32_t)(n - (uint64_t)b * p.tokens);
        Token w{};
        w.x = p.x.p + b * p.x.b + t * p.x.t;
        w.y = p.y.p + b * p.y.b + t * p.y.t;
        w.position = p.positions[b * p.position_stride + t];
        w.live = true;
        if (kAppend) {
            w.k = p.k.p + b * p.k.b + t * p.k.t;
            w.v = p.v.p + b * p.v.b + t * p.v.t;
            const Span sp = span_of(p.cache, p.counts, p.tokens, b);
            w.live = t < sp.fresh;
            w.place = w.live ? place_of(p.cache, b, sp.old + t) : Place{-1, 0};
        }
        tokens[tid] = w;
    }
    __syncthreads();
    Raw<T, V> a[kInFlight], bb[kInFlight];
    auto load = [&](const At& w, Raw<T, V>& va, Raw<T, V>& vb) {
        uint32_t ea, eb;
        columns(w.item, ea, eb);
        const uint32_t h = head0 + w.head;
        const char* row;
        if (!kAppend || h < p.q_heads)
            row = tokens[w.token].x + h * p.x.h;
        else if (h < p.q_heads + p.kv_heads)
            row = tokens[w.token].k + (h - p.q_heads) * p.k.h;
        else
            row = tokens[w.token].v + (h - p.q_heads - p.kv_heads) * p.v.h;
        va.load(row + ea * sizeof(T));
        if (eb < p.head_dim) vb.load(row + eb * sizeof(T));
    };

    At ahead = at;
    uint32_t loaded = tid;
#pragma unroll
    for (int u = 0; u < kInFlight; u++, loaded += kThreads) {
        if (loaded < total) load(ahead, a[u], bb[u]);
        next(ahead);
    }
    for (uint32_t i = tid; i < count * p.half; i += kThreads) {
        const uint32_t token = i / p.half;
        const uint64_t phase = (uint64_t)(int64_t)tokens[token].position * p.turns[i - token * p.half];
        float sn, cs;
        sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
        turned[i] = make_float2(cs * p.magnitude, sn * p.sign);
    }
    __syncthreads();

    for (uint32_t base = tid; base < total; base += kThreads * kInFlight) {
#pragma unroll
        for (int u = 0; u < kInFlight; u++) {
            if (base + u * kThreads >= total) break;
            uint32_t ea, eb;
            columns(at.item, ea, eb);
            const Token& w = tokens[at.token];
            const uint32_t h = head0 + at.head;
            const bool turn = at.item < turning, has_b = eb < p.head_dim;
            const float2* cs = turned + at.token * p.half + at.item * V;
            if (!kAppend || h < p.q_heads) {
                char* row = w.y + h * p.y.h;
                if (!kAppend || w.live) {
                    store_pairs<T, kHalf>(row, ea, eb, has_b, a[u], bb[u], turn, cs);
                } else {
                    const float z[V] = {};
                    put<T, V>(row + ea * sizeof(T), z);
                    if (has_b) put<T, V>(row + eb * sizeof(T), z);
                }
            } else if (w.place.page >= 0) {
                const bool is_k = h < p.q_heads + p.kv_heads;
                char* row = is_k ? k_row(p.cache, w.place, h - p.q_heads)
                                 : v_row(p.cache, w.place, h - p.q_heads - p.kv_heads);
                store_pairs<C, kHalf>(row, ea, eb, has_b, a[u], bb[u], turn && is_k, cs);
            }
            next(at);
            if (loaded < total) load(ahead, a[u], bb[u]);
            next(ahead);
            loaded += kThreads;
        }
    }
}

template <typename T, typename C, int V, bool kAppend>
int launch(Params& p, cudaStream_t stream) {
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    const uint32_t copied = p.head_dim - 2 * p.half;
    p.items = p.half / V + (copied + 2 * V - 1) / (2 * V);
    const uint32_t heads = p.q_heads + (kAppend ? 2 * p.kv_heads : 0);
    const uint64_t tokens = (uint64_t)p.sequences * p.tokens, items = (uint64_t)heads * p.items;
    // Many tokens: as many a CTA as give each thread about eight items (a CTA starts with two rounds of latency),
    // while four CTAs an SM remain. Few: several CTAs a token, while each thread has an item. Measured on 16,388
    // tokens of 72 heads of 128: 4 tokens a CTA 98 us, 6 99 us, 13 110 us; on 4,095 tokens of 48 heads, half of
    // each turned, to an E5M2 cache: one token 22 us, 3 17 us, 6 18 us.
    const uint64_t fill = (8 * kThreads + items - 1) / items, most = (items + kThreads - 1) / kThreads;
    p.group = (uint32_t)std::min<uint64_t>(std::min<uint64_t>(kMaxTokens, fill), std::max<uint64_t>(1, tokens / ((uint64_t)sms * 4)));
    const uint64_t want = std::min(most, std::max<uint64_t>(1, (uint64_t)sms * 16 / tokens));
    p.share = (uint32_t)((heads + want - 1) / want);
    p.splits = (heads + p.share - 1) / p.share;
    const uint64_t grid = (tokens + p.group - 1) / p.group * p.splits;
    if (grid > 0x7FFFFFFFull) return UZIP_ERR_ARG;
    const size_t smem = p.group * p.half * sizeof(float2);
    if (p.layout == UZKV_HALF)
        rotary_kernel<T, C, V, true, kAppend><<<(unsigned)grid, kThreads, smem, stream>>>(p);
    else
        rotary_kernel<T, C, V, false, kAppend><<<(unsigned)grid, kThreads, smem, stream>>>(p);
    UZIP_CUDA_TRY(cudaGetLastError());
    return UZIP_OK;
}

// Largest V of {8, 4, 1} (16-bit) or {4, 1} (32-bit) that all vectors of the call allow.
template <typename T, typename C, bool kAppend>
int dispatch(Params& p, cudaStream_t stream) {
    uint64_t a = p.half * sizeof(T) | p.head_dim * sizeof(T);
    auto add = [&](const Rows& r) { a |= reinterpret_cast<uintptr_t>(r.p) | (uint64_t)r.b | (uint64_t)r.t | (uint64_t)r.h; };
    add(p.x);
    add(p.y);
    if (kAppend) {
        add(p.k);
        add(p.v);
    }
    if (a % 16 == 0) return launch<T, C, 16 / sizeof(T), kAppend>(p, stream);
    if (sizeof(T) == 2 && a % 8 == 0) return launch<T, C, 4, kAppend>(p, stream);
    return launch<T, C, 1, kAppend>(p, stream);
}

int common(const int32_t* d_positions, int64_t position_stride, const uint64_t* d_turns, uint32_t rotary_dim,
           uint32_t layout, uint32_t head_dim, uint32_t tokens, uint32_t heads) {
    if (!d_positions || !d_turns || position_stride < 0) return UZIP_ERR_ARG;
    if (!head_dim || head_dim > UZKV_MAX_HEAD_DIM || !rotary_dim || rotary_dim % 2 || rotary_dim > head_dim) return UZIP_ERR_ARG;
    if (layout != UZKV_HALF && layout != UZKV_INTERLEAVED) return UZIP_ERR_ARG;
    if (!tokens || tokens > 0x7FFFFFFFu || !heads || heads > 65535) return UZIP_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(d_positions) & 3) || (reinterpret_cast<uintptr_t>(d_turns) & 7)) return UZIP_ERR_ALIGN;
    return UZIP_OK;
}

bool element_aligned(const Rows& r, uint32_t dtype) { return reinterpret_cast<uintptr_t>(r.p) % bytes_of(dtype) == 0; }

}  // namespace
}  // namespace uzkv

using namespace uzkv;

extern "C" UZIP_API int uzkv_rotary(const uzkv_rows_t* x, const uzkv_rows_t* y, uint32_t dtype, uint32_t sequences,
                                    uint32_t tokens, uint32_t heads, uint32_t head_dim, const int32_t* d_positions,
                                    int64_t position_stride, const uint64_t* d_turns, uint32_t rotary_dim,
                                    uint32_t layout, float magnitude, int backward, uzip_stream_t stream) {
    if (!rows_valid(x) || !rows_valid(y) || !sequences || dtype > UZKV_FP32) return UZIP_ERR_ARG;
    if (int rc = common(d_positions, position_stride, d_turns, rotary_dim, layout, head_dim, tokens, heads)) return rc;
    Params p{};
    p.x = rows_of(x, dtype, sequences, tokens, heads);
    p.y = rows_of(y, dtype, sequences, tokens, heads);
    if (!element_aligned(p.x, dtype) || !element_aligned(p.y, dtype)) return UZIP_ERR_ALIGN;
    p.positions = d_positions;
    p.position_stride = position_stride;
    p.turns = d_turns;
    p.sequences = sequences;
    p.tokens = tokens;
    p.q_heads = heads;
    p.head_dim = head_dim;
    p.half = rotary_dim / 2;
    p.layout = layout;
    p.magnitude = magnitude;
    p.sign = backward ? -magnitude : magnitude;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == UZKV_BF16) return dispatch<__nv_bfloat16, __nv_bfloat16, false>(p, s);
    if (dtype == UZKV_FP16) return dispatch<__half, __half, false>(p, s);
    return dispatch<float, float, false>(p, s);
}

extern "C" UZIP_API int uzkv_rotary_append(const uzkv_rows_t* q, const uzkv_rows_t* k, const uzkv_rows_t* v,
                                           const uzkv_rows_t* q_out, uint32_t dtype, uint32_t tokens,
                                           uint32_t q_heads, const int32_t* d_positions, int64_t position_stride,
                                           const uint64_t* d_turns, uint32_t rotary_dim, uint32_t layout,
                                           float magnitude, const int32_t* d_counts, const uzkv_cache_t* cache,
                                           uzip_stream_t stream) {
    if (!rows_valid(q) || !rows_valid(k) || !rows_valid(v) || !rows_valid(q_out) || dtype > UZKV_FP16) return UZIP_ERR_ARG;
    Params p{};
    if (int rc = cache_of(cache, &p.cache)) return rc;
    if (cache->dtype != dtype && cache->dtype != UZKV_E5M2) return UZIP_ERR_ARG;
    if (int rc = common(d_positions, position_stride, d_turns, rotary_dim, layout, cache->head_dim, tokens, q_heads)) return rc;
    p.x = rows_of(q, dtype, cache->sequences, tokens, q_heads);
    p.y = rows_of(q_out, dtype, cache->sequences, tokens, q_heads);
    p.k = rows_of(k, dtype, cache->sequences, tokens, cache->kv_heads);
    p.v = rows_of(v, dtype, cache->sequences, tokens, cache->kv_heads);
    for (const Rows* r : {&p.x, &p.y, &p.k, &p.v})
        if (!element_aligned(*r, dtype)) return UZIP_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(d_counts) & 3) return UZIP_ERR_ALIGN;
    p.positions = d_positions;
    p.position_stride = position_stride;
    p.turns = d_turns;
    p.counts = d_counts;
    p.sequences = cache->sequences;
    p.tokens = tokens;
    p.q_heads = q_heads;
    p.kv_heads = cache->kv_heads;
    p.head_dim = cache->head_dim;
    p.half = rotary_dim / 2;
    p.layout = layout;
    p.magnitude = p.sign = magnitude;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool fp8 = cache->dtype == UZKV_E5M2;
    if (dtype == UZKV_BF16)
        return fp8 ? dispatch<__nv_bfloat16, E5M2, true>(p, s) : dispatch<__nv_bfloat16, __nv_bfloat16, true>(p, s);
    return fp8 ? dispatch<__half, E5M2, true>(p, s) : dispatch<__half, __half, true>(p, s);
}
