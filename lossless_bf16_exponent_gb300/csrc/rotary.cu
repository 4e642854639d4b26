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
// multiply-adds. One warp takes one token: a lane keeps the cosines and sines
// of its V pairs in registers and walks the token's heads with them, so the
// angles are computed once a token and not once a head. A lane moves two
// vectors a head, the two halves of its pairs (half layout) or 2 V adjacent
// elements (interleaved), so both layouts are whole vectors. V is the widest
// of 16 bytes, 8 bytes and one element that the rotary dimension, strides and
// addresses allow.
#include <algorithm>

#include "kv_internal.cuh"

namespace uzkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTeams = kThreads / 32;
constexpr int kHeadsInFlight = 2;  // heads a lane loads before it stores the first

struct Params {
    Rows x, y, k, v;  // queries (or the tensor) and their result; new keys and values
    Cache cache;
    const int32_t* positions;
    const int32_t* counts;
    const uint64_t* turns;
    int64_t position_stride;
    uint32_t sequences, tokens, q_heads, kv_heads, head_dim, half;  // half: rotary_dim / 2
    uint32_t items, lanes, heads_at_once, splits;
    uint32_t layout;
    float magnitude, sign;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// Value copies keep their bits where the types agree.
template <typename C, typename T>
__device__ __forceinline__ C convert(T x) { return from_f32<C>(to_f32(x)); }
template <>
__device__ __forceinline__ float convert<float, float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 convert<__nv_bfloat16, __nv_bfloat16>(__nv_bfloat16 x) { return x; }
template <>
__device__ __forceinline__ __half convert<__half, __half>(__half x) { return x; }

template <typename D, typename T, int V>
__device__ __forceinline__ void store_pairs(char* row, uint32_t ea, uint32_t eb, bool has_b, const Vec<T, V>& a,
                                            const Vec<T, V>& b, bool turn, bool half_layout, const float* c,
                                            const float* s) {
    Vec<D, V> oa, ob;
    if (!turn) {
#pragma unroll
        for (int e = 0; e < V; e++) {
            oa.e[e] = convert<D, T>(a.e[e]);
            ob.e[e] = convert<D, T>(b.e[e]);
        }
    } else if (half_layout) {
#pragma unroll
        for (int e = 0; e < V; e++) {
            const float p = to_f32(a.e[e]), q = to_f32(b.e[e]);
            oa.e[e] = from_f32<D>(p * c[e] - q * s[e]);
            ob.e[e] = from_f32<D>(q * c[e] + p * s[e]);
        }
    } else {
        float x[2 * V];
#pragma unroll
        for (int e = 0; e < V; e++) {
            x[e] = to_f32(a.e[e]);
            x[V + e] = to_f32(b.e[e]);
        }
        D o[2 * V];
#pragma unroll
        for (int e = 0; e < V; e++) {
            o[2 * e] = from_f32<D>(x[2 * e] * c[e] - x[2 * e + 1] * s[e]);
            o[2 * e + 1] = from_f32<D>(x[2 * e + 1] * c[e] + x[2 * e] * s[e]);
        }
#pragma unroll
        for (int e = 0; e < V; e++) {
            oa.e[e] = o[e];
            ob.e[e] = o[V + e];
        }
    }
    *reinterpret_cast<Vec<D, V>*>(row + ea * sizeof(D)) = oa;
    if (has_b) *reinterpret_cast<Vec<D, V>*>(row + eb * sizeof(D)) = ob;
}

// One warp: one token (and, where tokens are few, one share of its heads).
template <typename T, typename C, int V, bool kAppend>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Params p) {
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t team = (uint64_t)blockIdx.x * kTeams + threadIdx.x / 32;
    const uint32_t split = (uint32_t)(team % p.splits);
    const uint64_t token = team / p.splits;
    if (token >= (uint64_t)p.sequences * p.tokens) return;
    const uint32_t b = (uint32_t)(token / p.tokens), t = (uint32_t)(token % p.tokens);
    const uint32_t mine = lane / p.lanes;
    if (mine >= p.heads_at_once) return;

    bool live = true;
    Place place{-1, 0};
    if (kAppend) {
        const Span sp = span_of(p.cache, p.counts, p.tokens, b);
        live = t < sp.fresh;
        if (live) place = place_of(p.cache, b, sp.old + t);
    }
    const uint64_t position = (uint64_t)(int64_t)p.positions[b * p.position_stride + t];
    const uint32_t heads = kAppend ? (live ? p.q_heads + 2 * p.kv_heads : p.q_heads) : p.q_heads;
    const uint32_t step = p.heads_at_once * p.splits;
    const bool half_layout = p.layout == UZKV_HALF;
    const uint32_t turning = p.half / V;  // items that turn; the rest copy

    for (uint32_t item = lane % p.lanes; item < p.items; item += p.lanes) {
        const bool turn = item < turning;
        uint32_t ea, eb;
        if (!turn) {
            ea = 2 * p.half + 2 * V * (item - turning);
            eb = ea + V;
        } else if (half_layout) {
            ea = item * V;
            eb = p.half + ea;
        } else {
            ea = 2 * V * item;
            eb = ea + V;
        }
        const bool has_b = eb < p.head_dim;
        float c[V], s[V];
        if (turn && live) {
#pragma unroll
            for (int e = 0; e < V; e++) {
                const uint64_t phase = position * p.turns[item * V + e];
                float sn, cs;
                sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
                c[e] = cs * p.magnitude;
                s[e] = sn * p.sign;
            }
        }
        for (uint32_t h0 = split * p.heads_at_once + mine; h0 < heads; h0 += step * kHeadsInFlight) {
            Vec<T, V> a[kHeadsInFlight], bb[kHeadsInFlight];
#pragma unroll
            for (int u = 0; u < kHeadsInFlight; u++) {
                const uint32_t h = h0 + u * step;
                if (h < heads && live) {
                    const char* row;
                    if (!kAppend || h < p.q_heads)
                        row = p.x.p + b * p.x.b + t * p.x.t + h * p.x.h;
                    else if (h < p.q_heads + p.kv_heads)
                        row = p.k.p + b * p.k.b + t * p.k.t + (h - p.q_heads) * p.k.h;
                    else
                        row = p.v.p + b * p.v.b + t * p.v.t + (h - p.q_heads - p.kv_heads) * p.v.h;
                    a[u] = *reinterpret_cast<const Vec<T, V>*>(row + ea * sizeof(T));
                    bb[u] = has_b ? *reinterpret_cast<const Vec<T, V>*>(row + eb * sizeof(T)) : a[u];
                }
            }
#pragma unroll
            for (int u = 0; u < kHeadsInFlight; u++) {
                const uint32_t h = h0 + u * step;
                if (h >= heads) continue;
                if (!kAppend || h < p.q_heads) {
                    char* row = p.y.p + b * p.y.b + t * p.y.t + h * p.y.h;
                    if (live) {
                        store_pairs<T>(row, ea, eb, has_b, a[u], bb[u], turn, half_layout, c, s);
                    } else {
                        Vec<T, V> z;
#pragma unroll
                        for (int e = 0; e < V; e++) z.e[e] = from_f32<T>(0.0f);
                        *reinterpret_cast<Vec<T, V>*>(row + ea * sizeof(T)) = z;
                        if (has_b) *reinterpret_cast<Vec<T, V>*>(row + eb * sizeof(T)) = z;
                    }
                } else if (place.page >= 0) {
                    const bool is_k = h < p.q_heads + p.kv_heads;
                    char* row = is_k ? k_row(p.cache, place, h - p.q_heads)
                                     : v_row(p.cache, place, h - p.q_heads - p.kv_heads);
                    store_pairs<C>(row, ea, eb, has_b, a[u], bb[u], turn && is_k, half_layout, c, s);
                }
            }
        }
    }
}

template <typename T, typename C, int V, bool kAppend>
int launch(Params& p, cudaStream_t stream) {
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    const uint32_t copied = p.head_dim - 2 * p.half;
    p.items = p.half / V + (copied + 2 * V - 1) / (2 * V);
    p.lanes = std::min(p.items, 32u);
    p.heads_at_once = 32 / p.lanes;
    const uint32_t heads = p.q_heads + (kAppend ? 2 * p.kv_heads : 0);
    const uint64_t tokens = (uint64_t)p.sequences * p.tokens;
    // Few tokens: several warps share a token's heads, up to one head batch each, until 32 warps an SM are there.
    const uint64_t most = (heads + p.heads_at_once - 1) / p.heads_at_once;
    p.splits = (uint32_t)std::min<uint64_t>(most, std::max<uint64_t>(1, (uint64_t)sms * 32 / tokens));
    const uint64_t grid = (tokens * p.splits + kTeams - 1) / kTeams;
    if (grid > 0x7FFFFFFFull) return UZIP_ERR_ARG;
    rotary_kernel<T, C, V, kAppend><<<(unsigned)grid, kThreads, 0, stream>>>(p);
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
    p.x = rows_of(x, dtype);
    p.y = rows_of(y, dtype);
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
    p.x = rows_of(q, dtype);
    p.y = rows_of(q_out, dtype);
    p.k = rows_of(k, dtype);
    p.v = rows_of(v, dtype);
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
