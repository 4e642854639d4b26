// attention.cu -- attention for a tree of drafted tokens over a paged cache,
// and the attention weight that each cached token collects.
//
// First form: one CTA a query row (attention), one thread a cached token
// (mass), in 32-bit floats.
#include <algorithm>

#include "kv_internal.cuh"

namespace uzkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

struct Params {
    Rows q, out;
    float* lse;
    const int64_t* mask;
    int64_t mask_b;
    uint32_t mask_words;
    const int32_t* counts;
    const float* weights;
    Cache cache;
    float scale;
    uint32_t tokens, q_heads, group;
    const float* mass_in;
    float* mass_out;
    float decay;
    int64_t mass_b, mass_h;
    uint32_t slots;
};

__device__ __forceinline__ const int64_t* mask_row(const Params& p, uint32_t b, uint32_t t) {
    return p.mask ? p.mask + b * p.mask_b + (uint64_t)t * p.mask_words : nullptr;
}

// Grid (tokens, q_heads, sequences).
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads) attend_rows_kernel(const __grid_constant__ Params p) {
    constexpr int kPer = UZKV_MAX_HEAD_DIM / 32;
    __shared__ float acc_s[kWarps][UZKV_MAX_HEAD_DIM];
    __shared__ float m_s[kWarps], l_s[kWarps];
    const uint32_t t = blockIdx.x, hq = blockIdx.y, b = blockIdx.z, h = hq / p.group;
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, d = p.cache.head_dim;
    const Span sp = span_of(p.cache, p.counts, p.tokens, b);
    const int64_t* mask = mask_row(p, b, t);
    const T* q = reinterpret_cast<const T*>(p.q.p + b * p.q.b + t * p.q.t + hq * p.q.h);
    float qr[kPer], o[kPer], m = -INFINITY, l = 0.0f;
    for (int i = 0; i < kPer; i++) {
        qr[i] = lane + 32 * i < d ? to_f32(q[lane + 32 * i]) * p.scale : 0.0f;
        o[i] = 0.0f;
    }
    const uint32_t n = t < sp.fresh ? sp.old + sp.fresh : 0;
    for (uint32_t j = warp; j < n; j += kWarps) {
        if (j >= sp.old && !mask_bit(mask, t, j - sp.old)) continue;
        const Place at = place_of(p.cache, b, j);
        if (at.page < 0) continue;
        const C* k = reinterpret_cast<const C*>(k_row(p.cache, at, h));
        const C* v = reinterpret_cast<const C*>(v_row(p.cache, at, h));
        float s = 0.0f;
        for (int i = 0; i < kPer; i++)
            if (lane + 32 * i < d) s += qr[i] * to_f32(k[lane + 32 * i]);
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
        const float mn = s > m ? s : m;  // NaN leaves m as it is and comes in through exp
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float f = expf(m - base), e = expf(s - base);
        m = mn;
        l = l * f + e;
        for (int i = 0; i < kPer; i++)
            if (lane + 32 * i < d) o[i] = o[i] * f + e * to_f32(v[lane + 32 * i]);
    }
    for (int i = 0; i < kPer; i++) acc_s[warp][lane + 32 * i] = o[i];
    if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < kWarps; w++) top = fmaxf(top, m_s[w]);
    const float base = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < kWarps; w++) sum += l_s[w] * expf(m_s[w] - base);
    T* out = reinterpret_cast<T*>(p.out.p + b * p.out.b + t * p.out.t + hq * p.out.h);
    for (uint32_t i = threadIdx.x; i < d; i += kThreads) {
        float x = 0.0f;
        for (int w = 0; w < kWarps; w++) x += acc_s[w][i] * expf(m_s[w] - base);
        out[i] = from_f32<T>(sum == 0.0f ? 0.0f : x / sum);
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[((uint64_t)b * p.tokens + t) * p.q_heads + hq] = sum == 0.0f ? -INFINITY : base + logf(sum);
}

// Grid (slots / kThreads, kv_heads, sequences).
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads) mass_rows_kernel(const __grid_constant__ Params p) {
    const uint32_t j = blockIdx.x * kThreads + threadIdx.x, h = blockIdx.y, b = blockIdx.z, d = p.cache.head_dim;
    if (j >= p.slots) return;
    const Span sp = span_of(p.cache, p.counts, p.tokens, b);
    const int64_t at_mass = b * p.mass_b + h * p.mass_h + j;
    float w = 0.0f;
    if (j < sp.old + sp.fresh) {
        const Place at = place_of(p.cache, b, j);
        const C* k = reinterpret_cast<const C*>(k_row(p.cache, at, h));
        for (uint32_t t = 0; t < sp.fresh && at.page >= 0; t++) {
            if (j >= sp.old && !mask_bit(mask_row(p, b, t), t, j - sp.old)) continue;
            const float weight = p.weights ? p.weights[b * p.tokens + t] : 1.0f;
            for (uint32_t g = 0; g < p.group; g++) {
                const uint32_t hq = h * p.group + g;
                const float lse = p.lse[((uint64_t)b * p.tokens + t) * p.q_heads + hq];
                if (lse == -INFINITY || weight == 0.0f) continue;
                const T* q = reinterpret_cast<const T*>(p.q.p + b * p.q.b + t * p.q.t + hq * p.q.h);
                float s = 0.0f;
                for (uint32_t i = 0; i < d; i++) s += to_f32(q[i]) * to_f32(k[i]);
                w += weight * expf(s * p.scale - lse);
            }
        }
    }
    if (p.mass_in && j < sp.old) w += p.decay * p.mass_in[at_mass];
    p.mass_out[at_mass] = w;
}

template <typename T, typename C>
int launch_attend(const Params& p, cudaStream_t s) {
    attend_rows_kernel<T, C><<<dim3(p.tokens, p.q_heads, p.cache.sequences), kThreads, 0, s>>>(p);
    UZIP_CUDA_TRY(cudaGetLastError());
    return UZIP_OK;
}
template <typename T, typename C>
int launch_mass(const Params& p, cudaStream_t s) {
    mass_rows_kernel<T, C><<<dim3((p.slots + kThreads - 1) / kThreads, p.cache.kv_heads, p.cache.sequences), kThreads, 0, s>>>(p);
    UZIP_CUDA_TRY(cudaGetLastError());
    return UZIP_OK;
}

// What attention and mass check alike.
int common(Params& p, const uzkv_rows_t* q, uint32_t dtype, uint32_t tokens, uint32_t q_heads, const int64_t* d_mask,
           int64_t mask_stride_b, const int32_t* d_counts, float scale, const uzkv_cache_t* cache) {
    if (int rc = cache_of(cache, &p.cache)) return rc;
    if (!rows_valid(q) || dtype > UZKV_FP16 || (cache->dtype != dtype && cache->dtype != UZKV_E5M2)) return UZIP_ERR_ARG;
    if (!tokens || tokens > UZKV_MAX_NEW_TOKENS || !q_heads || q_heads > 65535 || q_heads % cache->kv_heads) return UZIP_ERR_ARG;
    if (mask_stride_b < 0) return UZIP_ERR_ARG;
    p.q = rows_of(q, dtype);
    if (!rows_aligned16(p.q)) return UZIP_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(d_mask) & 7) || (reinterpret_cast<uintptr_t>(d_counts) & 3)) return UZIP_ERR_ALIGN;
    p.mask = d_mask;
    p.mask_b = mask_stride_b;
    p.mask_words = (tokens + 63) / 64;
    p.counts = d_counts;
    p.scale = scale;
    p.tokens = tokens;
    p.q_heads = q_heads;
    p.group = q_heads / cache->kv_heads;
    return UZIP_OK;
}

}  // namespace
}  // namespace uzkv

using namespace uzkv;

extern "C" UZIP_API size_t uzkv_tree_attention_workspace_bytes(uint32_t sequences, uint32_t tokens, uint32_t q_heads,
                                                               uint32_t kv_heads, uint32_t head_dim) {
    if (!sequences || !tokens || tokens > UZKV_MAX_NEW_TOKENS || !q_heads || !kv_heads || q_heads % kv_heads ||
        !head_dim || head_dim > UZKV_MAX_HEAD_DIM)
        return 0;
    return 16;
}

extern "C" UZIP_API int uzkv_tree_attention(const uzkv_rows_t* q, const uzkv_rows_t* out, float* d_lse, uint32_t dtype,
                                            uint32_t tokens, uint32_t q_heads, const int64_t* d_mask,
                                            int64_t mask_stride_b, const int32_t* d_counts, float scale,
                                            const uzkv_cache_t* cache, void* d_workspace, size_t workspace_bytes,
                                            uzip_stream_t stream) {
    Params p{};
    if (int rc = common(p, q, dtype, tokens, q_heads, d_mask, mask_stride_b, d_counts, scale, cache)) return rc;
    if (!rows_valid(out) || !d_workspace) return UZIP_ERR_ARG;
    p.out = rows_of(out, dtype);
    if (!rows_aligned16(p.out) || !aligned16(d_workspace) || (reinterpret_cast<uintptr_t>(d_lse) & 3)) return UZIP_ERR_ALIGN;
    if (workspace_bytes < uzkv_tree_attention_workspace_bytes(p.cache.sequences, tokens, q_heads, p.cache.kv_heads, p.cache.head_dim))
        return UZIP_ERR_CAPACITY;
    p.lse = d_lse;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool fp8 = cache->dtype == UZKV_E5M2;
    if (dtype == UZKV_BF16)
        return fp8 ? launch_attend<__nv_bfloat16, E5M2>(p, s) : launch_attend<__nv_bfloat16, __nv_bfloat16>(p, s);
    return fp8 ? launch_attend<__half, E5M2>(p, s) : launch_attend<__half, __half>(p, s);
}

extern "C" UZIP_API int uzkv_attention_mass(const uzkv_rows_t* q, const float* d_lse, uint32_t dtype, uint32_t tokens,
                                            uint32_t q_heads, const int64_t* d_mask, int64_t mask_stride_b,
                                            const int32_t* d_counts, const float* d_weights, float scale,
                                            const uzkv_cache_t* cache, const float* d_mass_in, float decay,
                                            float* d_mass_out, int64_t mass_stride_b, int64_t mass_stride_h,
                                            uint32_t slots, uzip_stream_t stream) {
    Params p{};
    if (int rc = common(p, q, dtype, tokens, q_heads, d_mask, mask_stride_b, d_counts, scale, cache)) return rc;
    if (!d_lse || !d_mass_out || mass_stride_b < 0 || mass_stride_h < 0 || !slots || slots > p.cache.capacity) return UZIP_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(d_lse) | reinterpret_cast<uintptr_t>(d_weights) |
         reinterpret_cast<uintptr_t>(d_mass_in) | reinterpret_cast<uintptr_t>(d_mass_out)) & 3)
        return UZIP_ERR_ALIGN;
    p.lse = const_cast<float*>(d_lse);
    p.weights = d_weights;
    p.mass_in = d_mass_in;
    p.mass_out = d_mass_out;
    p.decay = decay;
    p.mass_b = mass_stride_b;
    p.mass_h = mass_stride_h;
    p.slots = slots;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool fp8 = cache->dtype == UZKV_E5M2;
    if (dtype == UZKV_BF16)
        return fp8 ? launch_mass<__nv_bfloat16, E5M2>(p, s) : launch_mass<__nv_bfloat16, __nv_bfloat16>(p, s);
    return fp8 ? launch_mass<__half, E5M2>(p, s) : launch_mass<__half, __half>(p, s);
}
