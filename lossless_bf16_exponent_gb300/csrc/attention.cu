// attention.cu -- entry points of attention for a tree of drafted tokens over a
// paged cache and of the attention weight that each cached token collects; the
// kernel that joins the partial results of units that several CTAs shared.
#include <algorithm>

#include "kv_attention.cuh"

namespace uzkv {
namespace {

constexpr int kThreads = 128;
using Params = AttParams;

// Join: one warp a query row. Launched as a programmatic dependent of the attention kernel, so that finding its
// unit's share of the split overlaps that kernel; rows of units that one CTA finished are already written. Also
// writes the rows of sequences without new tokens, which have no tiles.
template <typename QT>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Params p) {
    const uint32_t lane = threadIdx.x % 32;
    const uint32_t w = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const uint32_t bh = w / p.rows, row = w - bh * p.rows, b = bh / p.cache.kv_heads, h = bh - b * p.cache.kv_heads;
    if (b >= p.cache.sequences) {
        uzip::pdl_wait();
        return;
    }
    uint64_t total = 0, before = 0;
    for (uint32_t i = lane; i < p.cache.sequences; i += 32) {
        const uint32_t n = width_of(p, tiles_of(p, i));
        total += n;
        before += i < b ? n : 0;
    }
    for (int o = 16; o; o >>= 1) {
        total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    }
    const uint32_t tiles = tiles_of(p, b), mt = row / p.m, r = row % p.m;
    const uint64_t units = (uint64_t)p.cache.kv_heads * p.mtiles;
    total *= units;
    const uint64_t start = before * units + ((uint64_t)h * p.mtiles + mt) * width_of(p, tiles) + p.unit_cost;  // of its tiles
    const uint64_t shares = min(total, (uint64_t)p.grid);
    uint32_t c0 = 0, c1 = 0;
    if (tiles) {
        c0 = share_of(start, shares, total);
        c1 = share_of(start + tiles - 1, shares, total);
    }
    uzip::pdl_wait();
    if (tiles && c0 == c1) return;
    const uint32_t t = row / p.group, hq = h * p.group + row % p.group;
    char* out = p.out.p + b * p.out.b + t * p.out.t + (uint64_t)hq * p.out.h;
    const uint64_t size = partial_floats(p);
    auto part_of = [&](uint32_t c) { return p.partial + ((uint64_t)c * 2 + (c == c0)) * size; };

    float top = -INFINITY;
    if (tiles)
        for (uint32_t c = c0 + lane; c <= c1; c += 32) {
            const float2 st = *reinterpret_cast<const float2*>(part_of(c) + (uint64_t)p.m * p.dp + 2 * r);
            if (st.y != 0.0f) top = fmaxf(top, st.x);
        }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float sum = 0.0f;
    float4 acc[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
    if (tiles)
#pragma unroll 4
        for (uint32_t c = c0; c <= c1; c++) {
            const float* part = part_of(c);
            const float2 st = *reinterpret_cast<const float2*>(part + (uint64_t)p.m * p.dp + 2 * r);
            const float f = st.y == 0.0f ? 0.0f : exp2_fast(st.x - top);
            sum += st.y * f;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint32_t d = 4 * lane + 128 * i;
                if (d >= p.cache.head_dim || st.y == 0.0f) continue;
                const float4 v = *reinterpret_cast<const float4*>(part + (uint64_t)r * p.dp + d);
                acc[i].x += v.x * f;
                acc[i].y += v.y * f;
                acc[i].z += v.z * f;
                acc[i].w += v.w * f;
            }
        }
    const bool none = sum == 0.0f;
    const float inv = none ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t d = 4 * lane + 128 * i;
        if (d >= p.cache.head_dim) continue;
        *reinterpret_cast<uint2*>(out + 2 * d) =
            none ? make_uint2(0, 0) : make_uint2(pack2<QT>(acc[i].x * inv, acc[i].y * inv), pack2<QT>(acc[i].z * inv, acc[i].w * inv));
    }
    if (p.lse && lane == 0)
        p.lse[((uint64_t)b * p.tokens + t) * p.q_heads + hq] = none ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <typename QT>
int launch_join(const Params& p, cudaStream_t s) {
    const uint64_t warps = (uint64_t)p.cache.sequences * p.cache.kv_heads * p.rows;
    const uint64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    UZIP_CUDA_TRY(cudaLaunchKernelEx(&cfg, join_kernel<QT>, p));
    return UZIP_OK;
}

// Rows of a (sequence, KV head) from which attention goes to the fifth-generation tensor cores: what the warp-level
// kernel takes at once ends at 32. Measured on 40 sequences of up to 16,384 tokens, 8 KV heads, pages of 16, warps /
// tensor cores: 32 rows, heads of 128 323 / 433 us, of 64 225 / 273; 40 rows 644 / 395 and 373 / 249 us (E5M2: 342 / 435
// and 236 / 345; 716 / 396 and 381 / 314).
constexpr uint32_t kManyRows = 33;

bool many(uint64_t rows, uint32_t head_dim) { return rows >= kManyRows && head_dim <= 128; }

// What attention and mass check alike.
int common(Params& p, const uzkv_rows_t* q, uint32_t dtype, uint32_t tokens, uint32_t q_heads, const int64_t* d_mask,
           int64_t mask_stride_b, const int32_t* d_counts, float scale, const uzkv_cache_t* cache) {
    if (int rc = cache_of(cache, &p.cache)) return rc;
    if (!rows_valid(q) || dtype > UZKV_FP16 || (cache->dtype != dtype && cache->dtype != UZKV_E5M2)) return UZIP_ERR_ARG;
    if (!tokens || tokens > UZKV_MAX_NEW_TOKENS || !q_heads || q_heads > 65535 || q_heads % cache->kv_heads) return UZIP_ERR_ARG;
    if (mask_stride_b < 0) return UZIP_ERR_ARG;
    p.q = rows_of(q, dtype, cache->sequences, tokens, q_heads);
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
    p.rows = tokens * p.group;
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
    const uint64_t rows = (uint64_t)tokens * (q_heads / kv_heads), m = many(rows, head_dim) ? (rows <= 128 ? 128 : 256) : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;  // at least a unit's rows
    const uint64_t dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    return (size_t)(kMaxAttGrid * 2 * m * (dp + 2) * 4);
}

extern "C" UZIP_API int uzkv_tree_attention(const uzkv_rows_t* q, const uzkv_rows_t* out, float* d_lse, uint32_t dtype,
                                            uint32_t tokens, uint32_t q_heads, const int64_t* d_mask,
                                            int64_t mask_stride_b, const int32_t* d_counts, float scale,
                                            const uzkv_cache_t* cache, void* d_workspace, size_t workspace_bytes,
                                            uzip_stream_t stream) {
    Params p{};
    if (int rc = common(p, q, dtype, tokens, q_heads, d_mask, mask_stride_b, d_counts, scale, cache)) return rc;
    if (!rows_valid(out) || !d_workspace) return UZIP_ERR_ARG;
    p.out = rows_of(out, dtype, cache->sequences, tokens, q_heads);
    if (!rows_aligned16(p.out) || !aligned16(d_workspace) || (reinterpret_cast<uintptr_t>(d_lse) & 3)) return UZIP_ERR_ALIGN;
    if (workspace_bytes < uzkv_tree_attention_workspace_bytes(p.cache.sequences, tokens, q_heads, p.cache.kv_heads, p.cache.head_dim))
        return UZIP_ERR_CAPACITY;
    // The join's grid: a warp a query row. Refused before anything is enqueued.
    if ((uint64_t)p.cache.sequences * p.cache.kv_heads * p.rows > 0x7FFFFFFFull) return UZIP_ERR_ARG;
    p.lse = d_lse;
    p.partial = static_cast<float*>(d_workspace);
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    using Launch = int (*)(AttParams&, const uzkv_cache_t*, int, cudaStream_t);
    static constexpr Launch kLaunch[2][2][2] = {  // [many rows][FP16][E5M2 cache]
        {{attend_bf16, attend_bf16_e5m2}, {attend_fp16, attend_fp16_e5m2}},
        {{attend_many_bf16, attend_many_bf16_e5m2}, {attend_many_fp16, attend_many_fp16_e5m2}}};
    if (int rc = kLaunch[many(p.rows, p.cache.head_dim)][dtype == UZKV_FP16][cache->dtype == UZKV_E5M2](p, cache, sms, s)) return rc;
    return dtype == UZKV_BF16 ? launch_join<__nv_bfloat16>(p, s) : launch_join<__half>(p, s);
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
    int sms = 0;
    if (int rc = sm_count(&sms)) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool fp8 = cache->dtype == UZKV_E5M2;
    if (dtype == UZKV_BF16) return fp8 ? mass_bf16_e5m2(p, cache, sms, s) : mass_bf16(p, cache, sms, s);
    return fp8 ? mass_fp16_e5m2(p, cache, sms, s) : mass_fp16(p, cache, sms, s);
}
