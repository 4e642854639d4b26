// kv_internal.cuh -- shared definitions of the KV-cache operators: the cache
// as kernels see it, element types, and the checks every entry point makes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "uzip_internal.cuh"
#include "uzip_kv.h"

namespace uzkv {

using uzip::aligned16;

struct E5M2 {
    uint8_t bits;
};

// E5M2 is the upper byte of an FP16 pattern, so it widens by a byte shift.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(E5M2 x) { return __half2float(__ushort_as_half((unsigned short)(x.bits << 8))); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
// Nearest even, infinity from 61440 on (halfway between the largest value and
// the next power of two), as an FP8 cache rounds; the conversion instruction
// alone would saturate.
template <>
__device__ __forceinline__ E5M2 from_f32<E5M2>(float x) {
    const uint32_t r = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E5M2);
    const uint32_t inf = 0x7Cu | ((__float_as_uint(x) >> 24) & 0x80u);
    return E5M2{(uint8_t)(fabsf(x) >= 61440.0f ? inf : r)};
}

// x / d for x < 2^32 by one 64-bit product: m = floor(2^64 / d) + 1.
struct Divisor {
    uint64_t m;
    uint32_t d;
    static Divisor of(uint32_t d) { return Divisor{d > 1 ? ~uint64_t(0) / d + 1 : 0, d}; }
    __device__ __forceinline__ uint32_t div(uint32_t x) const { return d > 1 ? (uint32_t)__umul64hi(x, m) : x; }
};

// A cache as kernels take it. Offsets are 64-bit: a pool may pass 2^32 elements.
struct Cache {
    char *k, *v;
    int64_t k_page, k_head, k_token, v_page, v_head, v_token;  // bytes
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lengths;
    uint32_t* status;
    Divisor page_tokens;
    uint32_t pages, kv_heads, head_dim, sequences, capacity;
};

struct Rows {
    char* p;
    int64_t b, t, h;  // bytes
};

__device__ __forceinline__ void corrupt(const Cache& c) {
    if (c.status) *c.status = UZIP_ERR_CORRUPT;
}

// Tokens of sequence b in the cache and new ones of the call, clamped to what is in bounds.
struct Span {
    uint32_t old, fresh;
};
__device__ __forceinline__ Span span_of(const Cache& c, const int32_t* counts, uint32_t tokens, uint32_t b) {
    const int32_t n = c.lengths[b], f = counts ? counts[b] : (int32_t)tokens;
    Span s;
    s.old = min((uint32_t)max(n, 0), c.capacity);
    s.fresh = min(min((uint32_t)max(f, 0), tokens), c.capacity - s.old);
    if ((int32_t)s.old != n || (int32_t)s.fresh != f) corrupt(c);
    return s;
}

// Page and row of slot j of sequence b; page < 0: there is no such page.
struct Place {
    int32_t page;
    uint32_t row;
};
// Looked up only: what looks ahead passes it through checked() where it is used, so that the load is not waited for
// before.
__device__ __forceinline__ Place look_up(const Cache& c, uint32_t b, uint32_t j) {
    const uint32_t q = c.page_tokens.div(j);
    return Place{c.table[b * c.table_stride + q], j - q * c.page_tokens.d};
}
__device__ __forceinline__ Place checked(const Cache& c, Place p) {
    if ((uint32_t)p.page >= c.pages) {
        corrupt(c);
        p.page = -1;
    }
    return p;
}
__device__ __forceinline__ Place place_of(const Cache& c, uint32_t b, uint32_t j) { return checked(c, look_up(c, b, j)); }
__device__ __forceinline__ char* k_row(const Cache& c, Place p, uint32_t h) {
    return c.k + p.page * c.k_page + h * c.k_head + p.row * c.k_token;
}
__device__ __forceinline__ char* v_row(const Cache& c, Place p, uint32_t h) {
    return c.v + p.page * c.v_page + h * c.v_head + p.row * c.v_token;
}

inline uint32_t bytes_of(uint32_t dtype) { return dtype == UZKV_FP32 ? 4 : dtype == UZKV_E5M2 ? 1 : 2; }

// The rows of b x t x h of them. A stride along a dimension of one is nothing: no alignment is asked of it.
inline Rows rows_of(const uzkv_rows_t* r, uint32_t dtype, uint32_t b, uint32_t t, uint32_t h) {
    const int64_t e = bytes_of(dtype);
    return Rows{static_cast<char*>(r->d), b > 1 ? r->stride_b * e : 0, t > 1 ? r->stride_t * e : 0, h > 1 ? r->stride_h * e : 0};
}

// Host checks of a cache; fills the kernels' form. cap is the width that must fit 31 bits.
inline int cache_of(const uzkv_cache_t* c, Cache* o) {
    if (!c || !c->d_k || !c->d_v || !c->d_lengths || !c->d_table) return UZIP_ERR_ARG;
    if (c->dtype != UZKV_BF16 && c->dtype != UZKV_FP16 && c->dtype != UZKV_E5M2) return UZIP_ERR_ARG;
    if (!c->pages || !c->kv_heads || !c->page_tokens || !c->sequences || !c->pages_per_sequence) return UZIP_ERR_ARG;
    const int64_t e = bytes_of(c->dtype);
    if (!c->head_dim || c->head_dim > UZKV_MAX_HEAD_DIM || c->head_dim * e % 16) return UZIP_ERR_ARG;
    const uint64_t cap = (uint64_t)c->page_tokens * c->pages_per_sequence;
    if (cap > 0x7FFFFF00ull || c->pages > 0x7FFFFFFFu || c->sequences > 65535 || c->kv_heads > 65535) return UZIP_ERR_ARG;
    if (c->table_stride < 0) return UZIP_ERR_ARG;
    int64_t st[6] = {c->k_page_stride, c->k_head_stride, c->k_token_stride,
                     c->v_page_stride, c->v_head_stride, c->v_token_stride};
    const uint32_t along[3] = {c->pages, c->kv_heads, c->page_tokens};
    for (int i = 0; i < 6; i++) {
        if (st[i] < 0) return UZIP_ERR_ARG;
        st[i] *= e;
        if (along[i % 3] == 1) st[i] = (st[i] + 15) / 16 * 16;  // along a dimension of one it only has to suit tensor maps
        if (st[i] % 16) return UZIP_ERR_ALIGN;
    }
    if (!aligned16(c->d_k) || !aligned16(c->d_v)) return UZIP_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(c->d_table) | reinterpret_cast<uintptr_t>(c->d_lengths) |
         reinterpret_cast<uintptr_t>(c->d_status)) & 3)
        return UZIP_ERR_ALIGN;
    o->k = static_cast<char*>(c->d_k);
    o->v = static_cast<char*>(c->d_v);
    o->k_page = st[0];
    o->k_head = st[1];
    o->k_token = st[2];
    o->v_page = st[3];
    o->v_head = st[4];
    o->v_token = st[5];
    o->table = c->d_table;
    o->table_stride = c->table_stride;
    o->lengths = c->d_lengths;
    o->status = c->d_status;
    o->page_tokens = Divisor::of(c->page_tokens);
    o->pages = c->pages;
    o->kv_heads = c->kv_heads;
    o->head_dim = c->head_dim;
    o->sequences = c->sequences;
    o->capacity = (uint32_t)cap;
    return UZIP_OK;
}

inline bool rows_valid(const uzkv_rows_t* r) { return r && r->d && r->stride_b >= 0 && r->stride_t >= 0 && r->stride_h >= 0; }

// Every row 16-byte aligned.
inline bool rows_aligned16(const Rows& r) { return aligned16(r.p) && (r.b | r.t | r.h) % 16 == 0; }

// SM count of the current device.
inline int sm_count(int* sms) {
    int dev = 0;
    UZIP_CUDA_TRY(cudaGetDevice(&dev));
    UZIP_CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
    return UZIP_OK;
}

}  // namespace uzkv
