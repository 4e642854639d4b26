// kv_maps.cu -- tensor maps of a cache's pools (kv_tma.cuh).
#include <algorithm>

#include "kv_tma.cuh"

namespace uzkv {
namespace {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once; null where it has none.
Encode encoder() {
    static const Encode found = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &how) != cudaSuccess) {
            cudaGetLastError();  // clear the error
            return (Encode) nullptr;
        }
        return how == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(fn) : (Encode) nullptr;
    }();
    return found;
}

}  // namespace

bool maps_of(const AttParams& p, const uzkv_cache_t* c, uint32_t tile, uint32_t least, Maps* m) {
    const uint32_t box = std::min(c->page_tokens & (0u - c->page_tokens), tile);  // largest power of two in both
    const uint32_t row = c->head_dim * bytes_of(c->dtype), wide = c->dtype == UZKV_E5M2 && c->head_dim <= 64 ? 64 : 128;
    if (box < 8 || box * wide < least || !encoder()) return false;
    m->box = box;
    const cuuint64_t dims[4] = {row, c->page_tokens, c->kv_heads, c->pages};
    const cuuint32_t boxes[4] = {wide, box, 1, 1}, steps[4] = {1, 1, 1, 1};
    for (int v = 0; v < 2; v++) {
        const cuuint64_t strides[3] = {(cuuint64_t)(v ? p.cache.v_token : p.cache.k_token), (cuuint64_t)(v ? p.cache.v_head : p.cache.k_head),
                                       (cuuint64_t)(v ? p.cache.v_page : p.cache.k_page)};
        if (encoder()(v ? &m->v : &m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, v ? p.cache.v : p.cache.k, dims, strides, boxes, steps,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, wide == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    return true;
}

}  // namespace uzkv
