// attend_bf16_e5m2.cu -- attention kernels of BF16 queries over a cache of E5M2.
#include "kv_attend.cuh"

int uzkv::attend_bf16_e5m2(AttParams& p, const uzkv_cache_t*, int sms, cudaStream_t s) {
    return launch_attend<__nv_bfloat16, true>(p, sms, s);
}
