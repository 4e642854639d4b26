// attend_bf16.cu -- attention kernels of BF16 queries over a cache of BF16.
#include "kv_attend.cuh"

int uzkv::attend_bf16(AttParams& p, const uzkv_cache_t*, int sms, cudaStream_t s) {
    return launch_attend<__nv_bfloat16, false>(p, sms, s);
}
