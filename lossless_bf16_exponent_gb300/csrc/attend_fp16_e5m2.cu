// attend_fp16_e5m2.cu -- attention kernels of FP16 queries over a cache of E5M2.
#include "kv_attend.cuh"

int uzkv::attend_fp16_e5m2(AttParams& p, const uzkv_cache_t*, int sms, cudaStream_t s) {
    return launch_attend<__half, true>(p, sms, s);
}
