// attend_fp16.cu -- attention kernels of FP16 queries over a cache of FP16.
#include "kv_attend.cuh"

int uzkv::attend_fp16(AttParams& p, const uzkv_cache_t*, int sms, cudaStream_t s) {
    return launch_attend<__half, false>(p, sms, s);
}
