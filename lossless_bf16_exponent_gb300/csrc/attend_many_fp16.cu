// attend_many_fp16.cu -- attention kernels of many FP16 query rows.
#include "kv_attend_many.cuh"

int uzkv::attend_many_fp16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return launch_many<__half, false>(p, c, sms, s);
}
int uzkv::attend_many_fp16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return launch_many<__half, true>(p, c, sms, s);
}
