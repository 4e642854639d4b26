// attend_many_bf16.cu -- attention kernels of many BF16 query rows.
#include "kv_attend_many.cuh"

int uzkv::attend_many_bf16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return launch_many<__nv_bfloat16, false>(p, c, sms, s);
}
int uzkv::attend_many_bf16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return launch_many<__nv_bfloat16, true>(p, c, sms, s);
}
