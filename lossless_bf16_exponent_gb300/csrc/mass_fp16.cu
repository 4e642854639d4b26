// mass_fp16.cu -- mass kernels of FP16 queries.
#include "kv_mass.cuh"

int uzkv::mass_fp16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return launch_mass<__half, false>(p, c, sms, s);
}
int uzkv::mass_fp16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return launch_mass<__half, true>(p, c, sms, s);
}
