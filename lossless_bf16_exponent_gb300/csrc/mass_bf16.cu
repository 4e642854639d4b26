// mass_bf16.cu -- mass kernels of BF16 queries.
#include "kv_mass.cuh"

int uzkv::mass_bf16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return launch_mass<__nv_bfloat16, false>(p, c, sms, s);
}
int uzkv::mass_bf16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return launch_mass<__nv_bfloat16, true>(p, c, sms, s);
}
