// attend_many_bf16.cu -- attention kernels of many BF16 query rows.
#include "kv_attend_many.cuh"

int uzkv::attend_many_bf16(AttParams& p, int sms, cudaStream_t s) { return launch_many<__nv_bfloat16, false>(p, sms, s); }
int uzkv::attend_many_bf16_e5m2(AttParams& p, int sms, cudaStream_t s) { return launch_many<__nv_bfloat16, true>(p, sms, s); }
