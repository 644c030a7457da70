// rb_add_rms_norm for rows of bf16.
#include "rms_norm.cuh"

template rb_status rb::norm::run_norm<__nv_bfloat16>(const NormArgs&, bool, cudaStream_t);
