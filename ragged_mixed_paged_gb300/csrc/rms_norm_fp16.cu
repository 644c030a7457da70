// rb_add_rms_norm for rows of fp16.
#include "rms_norm.cuh"

template rb_status rb::norm::run_norm<__half>(const NormArgs&, bool, cudaStream_t);
