// rb_add_rms_norm for rows of fp32.
#include "rms_norm.cuh"

template rb_status rb::norm::run_norm<float>(const NormArgs&, bool, cudaStream_t);
