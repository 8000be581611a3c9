// msa_attend_scaled.cu -- the attend kernels for a cache with page scales
// (launch_attend_scaled).
#define MSA_KV_SCALES 1
#include "msa_attend.cu"
