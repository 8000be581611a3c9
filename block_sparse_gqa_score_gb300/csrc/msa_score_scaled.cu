// msa_score_scaled.cu -- the scorer for a cache with page scales
// (launch_score_scaled).
#define MSA_KV_SCALES 1
#include "msa_score.cu"
