// msa_union_scaled.cu -- the union attend and dense decode for a cache with page
// scales (launch_union_attend_scaled).
#define MSA_KV_SCALES 1
#include "msa_union.cu"
