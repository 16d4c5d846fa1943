// The fp16 instances of the wide 4-bit products (q4_wide.cuh).
#include "q4_wide.cuh"

bsp_status_t bsp_run_q4_wide_f16(const bspq4::Problem& p, cudaStream_t s) { return run_wide<__half>(p, s); }
