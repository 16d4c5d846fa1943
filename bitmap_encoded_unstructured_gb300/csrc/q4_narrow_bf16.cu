// The bf16 instances of the narrow 4-bit products (q4_narrow.cuh).
#include "q4_narrow.cuh"

bsp_status_t bsp_run_q4_narrow_bf16(const bspq4::Problem& p, cudaStream_t s) { return by_group<__nv_bfloat16>(p, s); }
