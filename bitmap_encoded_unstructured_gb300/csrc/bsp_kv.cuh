// Internal declarations of the paged 8-bit KV cache (kv_cache.cu,
// kv_attention.cu): the handle, the device view of the caller's arrays and
// the searches that map work items to requests.
#pragma once

#include "bsp_internal.cuh"

#include <cuda.h>
#include <cuda_bf16.h>

#define BSP_KV_MAGIC 0xB5B1CAC8u

// What the kernels read of a bsp_kv_desc_t.
struct KvView {
    int8_t *k, *v;
    float *k_scale, *v_scale;
    int32_t pages, heads, page_shift, dim;
    int64_t page_stride, head_stride, row_stride, scale_stride;
};

// What they read of a bsp_kv_step_t, and the rows of the call's tensors.
struct KvStepView {
    const int32_t *table, *seq_len, *q_start;
    int64_t table_stride;
    int32_t batch, width;
    int64_t rows;
};

struct bsp_kv {
    uint32_t magic;
    int device, num_sms;
    KvView view;
    // the codes as 4-D tensors {dim, row, head, page}: boxes of up to 32
    // rows of a page by 64 or 128 dims, swizzled by their width (kv_decode)
    CUtensorMap map_k, map_v;
    int* ticket;  // arrivals of a plan whose count is updated in place; zero between calls
    int* err;     // as bsp_handle::err
    // decode: partial results of segments split between CTAs, two slots a
    // CTA, and the arrivals of each split segment (zero between calls)
    float* parts;
    int* arrivals;
    int decode_ctas;
};

namespace bspkv {

inline bool valid(const bsp_kv* h) { return h != nullptr && h->magic == BSP_KV_MAGIC; }
inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Run on the handle's device, restoring the caller's current device after.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

// Checks of a step and of the row tensors' strides, before any CUDA call.
bsp_status_t check_step(const bsp_kv_step_t* st, int64_t rows);
KvStepView view_of(const bsp_kv_step_t* st, int64_t rows);

// The request's lengths, held inside its block table row and the call's
// rows whatever the arrays say: n new rows from row r0 on, the last of them
// at position len - 1 (rows at negative positions see and store nothing).
struct Request {
    int32_t r0, n, len;
};

__device__ __forceinline__ Request request_of(const KvStepView& s, int page_shift, int b)
{
    Request r;
    const int64_t lo = s.q_start[b], hi = s.q_start[b + 1];
    const int64_t len = s.seq_len[b], room = (int64_t)s.width << page_shift;
    r.r0 = (int32_t)(lo < 0 ? 0 : lo);
    r.len = (int32_t)(len < 0 ? 0 : (len > room ? room : len));
    const int64_t n = (hi < s.rows ? hi : s.rows) - r.r0;
    r.n = (int32_t)(n < 0 ? 0 : n);
    return r;
}

template <class T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

// Encode the tensor maps and allocate the decode scratch of a new handle.
bsp_status_t attention_setup(bsp_kv* h, cudaStream_t s);
void attention_free(bsp_kv* h);

}  // namespace bspkv

bsp_status_t bsp_run_kv_attention(const bsp_kv* h, const KvStepView& st, int64_t max_new, const void* q,
                                  bsp_dtype_t dtype, int32_t heads, int64_t q_row, int64_t q_head, float scale,
                                  int32_t window, void* out, int64_t o_row, int64_t o_head, float* lse,
                                  cudaStream_t s);
