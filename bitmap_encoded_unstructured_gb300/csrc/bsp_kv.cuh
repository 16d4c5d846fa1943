// Internal declarations of the paged 8-bit KV cache (kv_cache.cu,
// kv_attention.cu): the handle, the device view of the caller's arrays and
// the searches that map work items to requests.
#pragma once

#include "bsp_internal.cuh"
#include "bsp_ptx.cuh"

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

// A segment (request, KV head, group of query rows) whose cached rows were
// shared by warps from its own index to `last`, `per_cta` to a CTA.
struct KvCut {
    int32_t last, per_cta;
    int32_t r0, n, h, rg;  // the request's first row and new rows, KV head, group
    int32_t pad[2];
};

struct bsp_kv {
    uint32_t magic;
    int device, num_sms;
    KvView view;
    // the codes as 4-D tensors {dim, row, head, page}: boxes of up to 32
    // rows of a page by 64 or 128 dims, swizzled by their width (kv_decode)
    CUtensorMap map_k, map_v;
    int* ticket;  // arrivals of a plan whose count is updated in place; zero between calls
    int* ready;   // 1 while the prompt kernel of an attention call runs, 0 between calls
    int* err;     // as bsp_handle::err
    // few queries: parts of segments cut between warps, two slots a warp, and
    // the cut segments by the warp that begins them (last = -1: none)
    float* parts;
    size_t part_floats;
    KvCut* cuts;
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

// Rows of a call and rows a block table row can name: positions, and their
// differences to a window, stay in 32 bits.
constexpr int64_t MOST_ROWS = (int64_t)1 << 30;
// Launch a kernel that may be set up while the kernel before it in the
// stream ends (programmatic dependent launch).  It calls wait_prior_grids()
// before it touches global memory, so nothing but the launch overlaps.
template <class... P, class... A>
bool launch_early(void (*kernel)(P...), dim3 grid, dim3 block, int smem, cudaStream_t s, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess;
}

// Checks of a step, before any CUDA call.
bsp_status_t check_step(const bsp_kv_step_t* st, int64_t rows, int page_shift);
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

struct AttnArgs {
    KvView c;
    KvStepView s;
    const void* q;
    void* out;
    float* lse;
    int64_t q_row, q_head, o_row, o_head;
    float scale;
    int32_t heads, group, window;
};

// Softmax statistics, in powers of two.  A row keeps the largest logit seen
// (m), the largest logit + log2(V scale) seen (mw), l = sum of 2^(x - m) and
// O = sum of 2^(x - mw) * V scale * codes; both maxima may lag, so that the
// sums are rescaled a few times a row, not at every tile.  Two maxima,
// because the weights 2^(x - mw) * V scale go through fp16: they stay in its
// range whatever the V scales are.
constexpr float NONE = -1e30f;           // running maximum before any row is seen
constexpr float LAZY = 8.f;              // a maximum may lag by 2^8 before sums are rescaled
constexpr float DEEP = 120.f;            // mw is not held further below m: 2^(m - mw) stays finite
constexpr float LIFT = 64.f;             // weights are held 2^6 up, away from fp16's subnormals

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What p is multiplied by for its weight: 2^(m - mw) (lifted) times the V scale.
// Rows that are not seen, or far below the maximum, have p = 0 and any scale:
// the product stays finite for them, so that the weight is 0.  (A NaN stays one.)
__device__ __forceinline__ float weight_of(float lift, float v_scale)
{
    float y;
    asm("min.NaN.f32 %0, %1, 0f7F7FFFFF;" : "=f"(y) : "f"(lift * v_scale));
    return y;
}

__device__ __forceinline__ uint32_t h2bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Two fp16 from bytes of w (already offset by 128) picked by sel.
__device__ __forceinline__ uint32_t widen(uint32_t w, uint32_t sel)
{
    const uint32_t h = __byte_perm(w, 0x64646464u, sel);
    return h2bits(__hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480))));
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(bspx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bspx::smem_u32(bar))
        : "memory");
}

// Wait until the grids this one depends on (programmatic dependent launch)
// have completed and their memory is visible; returns at once otherwise.
__device__ __forceinline__ void wait_prior_grids() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Encode the tensor maps and allocate the decode scratch of a new handle.
bsp_status_t attention_setup(bsp_kv* h, cudaStream_t s);
void attention_free(bsp_kv* h);

}  // namespace bspkv

// Attention of the requests with more than `few` query rows per KV head
// (kv_prompt.cu); dim <= 128.  `beside`: the kernel launched next may start
// while this one runs, see bsp_kv::ready; otherwise it starts behind it.
bsp_status_t bsp_run_kv_prompt(const bsp_kv* h, const bspkv::AttnArgs& a, bsp_dtype_t dtype, int32_t few, bool* beside,
                               cudaStream_t s);

bsp_status_t bsp_run_kv_attention(const bsp_kv* h, const KvStepView& st, int64_t max_new, const void* q,
                                  bsp_dtype_t dtype, int32_t heads, int64_t q_row, int64_t q_head, float scale,
                                  int32_t window, void* out, int64_t o_row, int64_t o_head, float* lse,
                                  cudaStream_t s);
