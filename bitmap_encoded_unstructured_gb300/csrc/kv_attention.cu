// Attention of a step's new rows over the paged 8-bit cache.
//
// A cached value is code * scale with one scale for each page and KV head,
// so the scales stay out of the inner sums: q . k_j = s_k(page of j) *
// (q . codes_j), and p_j v_j = (p_j s_v(page of j)) codes_j.
#include "bsp_kv.cuh"

#include <algorithm>

namespace {

using namespace bspkv;

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

// One warp per (row, head): lane i takes token i of a run of 32, softmax
// statistics are the warp's, then lane i owns dims i, i + 32, ...
template <class T>
__global__ void __launch_bounds__(128) kv_attention_rows_kernel(const AttnArgs a)
{
    __shared__ __align__(16) float qs[4][256];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, dim = a.c.dim, sh = a.c.page_shift;
    const int64_t unit = (int64_t)blockIdx.x * 4 + w;
    if (unit >= a.s.rows * a.heads) return;
    const int row = (int)(unit / a.heads), head = (int)(unit % a.heads), kvh = head / a.group;
    int lo = 0, hi = a.s.batch;
    while (hi - lo > 1) {  // the request of the row
        const int mid = (lo + hi) >> 1;
        if (a.s.q_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    int pos = -1;
    if (a.s.batch) {
        const Request r = request_of(a.s, sh, lo);
        if (row >= r.r0 && row < r.r0 + r.n) pos = r.len - r.n + row - r.r0;
    }
    const T* q = (const T*)a.q + row * a.q_row + head * a.q_head;
    for (int d = lane; d < dim; d += 32) qs[w][d] = to_float(q[d]) * a.scale;
    __syncwarp();
    const int first = a.window ? max(0, pos - a.window + 1) : 0;
    float m = -INFINITY, l = 0.f, o[8] = {};
    for (int j0 = first; j0 <= pos; j0 += 32) {
        const int j = j0 + lane;
        int p = -1;
        float x = -INFINITY, vs = 0.f;
        if (j <= pos) {
            p = a.s.table[(int64_t)lo * a.s.table_stride + (j >> sh)];
            if (p >= a.c.pages) p = -1;
        }
        const int64_t at = (int64_t)(p < 0 ? 0 : p) * a.c.page_stride + (int64_t)kvh * a.c.head_stride +
                           (int64_t)(j & ((1 << sh) - 1)) * a.c.row_stride;
        if (p >= 0) {
            float sum = 0.f;
            for (int d = 0; d < dim; d += 16) {
                const int4 raw = *reinterpret_cast<const int4*>(a.c.k + at + d);
                const int8_t* e = reinterpret_cast<const int8_t*>(&raw);
#pragma unroll
                for (int c = 0; c < 16; ++c) sum += qs[w][d + c] * (float)e[c];
            }
            x = sum * a.c.k_scale[(int64_t)p * a.c.scale_stride + kvh];
            vs = a.c.v_scale[(int64_t)p * a.c.scale_stride + kvh];
        }
        float top = x;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        top = fmaxf(top, m);
        if (top == -INFINITY) continue;  // nothing seen yet
        const float back = __expf(m - top), e = p >= 0 ? __expf(x - top) : 0.f;
        m = top;
        float sum = e;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        l = l * back + sum;
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] *= back;
        const float pv = e * vs;
        for (int t = 0; t < 32; ++t) {
            const float f = __shfl_sync(0xFFFFFFFFu, pv, t);
            const int64_t vat = __shfl_sync(0xFFFFFFFFu, at, t);
            if (__shfl_sync(0xFFFFFFFFu, p, t) < 0) continue;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (lane + 32 * c < dim) o[c] += f * (float)a.c.v[vat + lane + 32 * c];
        }
    }
    T* out = (T*)a.out + row * a.o_row + head * a.o_head;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (lane + 32 * c < dim) out[lane + 32 * c] = from_float<T>(l > 0.f ? o[c] / l : 0.f);
    if (a.lse && lane == 0) a.lse[(int64_t)row * a.heads + head] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

bsp_status_t bsp_run_kv_attention(const bsp_kv* h, const KvStepView& st, int64_t max_new, const void* q,
                                  bsp_dtype_t dtype, int32_t heads, int64_t q_row, int64_t q_head, float scale,
                                  int32_t window, void* out, int64_t o_row, int64_t o_head, float* lse,
                                  cudaStream_t s)
{
    (void)max_new;
    const AttnArgs a = {h->view, st, q, out, lse, q_row, q_head, o_row, o_head, scale, heads, heads / h->view.heads,
                        window};
    const int64_t grid = (st.rows * heads + 3) / 4;
    if (grid > 0x7FFFFFFF) return BSP_ERR_INVALID_ARG;
    if (dtype == BSP_FP16) kv_attention_rows_kernel<__half><<<(unsigned)grid, 128, 0, s>>>(a);
    else kv_attention_rows_kernel<__nv_bfloat16><<<(unsigned)grid, 128, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}
