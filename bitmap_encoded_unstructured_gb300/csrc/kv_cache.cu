// Paged 8-bit KV cache: the handle, the plan of a step (pages, slots), the
// quantising append and the read-back.  The attention is in
// kv_attention.cu.
#include "bsp_kv.cuh"

#include <algorithm>
#include <climits>
#include <new>

namespace {

using namespace bspkv;

// ------------------------------------------------------------------- plan

struct PlanArgs {
    const int32_t *ctx_len, *new_len, *free_count;
    int32_t *table, *free_list, *seq_len, *q_start, *granted, *positions, *free_count_out;
    int64_t* slots;
    int64_t table_stride;
    int32_t batch, width, capacity, tokens, page_shift;
    int* ticket;  // null: free_count_out is another word than free_count
};

constexpr int PLAN_THREADS = 512;

// Sum of two counts >= 0, held at INT_MAX (associative, so a scan may use
// it): lengths that no page table could hold then simply do not fit.
__device__ __forceinline__ int sat_add(int a, int b)
{
    return (int)min((unsigned)a + (unsigned)b, (unsigned)INT_MAX);
}

struct Ask {
    int ctx, have, rows, pages, back;  // cached rows, their pages; rows and pages asked for; pages given back
};

__device__ __forceinline__ Ask ask_of(const PlanArgs& a, int b)
{
    Ask r;
    const int64_t room = (int64_t)a.width << a.page_shift;
    const int64_t mask = ((int64_t)1 << a.page_shift) - 1;
    const int64_t ctx = min(max((int64_t)a.ctx_len[b], (int64_t)0), room);
    const int n = a.new_len[b];
    const int64_t rows = n > 0 && ctx + n <= room ? n : 0;
    r.ctx = (int)ctx;
    r.have = (int)((ctx + mask) >> a.page_shift);
    r.rows = (int)rows;
    r.pages = n < 0 ? 0 : (int)((ctx + rows + mask) >> a.page_shift) - r.have;
    r.back = n < 0 ? r.have : 0;
    return r;
}

// The request that holds item x of a rising prefix P[0..n]: the b < n with
// P[b] <= x < P[b + 1].
__device__ __forceinline__ int holder(const int* P, int n, int x)
{
    int lo = 0, hi = n;  // P[lo] <= x < P[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (P[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Every CTA scans the whole batch (three sums, in shared memory) and then
// takes its share of the requests, granted pages, returned pages and rows:
// no CTA waits for another, and one launch does it all.  Granted pages that
// are being returned in the same step are read from the returning request's
// block table row, which nobody writes, not from the stack.
__global__ void __launch_bounds__(PLAN_THREADS) kv_plan_kernel(const PlanArgs a)
{
    extern __shared__ int sm[];
    const int B = a.batch, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* rows = sm;              // [B + 1] rows asked for before request b
    int* pages = rows + B + 1;   // [B + 1] pages asked for
    int* back = pages + B + 1;   // [B + 1] pages given back
    __shared__ int part[3][PLAN_THREADS / 32];
    int carry[3] = {0, 0, 0};
    if (tid == 0) rows[0] = pages[0] = back[0] = 0;
    for (int base = 0; base < B; base += PLAN_THREADS) {
        const int b = base + tid;
        int v[3] = {0, 0, 0};
        if (b < B) {
            const Ask r = ask_of(a, b);
            v[0] = r.rows;
            v[1] = r.pages;
            v[2] = r.back;
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, v[i], d);
                if (lane >= d) v[i] = sat_add(v[i], o);
            }
            if (lane == 31) part[i][warp] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            int before = carry[i];
            for (int w = 0; w < PLAN_THREADS / 32; ++w) {
                if (w < warp) before = sat_add(before, part[i][w]);
                carry[i] = sat_add(carry[i], part[i][w]);
            }
            if (b < B) (i == 0 ? rows : i == 1 ? pages : back)[b + 1] = sat_add(before, v[i]);
        }
        __syncthreads();
    }
    __syncthreads();
    const int live = min(max(*a.free_count, 0), a.capacity);
    const int avail = sat_add(live, back[B]);
    // requests 0 .. G-1 are granted what they ask for
    int G = 0;
    for (int lo = 0, hi = B; lo < hi;) {
        const int mid = (lo + hi) >> 1;
        if (pages[mid + 1] <= avail && rows[mid + 1] <= a.tokens) lo = mid + 1;
        else hi = mid;
        G = lo;
    }
    const int granted_pages = pages[G], granted_rows = rows[G];
    const int left = min(avail - granted_pages, a.capacity);
    const int mask = (1 << a.page_shift) - 1;
    const int first = blockIdx.x * PLAN_THREADS + tid, step = gridDim.x * PLAN_THREADS;

    auto returned = [&](int i) {  // the i-th page given back
        const int b = holder(back, B, i);
        return a.table[(int64_t)b * a.table_stride + (i - back[b])];
    };
    auto granted_page = [&](int i) {  // the i-th page taken off the stack
        const int at = avail - 1 - i;
        return at < live ? a.free_list[at] : returned(at - live);
    };
    for (int b = first; b < B; b += step) {
        const Ask r = ask_of(a, b);
        const int n = b < G ? r.rows : 0;
        a.granted[b] = n;
        a.seq_len[b] = a.new_len[b] < 0 ? 0 : r.ctx + n;
        a.q_start[b] = rows[min(b, G)];
    }
    if (first == 0) a.q_start[B] = granted_rows;
    for (int i = first; i < granted_pages; i += step) {
        const int b = holder(pages, G, i);
        const int ctx = ask_of(a, b).have;
        a.table[(int64_t)b * a.table_stride + ctx + (i - pages[b])] = granted_page(i);
    }
    for (int64_t i = (int64_t)live + first; i < left; i += step) a.free_list[i] = returned((int)i - live);
    for (int64_t t = first; t < a.tokens; t += step) {
        int64_t slot = -1;
        int pos = -1;
        if (t < granted_rows) {
            const int b = holder(rows, G, (int)t);
            const Ask r = ask_of(a, b);
            pos = r.ctx + ((int)t - rows[b]);
            const int j = pos >> a.page_shift;
            const int p = j < r.have ? a.table[(int64_t)b * a.table_stride + j] : granted_page(pages[b] + j - r.have);
            slot = p < 0 ? -1 : ((int64_t)p << a.page_shift) + (pos & mask);
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
    if (!a.ticket) {
        if (first == 0) *a.free_count_out = left;
    } else {  // updated in place: by the last CTA, when every one has read it
        __syncthreads();
        if (tid == 0 && atomicAdd(a.ticket, 1) == (int)gridDim.x - 1) {
            *a.ticket = 0;
            *a.free_count_out = left;
        }
    }
}

// ----------------------------------------------------------------- append

struct AppendArgs {
    KvView c;
    KvStepView s;
    const void *k, *v;
    int64_t k_row, k_head, v_row, v_head;
};

// Work items of a step, one per page that receives rows.  Request b's items
// start at F(b) = q_start[b] / page + 2 b: it touches at most n / page + 2
// pages, so F leaves room for them without a scan of the batch; items past a
// request's last page have nothing to do.
__device__ __forceinline__ int item_request(const KvStepView& s, int page_shift, int item)
{
    int lo = 0, hi = s.batch;  // F(lo) <= item < F(hi), or hi = batch
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((s.q_start[mid] >> page_shift) + 2 * mid <= item) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One warp per (page that receives rows, head, K or V).
template <class T>
__global__ void __launch_bounds__(128) kv_append_kernel(const AppendArgs a)
{
    const int unit = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (unit >= 2 * a.c.heads) return;
    const int head = unit >> 1, sh = a.c.page_shift, page = 1 << sh;
    const bool is_v = unit & 1;
    const int b = item_request(a.s, sh, blockIdx.x);
    const Request r = request_of(a.s, sh, b);
    const int start = r.len - r.n, from = max(start, 0);  // position of the first new row; of the first stored
    const int64_t jj = (from >> sh) + (int64_t)blockIdx.x - ((a.s.q_start[b] >> sh) + 2 * (int64_t)b);
    if (jj < (from >> sh) || jj << sh >= r.len) return;
    const int j = (int)jj;
    const int lo = max(from, j << sh), hi = (int)min((int64_t)r.len, (jj + 1) << sh);  // new rows of this page
    if (lo >= hi) return;
    const int p = a.s.table[(int64_t)b * a.s.table_stride + j];
    if (p < 0 || p >= a.c.pages) return;
    const int vecs = a.c.dim / 8;                        // 16-byte vectors of a row
    const int64_t row_step = is_v ? a.v_row : a.k_row;
    const T* x = (const T*)(is_v ? a.v : a.k) + (int64_t)(r.r0 + lo - start) * row_step +
                 (int64_t)head * (is_v ? a.v_head : a.k_head);
    int8_t* codes = (is_v ? a.c.v : a.c.k) + (int64_t)p * a.c.page_stride + (int64_t)head * a.c.head_stride;
    float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + (int64_t)p * a.c.scale_stride + head;
    const int total = (hi - lo) * vecs;

    float top = 0.f;
    for (int i = lane; i < total; i += 32) {
        const uint4 raw = *reinterpret_cast<const uint4*>(x + (i / vecs) * row_step + (i % vecs) * 8);
        const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float f = fabsf(to_float(e[c]));
            if (f < INFINITY) top = fmaxf(top, f);       // false for NaN and infinities
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const int kept = lo & (page - 1);                    // earlier rows of the page
    const float old = kept ? *scale : 0.f;
    const float now = fmaxf(old, __fdiv_rn(top, 127.f));
    if (kept && now != old) {
        const float ratio = now > 0.f ? __fdiv_rn(old, now) : 0.f;
        for (int i = lane; i < kept * (a.c.dim / 16); i += 32) {
            int4* at = reinterpret_cast<int4*>(codes + (i / (a.c.dim / 16)) * a.c.row_stride + (i % (a.c.dim / 16)) * 16);
            int4 w = *at;
            int8_t* e = reinterpret_cast<int8_t*>(&w);
#pragma unroll
            for (int c = 0; c < 16; ++c) e[c] = (int8_t)__float2int_rn(__fmul_rn((float)e[c], ratio));
            *at = w;
        }
    }
    for (int i = lane; i < total; i += 32) {
        const uint4 raw = *reinterpret_cast<const uint4*>(x + (i / vecs) * row_step + (i % vecs) * 8);
        const T* e = reinterpret_cast<const T*>(&raw);
        alignas(8) int8_t q[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float f = to_float(e[c]);
            // NaN converts to 0; infinities meet the clamp
            const float t = now > 0.f ? __fdiv_rn(f, now) : 0.f;
            q[c] = (int8_t)(t != t ? 0 : __float2int_rn(fminf(fmaxf(t, -127.f), 127.f)));
        }
        *reinterpret_cast<int2*>(codes + ((lo & (page - 1)) + i / vecs) * a.c.row_stride + (i % vecs) * 8) =
            *reinterpret_cast<const int2*>(q);
    }
    __syncwarp();
    if (lane == 0) *scale = now;
}

// ------------------------------------------------------------------- read

struct ReadArgs {
    KvView c;
    const int64_t* slots;
    void *k, *v;
    int64_t n;
};

// One thread per 16 codes of a row, K and V by blockIdx.y.
template <class T>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadArgs a)
{
    const int per = a.c.dim / 16;                        // threads of a row
    const int64_t all = a.n * a.c.heads * per;
    const int8_t* codes = blockIdx.y ? a.c.v : a.c.k;
    const float* scales = blockIdx.y ? a.c.v_scale : a.c.k_scale;
    T* out = (T*)(blockIdx.y ? a.v : a.k);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int part = (int)(i - row * per), head = (int)(row % a.c.heads);
        const int64_t slot = a.slots[row / a.c.heads], p = slot >> a.c.page_shift;
        alignas(16) T o[16];
        if (slot >= 0 && p < a.c.pages) {
            const int64_t off = slot - (p << a.c.page_shift);
            const int4 w = *reinterpret_cast<const int4*>(codes + p * a.c.page_stride + head * a.c.head_stride +
                                                          off * a.c.row_stride + part * 16);
            const float s = scales[p * a.c.scale_stride + head];
            const int8_t* e = reinterpret_cast<const int8_t*>(&w);
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = from_float<T>((float)e[c] * s);
        } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = from_float<T>(0.f);
        }
        uint4* to = reinterpret_cast<uint4*>(out + i * 16);
        to[0] = reinterpret_cast<const uint4*>(o)[0];
        to[1] = reinterpret_cast<const uint4*>(o)[1];
    }
}

void free_kv(bsp_kv* h)
{
    if (!h) return;
    attention_free(h);
    cudaFree(h->ticket);
    cudaFree(h->err);
    h->magic = 0;
    delete h;
}

bool good_strides(int64_t row, int64_t head, int32_t dim, int64_t rows, int32_t heads)
{
    return (row % 8) == 0 && (head % 8) == 0 && (rows < 2 || row >= 0) && (heads < 2 || head >= dim);
}

}  // namespace

namespace bspkv {

bsp_status_t check_step(const bsp_kv_step_t* st, int64_t rows, int page_shift)
{
    if (!st || rows < 0 || rows > MOST_ROWS) return BSP_ERR_INVALID_ARG;
    if (st->batch < 0 || st->batch > BSP_KV_MAX_BATCH || st->max_new < 0) return BSP_ERR_INVALID_ARG;
    if (st->batch && (!st->block_table || !st->seq_len || !st->q_start)) return BSP_ERR_INVALID_ARG;
    if (st->batch && (st->width < 1 || st->table_stride < st->width ||
                      (int64_t)st->width << page_shift > MOST_ROWS))
        return BSP_ERR_SHAPE;
    return BSP_OK;
}

KvStepView view_of(const bsp_kv_step_t* st, int64_t rows)
{
    return {st->block_table, st->seq_len, st->q_start, st->table_stride, st->batch, st->width, rows};
}

}  // namespace bspkv

extern "C" {

bsp_status_t bsp_kv_create(const bsp_kv_desc_t* d, bsp_stream_t stream, bsp_kv_t* out)
{
    if (!out) return BSP_ERR_INVALID_ARG;
    *out = nullptr;
    if (!d || !d->k || !d->v || !d->k_scale || !d->v_scale) return BSP_ERR_INVALID_ARG;
    int shift = 4;
    while (shift < 8 && (1 << shift) != d->page) ++shift;
    if ((1 << shift) != d->page || d->pages < 1 || d->pages > INT32_MAX || d->heads < 1 || d->heads > 32767 ||
        d->dim < 16 || d->dim > 256 || d->dim % 16)
        return BSP_ERR_SHAPE;
    if (d->row_stride < d->dim || d->row_stride % 16 || d->head_stride < 0 || d->head_stride % 16 ||
        d->page_stride < 0 || d->page_stride % 16 || (d->heads > 1 && d->head_stride < d->dim) ||
        (d->pages > 1 && (d->page_stride < d->dim || d->scale_stride < d->heads)))
        return BSP_ERR_SHAPE;
    if (!aligned(d->k, 16) || !aligned(d->v, 16) || !aligned(d->k_scale, 4) || !aligned(d->v_scale, 4))
        return BSP_ERR_ALIGN;
    bsp_kv* h = new (std::nothrow) bsp_kv{};
    if (!h) return BSP_ERR_OOM;
    h->magic = BSP_KV_MAGIC;
    h->view = {d->k, d->v, d->k_scale, d->v_scale, (int32_t)d->pages, d->heads, shift, d->dim,
               d->page_stride, d->head_stride, d->row_stride, d->scale_stride};
    cudaStream_t s = (cudaStream_t)stream;
    bsp_status_t st = BSP_OK;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess)
        st = BSP_ERR_CUDA;
    else if (cudaMalloc(&h->ticket, sizeof(int)) != cudaSuccess || cudaMalloc(&h->err, sizeof(int)) != cudaSuccess)
        st = BSP_ERR_OOM;
    else if (cudaMemsetAsync(h->ticket, 0, sizeof(int), s) != cudaSuccess ||
             cudaMemsetAsync(h->err, 0, sizeof(int), s) != cudaSuccess)
        st = BSP_ERR_CUDA;
    else
        st = attention_setup(h, s);
    if (st == BSP_OK && cudaStreamSynchronize(s) != cudaSuccess) st = BSP_ERR_CUDA;
    if (st != BSP_OK) {
        free_kv(h);
        return st;
    }
    *out = h;
    return BSP_OK;
}

bsp_status_t bsp_kv_destroy(bsp_kv_t h)
{
    if (!valid(h)) return BSP_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    cudaDeviceSynchronize();
    free_kv(h);
    return BSP_OK;
}

bsp_status_t bsp_kv_check(bsp_kv_t h, bsp_stream_t stream)
{
    if (!valid(h)) return BSP_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    int e = 0;
    if (cudaMemcpyAsync(&e, h->err, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemsetAsync(h->err, 0, sizeof(int), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
        return BSP_ERR_CUDA;
    return e ? (bsp_status_t)e : BSP_OK;
}

bsp_status_t bsp_kv_plan(bsp_kv_t h, const int32_t* ctx_len, const int32_t* new_len, int32_t batch,
                         int32_t* block_table, int32_t width, int64_t table_stride, int32_t* free_list,
                         int32_t free_capacity, const int32_t* free_count, int64_t tokens, int32_t* seq_len,
                         int32_t* q_start, int32_t* granted, int64_t* slots, int32_t* positions,
                         int32_t* free_count_out, bsp_stream_t stream)
{
    if (!valid(h) || !free_count || !free_count_out || !q_start) return BSP_ERR_INVALID_ARG;
    if (batch < 0 || batch > BSP_KV_MAX_BATCH || free_capacity < 0 || tokens < 0 || tokens > INT32_MAX)
        return BSP_ERR_INVALID_ARG;
    if (batch && (!ctx_len || !new_len || !block_table || !seq_len || !granted)) return BSP_ERR_INVALID_ARG;
    if ((free_capacity && !free_list) || (tokens && (!slots || !positions))) return BSP_ERR_INVALID_ARG;
    if (batch && (width < 1 || table_stride < width)) return BSP_ERR_SHAPE;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    static bsp_attr_once attr_once;
    const int smem_most = 3 * (BSP_KV_MAX_BATCH + 1) * (int)sizeof(int);
    if (!attr_once.run(h->device, [&] {
            return cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_most);
        }))
        return BSP_ERR_CUDA;
    const PlanArgs a = {ctx_len, new_len, free_count, block_table, free_list, seq_len, q_start, granted, positions,
                        free_count_out, slots, table_stride, batch, width, free_capacity, (int32_t)tokens,
                        h->view.page_shift, free_count == free_count_out ? h->ticket : nullptr};
    const int64_t want = (std::max<int64_t>(tokens, batch) + PLAN_THREADS - 1) / PLAN_THREADS;
    const int grid = (int)std::clamp<int64_t>(want, 1, h->num_sms);
    kv_plan_kernel<<<grid, PLAN_THREADS, 3 * (batch + 1) * sizeof(int), (cudaStream_t)stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

bsp_status_t bsp_kv_append(bsp_kv_t h, const bsp_kv_step_t* step, const void* k, const void* v, bsp_dtype_t dtype,
                           int64_t rows, int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head,
                           bsp_stream_t stream)
{
    if (!valid(h)) return BSP_ERR_INVALID_ARG;
    if (const bsp_status_t st = check_step(step, rows, h->view.page_shift)) return st;
    if (dtype != BSP_FP16 && dtype != BSP_BF16) return BSP_ERR_DTYPE;
    if (!rows || !step->batch) return BSP_OK;
    if (!k || !v) return BSP_ERR_INVALID_ARG;
    if (!good_strides(k_row, k_head, h->view.dim, rows, h->view.heads) ||
        !good_strides(v_row, v_head, h->view.dim, rows, h->view.heads))
        return BSP_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16)) return BSP_ERR_ALIGN;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    const AppendArgs a = {h->view, view_of(step, rows), k, v, k_row, k_head, v_row, v_head};
    const int64_t items = (rows >> h->view.page_shift) + 2 * (int64_t)step->batch;
    const dim3 grid((unsigned)items, (unsigned)((2 * h->view.heads + 3) / 4));
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == BSP_FP16) kv_append_kernel<__half><<<grid, 128, 0, s>>>(a);
    else kv_append_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

bsp_status_t bsp_kv_read(bsp_kv_t h, const int64_t* slots, int64_t n, void* k, void* v, bsp_dtype_t dtype,
                         bsp_stream_t stream)
{
    if (!valid(h) || n < 0 || n > INT32_MAX) return BSP_ERR_INVALID_ARG;
    if (dtype != BSP_FP16 && dtype != BSP_BF16) return BSP_ERR_DTYPE;
    if (!n) return BSP_OK;
    if (!slots || !k || !v) return BSP_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return BSP_ERR_ALIGN;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    const ReadArgs a = {h->view, slots, k, v, n};
    const int64_t want = (n * h->view.heads * (h->view.dim / 16) + 255) / 256;
    const dim3 grid((unsigned)std::min<int64_t>(want, (int64_t)h->num_sms * 8), 2);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == BSP_FP16) kv_read_kernel<__half><<<grid, 256, 0, s>>>(a);
    else kv_read_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

bsp_status_t bsp_kv_attention(bsp_kv_t h, const bsp_kv_step_t* step, const void* q, bsp_dtype_t dtype, int64_t rows,
                              int32_t heads, int64_t q_row, int64_t q_head, float scale, int32_t window, void* out,
                              int64_t o_row, int64_t o_head, float* lse, bsp_stream_t stream)
{
    if (!valid(h)) return BSP_ERR_INVALID_ARG;
    if (const bsp_status_t st = check_step(step, rows, h->view.page_shift)) return st;
    if (dtype != BSP_FP16 && dtype != BSP_BF16) return BSP_ERR_DTYPE;
    // scale: finite and not negative (a comparison that NaN fails)
    if (window < 0 || !(scale >= 0.f && scale < INFINITY)) return BSP_ERR_INVALID_ARG;
    if (heads < 1 || heads > 32767 || heads % h->view.heads) return BSP_ERR_SHAPE;
    if (!rows) return BSP_OK;
    if (!q || !out) return BSP_ERR_INVALID_ARG;
    if (!good_strides(q_row, q_head, h->view.dim, rows, heads) ||
        !good_strides(o_row, o_head, h->view.dim, rows, heads))
        return BSP_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4))) return BSP_ERR_ALIGN;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    const int64_t most = step->max_new && step->max_new < rows ? step->max_new : rows;
    return bsp_run_kv_attention(h, view_of(step, rows), most, q, dtype, heads, q_row, q_head, scale, window, out,
                                o_row, o_head, lse, (cudaStream_t)stream);
}

}  // extern "C"
