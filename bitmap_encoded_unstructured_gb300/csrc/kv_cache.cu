// Paged 8-bit KV cache: the handle, the plan of a step (pages, slots), the
// quantising append and the read-back.  The attention is in
// kv_attention.cu.
#include "bsp_kv.cuh"

#include <algorithm>
#include <climits>
#include <new>
#include <type_traits>

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
// block table row, which nobody writes, not from the stack.  Bound by the
// launch and the chain of sums: 5.6 us for 64 requests, 6.7 us for 1024.
__global__ void __launch_bounds__(PLAN_THREADS) kv_plan_kernel(const PlanArgs a)
{
    wait_prior_grids();
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
// request's last page have nothing to do.  The warp looks 32 requests at a
// time, so that a search costs one or two loads.
__device__ __forceinline__ int item_request(const KvStepView& s, int page_shift, int item, int lane)
{
    int lo = 0, n = s.batch;  // F(lo) <= item, among lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32, at = lane * step;
        const bool below = at < n && (s.q_start[lo + at] >> page_shift) + 2 * (lo + at) <= item;
        const uint32_t set = __ballot_sync(0xFFFFFFFFu, below || lane == 0);
        const int last = 31 - __clz(set);
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

constexpr int APPEND_THREADS = 128, CACHED = 8;

__device__ __forceinline__ __half2 larger(__half2 a, uint32_t b) { return __hmax2(a, __habs2(*reinterpret_cast<__half2*>(&b))); }
__device__ __forceinline__ __nv_bfloat162 larger(__nv_bfloat162 a, uint32_t b)
{
    return __hmax2(a, __habs2(*reinterpret_cast<__nv_bfloat162*>(&b)));
}
__device__ __forceinline__ float larger_of(__half2 a) { return fmaxf(__low2float(a), __high2float(a)); }
__device__ __forceinline__ float larger_of(__nv_bfloat162 a) { return fmaxf(__low2float(a), __high2float(a)); }

// Eight codes round(x / scale), as the IEEE quotient rounds, from products
// with the reciprocal: adding 1.5 2^23 rounds them to even.  Where one is near
// a tie (the product is off by less than 3e-5 at 127) or not finite, the
// eight are divided.
template <class T>
__device__ __forceinline__ uint2 codes_of(const uint4& raw, float scale, float inv)
{
    constexpr float ROUND = 12582912.f;
    const T* e = reinterpret_cast<const T*>(&raw);
    uint32_t q[8];
    bool fine = true;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float t = __fmul_rn(to_float(e[c]), inv), r = __fadd_rn(t, ROUND);
        fine = fine && fabsf(__fsub_rn(t, __fsub_rn(r, ROUND))) <= 0.49995f;  // false for NaN
        q[c] = __float_as_uint(r);
    }
    if (!fine) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float t = __fdiv_rn(to_float(e[c]), scale);
            q[c] = t != t ? 0u : (uint32_t)__float2int_rn(fminf(fmaxf(t, -127.f), 127.f));
        }
    }
    uint2 o;
    o.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
    return o;
}

// WARPS warps (1 or 4) per unit: a page that receives rows, a head, K or V.
// Two passes over the unit's rows, its largest value and its codes; the first
// CACHED vectors of a thread stay in registers between them.  1 << lane_shift
// threads share a row, one 16-byte vector each.  2 bytes in and 1 out a value:
// 15879 bfloat16 rows of 8 heads of 128 take 28.5 us, 3.4 TB/s, 0.50 of the copy
// rate.  Bound by instructions: the largest stall is the wait for them (the
// codes' products, tie checks and divisions stand at each of nine stores), and
// 66% of the issue slots are taken.  Single rows are bound by the latency of
// request search, scale, rows and codes (4 us).
template <class T, int WARPS>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_kernel(const AppendArgs a, const int lane_shift)
{
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    constexpr int THREADS = WARPS * 32;
    wait_prior_grids();
    const int lane = threadIdx.x & 31, tid = threadIdx.x % THREADS;
    const int unit = blockIdx.y * (APPEND_THREADS / THREADS) + threadIdx.x / THREADS;
    if (unit >= 2 * a.c.heads) return;
    const int head = unit >> 1, sh = a.c.page_shift, page = 1 << sh;
    const bool is_v = unit & 1;
    const int b = item_request(a.s, sh, blockIdx.x, lane);
    const Request r = request_of(a.s, sh, b);
    const int start = r.len - r.n, from = max(start, 0);  // position of the first new row; of the first stored
    const int64_t jj = (from >> sh) + (int64_t)blockIdx.x - ((a.s.q_start[b] >> sh) + 2 * (int64_t)b);
    if (jj < (from >> sh) || jj << sh >= r.len) return;
    const int j = (int)jj;
    const int lo = max(from, j << sh), hi = (int)min((int64_t)r.len, (jj + 1) << sh);  // new rows of this page
    if (lo >= hi) return;
    const int p = a.s.table[(int64_t)b * a.s.table_stride + j];
    if (p < 0 || p >= a.c.pages) return;
    const int64_t row_step = is_v ? a.v_row : a.k_row;
    const int kept = lo & (page - 1), rows = hi - lo;    // earlier rows of the page; new ones
    const int col = (tid & ((1 << lane_shift) - 1)) * 8, row0 = tid >> lane_shift, step = THREADS >> lane_shift;
    const bool mine = col < a.c.dim;
    const T* x = (const T*)(is_v ? a.v : a.k) + (int64_t)(r.r0 + lo - start) * row_step +
                 (int64_t)head * (is_v ? a.v_head : a.k_head) + col;
    int8_t* codes = (is_v ? a.c.v : a.c.k) + (int64_t)p * a.c.page_stride + (int64_t)head * a.c.head_stride;
    float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + (int64_t)p * a.c.scale_stride + head;
    const float old = kept ? *scale : 0.f;
    auto load = [&](int row) {
        return mine && row < rows ? *reinterpret_cast<const uint4*>(x + row * row_step) : make_uint4(0, 0, 0, 0);
    };
    auto most = [&](float f) {  // over the unit's threads
#pragma unroll
        for (int d = 16; d; d >>= 1) f = fmaxf(f, __shfl_xor_sync(0xFFFFFFFFu, f, d));
        if constexpr (WARPS > 1) {
            __shared__ float tops[WARPS];
            __syncthreads();
            if (lane == 0) tops[tid >> 5] = f;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WARPS; ++w) f = fmaxf(f, tops[w]);
        }
        return f;
    };

    uint4 held[CACHED];
#pragma unroll
    for (int c = 0; c < CACHED; ++c) held[c] = load(row0 + c * step);
    T2 big;
    big.x = big.y = from_float<T>(0.f);
    auto look = [&](const uint4& v) { big = larger(larger(larger(larger(big, v.x), v.y), v.z), v.w); };
#pragma unroll
    for (int c = 0; c < CACHED; ++c) look(held[c]);
    for (int row = row0 + CACHED * step; row < rows; row += step) look(load(row));
    float top = most(larger_of(big));
    if (top == INFINITY) {  // again, without the infinities
        top = 0.f;
        for (int row = row0; row < rows; row += step) {
            const uint4 v = load(row);
            const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float f = fabsf(to_float(e[c]));
                if (f < INFINITY) top = fmaxf(top, f);   // false for NaN too
            }
        }
        top = most(top);
    }
    const float now = fmaxf(old, __fdiv_rn(top, 127.f));
    if (kept && now != old) {
        const float ratio = now > 0.f ? __fdiv_rn(old, now) : 0.f;
        for (int i = tid; i < kept * (a.c.dim / 16); i += THREADS) {
            int4* at = reinterpret_cast<int4*>(codes + (i / (a.c.dim / 16)) * a.c.row_stride + (i % (a.c.dim / 16)) * 16);
            int4 w = *at;
            int8_t* e = reinterpret_cast<int8_t*>(&w);
#pragma unroll
            for (int c = 0; c < 16; ++c) e[c] = (int8_t)__float2int_rn(__fmul_rn((float)e[c], ratio));
            *at = w;
        }
    }
    if (kept && now == 0.f)  // no codes under a scale of 0 (apart: in the loop above it costs 7 registers)
        for (int i = tid; i < kept * (a.c.dim / 16); i += THREADS)
            *reinterpret_cast<int4*>(codes + (i / (a.c.dim / 16)) * a.c.row_stride + (i % (a.c.dim / 16)) * 16) =
                make_int4(0, 0, 0, 0);
    // no reciprocal of a scale below 2^-126: NaN makes every code a quotient
    const float inv = now < 1.2e-38f ? __int_as_float(0x7FC00000) : __fdiv_rn(1.f, now);
    auto store = [&](int row, const uint4& v) {
        if (mine && row < rows)
            *reinterpret_cast<uint2*>(codes + (kept + row) * a.c.row_stride + col) =
                now > 0.f ? codes_of<T>(v, now, inv) : make_uint2(0, 0);
    };
#pragma unroll
    for (int c = 0; c < CACHED; ++c) store(row0 + c * step, held[c]);
    for (int row = row0 + CACHED * step; row < rows; row += step) store(row, load(row));
    if (tid == 0) *scale = now;
}

// ------------------------------------------------------------------- read

// x / d for x < 2^31 by a multiplication: with 2^s the power of two at or
// above d, q = (floor(x m / 2^32) + x) / 2^s where m = floor(2^32 (2^s - d) / d) + 1
// (division by an invariant integer, Granlund and Montgomery 1994).
struct Divide {
    uint32_t d, m, s;
    explicit Divide(uint32_t by = 1) : d(by), s(0)
    {
        while ((1u << s) < d) ++s;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1);
    }
    __device__ uint32_t operator()(uint32_t x) const { return (__umulhi(x, m) + x) >> s; }
};

struct ReadArgs {
    KvView c;
    const int64_t* slots;
    void *k, *v;
    int64_t n;       // rows
    uint32_t units;  // of 8 values in a row of all heads
    Divide by_units, by_head;
    int rows;        // of a CTA's piece: rows * units < 2^31
};

constexpr int READ_AT_ONCE = 4;  // units of a thread in flight

// A thread takes units of 8 values, so that a warp's loads and stores are
// whole lines; K and V by blockIdx.y.  CTA x takes
// pieces x, x + gridDim.x, ... of `rows` rows each.  Bound by memory: 15879
// rows of 8 heads of 128, 98 MB, take 18.9 us (5.2 TB/s), 30011 rows 33.6 us.
template <class T>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadArgs a)
{
    wait_prior_grids();
    const int8_t* codes = blockIdx.y ? a.c.v : a.c.k;
    const float* scales = blockIdx.y ? a.c.v_scale : a.c.k_scale;
    for (int64_t r0 = (int64_t)blockIdx.x * a.rows; r0 < a.n; r0 += (int64_t)gridDim.x * a.rows) {
        const uint32_t all = (uint32_t)min((int64_t)a.rows, a.n - r0) * a.units;
        T* out = (T*)(blockIdx.y ? a.v : a.k) + r0 * a.units * 8;
        for (uint32_t u0 = threadIdx.x; u0 < all; u0 += 256 * READ_AT_ONCE) {
            int2 w[READ_AT_ONCE];
            float sc[READ_AT_ONCE];
#pragma unroll
            for (int x = 0; x < READ_AT_ONCE; ++x) {
                const uint32_t u = u0 + 256 * x;
                w[x] = make_int2(0, 0);
                sc[x] = 0.f;
                if (u < all) {
                    const uint32_t row = a.by_units(u), unit = u - row * a.units, head = a.by_head(unit);
                    const int64_t slot = a.slots[r0 + row], p = slot >> a.c.page_shift;
                    if (slot >= 0 && p < a.c.pages) {
                        const int64_t off = slot - (p << a.c.page_shift);
                        w[x] = *reinterpret_cast<const int2*>(codes + p * a.c.page_stride + head * a.c.head_stride +
                                                              off * a.c.row_stride + (unit - head * a.by_head.d) * 8);
                        sc[x] = scales[p * a.c.scale_stride + head];
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < READ_AT_ONCE; ++x) {
                const uint32_t u = u0 + 256 * x;
                if (u < all) {
                    alignas(16) T o[8];
                    const int8_t* e = reinterpret_cast<const int8_t*>(&w[x]);
#pragma unroll
                    for (int c = 0; c < 8; ++c) o[c] = from_float<T>((float)e[c] * sc[x]);
                    *reinterpret_cast<uint4*>(out + (int64_t)u * 8) = *reinterpret_cast<const uint4*>(o);
                }
            }
        }
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

// Do bytes [p, p + n) meet one of `rows` pieces of `len` bytes, `stride` apart
// from q on?
bool meet(const void* p, int64_t n, const void* q, int64_t len, int64_t rows = 1, int64_t stride = 0)
{
    if (n <= 0 || len <= 0 || rows <= 0) return false;
    const int64_t lo = (int64_t)((uintptr_t)p - (uintptr_t)q), hi = lo + n;
    if (rows == 1 || stride <= 0) return lo < len && hi > 0;
    if (hi <= 0 || lo >= (rows - 1) * stride + len) return false;
    // the row that p lies in or behind, and the next one
    const int64_t b = std::max<int64_t>(lo, 0) / stride;
    return lo < b * stride + len || (b + 1 < rows && hi > (b + 1) * stride);
}

// A stride that is never used (one row, one head) may be anything.
bool good_strides(int64_t row, int64_t head, int32_t dim, int64_t rows, int32_t heads)
{
    return (rows < 2 || (row >= 0 && row % 8 == 0)) && (heads < 2 || (head >= dim && head % 8 == 0));
}

// Rows and heads of an output each have memory of their own.
bool apart(int64_t row, int64_t head, int32_t dim, int64_t rows, int32_t heads)
{
    if (rows < 2) return true;
    if (row < dim) return false;
    return heads < 2 || row >= (heads - 1) * head + dim || head >= (rows - 1) * row + dim;
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
    if (d->row_stride < d->dim || d->row_stride % 16 ||
        (d->heads > 1 && (d->head_stride < d->dim || d->head_stride % 16)) ||
        (d->pages > 1 && (d->page_stride < d->dim || d->page_stride % 16 || d->scale_stride < d->heads)))
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
    else if (cudaMalloc(&h->ticket, 2 * sizeof(int)) != cudaSuccess || cudaMalloc(&h->err, sizeof(int)) != cudaSuccess)
        st = BSP_ERR_OOM;
    else if (cudaMemsetAsync(h->ticket, 0, 2 * sizeof(int), s) != cudaSuccess ||
             cudaMemsetAsync(h->err, 0, sizeof(int), s) != cudaSuccess)
        st = BSP_ERR_CUDA;
    else
        st = attention_setup(h, s);
    h->ready = h->ticket + 1;
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
    // every CTA reads the lengths and the stack while others write their
    // shares: what is written shares memory with nothing else of the call (but
    // the count, which the last CTA writes)
    struct Piece {
        const void* at;
        int64_t bytes;
    };
    const Piece of[] = {{seq_len, 4 * (int64_t)batch},      {q_start, 4 * ((int64_t)batch + 1)},
                        {granted, 4 * (int64_t)batch},      {slots, 8 * tokens},
                        {positions, 4 * tokens},            {free_list, 4 * (int64_t)free_capacity},
                        {free_count_out, 4},                {free_count, 4},
                        {ctx_len, 4 * (int64_t)batch},      {new_len, 4 * (int64_t)batch}};
    constexpr int WRITTEN = 7, ALL = 10;
    for (int i = 0; i < ALL; ++i) {
        if (meet(of[i].at, of[i].bytes, block_table, 4 * (int64_t)width, batch, 4 * table_stride))
            return BSP_ERR_INVALID_ARG;
        for (int j = i + 1; i < WRITTEN && j < ALL; ++j)
            if (meet(of[i].at, of[i].bytes, of[j].at, of[j].bytes) && !(i == 6 && j == 7 && of[i].at == of[j].at))
                return BSP_ERR_INVALID_ARG;
    }
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
    return launch_early(kv_plan_kernel, dim3(grid), dim3(PLAN_THREADS), 3 * (batch + 1) * (int)sizeof(int),
                        (cudaStream_t)stream, a)
               ? BSP_OK
               : BSP_ERR_CUDA;
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
    int lane_shift = 1;
    while ((8 << lane_shift) < h->view.dim) ++lane_shift;
    // a block a unit where units are large on average (more rows than a warp
    // holds in registers), a warp a unit where they are single rows
    const bool large = std::min<int64_t>(rows / step->batch, 1 << h->view.page_shift) > CACHED * (32 >> lane_shift);
    const dim3 grid((unsigned)items, (unsigned)(large ? 2 * h->view.heads : (2 * h->view.heads + 3) / 4));
    const dim3 block(APPEND_THREADS);
    cudaStream_t s = (cudaStream_t)stream;
    auto go = [&](auto kernel) { return launch_early(kernel, grid, block, 0, s, a, lane_shift); };
    const bool ok = dtype == BSP_FP16 ? large ? go(kv_append_kernel<__half, 4>) : go(kv_append_kernel<__half, 1>)
                    : large           ? go(kv_append_kernel<__nv_bfloat16, 4>)
                                      : go(kv_append_kernel<__nv_bfloat16, 1>);
    return ok ? BSP_OK : BSP_ERR_CUDA;
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
    const uint32_t per_head = (uint32_t)h->view.dim / 8, units = (uint32_t)h->view.heads * per_head;
    // pieces of about 4096 units: enough CTAs for a small call, and few
    // searches for a large one
    const int piece = (int)std::max<uint32_t>(1, 4096 / units);
    const ReadArgs a = {h->view, slots, k, v, n, units, Divide(units), Divide(per_head), piece};
    const dim3 grid((unsigned)std::min<int64_t>((n + piece - 1) / piece, (int64_t)h->num_sms * 16), 2);
    cudaStream_t s = (cudaStream_t)stream;
    const bool ok = dtype == BSP_FP16 ? launch_early(kv_read_kernel<__half>, grid, dim3(256), 0, s, a)
                                      : launch_early(kv_read_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, a);
    return ok ? BSP_OK : BSP_ERR_CUDA;
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
        !good_strides(o_row, o_head, h->view.dim, rows, heads) || !apart(o_row, o_head, h->view.dim, rows, heads))
        return BSP_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4))) return BSP_ERR_ALIGN;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    const int64_t most = step->max_new && step->max_new < rows ? step->max_new : rows;
    return bsp_run_kv_attention(h, view_of(step, rows), most, q, dtype, heads, q_row, q_head, scale, window, out,
                                o_row, o_head, lse, (cudaStream_t)stream);
}

}  // extern "C"
