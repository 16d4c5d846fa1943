// Attention of a step's new rows over the paged 8-bit cache.
//
// A cached value is code * scale with one scale for each page and KV head,
// so the scales stay out of the inner sums: q . k_j = s_k(page of j) *
// (q . codes_j), and p_j v_j = (p_j s_v(page of j)) codes_j.
#include "bsp_kv.cuh"
#include "bsp_ptx.cuh"

#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

namespace {

using namespace bspkv;

// ------------------------------------------------------------ few queries
//
// One kernel for requests with few query rows per KV head (decoding,
// drafts): bound by the bytes of the codes.  A segment is one request, KV
// head and group of Q query rows; its cached rows are taken in sub-tiles of
// 32.  The warps of the grid share all sub-tiles evenly, each a contiguous
// run of them in order of request, head and group, so that neither ragged
// lengths nor few requests leave SMs idle.  A segment counts OVER sub-tiles
// more than it has, the price of starting and finishing one.
//
// A warp works alone: it streams its sub-tiles through a ring of its own
// (TMA boxes of the paged codes, across segment ends), with no block-wide
// barrier until its run is done, and writes the segments that it has whole.
// Of a segment cut between warps each leaves a part (the warps of a CTA add
// theirs first), and a second kernel joins the parts in order.
//
//   S^T[row][query] = codes_K . q     mma m16n8k16, A = codes as exact fp16
//   O^T[dim][query] += codes_V^T . W  W = p * V scale
// Codes become fp16 by a byte permute under the exponent of 1024 and one
// subtraction (1024 + 128 + c - 1152, exact).  The dims a thread multiplies
// are chosen so that its operands are whole 16-byte chunks: the k index of a
// product may be permuted freely as long as both sides agree.
constexpr int DEC_WARPS = 4;
constexpr int SUB = 32;                  // rows of a sub-tile
// OVER: sub-tiles a segment's start and end are worth.  LEAST: a warp's run is
// at least this long (more than OVER).  Cold, 64 ragged streams of 64 over 8
// heads | 256 streams of 100 .. 900 rows | one of 517: 2 and 3 take 135 | 78 |
// 20.5 us, 0 and 1 141 | 82 | 18.4, 3 and 4 131 | 78 | 20.5, 4 and 5 137 | 80 |
// 22.5, 2 and 10 131 | 78 | 26.6.
constexpr int OVER = 2;
constexpr int LEAST = 3;
constexpr int RUN = 32, FILL = 16;       // entries of the run that a warp looks ahead, and fills at a time later

template <int DP, int NT>
struct DecCfg {
    static constexpr int BOX = DP < 128 ? DP : 128;    // bytes of a smem row
    static constexpr int REGIONS = DP / BOX;
    static constexpr int HALF = SUB * DP;              // K (or V) codes of a stage
    static constexpr int STAGE = 2 * HALF;
    // CTAs that an SM holds (by registers and shared memory), and stages of a
    // warp's ring: with three CTAs two stages of 8 KB keep more bytes in
    // flight than the memory needs
    static constexpr int CTAS = NT == 1 && DP <= 128 ? 3 : 2;
    // queries too many for the registers beside the sums wait in shared memory
    static constexpr bool QSMEM = NT * DP > 256;
    static constexpr int STAGES = DP == 64 ? 4 : CTAS == 3 || QSMEM ? 2 : 3;
    static constexpr int QBYTES = QSMEM ? NT * DP * 16 : 0;  // of a warp
    static constexpr int RING = DEC_WARPS * STAGES * STAGE;
    static constexpr int Q = 8 * NT;                   // query rows of a segment
    static constexpr int OPAD = DP + 4;                // floats of a row of the joining buffer
    static constexpr int PART = Q * (DP + 4);          // floats of a part: O, then m, l, mw of the rows
    static constexpr int OFF_RUN = RING;               // entries of each warp's run
    static constexpr int OFF_Q = OFF_RUN + DEC_WARPS * RUN * 64;
    static constexpr int OFF_STAT = OFF_Q + DEC_WARPS * QBYTES;  // m, l, mw of each warp
    static constexpr int OFF_BAR = OFF_STAT + DEC_WARPS * Q * 3 * 4;
    // (all of it dynamic: static arrays would be rounded up to its alignment)
    static constexpr int OFF_PRE = OFF_BAR + DEC_WARPS * STAGES * 8;         // what comes before each thread's requests
    static constexpr int OFF_SEG = OFF_PRE + (DEC_WARPS * 32 + 2) * 8;       // the warps' open segments
    static constexpr int OFF_SUMS = OFF_SEG + DEC_WARPS * 64;
    static constexpr int OFF_AT = OFF_SUMS + DEC_WARPS * 8;
    static constexpr int SMEM = OFF_AT + DEC_WARPS * 8 + 1024;
    static_assert(OFF_SEG % 16 == 0, "alignment of the entries");
    static_assert(SMEM + 1024 + 128 <= 228 * 1024 / (DP == 256 ? 1 : CTAS), "shared memory of the resident CTAs");
    static_assert(DEC_WARPS * Q * OPAD * 4 <= RING, "joining buffer in the idle ring");
};

struct DecodeArgs {
    AttnArgs a;
    float* parts;
    KvCut* cuts;
    int* err;
    uint32_t spin_cap;
    int32_t most_rows;  // requests with more query rows than this (per KV head) are not this kernel's
    int* ready;         // set by the prompt kernel of this call (null: there is none)
    bool beside;        // runs beside the prompt kernel
    bool stall;         // test only: each warp skips the copies of its first sub-tile
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A request's share of the work: cached rows [lo, len) that some query sees
// (lo rounded down to whole sub-tiles); row groups of Q queries.
struct Share {
    Request r;
    int seen, lo, subs, groups;  // first cached row that a query sees, and the sub-tile it starts in
    __device__ int64_t cost(int heads) const { return (int64_t)groups * heads * (subs + OVER); }
};

template <int Q>
__device__ __forceinline__ Share share_of(const DecodeArgs& d, Request r)
{
    const AttnArgs& a = d.a;
    Share s;
    s.r = r;
    const int64_t rows = (int64_t)s.r.n * a.group;
    if (rows > d.most_rows) s.r.n = 0;
    const int first = s.r.len - s.r.n;
    s.seen = a.window ? max(0, first - a.window + 1) : 0;
    s.lo = s.seen & ~(SUB - 1);
    s.groups = s.r.n ? (int)((rows + Q - 1) / Q) : 0;
    s.subs = max(1, (s.r.len - s.lo + SUB - 1) / SUB);  // at least one: it writes the zeros of rows that see nothing
    return s;
}

// One sub-tile of a warp's run (or a place that OVER reserves: tok < 0).
struct Entry {
    int tok, p0, p1, h;      // first row, its page and (pages of 16 rows) the next one's, KV head
    int len, n, r0, rg;      // the request, the group of query rows
    float ks[2], vs[2];
    int i, subs;             // which sub-tile of how many
    float lv[2];             // log2 vs
};
static_assert(sizeof(Entry) == 64, "run entries");

// x / y for x >= 0, y > 0: 64-bit division is a long subroutine, and the
// numbers nearly always fit 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y)
{
    return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// The shared run of `total` places among P workers (warps): the first
// `longer` have one place more than the others.
struct Split {
    int64_t each, longer;
    __device__ Split(int64_t total, int64_t P)
    {
        each = quotient(total, P);
        longer = total - each * P;
    }
    __device__ int64_t begin(int64_t w) const { return w * each + min(w, longer); }
    __device__ int worker(int64_t x) const
    {
        const int64_t head = longer * (each + 1);
        return (int)(x < head ? quotient(x, each + 1) : longer + quotient(x - head, each));
    }
};

// Four dims of one query row, joined: out = O 2^(mw - m) / l.  A sum of 0 is a
// row that sees nothing; a NaN query's sum is NaN, and so is its row.
template <class T>
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t row, int64_t head, int dim, float4 o, float top,
                                          float topw, float sum)
{
    const float f = sum != 0.f ? ex2(topw - top) / sum : 0.f;
    if (dim < a.c.dim) {
        alignas(8) T y[4] = {from_float<T>(o.x * f), from_float<T>(o.y * f), from_float<T>(o.z * f),
                             from_float<T>(o.w * f)};
        *reinterpret_cast<uint2*>((T*)a.out + row * a.o_row + head * a.o_head + dim) = *reinterpret_cast<const uint2*>(y);
    }
    if (a.lse && dim == 0)
        a.lse[row * a.heads + head] = sum != 0.f ? (top + __log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

constexpr int JOIN_WARPS = 8, JOIN_ROWS = 2, ROW_WARPS = JOIN_WARPS / JOIN_ROWS, JOIN_CTAS = 2;
constexpr int MANY = 8;  // parts of a segment from which several warps share a row

// The parts of a row of one cut segment: the first worker's, one of each
// further CTA's, and the last worker's; every step-th from `from` on.  L lanes
// share a row (RPW rows a warp, each of a segment of its own): a lane adds up
// dims 4 i .. and DP / 2 + 4 i .., and looks after the maxima and sum of one
// part of those whose loads are in flight together.
template <class C, int DP>
struct RowSum {
    static constexpr int L = DP / 8, RPW = 32 / L, V = 2, AT_ONCE = 4;
    float top = NONE, topw = NONE, sum = 0.f;
    float4 o[V];

    __device__ void add(float m, float l, float mw, const float4 (&x)[V])
    {
        const float t = fmaxf(top, m), tw = fmaxf(topw, mw);
        sum = sum * ex2(top - t) + l * ex2(m - t);
        const float f = ex2(topw - tw), g = ex2(mw - tw);
#pragma unroll
        for (int v = 0; v < V; ++v)
            o[v] = make_float4(o[v].x * f + x[v].x * g, o[v].y * f + x[v].y * g, o[v].z * f + x[v].z * g,
                               o[v].w * f + x[v].w * g);
        top = t;
        topw = tw;
    }

    // n = 0: no row
    __device__ RowSum(const float* parts, const KvCut& cut, int w, int n, int qr, int lane, int from, int step)
    {
        constexpr int Q = C::Q;
        constexpr uint32_t FULL = 0xFFFFFFFFu;
        const int dim = lane % L * 4, cta = n ? w / cut.per_cta : 0, most = __reduce_max_sync(FULL, n);
        auto part = [&](int k) {
            const int slot = k == n - 1 ? 2 * cut.last + 1 : 2 * (k ? (cta + k) * cut.per_cta : w);
            return parts + (int64_t)slot * C::PART;
        };
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = from; k0 < most; k0 += AT_ONCE * step) {
            const int mine = k0 + lane % AT_ONCE * step;
            float m = NONE, l = 0.f, mw = NONE;
            if (mine < n) {
                const float* p = part(mine) + Q * DP + qr;
                m = __ldcg(p);
                l = __ldcg(p + Q);
                mw = __ldcg(p + 2 * Q);
            }
            float4 x[AT_ONCE][V];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) x[i][v] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + i * step < n) {
                    const float* p = part(k0 + i * step) + qr * DP + dim;
#pragma unroll
                    for (int v = 0; v < V; ++v) x[i][v] = __ldcg(reinterpret_cast<const float4*>(p + v * (DP / 2)));
                }
            }
            float t = fmaxf(top, m), tw = fmaxf(topw, mw);
#pragma unroll
            for (int i = 1; i < AT_ONCE; i <<= 1) {
                t = fmaxf(t, __shfl_xor_sync(FULL, t, i));
                tw = fmaxf(tw, __shfl_xor_sync(FULL, tw, i));
            }
            l *= ex2(m - t);
#pragma unroll
            for (int i = 1; i < AT_ONCE; i <<= 1) l += __shfl_xor_sync(FULL, l, i);
            sum = sum * ex2(top - t) + l;
            const float f = ex2(topw - tw), g = ex2(mw - tw);
            top = t;
            topw = tw;
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = make_float4(o[v].x * f, o[v].y * f, o[v].z * f, o[v].w * f);
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const float gi = __shfl_sync(FULL, g, i, L);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    o[v].x += x[i][v].x * gi;
                    o[v].y += x[i][v].y * gi;
                    o[v].z += x[i][v].z * gi;
                    o[v].w += x[i][v].w * gi;
                }
            }
        }
    }
};

// Joins the parts of the segments that were cut, in order.  A CTA looks at 32
// entries of the list (or 32 of every lists * 32) with team - 1 others and
// takes rows of their segments: L lanes a row, or for segments of many parts
// ROW_WARPS warps that add up in shared memory.  Bound by latency, 1.5 us for
// the list and 2 us for a row's parts: 5 us behind 64 ragged streams of 64
// heads (4096 rows).  Two rows a warp and JOIN_CTAS = 2 leave most warps one
// turn: 80.0 us a call, against 84 with 1, 83 with 3 (spills) and 84 with 4.
template <class T, int DP, int NT>
__global__ void __launch_bounds__(JOIN_WARPS * 32, JOIN_CTAS) kv_join_kernel(const DecodeArgs d, int workers)
{
    using C = DecCfg<DP, NT>;
    using Sum = RowSum<C, DP>;
    constexpr int Q = C::Q, V = Sum::V, L = Sum::L, RPW = Sum::RPW;
    constexpr uint32_t FULL = 0xFFFFFFFFu;
    const AttnArgs& a = d.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / L;
    const int ri = warp / ROW_WARPS, rw = warp % ROW_WARPS;
    const int lists = min((workers + 31) / 32, (int)gridDim.x), team = (int)gridDim.x / lists;
    const int member = (int)blockIdx.x / lists;
    __shared__ float stat[JOIN_ROWS][ROW_WARPS][RPW][3];
    __shared__ float4 sums[JOIN_ROWS][ROW_WARPS][V][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    wait_prior_grids();
    if (d.ready && blockIdx.x == 0 && threadIdx.x == 0) *d.ready = 0;
    if (member >= team) return;
    auto out = [&](const Sum& s, const KvCut& cut, int qr) {
        const int r = cut.rg * Q + qr, of = r / a.group;
#pragma unroll
        for (int v = 0; v < V; ++v)
            store_out<T>(a, cut.r0 + of, cut.h * a.group + r - of * a.group, lane % L * 4 + v * (DP / 2), s.o[v], s.top,
                         s.topw, s.sum);
    };
    for (int w0 = (int)blockIdx.x % lists * 32; w0 < workers; w0 += lists * 32) {
        KvCut mine = {-1, 1, 0, 0, 0, 0, {0, 0}};
        if (w0 + lane < workers) mine = d.cuts[w0 + lane];
        int n_mine = 0, rows_mine = 0;  // parts and rows of this lane's segment
        if (mine.last >= 0) {
            n_mine = (mine.last - 1) / mine.per_cta - (w0 + lane) / mine.per_cta + 2;
            rows_mine = min(Q, mine.n * a.group - mine.rg * Q);
        }
        auto cut_of = [&](int e) {
            return KvCut{__shfl_sync(FULL, mine.last, e), __shfl_sync(FULL, mine.per_cta, e),
                         __shfl_sync(FULL, mine.r0, e),   __shfl_sync(FULL, mine.n, e),
                         __shfl_sync(FULL, mine.h, e),    __shfl_sync(FULL, mine.rg, e), {0, 0}};
        };
        // segments of few parts: their rows in order, each to the next L lanes
        int upto = n_mine <= MANY ? rows_mine : 0;
        const int few = upto;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int y = __shfl_up_sync(FULL, upto, i);
            if (lane >= i) upto += y;
        }
        const int all = __shfl_sync(FULL, upto, 31);
        for (int i0 = (member * JOIN_WARPS + warp) * RPW; i0 < all; i0 += team * JOIN_WARPS * RPW) {
            const int i = i0 + sub;
            int e = 0;  // the first lane whose `upto` is beyond i
#pragma unroll
            for (int y = 16; y; y >>= 1)
                if (__shfl_sync(FULL, upto, e + y - 1) <= i) e += y;
            const int qr = i - __shfl_sync(FULL, upto - few, e), n = __shfl_sync(FULL, n_mine, e);
            const KvCut cut = cut_of(e);
            const Sum s(d.parts, cut, w0 + e, i < all ? n : 0, qr, lane, 0, 1);
            if (i < all) out(s, cut, qr);
        }
        for (uint32_t todo = __ballot_sync(FULL, n_mine > MANY); todo; todo &= todo - 1) {
            const int e = __ffs(todo) - 1, n = __shfl_sync(FULL, n_mine, e), rows = __shfl_sync(FULL, rows_mine, e);
            const KvCut cut = cut_of(e);
            for (int q0 = member * JOIN_ROWS * RPW; q0 < rows; q0 += team * JOIN_ROWS * RPW) {
                const int qr = q0 + ri * RPW + sub;
                Sum s(d.parts, cut, w0 + e, qr < rows ? n : 0, qr, lane, rw, ROW_WARPS);
                __syncthreads();  // the rows before are read
                if (lane % L == 0) {
                    stat[ri][rw][sub][0] = s.top;
                    stat[ri][rw][sub][1] = s.sum;
                    stat[ri][rw][sub][2] = s.topw;
                }
#pragma unroll
                for (int v = 0; v < V; ++v) sums[ri][rw][v][lane] = s.o[v];
                __syncthreads();
                if (rw == 0 && qr < rows) {
#pragma unroll
                    for (int i = 1; i < ROW_WARPS; ++i) {
                        const float4 y[V] = {sums[ri][i][0][lane], sums[ri][i][1][lane]};
                        s.add(stat[ri][i][sub][0], stat[ri][i][sub][1], stat[ri][i][sub][2], y);
                    }
                    out(s, cut, qr);
                }
            }
        }
    }
}

__device__ __forceinline__ bool is_ready(const int* ready)
{
    int r;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(r) : "l"(ready) : "memory");
    return r != 0;
}

// Bound by memory at 8 queries: 64 ragged streams of 8 KV heads, 391 MB of
// codes, take 72 us (5.4 TB/s; 6.1 TB/s while warps work, the rest is the
// start and uneven ends).  At 24 queries by the latency of two warps a
// scheduler (253 registers hold the sums): 595 MB in 142 us, 4.2 TB/s.
template <class T, int DP, int NT>
__global__ void __launch_bounds__(DEC_WARPS * 32, DecCfg<DP, NT>::CTAS)
kv_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const DecodeArgs d)
{
    using C = DecCfg<DP, NT>;
    constexpr int Q = C::Q, CH = DP / 64, MT = DP / 16;
    constexpr uint32_t FULL = 0xFFFFFFFFu;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (bspx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const AttnArgs& a = d.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int H = a.c.heads, B = a.s.batch, sh = a.c.page_shift;
    float* stat = reinterpret_cast<float*>(smem + C::OFF_STAT);  // [warp][3][Q]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * C::STAGES;
    uint8_t* ring = smem + warp * C::STAGES * C::STAGE;
    Entry* run = reinterpret_cast<Entry*>(smem + C::OFF_RUN) + warp * RUN;

    if (lane < C::STAGES) bspx::mbar_init(full + lane, 1);
    bspx::fence_mbar_init();
    // launched before the kernel ahead of it is done; beside the prompt kernel
    // it only has to end after it, but it has to see what the kernels before
    // both wrote: through `ready`, or (not set yet) by waiting all the same
    if (d.beside && is_ready(d.ready)) asm volatile("fence.proxy.async.global;" ::: "memory");  // codes come by TMA
    else wait_prior_grids();
    __syncwarp();

    // the shared run: each thread sums some requests; pre[i] is what comes
    // before thread i's
    int64_t* pre = reinterpret_cast<int64_t*>(smem + C::OFF_PRE);
    int64_t* sums = reinterpret_cast<int64_t*>(smem + C::OFF_SUMS);
    const int per = (B + DEC_WARPS * 32 - 1) / (DEC_WARPS * 32);
    int64_t upto = 0;
    for (int b = min(B, tid * per); b < min(B, (tid + 1) * per); ++b)
        upto += share_of<Q>(d, request_of(a.s, sh, b)).cost(H);
    const int64_t mine = upto;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int64_t o = __shfl_up_sync(FULL, upto, i);
        if (lane >= i) upto += o;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < DEC_WARPS; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
    }
    pre[tid] = upto - mine;
    if (tid == 0) pre[DEC_WARPS * 32] = total;
    __syncthreads();

    // P workers; fewer than there are warps are spread over the CTAs
    const int P = (int)max((int64_t)1, min((int64_t)gridDim.x * DEC_WARPS, quotient(total, LEAST)));
    const int wpc = min(DEC_WARPS, (P + (int)gridDim.x - 1) / (int)gridDim.x);
    const Split split(total, P);
    const int worker = blockIdx.x * wpc + warp;
    const bool works = total > 0 && warp < wpc && worker < P;
    const int64_t x0 = works ? split.begin(worker) : 0;
    const int N = works ? (int)(split.begin(worker + 1) - x0) : 0;

    int filled = 0;
    uint32_t stage = 0, phase = 0, next = 0;  // ring: stage being read, stage of the next load
    int ahead = 0, loading = 0;               // entries looked at for loading; loads in flight
    bool failed = false, stall = d.stall;
    auto load = [&]() {
        while (ahead < min(N, filled) && loading < C::STAGES) {
            const Entry& e = run[ahead % RUN];
            ++ahead;
            if (e.tok < 0) continue;
            if (lane == 0 && !stall) {
                uint8_t* st = ring + next * C::STAGE;
                const int p0 = e.p0, p1 = sh == 4 ? e.p1 : -1;
                const uint32_t rows = sh == 4 ? 16 * ((p0 >= 0) + (p1 >= 0)) : p0 >= 0 ? SUB : 0;
                if (rows) bspx::mbar_arrive_expect_tx(full + next, rows * 2 * DP);
                else bspx::mbar_arrive(full + next);
                const int row = sh == 4 ? 0 : e.tok & ((1 << sh) - 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int p = i ? p1 : p0;
                    if (p < 0) continue;
#pragma unroll
                    for (int rgn = 0; rgn < C::REGIONS; ++rgn) {
                        uint8_t* to = st + rgn * SUB * C::BOX + i * 16 * C::BOX;
                        tma_load_4d(to, &map_k, rgn * 128, row, e.h, p, full + next);
                        tma_load_4d(to + C::HALF, &map_v, rgn * 128, row, e.h, p, full + next);
                    }
                }
            }
            stall = false;
            ++loading;
            if (++next == C::STAGES) next = 0;
        }
        __syncwarp();
    };
    auto fill = [&](int count) {  // the next entries of the run, one per lane
        const bool keep = lane < count && filled + lane < N;
        Entry e;
        e.tok = e.p0 = e.p1 = -1;
        e.ks[0] = e.ks[1] = e.vs[0] = e.vs[1] = 0.f;
        e.lv[0] = e.lv[1] = NONE;
        if (keep) {
            const int64_t x = x0 + filled + lane;
            int t = 0;  // the thread whose requests hold place x, then the request
#pragma unroll
            for (int i = DEC_WARPS * 16; i; i >>= 1)
                if (pre[t + i] <= x) t += i;
            int b = t * per;
            int64_t off = x - pre[t];
            Share s = share_of<Q>(d, request_of(a.s, sh, b));
            while (off >= s.cost(H) && b + 1 < B) {
                off -= s.cost(H);
                s = share_of<Q>(d, request_of(a.s, sh, ++b));
            }
            const int64_t seg = quotient(off, s.subs + OVER);
            e.i = (int)(off - seg * (s.subs + OVER)) - OVER;
            e.subs = s.subs;
            e.h = (int)quotient(seg, max(s.groups, 1));
            e.rg = (int)(seg - (int64_t)e.h * s.groups);
            e.len = s.r.len;
            e.n = s.r.n;
            e.r0 = s.r.r0;
            if (e.i >= 0 && e.h < H) {
                e.tok = s.lo + e.i * SUB;
                const int32_t* table = a.s.table + (int64_t)b * a.s.table_stride;
                if (e.tok < s.r.len && ((e.tok >> sh) + 1) << sh > s.seen) e.p0 = table[e.tok >> sh];
                if (sh == 4 && e.tok + 16 < s.r.len && e.tok + 32 > s.seen) e.p1 = table[(e.tok >> 4) + 1];
                if (e.p0 >= a.c.pages) e.p0 = -1;
                if (e.p1 >= a.c.pages) e.p1 = -1;
                if (sh != 4) e.p1 = e.p0;
            }
        }
        Entry* to = run + (filled + lane) % RUN;
        __syncwarp();
        if (keep) *to = e;
        __syncwarp();
        filled += count;
        load();  // before the scales, whose addresses also wait for the pages
        if (keep && e.tok >= 0) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int p = y ? e.p1 : e.p0;
                if (p < 0) continue;
                to->ks[y] = a.c.k_scale[(int64_t)p * a.c.scale_stride + e.h];
                const float vs = a.c.v_scale[(int64_t)p * a.c.scale_stride + e.h];
                to->vs[y] = vs;
                if (vs != 0.f) to->lv[y] = __log2f(fabsf(vs));
            }
        }
        __syncwarp();
    };
    if (works) fill(RUN);

    // the segment being worked on
    uint32_t qf[C::QSMEM ? 1 : NT][CH][8];  // queries: a thread's chunks of its row
    uint2* qm = reinterpret_cast<uint2*>(smem + C::OFF_Q + warp * C::QBYTES) + lane;
    float qs[NT][2];          // scale of its columns' logits
    int pos[NT][2];           // positions of the columns' queries
    float acc[MT][NT][4];
    float m[NT][2], mw[NT][2], l[NT][2], lift[NT][2];
    bool open = false;        // a segment that goes on in the next worker's run
    int begun = 0;            // its first sub-tile here
    int last_at = 0;          // the place of its last entry here

    for (int k = 0; k < N; ++k) {
        if (filled < N && filled - k <= RUN - FILL) fill(FILL);
        const Entry& e = run[k % RUN];
        const int tok = e.tok;
        if (tok < 0) continue;
        const int first = e.len - e.n, rows = e.n * a.group;
        if (!open) {
            open = true;
            begun = e.i;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = e.rg * Q + nt * 8 + g;
                float top = 0.f, x[CH][16];
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    const int ch = DP == 64 ? c : 8 * (j >> 1) + 2 * c + (j & 1);
                    if (r < rows && ch * 16 < a.c.dim) {
                        const T* q = (const T*)a.q + (int64_t)(e.r0 + r / a.group) * a.q_row +
                                     (int64_t)(e.h * a.group + r % a.group) * a.q_head + ch * 16;
                        const uint4 v0 = *reinterpret_cast<const uint4*>(q), v1 = *reinterpret_cast<const uint4*>(q + 8);
                        const T* e0 = reinterpret_cast<const T*>(&v0);
                        const T* e1 = reinterpret_cast<const T*>(&v1);
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            x[j][y] = to_float(e0[y]);
                            x[j][8 + y] = to_float(e1[y]);
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 16; ++y) x[j][y] = 0.f;
                    }
#pragma unroll
                    for (int y = 0; y < 16; ++y) top = fmaxf(top, fabsf(x[j][y]));
                }
                // bfloat16 rows are brought into fp16's range by a power of
                // two: exact down to 2^-17 of it, below that off by at most
                // 2^-25 of it
                float unit = 1.f;
                if constexpr (!std::is_same<T, __half>::value) {
                    top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
                    const uint32_t ex = min(max(__float_as_uint(top) >> 23, 1u), 253u);
                    unit = __uint_as_float(ex << 23);
                    const float inv = __uint_as_float((254u - ex) << 23);
#pragma unroll
                    for (int j = 0; j < CH; ++j)
#pragma unroll
                        for (int y = 0; y < 16; ++y) x[j][y] *= inv;
                }
#pragma unroll
                for (int j = 0; j < CH; ++j)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint2 v = make_uint2(h2bits(__floats2half2_rn(x[j][4 * y], x[j][4 * y + 1])),
                                                   h2bits(__floats2half2_rn(x[j][4 * y + 2], x[j][4 * y + 3])));
                        if constexpr (C::QSMEM) {
                            qm[((nt * CH + j) * 4 + y) * 32] = v;  // read by the same thread only
                        } else {
                            qf[nt][j][2 * y] = v.x;
                            qf[nt][j][2 * y + 1] = v.y;
                        }
                    }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    qs[nt][y] = __shfl_sync(FULL, unit, (2 * c + y) * 4) * (a.scale * 1.4426950408889634f);
                    pos[nt][y] = first + (e.rg * Q + nt * 8 + 2 * c + y) / a.group;
                    m[nt][y] = mw[nt][y] = NONE;
                    l[nt][y] = 0.f;
                    lift[nt][y] = LIFT;
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int y = 0; y < 4; ++y) acc[i][nt][y] = 0.f;
            }
        }

        failed = __any_sync(FULL, !bspx::mbar_wait_bounded(full + stage, phase, d.spin_cap));
        if (failed) {
            // nothing more is loaded, and no copy may land in the ring (which
            // the CTA goes on to use) or after the CTA is gone; the rows of
            // this segment and of the warp's later ones are not written
            bool none = d.stall && k <= OVER;  // the first sub-tile's copies were skipped
            for (; loading; --loading) {
                if (!none) bspx::mbar_wait_bounded(full + stage, phase);
                none = false;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            __syncwarp();
            open = false;
            break;
        }
        const uint8_t* kt = ring + stage * C::STAGE;
        const uint8_t* vt = kt + C::HALF;
        const int p0 = e.p0, p1 = e.p1;
        if (p0 >= 0 || p1 >= 0) {
            const float kscale[2] = {e.ks[0], e.ks[1]}, vscale[2] = {e.vs[0], e.vs[1]};
            // S^T
            float sc[2][NT][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 4; ++y) sc[i][nt][y] = 0.f;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int ch = DP == 64 ? c : 2 * c + (j & 1);
                const uint8_t* reg = kt + (j >> 1) * SUB * C::BOX;
                uint4 v[2][2];  // rows g and g + 8 of each half
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 8 * i + g, sw = DP == 64 ? (row >> 1) & 3 : row & 7;
                    v[i >> 1][i & 1] = *reinterpret_cast<const uint4*>(reg + row * C::BOX + ((ch ^ sw) << 4));
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t z = (&v[i][y].x)[w] ^ 0x80808080u;
                            f[i][y] = widen(z, 0x4140);
                            f[i][2 + y] = widen(z, 0x4342);
                        }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint2 q;
                        if constexpr (C::QSMEM) q = qm[((nt * CH + j) * 4 + w) * 32];
                        else q = make_uint2(qf[nt][j][2 * w], qf[nt][j][2 * w + 1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            mma16816(sc[i][nt], f[i][0], f[i][1], f[i][2], f[i][3], q.x, q.y);
                    }
                }
            }
            // factors of the logits (in powers of two); where a query does not
            // see every row the masked logits themselves, and a factor of one
            const bool edge = tok + SUB - 1 > first || (a.window && tok <= e.len - 1 - a.window) || p0 < 0 || p1 < 0;
            const float lv[2] = {e.lv[0], e.lv[1]};
            float kf[2][NT][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) kf[i][nt][y] = kscale[i] * qs[nt][y];
            if (edge)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int j = tok + 16 * i + g + (y >> 1) * 8, p = pos[nt][y & 1];
                            const bool see = (i ? p1 : p0) >= 0 && j <= p && (!a.window || j > p - a.window);
                            sc[i][nt][y] = see ? sc[i][nt][y] * kf[i][nt][y & 1] : -INFINITY;
                        }
                        kf[i][nt][0] = kf[i][nt][1] = 1.f;
                    }
            // running maxima, allowed to lag
            bool lag = false;
            float hi[NT][2][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        hi[nt][y][i] = fmaxf(sc[i][nt][y], sc[i][nt][y + 2]) * kf[i][nt][y];
                    lag |= fmaxf(hi[nt][y][0], hi[nt][y][1]) > m[nt][y] + LAZY;
                    lag |= fmaxf(hi[nt][y][0] + lv[0], hi[nt][y][1] + lv[1]) > mw[nt][y] + LAZY;
                }
            if (__any_sync(FULL, lag)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float t = fmaxf(hi[nt][y][0], hi[nt][y][1]);
                        float tw = fmaxf(hi[nt][y][0] + lv[0], hi[nt][y][1] + lv[1]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) {
                            t = fmaxf(t, __shfl_xor_sync(FULL, t, x));
                            tw = fmaxf(tw, __shfl_xor_sync(FULL, tw, x));
                        }
                        t = fmaxf(t, m[nt][y]);
                        tw = fmaxf(fmaxf(tw, mw[nt][y]), t - DEEP);
                        l[nt][y] *= ex2(m[nt][y] - t);
                        const float back = ex2(mw[nt][y] - tw);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            acc[i][nt][y] *= back;
                            acc[i][nt][y + 2] *= back;
                        }
                        m[nt][y] = t;
                        mw[nt][y] = tw;
                        lift[nt][y] = ex2(t - tw) * LIFT;
                    }
            }
            // weights, as the B operand of the second product
            uint32_t wf[2][NT][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float p[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        p[y] = ex2(fmaf(sc[i][nt][y], kf[i][nt][y & 1], -m[nt][y & 1]));
                        l[nt][y & 1] += p[y];
                        p[y] *= weight_of(lift[nt][y & 1], vscale[i]);
                    }
                    wf[i][nt][0] = movmatrix(h2bits(__floats2half2_rn(p[0], p[1])));
                    wf[i][nt][1] = movmatrix(h2bits(__floats2half2_rn(p[2], p[3])));
                }
            // O^T
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * i + 2 * c;
#pragma unroll
                for (int rgn = 0; rgn < C::REGIONS; ++rgn) {
                    constexpr int WORDS = DP == 64 ? 2 : 4;  // of each row, a thread's dims
                    uint32_t t[4][4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int row = r + (x & 1) + 8 * (x >> 1);
                        const uint8_t* base = vt + rgn * SUB * C::BOX + row * C::BOX;
                        if constexpr (DP == 64) {
                            const uint2 v = *reinterpret_cast<const uint2*>(
                                base + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
                            t[x][0] = v.x ^ 0x80808080u;
                            t[x][1] = v.y ^ 0x80808080u;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(base + ((g ^ (row & 7)) << 4));
                            t[x][0] = v.x ^ 0x80808080u;
                            t[x][1] = v.y ^ 0x80808080u;
                            t[x][2] = v.z ^ 0x80808080u;
                            t[x][3] = v.w ^ 0x80808080u;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < WORDS; ++w)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t sel = half ? 0x7362 : 0x5140;
                            const uint32_t z0 = __byte_perm(t[0][w], t[1][w], sel);
                            const uint32_t z1 = __byte_perm(t[2][w], t[3][w], sel);
                            const uint32_t a0 = widen(z0, 0x4140), a1 = widen(z0, 0x4342);
                            const uint32_t a2 = widen(z1, 0x4140), a3 = widen(z1, 0x4342);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(acc[rgn * 8 + 2 * w + half][nt], a0, a1, a2, a3, wf[i][nt][0], wf[i][nt][1]);
                        }
                }
            }
        }
        __syncwarp();  // the stage is read: it may be filled again
        if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
        }
        --loading;
        load();
        last_at = k;
        if (e.i + 1 < e.subs) continue;

        // the segment ends here: its rows out, or the last part of it
        open = false;
        const bool whole = begun == 0;
        float* part = d.parts + (2 * (int64_t)worker + 1) * C::PART;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float sum = l[nt][y];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(FULL, sum, x);
                const int qr = nt * 8 + 2 * c + y, r = e.rg * Q + qr;
                const int64_t row = e.r0 + r / a.group, head = e.h * a.group + r % a.group;
#pragma unroll
                for (int i = 0; i < MT; i += 2) {
                    const int dim = DP == 64 ? g * 8 + 2 * i : (i >> 3) * 128 + g * 16 + 2 * (i & 7);
                    constexpr float f = 1.f / LIFT;
                    const float4 o = make_float4(acc[i][nt][y] * f, acc[i][nt][y + 2] * f, acc[i + 1][nt][y] * f,
                                                 acc[i + 1][nt][y + 2] * f);
                    if (!whole) *reinterpret_cast<float4*>(part + qr * DP + dim) = o;
                    else if (r < rows) store_out<T>(a, row, head, dim, o, m[nt][y], mw[nt][y], sum);
                }
                if (!whole && g == 0) {
                    part[Q * DP + qr] = m[nt][y];
                    part[Q * DP + Q + qr] = sum;
                    part[Q * DP + 2 * Q + qr] = mw[nt][y];
                }
            }
    }
    if (failed && lane == 0) atomicExch(d.err, (int)BSP_ERR_TIMEOUT);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel, as SMs fall free

    // rows past the step's
    {
        const int64_t live = B ? min((int64_t)max(a.s.q_start[B], 0), a.s.rows) : (int64_t)0;
        const int64_t vec = a.c.dim / 8, all = (a.s.rows - live) * a.heads * vec;
        for (int64_t i = (int64_t)blockIdx.x * blockDim.x + tid; i < all; i += (int64_t)gridDim.x * blockDim.x) {
            const int64_t row = live + i / (a.heads * vec), head = i / vec % a.heads;
            *reinterpret_cast<uint4*>((T*)a.out + row * a.o_row + head * a.o_head + i % vec * 8) = make_uint4(0, 0, 0, 0);
            if (a.lse && i % vec == 0) a.lse[row * a.heads + head] = -INFINITY;
        }
    }

    // Segments that go on beyond the warps' runs.  The warps of a CTA that
    // are on the same one add their sums in shared memory (the ring is idle).
    int64_t* seg_at = reinterpret_cast<int64_t*>(smem + C::OFF_AT);  // place of the segment's first sub-tile, -1: none
    Entry* seg_entry = reinterpret_cast<Entry*>(smem + C::OFF_SEG);
    if (lane == 0) {
        seg_at[warp] = -1;
        if (open) {
            seg_entry[warp] = run[last_at % RUN];
            seg_at[warp] = x0 + last_at - seg_entry[warp].i;
        }
    }
    if (open)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float sum = l[nt][y];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(FULL, sum, x);
                if (g == 0) {
                    float* st = stat + warp * 3 * Q + nt * 8 + 2 * c + y;
                    st[0] = m[nt][y];
                    st[Q] = sum;
                    st[2 * Q] = mw[nt][y];
                }
            }
    __syncthreads();
    float* join = reinterpret_cast<float*>(smem);  // [warp][Q][OPAD]
    if (open)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int qr = nt * 8 + 2 * c + y;
                float top = NONE;
                for (int w = 0; w < DEC_WARPS; ++w)
                    if (seg_at[w] == seg_at[warp]) top = fmaxf(top, stat[w * 3 * Q + 2 * Q + qr]);
                const float f = ex2(mw[nt][y] - top) * (1.f / LIFT);
                float* o = join + (warp * Q + qr) * C::OPAD;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int dim = DP == 64 ? g * 8 + 2 * i : (i >> 3) * 128 + g * 16 + 2 * (i & 7);
                    *reinterpret_cast<float2*>(o + dim) = make_float2(acc[i][nt][y] * f, acc[i][nt][y + 2] * f);
                }
            }
    __syncthreads();
    if (tid == 0)  // this CTA's share of the list: its workers', and of those that there are not
        for (int i = 0; i < DEC_WARPS; ++i)
            d.cuts[i < wpc ? blockIdx.x * wpc + i : gridDim.x * wpc + blockIdx.x * (DEC_WARPS - wpc) + i - wpc].last = -1;
    for (int w0 = 0; w0 < wpc;) {
        const int64_t at = seg_at[w0];
        int w1 = w0 + 1;
        while (w1 < wpc && seg_at[w1] == at) ++w1;
        if (at >= 0) {
            float* part = d.parts + 2 * (int64_t)(blockIdx.x * wpc + w0) * C::PART;
            for (int i = tid; i < Q * (DP / 4); i += DEC_WARPS * 32) {
                const int qr = i / (DP / 4), dim = i % (DP / 4) * 4;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                float top = NONE, sum = 0.f, topw = NONE;
                for (int w = w0; w < w1; ++w) {
                    const float4 x = *reinterpret_cast<const float4*>(join + (w * Q + qr) * C::OPAD + dim);
                    o.x += x.x;
                    o.y += x.y;
                    o.z += x.z;
                    o.w += x.w;
                    top = fmaxf(top, stat[w * 3 * Q + qr]);
                    topw = fmaxf(topw, stat[w * 3 * Q + 2 * Q + qr]);
                }
                for (int w = w0; w < w1; ++w) sum += stat[w * 3 * Q + Q + qr] * ex2(stat[w * 3 * Q + qr] - top);
                *reinterpret_cast<float4*>(part + qr * DP + dim) = o;
                if (dim == 0) {
                    part[Q * DP + qr] = top;
                    part[Q * DP + Q + qr] = sum;
                    part[Q * DP + 2 * Q + qr] = topw;
                }
            }
            // the worker that begins the segment says who ends it
            const Entry& e = seg_entry[w0];
            const int me = blockIdx.x * wpc + w0;
            if (tid == 0 && split.worker(at) == me)
                d.cuts[me] = {split.worker(at + e.subs - 1), wpc, e.r0, e.n, e.h, e.rg, {0, 0}};
        }
        w0 = w1;
    }
    if (d.beside) wait_prior_grids();
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

template <class T, int DP, int NT>
bsp_status_t launch_decode(const bsp_kv* h, const DecodeArgs& d, cudaStream_t s)
{
    using C = DecCfg<DP, NT>;
    static bsp_attr_once attr_once;
    static int per_sm[64];
    const int dev = h->device;
    if (!attr_once.run(dev, [&] {
            cudaError_t e = cudaFuncSetAttribute(kv_decode_kernel<T, DP, NT>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm[dev], kv_decode_kernel<T, DP, NT>,
                                                                  DEC_WARPS * 32, C::SMEM);
            return e;
        }))
        return BSP_ERR_CUDA;
    const int grid = h->num_sms * std::min(std::max(per_sm[dev], 1), C::CTAS);
    if (!launch_early(kv_decode_kernel<T, DP, NT>, dim3((unsigned)grid), dim3(DEC_WARPS * 32), C::SMEM, s, h->map_k,
                      h->map_v, d))
        return BSP_ERR_CUDA;
    return launch_early(kv_join_kernel<T, DP, NT>, dim3((unsigned)(h->num_sms * JOIN_CTAS)), dim3(JOIN_WARPS * 32), 0, s,
                        d, grid * DEC_WARPS)
               ? BSP_OK
               : BSP_ERR_CUDA;
}

template <class T>
bsp_status_t run(const bsp_kv* h, const AttnArgs& a, int64_t max_new, cudaStream_t s)
{
    // Query blocks of 8, 16 or 24 rows: the smallest that holds the largest
    // request.  Requests with more rows are the prompt kernel's, whose row
    // tiles have 128 rows and whose dims end at 128.
    //
    // Steps of few rows in all stay here, in several blocks, each of which
    // reads the codes again.  One request, 64 over 8 heads of 128, here |
    // prompt kernel, cold: 16 rows (1024 rows x heads) 20.5 | 44 us with nothing
    // cached, 27 | 44 with 500, 39 | 48 with 4000, 184 | 87 with 60000; 64 rows
    // 25 | 38, 31 | 40, 64 | 46, 582 | 159.  The host does not know the lengths
    // in the device's arrays: 1024 costs short requests of up to 4096 at most
    // 24 us, and long ones of up to 1024 twice their time.
    //
    // A step with prompts is taken for one of prompts and single tokens, and
    // the block for a single token's rows.  A chunk of 513 beside 16 single
    // tokens in groups of 8: 48 us with blocks of 8, 58 with 24; beside 64 single
    // heads' tokens 497 and 685.  Drafts of more rows then go to the prompt
    // kernel: 16 of 5 tokens in groups of 4 56 and 62 us, but 3 of them over
    // 60k .. 120k rows 1293 and 177.
    const int64_t most = max_new * a.group;
    const bool prompts = most > 24 && a.c.dim <= 128 && a.s.batch > 0 && a.s.rows * a.heads > 1024;
    const int64_t block = prompts ? std::min<int64_t>(a.group, 24) : most;
    const int few = block <= 8 ? 8 : block <= 16 ? 16 : 24;
    bool beside = false;
    if (prompts) {
        const bsp_status_t st =
            bsp_run_kv_prompt(h, a, std::is_same<T, __half>::value ? BSP_FP16 : BSP_BF16, few, &beside, s);
        if (st != BSP_OK) return st;
    }
    const DecodeArgs d = {a, h->parts, h->cuts, h->err, bsp_spin_cap(), prompts ? few : INT32_MAX,
                          prompts ? h->ready : nullptr, beside, bsp_test_stall() != 0};
    if (a.c.dim <= 64)
        return few == 8 ? launch_decode<T, 64, 1>(h, d, s) : few == 16 ? launch_decode<T, 64, 2>(h, d, s)
                                                                       : launch_decode<T, 64, 3>(h, d, s);
    if (a.c.dim <= 128)
        return few == 8 ? launch_decode<T, 128, 1>(h, d, s) : few == 16 ? launch_decode<T, 128, 2>(h, d, s)
                                                                        : launch_decode<T, 128, 3>(h, d, s);
    return few == 8 ? launch_decode<T, 256, 1>(h, d, s) : launch_decode<T, 256, 2>(h, d, s);
}

}  // namespace

namespace bspkv {

bsp_status_t attention_setup(bsp_kv* h, cudaStream_t s)
{
    auto encode = encode_fn();
    if (!encode) return BSP_ERR_CUDA;
    const KvView& c = h->view;
    const int page = 1 << c.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)page, (cuuint64_t)c.heads, (cuuint64_t)c.pages};
    // a stride that is never used (one head, one page) is any valid one
    const cuuint64_t row = (cuuint64_t)c.row_stride;
    const cuuint64_t head = c.heads > 1 ? (cuuint64_t)c.head_stride : row * page;
    const cuuint64_t pg = c.pages > 1 ? (cuuint64_t)c.page_stride : head * c.heads;
    const cuuint64_t strides[3] = {row, head, pg};
    const cuuint32_t box[4] = {(cuuint32_t)(c.dim <= 64 ? 64 : 128), (cuuint32_t)std::min(page, SUB), 1, 1};
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    for (int i = 0; i < 2; ++i)
        if (encode(i ? &h->map_v : &h->map_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, i ? c.v : c.k, dims, strides, box, unit,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, c.dim <= 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return BSP_ERR_SHAPE;
    const size_t workers = (size_t)h->num_sms * 3 * DEC_WARPS;  // at most
    auto floats = [](auto cfg) { return (size_t)decltype(cfg)::CTAS * decltype(cfg)::PART; };
    const size_t part = c.dim <= 64 ? std::max(floats(DecCfg<64, 1>{}), floats(DecCfg<64, 3>{}))
                        : c.dim <= 128 ? std::max(floats(DecCfg<128, 1>{}), floats(DecCfg<128, 3>{}))
                                       : floats(DecCfg<256, 2>{});
    h->part_floats = (size_t)h->num_sms * DEC_WARPS * 2 * part;
    if (cudaMalloc(&h->parts, h->part_floats * sizeof(float)) != cudaSuccess ||
        cudaMalloc(&h->cuts, workers * sizeof(KvCut)) != cudaSuccess)
        return BSP_ERR_OOM;
    if (cudaMemsetAsync(h->cuts, 0, workers * sizeof(KvCut), s) != cudaSuccess) return BSP_ERR_CUDA;
    return BSP_OK;
}

void attention_free(bsp_kv* h)
{
    cudaFree(h->parts);
    cudaFree(h->cuts);
}

}  // namespace bspkv

bsp_status_t bsp_run_kv_attention(const bsp_kv* h, const KvStepView& st, int64_t max_new, const void* q,
                                  bsp_dtype_t dtype, int32_t heads, int64_t q_row, int64_t q_head, float scale,
                                  int32_t window, void* out, int64_t o_row, int64_t o_head, float* lse,
                                  cudaStream_t s)
{
    // a window no row can look beyond is none (and positions minus a window stay in 32 bits)
    if (window >= (int64_t)st.width << h->view.page_shift) window = 0;
    const AttnArgs a = {h->view, st, q, out, lse, q_row, q_head, o_row, o_head, scale, heads, heads / h->view.heads,
                        window};
    return dtype == BSP_FP16 ? run<__half>(h, a, max_new, s) : run<__nv_bfloat16>(h, a, max_new, s);
}
