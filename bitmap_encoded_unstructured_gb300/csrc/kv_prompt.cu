// Attention of many queries (prompts, chunks of prompts) over the paged
// 8-bit cache, on the 5th-generation tensor cores.
//
// A CTA takes 256 query rows of one request and KV head (a row = a query
// token and one of the heads that share the KV head) as two row tiles of
// 128, and walks the cached rows they see in tiles of 128:
//   S = Q . codes_K^T     tcgen05.mma 128 x 128 x dim, Q and K in shared memory
//   P = 2^(S * k scale - m), W = fp16(P * V scale)      one thread per row
//   O += W . codes_V      tcgen05.mma 128 x dim x 128, W in tensor memory
// The codes are exact in fp16, so the products see them unrounded; the
// scales (one for each page) are factors of 16 or more columns and are
// applied to S and P.  While one row tile's softmax runs, the tensor cores
// work on the other's.
//
// Warps: 0 loads codes (TMA boxes of the paged cache) and scales; 1 issues
// the MMAs; 4-7 turn codes into fp16 tiles; 8-11 and 12-15 are the softmax
// of row tiles 0 and 1 (a warp reaches the 32 tensor-memory lanes 32 (w % 4)
// .. + 31).  Rings of tiles in the order the products need them, K0 V0 K1 V1
// ..: codes (four deep) and fp16 tiles (three: V of a tile and K of the next
// are live while the next V is made).  Both fp16 tiles have one layout, rows
// of 64 dims swizzled by 128 bytes: K-major for the first product, MN-major
// for the second.
// Tensor memory: S0, S1 (128 fp32 columns each; W takes the lower half of
// its own S), O0, O1.  Products of one thread run in order, so the next S
// may be asked for right after the product that reads W.
//
// Bound by each row tile's chain S -> P -> W -> S (issue slots are 55% busy, the
// tensor pipe 56%): a prompt of 8101 rows, 64 heads over 8 KV heads of 128,
// takes 845 us (1.075 TFLOP at 1273 TFLOP/s, 0.65 of the library's bf16
// product).  Two threads a row (16
// softmax warps of 96 registers) were slower, 1070 us: a barrier a tile joins
// the halves, and half the registers spill.
#include "bsp_kv.cuh"

#include <algorithm>
#include <type_traits>

namespace {

using namespace bspkv;

constexpr uint32_t FULL = 0xFFFFFFFFu;
constexpr int ROWS = 256;      // query rows of a CTA
constexpr int TOK = 128;       // cached rows of a tile
constexpr int GROUPS = TOK / 16;
constexpr int NC = 4, NF = 3, NM = 8;  // rings: codes, fp16 tiles, scales
constexpr int THREADS = 512;
// Registers of a thread after the roles part, from 128 of each at launch: the
// softmax keeps a row of 128 logits.
constexpr int REG_CONTROL = 48, REG_CONVERT = 48, REG_SOFTMAX = 208;
static_assert(REG_CONTROL + REG_CONVERT + 2 * REG_SOFTMAX == 4 * 128, "shares of the launch's registers");

template <int DP>
struct Cfg {
    static constexpr int QBLK = 128 * 128, BLK = TOK * 128;  // 64 dims of a row tile's Q, of an fp16 tile
    static constexpr int QT = QBLK * (DP / 64);         // Q of a row tile
    static constexpr int FT = BLK * (DP / 64);          // fp16 K or V tile
    static constexpr int CT = TOK * DP;                 // codes of a tile
    static constexpr int OFF_F = 2 * QT;
    static constexpr int OFF_C = OFF_F + NF * FT;
    static constexpr int OFF_META = OFF_C + NC * CT;    // per scale slot: ks, vs, log2 vs [8] each, mask
    static constexpr int META = 3 * GROUPS + 4;         // floats
    static constexpr int OFF_BAR = OFF_META + NM * META * 4;
    static constexpr int NBAR = 2 * NC + 2 * NF + NM + 1 + 3 * 2 + 2;
    static constexpr int END = OFF_BAR + NBAR * 8 + 16;
    // one CTA per SM: it may take all of the tensor memory
    static constexpr int SMEM = (END > 120 * 1024 ? END : 120 * 1024) + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

constexpr int MOST_SPLITS = 16;

struct PromptArgs {
    AttnArgs a;
    int *err, *ready;
    uint32_t spin_cap;
    int32_t few;
    int32_t splits;  // CTAs that share the cached rows of a row tile pair
    int64_t items;   // row tile pairs of one KV head
    float* parts;    // splits > 1: of CTA i and row r, O, m, l, mw at (i ROWS + r) (DP + 4)
    bool stall;      // test only: the copies of the first tile are skipped
};

// The item a CTA (or its part) works on: request b, its first query row.
struct Item {
    int b;
    int64_t row0;
};

// Request b's items start at F(b) = q_start[b] * group / ROWS + b: it has at
// most n * group / ROWS + 1, so F leaves room for them without a scan.
__device__ __forceinline__ Item item_of(const AttnArgs& a, int64_t item)
{
    int b = 0, hi = a.s.batch;
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if ((int64_t)a.s.q_start[mid] * a.group / ROWS + mid <= item) b = mid;
        else hi = mid;
    }
    return {b, (item - ((int64_t)a.s.q_start[b] * a.group / ROWS + b)) * ROWS};
}

// kind::f16 instruction descriptor: D fp32, A and B fp16, M = 128.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn_major)
{
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// Shared-memory matrix descriptor, rows of 128 B swizzled by 128 B, 8-row
// atoms of 1 KB.  K-major: the rows are M or N, the stride between atoms is
// 1 KB, the leading offset is not used.  MN-major: the rows are K, the
// stride between 8-row atoms is 1 KB and the leading offset is the distance
// of the next 64 columns.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t leading)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((leading >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((1024u >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1u << 46;  // descriptor version of sm_100
    d |= (uint64_t)2u << 61;  // SWIZZLE_128B
    return d;
}

// Products and commits are written for the whole warp, with the one thread
// that issues them elected inside: the operands then stay in uniform
// registers.  Issued under a branch on the lane, each product would wait for
// its descriptors to be moved there (86 cycles a product, more than it takes).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}

__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bspx::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}

// 32 consecutive tensor-memory columns of this thread's lane; they are there
// after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}

// The loaded registers pass through, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r, int n)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < n; ++i) asm volatile("" : "+r"(r[i]));
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <int REGS>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// The whole warp waits; false if the wait ran out.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t cap)
{
    return __all_sync(FULL, bspx::mbar_wait_bounded(bar, parity, cap));
}

template <class T, int DP>
__global__ void __launch_bounds__(THREADS, 1)
kv_prompt_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const PromptArgs d)
{
    using C = Cfg<DP>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (bspx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const AttnArgs& a = d.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sh = a.c.page_shift, dim = a.c.dim;
    const int H = a.c.heads;

    wait_prior_grids();
    // for the kernel that may start beside this one (below): the kernels before
    // this one are done
    if (blockIdx.x == 0 && threadIdx.x == 0)
        asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(d.ready) : "memory");

    // the item: long rows first (later rows of a causal prompt see more),
    // the heads of one row tile pair side by side
    const int piece = (int)(blockIdx.x % d.splits), h = (int)(blockIdx.x / d.splits % H);
    const Item it = item_of(a, d.items - 1 - (int64_t)(blockIdx.x / d.splits / H));
    const int b = it.b;
    const int64_t row0 = it.row0;
    const Request rq = request_of(a.s, sh, b);
    const int64_t rows = (int64_t)rq.n * a.group;
    if (row0 < 0 || row0 >= rows || rows <= d.few) return;
    const int n_rows = (int)min((int64_t)ROWS, rows - row0);
    const bool two = n_rows > 128;
    const int first = rq.len - rq.n;                                 // position of the request's first query
    const int pos0 = first + (int)(row0 / a.group), pos1 = first + (int)((row0 + n_rows - 1) / a.group);
    const int seen = a.window ? max(0, pos0 - a.window + 1) : 0;    // first cached row that a query sees
    const int all_tiles = pos1 >= 0 ? (pos1 + 1 - (seen & ~(TOK - 1)) + TOK - 1) / TOK : 0;
    const int first_tile = (int)((int64_t)all_tiles * piece / d.splits);
    const int tiles = (int)((int64_t)all_tiles * (piece + 1) / d.splits) - first_tile;
    const int t0 = (seen & ~(TOK - 1)) + first_tile * TOK;
    const uint32_t cap = d.spin_cap;

    uint64_t* c_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* c_empty = c_full + NC;
    uint64_t* f_full = c_empty + NC;
    uint64_t* f_empty = f_full + NF;
    uint64_t* m_full = f_empty + NF;
    uint64_t* q_full = m_full + NM;
    uint64_t* s_full = q_full + 1;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_done = p_full + 2;
    uint64_t* drain = o_done + 2;
    uint64_t* read = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(read + 1);
    float* meta = reinterpret_cast<float*>(smem + C::OFF_META);

    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         bspx::smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NC; ++i) {
            bspx::mbar_init(c_full + i, 1);
            bspx::mbar_init(c_empty + i, 4);
        }
        for (int i = 0; i < NF; ++i) {
            bspx::mbar_init(f_full + i, 4);
            bspx::mbar_init(f_empty + i, 1);
        }
        for (int i = 0; i < NM; ++i) bspx::mbar_init(m_full + i, 1);
        bspx::mbar_init(q_full, 8);
        for (int i = 0; i < 2; ++i) {
            bspx::mbar_init(s_full + i, 1);
            bspx::mbar_init(p_full + i, 4);
            bspx::mbar_init(o_done + i, 1);
        }
        bspx::mbar_init(drain, 1);
        bspx::mbar_init(read, 8);
        bspx::fence_mbar_init();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    bool failed = false;
    // What comes next (the kernel of the other requests) may fill the SMs that
    // this one leaves idle.  Its launch orders no memory: what was written
    // before this kernel it sees through `ready`.  Not before the tensor memory
    // is ours: the kernels behind start early in their turn, and a product
    // kernel that took some of it here first, waiting for this grid to end,
    // would never let this CTA have it.
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp < 4) fewer_registers<REG_CONTROL>();
    if (warp == 0) {
        // ---------------- codes and scales: lane l < 8 looks after rows 16 l ..
        const int32_t* table = a.s.table + (int64_t)b * a.s.table_stride;
        const int box = min(32, 1 << sh);
        auto page_of = [&](int j) {
            const int tok = t0 + j * TOK + 16 * lane;
            int p = -1;
            if (lane < GROUPS && j < tiles && tok < rq.len && ((tok >> sh) + 1) << sh > seen) {
                p = table[tok >> sh];
                if (p >= a.c.pages) p = -1;
            }
            return p;
        };
        int n = 0;  // tiles issued
        auto load = [&](const CUtensorMap* map, int j, int p) {
            const int slot = n % NC;
            if (failed || (n >= NC && !wait(c_empty + slot, (n / NC - 1) & 1, cap))) {
                failed = true;
                return;
            }
            const bool mine = p >= 0 && (box == 16 || (lane & 1) == 0);
            const uint32_t bytes = __popc(__ballot_sync(FULL, mine)) * box * DP;
            const bool skip = d.stall && n == 0;
            if (lane == 0 && !skip) {
                if (bytes) bspx::mbar_arrive_expect_tx(c_full + slot, bytes);
                else bspx::mbar_arrive(c_full + slot);
            }
            __syncwarp();
            if (mine && !skip)
                tma_load_4d(smem + C::OFF_C + slot * C::CT + 16 * lane * DP, map, 0,
                            (t0 + j * TOK + 16 * lane) & ((1 << sh) - 1), h, p, c_full + slot);
            ++n;
        };
        // what is looked up for a tile travels ahead of its loads, so that no
        // step waits for the table or the scales
        auto scale_of = [&](const float* scale, int p) {
            return p >= 0 ? scale[(int64_t)p * a.c.scale_stride + h] : 0.f;
        };
        auto load_k = [&](int j, int p, float ks, float vs) {
            load(&map_k, j, p);
            if (failed) return;
            // slot j % NM was last read for tile j - NM, whose products are
            // done: the codes of tile j could not have been asked for otherwise
            float* mt = meta + (j % NM) * C::META;
            const uint32_t there = __ballot_sync(FULL, p >= 0);
            if (lane < GROUPS) {
                mt[lane] = ks;
                mt[GROUPS + lane] = vs;
                mt[2 * GROUPS + lane] = vs != 0.f ? __log2f(fabsf(vs)) : NONE;
            }
            if (lane == 0) reinterpret_cast<uint32_t*>(mt)[3 * GROUPS] = there;
            __syncwarp();
            if (lane == 0) bspx::mbar_arrive(m_full + j % NM);
        };
        int p0 = page_of(0), p1 = page_of(1), p2 = page_of(2);  // of tiles j .. j + 2
        float ks0 = scale_of(a.c.k_scale, p0), vs0 = scale_of(a.c.v_scale, p0);  // of tiles j, j + 1
        float ks1 = scale_of(a.c.k_scale, p1), vs1 = scale_of(a.c.v_scale, p1);
        for (int j = 0; j < tiles && !failed; ++j) {
            const int p3 = page_of(j + 3);
            const float ks2 = scale_of(a.c.k_scale, p2), vs2 = scale_of(a.c.v_scale, p2);
            load_k(j, p0, ks0, vs0);
            load(&map_v, j, p0);
            p0 = p1;
            p1 = p2;
            p2 = p3;
            ks0 = ks1;
            vs0 = vs1;
            ks1 = ks2;
            vs1 = vs2;
        }
        // no copy may land after the CTA is gone (the full cap, whatever `cap` is)
        for (int i = std::max(d.stall ? 1 : 0, n - NC); i < n; ++i)
            bspx::mbar_wait_bounded(c_full + i % NC, (i / NC) & 1);
        if (failed && lane == 0) atomicExch(d.err, (int)BSP_ERR_TIMEOUT);
        return;
    }
    if (warp == 1) {
        // ---------------- MMA issuer (control flow and operands uniform)
        const int n_tiles = __shfl_sync(FULL, tiles, 0);
        const bool pair_of = __any_sync(FULL, two);
        const uint32_t tm = __shfl_sync(FULL, tmem, 0);
        if (n_tiles) {
            const uint64_t q_desc = smem_desc(bspx::smem_u32(smem), 16);
            const uint64_t k_desc = smem_desc(bspx::smem_u32(smem + C::OFF_F), 16);
            const uint64_t v_desc = smem_desc(bspx::smem_u32(smem + C::OFF_F), C::BLK);
            const uint32_t id_s = idesc(TOK, false), id_o = idesc(dim, true);
            // (the fence orders products after other threads' tensor-memory
            // accesses, and stops their overlap: only where there are some)
            auto ready = [&](uint64_t* bar, uint32_t parity) {
                if (!wait(bar, parity, cap)) failed = true;
                return !failed;
            };
            auto ready_w = [&](int t, int j) {
                const bool ok = ready(p_full + t, j & 1);
                tc_after();
                return ok;
            };
            auto product_s = [&](int t, int slot) {  // S of row tile t, from a slot of the fp16 ring
                const uint64_t qd = q_desc + t * (C::QT >> 4), kd = k_desc + slot * (C::FT >> 4);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)  // dims past dim are zeros
                    mma_ss(tm + t * TOK, qd + ((k >> 2) * (C::QBLK >> 4) + (k & 3) * 2),
                           kd + ((k >> 2) * (C::BLK >> 4) + (k & 3) * 2), id_s, k ? 1u : 0u);
                commit(s_full + t);
            };
            auto product_o = [&](int t, int j, int slot) {
                const uint64_t vd = v_desc + slot * (C::FT >> 4);
#pragma unroll
                for (int k = 0; k < TOK / 16; ++k)
                    mma_ts(tm + 2 * TOK + t * DP, tm + t * TOK + 8 * k, vd + k * (2048 >> 4), id_o,
                           (j || k) ? 1u : 0u);
                // earlier products of O are known to be done by the S after them
                if (j == n_tiles - 1) commit(o_done + t);
            };
            int slot = 0;           // of the fp16 ring
            uint32_t phase = 0;     // and its phase
            auto next = [&]() {
                if (++slot == NF) {
                    slot = 0;
                    phase ^= 1u;
                }
            };
            if (ready(q_full, 0) && ready(f_full, 0)) {
                product_s(0, 0);
                if (pair_of) product_s(1, 0);
                commit(f_empty);
                next();
                for (int j = 0; j < n_tiles; ++j) {
                    const bool more = j + 1 < n_tiles;
                    const int v = slot;
                    if (!ready(f_full + v, phase) || !ready_w(0, j)) break;
                    product_o(0, j, v);
                    next();
                    if (more) {
                        if (!ready(f_full + slot, phase)) break;
                        product_s(0, slot);
                    }
                    if (pair_of) {
                        if (!ready_w(1, j)) break;
                        product_o(1, j, v);
                    }
                    commit(f_empty + v);
                    if (more) {
                        if (pair_of) product_s(1, slot);
                        commit(f_empty + slot);
                        next();
                    }
                }
            }
        }
        // no product in flight (after a wait ran out) and nobody reading when
        // the tensor memory is given back: with the full cap, and for readers
        // that may be in two waits of their own before they say so
        __syncwarp();
        commit(drain);
        if (!wait(drain, 0, bspx::kSpinCap)) failed = true;
        bool done = false;
        for (int i = 0; i < 4 && !done; ++i) done = wait(read, 0, bspx::kSpinCap);
        if (!done) failed = true;
        if (failed && lane == 0) atomicExch(d.err, (int)BSP_ERR_TIMEOUT);
        tc_after();
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
        return;
    }
    if (warp < 4) return;
    if (warp < 8) {
        fewer_registers<REG_CONVERT>();
        // ---------------- codes -> fp16.  A thread's chunk of 16 codes and the
        // rows of its eight-lane phase (r and r ^ 5) are such that both the
        // loads and the two stores of a phase fall into distinct banks.
        const int w = warp & 3, c = lane & 3, r8 = ((lane >> 3) & 3) ^ ((lane & 4) ? 5 : 0);
        for (int n = 0; n < 2 * tiles; ++n) {
            const int from = n % NC, to = n % NF;
            if (!wait(c_full + from, (n / NC) & 1, cap) || (n >= NF && !wait(f_empty + to, (n / NF - 1) & 1, cap))) {
                failed = true;
                break;
            }
            const uint8_t* src = smem + C::OFF_C + from * C::CT;
            uint8_t* dst = smem + C::OFF_F + to * C::FT;
#pragma unroll
            for (int i = 0; i < TOK / 32; ++i) {
                const int row = 8 * (w + 4 * i) + r8;
#pragma unroll
                for (int half = 0; half < DP / 64; ++half) {
                    const int ch = c + 4 * half;
                    const int sw = DP == 64 ? (row >> 1) & 3 : row & 7;
                    const uint4 v = *reinterpret_cast<const uint4*>(src + row * DP + ((ch ^ sw) << 4));
                    const uint32_t x[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
                    uint8_t* at = dst + half * C::BLK + row * 128;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<uint4*>(at + (((2 * c + e) ^ (row & 7)) << 4)) =
                            make_uint4(widen(x[2 * e], 0x4140), widen(x[2 * e], 0x4342), widen(x[2 * e + 1], 0x4140),
                                       widen(x[2 * e + 1], 0x4342));
                }
            }
            bspx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                bspx::mbar_arrive(f_full + to);
                bspx::mbar_arrive(c_empty + from);
            }
        }
        if (failed && lane == 0) atomicExch(d.err, (int)BSP_ERR_TIMEOUT);
        return;
    }
    more_registers<REG_SOFTMAX>();
    {
        // ---------------- softmax of one row per thread
        const int t = (warp - 8) >> 2, quad = warp & 3;
        const int tr = 32 * quad + lane;                     // row of the tile
        const int64_t r = row0 + 128 * t + tr;               // row of the request
        const bool mine = 128 * t + tr < n_rows;
        const int64_t q_tok = rq.r0 + r / a.group;
        const int head = h * a.group + (int)(r % a.group);
        // the warp's 32 query rows to shared memory, DP / 8 lanes to a row;
        // bfloat16 rows are brought into fp16's range by a power of two (exact
        // down to 2^-17 of it, below that off by at most 2^-25 of it)
        float unit = 1.f;
        {
            constexpr int LANES = DP / 8, STEP = 32 / LANES;
            const int col = lane % LANES;
            const int64_t at = q_tok * a.q_row + (int64_t)head * a.q_head;  // of this thread's row
            uint4 v[32 / STEP];
#pragma unroll
            for (int i = 0; i < 32 / STEP; ++i) {
                const int src = STEP * i + lane / LANES;  // row of the warp
                const int64_t from = __shfl_sync(FULL, at, src);
                v[i] = make_uint4(0, 0, 0, 0);
                if (128 * t + 32 * quad + src < n_rows && 8 * col < dim)
                    v[i] = *reinterpret_cast<const uint4*>((const T*)a.q + from + 8 * col);
            }
#pragma unroll
            for (int i = 0; i < 32 / STEP; ++i) {
                const int src = STEP * i + lane / LANES, row = 32 * quad + src;
                if constexpr (!std::is_same<T, __half>::value) {
                    const T* e = reinterpret_cast<const T*>(&v[i]);
                    float top = 0.f;
#pragma unroll
                    for (int x = 0; x < 8; ++x) top = fmaxf(top, fabsf(to_float(e[x])));
#pragma unroll
                    for (int x = 1; x < LANES; x <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, x));
                    const uint32_t ex = min(max(__float_as_uint(top) >> 23, 1u), 253u);
                    const float inv = __uint_as_float((254u - ex) << 23);
                    uint32_t y[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        y[x] = h2bits(__floats2half2_rn(to_float(e[2 * x]) * inv, to_float(e[2 * x + 1]) * inv));
                    v[i] = make_uint4(y[0], y[1], y[2], y[3]);
                    // row src's unit to its thread
                    const float u = __shfl_sync(FULL, __uint_as_float(ex << 23), (lane % STEP) * LANES);
                    if (lane / STEP == i) unit = u;
                }
                *reinterpret_cast<uint4*>(smem + t * C::QT + (col >> 3) * C::QBLK + row * 128 +
                                          (((col & 7) ^ (row & 7)) << 4)) = v[i];
            }
            bspx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) bspx::mbar_arrive(q_full);
        }
        const float unit_scale = unit * (a.scale * 1.4426950408889634f);
        const int pos = mine ? first + (int)(r / a.group) : -1;
        const int tile_pos0 = first + (int)((row0 + 128 * t) / a.group);
        const int tile_pos1 = first + (int)((row0 + min(128 * t + 127, n_rows - 1)) / a.group);
        const uint32_t s_at = tmem + t * TOK + ((uint32_t)(32 * quad) << 16);
        const uint32_t o_at = tmem + 2 * TOK + t * DP + ((uint32_t)(32 * quad) << 16);
        float m = NONE, mw = NONE, l = 0.f, lift = LIFT;
        const int my_tiles = t == 0 || two ? tiles : 0;
        for (int j = 0; j < my_tiles; ++j) {
            if (!wait(m_full + j % NM, (j / NM) & 1, cap) || !wait(s_full + t, j & 1, cap)) {
                failed = true;
                break;
            }
            tc_after();
            const float* mt = meta + (j % NM) * C::META;
            const uint32_t there = reinterpret_cast<const uint32_t*>(mt)[3 * GROUPS];
            const int tok = t0 + j * TOK;
            const bool edge = tok + TOK - 1 > tile_pos0 || (a.window && tok <= tile_pos1 - a.window) || there != (1u << GROUPS) - 1u;
            // columns lo .. hi of this tile are this row's
            const int hi = pos - tok, lo = (a.window ? max(pos - a.window + 1, 0) : 0) - tok;
            uint32_t x[TOK];
            __syncwarp();
#pragma unroll
            for (int cb = 0; cb < TOK; cb += 32) tmem_ld32(s_at + cb, x + cb);
            float kf[GROUPS];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) kf[g] = fmaxf(mt[g] * unit_scale, 1e-30f);  // a masked -inf stays one
            tmem_wait_ld(x, TOK);
            if (edge) {
#pragma unroll
                for (int w = 0; w < TOK / 32; ++w) {
                    // bits lo .. hi of this word, and the pages that are there
                    const int h = hi - 32 * w, o = lo - 32 * w;
                    uint32_t see = h < 0 ? 0u : h >= 31 ? FULL : (2u << h) - 1u;
                    see &= o <= 0 ? FULL : o >= 32 ? 0u : FULL << o;
                    see &= ((there >> (2 * w)) & 1u ? 0x0000FFFFu : 0u) | ((there >> (2 * w + 1)) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 t;\n\tand.b32 t, %1, %2;\n\t"
                                     "setp.eq.u32 p, t, 0;\n\t@p mov.b32 %0, 0xFF800000;\n\t}"
                                     : "+r"(x[32 * w + i])
                                     : "r"(see), "r"(1u << i));  // -inf
                }
            }
            // weights with the maxima of the tiles before, two at a time; the
            // sum of the tile then tells whether the maxima lagged too far
            float most_v = 0.f;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) most_v = fmaxf(most_v, fabsf(mt[GROUPS + g]));
            float sum;
            auto weigh = [&]() {
                const uint64_t minus = pair(-m, -m);
                uint64_t part[4] = {0, 0, 0, 0};
                uint32_t y[16];
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    const float v = weight_of(lift, mt[GROUPS + g]);
                    const uint64_t kk = pair(kf[g], kf[g]), vv = pair(v, v);
#pragma unroll
                    for (int i = 16 * g; i < 16 * g + 16; i += 2) {
                        float a0, a1;
                        unpair(fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), kk, minus), a0, a1);
                        const uint64_t p = pair(ex2(a0), ex2(a1));
                        part[(i / 2) & 3] = add2(part[(i / 2) & 3], p);
                        unpair(mul2(p, vv), a0, a1);
                        y[(i / 2) % 16] = h2bits(__floats2half2_rn(a0, a1));
                    }
                    if (g & 1) {
                        __syncwarp();
                        tmem_st16(s_at + 8 * (g - 1), y);
                    }
                }
                float a0, a1;
                unpair(add2(add2(part[0], part[1]), add2(part[2], part[3])), a0, a1);
                sum = a0 + a1;
            };
            weigh();
            // every p is at most the sum, every weight at most the sum times the
            // largest V scale times lift, which must stay within fp16
            if (__any_sync(FULL, !(sum <= 256.f) || !(sum * (most_v * lift) <= 32768.f))) {
                float top = m, topw = mw;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    float big = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 16; ++i) big = fmaxf(big, __uint_as_float(x[16 * g + i]));
                    big *= kf[g];
                    top = fmaxf(top, big);
                    topw = fmaxf(topw, big + mt[2 * GROUPS + g]);
                }
                topw = fmaxf(topw, top - DEEP);
                const float fade = ex2(m - top), back = ex2(mw - topw);
                l *= fade;
                m = top;
                mw = topw;
                lift = ex2(m - mw) * LIFT;
                if (j) {  // the product of the tile before is done: this S was asked for after it
                    for (int cb = 0; cb < DP; cb += 16) {
                        uint32_t o[16];
                        __syncwarp();
                        tmem_ld16(o_at + cb, o);
                        tmem_wait_ld(o, 16);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * back);
                        tmem_st16(o_at + cb, o);
                    }
                }
                weigh();
            }
            l += sum;
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_before();
            __syncwarp();
            if (lane == 0) bspx::mbar_arrive(p_full + t);
        }
        // ---------------- the rows out (l = 0: the row sees nothing; NaN: so is its query)
        if (my_tiles && !failed && !wait(o_done + t, 0, cap)) failed = true;
        tc_after();
        const bool parts = d.splits > 1;
        const float f = parts ? 1.f / LIFT : l != 0.f ? ex2(mw - m) / (l * LIFT) : 0.f;
        T* out = (T*)a.out + q_tok * a.o_row + (int64_t)head * a.o_head;
        float* part = d.parts + ((int64_t)blockIdx.x * ROWS + 128 * t + tr) * (DP + 4);
        if (!failed && (t == 0 || two)) {
            for (int cb = 0; cb < dim; cb += 32) {
                uint32_t x[32];
                __syncwarp();
                if (my_tiles) {
                    tmem_ld32(o_at + cb, x);
                    tmem_wait_ld(x, 32);
                }
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = l != 0.f ? __uint_as_float(x[i]) * f : 0.f;
                if (!mine) continue;
                if (parts) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4*>(part + cb + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        alignas(16) T y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = from_float<T>(o[i + e]);
                        if (cb + i < dim) *reinterpret_cast<uint4*>(out + cb + i) = *reinterpret_cast<const uint4*>(y);
                    }
                }
            }
            if (mine && parts)
                *reinterpret_cast<float4*>(part + DP) = make_float4(m, l, mw, 0.f);
            else if (mine && a.lse)
                a.lse[q_tok * a.heads + head] = l != 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
    }
    tc_before();
    __syncwarp();
    if (lane == 0) bspx::mbar_arrive(read);
    if (failed && lane == 0) atomicExch(d.err, (int)BSP_ERR_TIMEOUT);
}

// The parts of each row of split items joined, a warp a row: O and l weighed by
// 2 to the part's maximum less the row's.  Bound by latency (a few loads in
// a row); it runs only where few row tiles left SMs idle.
constexpr int JOIN_THREADS = 256;

template <class T, int DP>
__global__ void __launch_bounds__(JOIN_THREADS) kv_prompt_join_kernel(const PromptArgs d)
{
    wait_prior_grids();
    const AttnArgs& a = d.a;
    const int lane = threadIdx.x & 31, H = a.c.heads;
    const int64_t cta = blockIdx.x / (ROWS / 32);        // of the prompt kernel, before its splits
    const int h = (int)(cta % H);
    const Item it = item_of(a, d.items - 1 - cta / H);
    const Request rq = request_of(a.s, a.c.page_shift, it.b);
    const int64_t rows = (int64_t)rq.n * a.group;
    if (it.row0 < 0 || it.row0 >= rows || rows <= d.few) return;
    for (int i = threadIdx.x / 32; i < 32; i += JOIN_THREADS / 32) {
        const int tr = (int)(blockIdx.x % (ROWS / 32)) * 32 + i;
        const int64_t r = it.row0 + tr;
        if (r >= rows) return;
        const float* part = d.parts + (cta * d.splits * ROWS + tr) * (DP + 4);
        const int64_t stride = (int64_t)ROWS * (DP + 4);
        float m = NONE, mw = NONE, l = 0.f;
        for (int s = 0; s < d.splits; ++s) {
            const float4 st = __ldcg(reinterpret_cast<const float4*>(part + s * stride + DP));
            m = fmaxf(m, st.x);
            mw = fmaxf(mw, st.z);
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const int dim = lane * 4;
#pragma unroll 4
        for (int s = 0; s < d.splits; ++s) {
            const float4 st = __ldcg(reinterpret_cast<const float4*>(part + s * stride + DP));
            l += st.y * ex2(st.x - m);
            if (dim < a.c.dim) {
                const float f = ex2(st.z - mw);
                const float4 y = __ldcg(reinterpret_cast<const float4*>(part + s * stride + dim));
                o.x += y.x * f;
                o.y += y.y * f;
                o.z += y.z * f;
                o.w += y.w * f;
            }
        }
        const int64_t tok = rq.r0 + r / a.group, head = (int64_t)h * a.group + r % a.group;
        const float f = l != 0.f ? ex2(mw - m) / l : 0.f;
        if (dim < a.c.dim) {
            alignas(8) T y[4] = {from_float<T>(o.x * f), from_float<T>(o.y * f), from_float<T>(o.z * f), from_float<T>(o.w * f)};
            *reinterpret_cast<uint2*>((T*)a.out + tok * a.o_row + head * a.o_head + dim) = *reinterpret_cast<const uint2*>(y);
        }
        if (a.lse && lane == 0) a.lse[tok * a.heads + head] = l != 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

template <class T, int DP>
bsp_status_t launch(const bsp_kv* h, const PromptArgs& d, cudaStream_t s)
{
    using C = Cfg<DP>;
    static bsp_attr_once attr_once;
    if (!attr_once.run(h->device, [] {
            return cudaFuncSetAttribute(kv_prompt_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        }))
        return BSP_ERR_CUDA;
    const int64_t ctas = d.items * h->view.heads * d.splits;
    if (ctas > 0x7FFFFFFF) return BSP_ERR_INVALID_ARG;
    if (!launch_early(kv_prompt_kernel<T, DP>, dim3((unsigned)ctas), dim3(THREADS), C::SMEM, s, h->map_k, h->map_v, d))
        return BSP_ERR_CUDA;
    if (d.splits > 1 && !launch_early(kv_prompt_join_kernel<T, DP>, dim3((unsigned)(d.items * h->view.heads * (ROWS / 32))),
                                      dim3(JOIN_THREADS), 0, s, d))
        return BSP_ERR_CUDA;
    return BSP_OK;
}

}  // namespace

bsp_status_t bsp_run_kv_prompt(const bsp_kv* h, const bspkv::AttnArgs& a, bsp_dtype_t dtype, int32_t few, bool* beside,
                               cudaStream_t s)
{
    // Few row tiles leave SMs idle: then several CTAs share the cached rows of
    // each, as many as there are SMs for and the scratch holds
    const int64_t items = a.s.rows * a.group / ROWS + a.s.batch;
    const int64_t room = (int64_t)(h->part_floats / ((size_t)ROWS * (a.c.dim > 64 ? 132 : 68)));
    const int64_t ctas = std::min<int64_t>(h->num_sms, room) / std::max<int64_t>(1, items * a.c.heads);
    const PromptArgs d = {a, h->err, h->ready, bsp_spin_cap(), few, (int32_t)std::clamp<int64_t>(ctas, 1, MOST_SPLITS),
                          items, h->parts, bsp_test_stall() != 0};
    *beside = d.splits == 1;  // else the joining kernel is in between
    const bool wide = a.c.dim > 64;
    if (dtype == BSP_FP16) return wide ? launch<__half, 128>(h, d, s) : launch<__half, 64>(h, d, s);
    return wide ? launch<__nv_bfloat16, 128>(h, d, s) : launch<__nv_bfloat16, 64>(h, d, s);
}
