// Products of 4-bit weights with many activation rows (prompts, batches of
// more than a few), and the gated form over two weights, on the
// 5th-generation tensor cores.
//
// A CTA takes one strip of 128 rows of W (the gated form: the strips of both
// weights) and BN rows of X, and walks the columns in steps of 64:
//   A  codes less zero points as fp16 or bf16, exact small integers, made
//      by the widening warps in shared memory (K-major, swizzled by 128
//      bytes: a lane's eight columns of a row are one 16-byte chunk)
//   B  X by TMA, the same layout
//   D  sums of one group of columns, in tensor memory, two buffers
// Scales are applied to D: the promoting warps read a group's sums while
// the next group's products run, and add s D to fp32 sums in registers, two
// values at a time.  So no weight is rounded, whatever its scale; weights
// multiplied out and rounded to the type would leave an error of 1.3 times
// the output's own rounding (the gated form 1.55 times).
// Warps: 0 loads X, 1 issues the products, 3 loads codes and scales, DW widen,
// PW promote (a warp reaches the tensor-memory lanes 32 (w % 4) ..
// + 31, so a thread has one row of each strip).  Where few tiles leave SMs idle, the CTAs of a cluster
// share a tile's columns and add their parts in order through shared memory.
#pragma once

#include "bsp_q4.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

// (Anonymous: the test library has the same kernels, and a process may load
// both.)
namespace {

using namespace bspq4;

constexpr uint32_t FULL = 0xFFFFFFFFu;
constexpr int BM = 128, BK = 64;
constexpr int A_BYTES = BM * BK * 2;  // of a strip's step

// BN columns of Y and MS strips a CTA, G columns of a group.  Registers of a
// thread by role, from REGS of each at launch (their sum over warpgroups is
// the launch's).
template <int G, int BN, int MS>
struct Wide {
    static constexpr int SIZE = BN * MS;
    static constexpr int CTAS = SIZE <= 64 && MS == 1 ? 2 : 1;  // an SM
    static constexpr int DW = SIZE == 256 ? 4 : 8, PW = SIZE <= 64 ? 4 : 8;
    static constexpr int WARPS = 4 + DW + PW, THREADS = 32 * WARPS;
    static constexpr int REGS = SIZE == 256 ? 128 : SIZE == 128 ? 96 : CTAS == 1 ? 128 : 64;
    static constexpr int R_CONTROL = SIZE == 256 ? 40 : SIZE == 128 ? 32 : CTAS == 1 ? 128 : SIZE == 64 ? 24 : 40;
    static constexpr int R_WIDEN = SIZE == 256 ? 72 : SIZE == 128 ? 72 : CTAS == 1 ? 128 : SIZE == 64 ? 64 : 72;
    static constexpr int R_PROMOTE = SIZE == 256 ? 200 : SIZE == 128 ? 152 : CTAS == 1 ? 128 : SIZE == 64 ? 104 : 72;
    static_assert(4 * R_CONTROL + DW * R_WIDEN + PW * R_PROMOTE == WARPS * REGS, "shares of the launch's registers");
    static constexpr int TILES = 8 * MS / DW;             // row tiles of a widening warp and step
    static constexpr int COLS = BN / (PW / 4);            // columns of a promoting thread, of each strip
    // rings: A and B in steps of 64 columns, codes (with zero points) and
    // scales in blocks of 128
    static constexpr int SA = SIZE == 256 ? (MS == 2 ? 2 : 3) : SIZE == 128 ? (MS == 2 ? 3 : 4) : BN == 64 ? 2 : 3;
    static constexpr int SB = 4, SC = SIZE == 128 && MS == 1 ? 6 : 4, SS = 8;
    static constexpr int B_BYTES = BN * BK * 2;
    static constexpr int Z_BYTES = 128 / G * 64, C_BYTES = MS * (8192 + Z_BYTES), S_BYTES = MS * (128 / G * 256);
    static constexpr int OFF_B = 0, OFF_A = SB * B_BYTES;
    static constexpr int OFF_C = OFF_A + SA * MS * A_BYTES, OFF_S = OFF_C + SC * C_BYTES;
    static constexpr int OFF_BAR = OFF_S + SS * S_BYTES;
    static constexpr int NBAR = 2 * (SA + SB + SC + SS) + 4 + 2;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr uint32_t TMEM = 2 * SIZE;
    static_assert(SMEM <= (CTAS == 2 ? 113 : 227) * 1024, "shared memory");
    static_assert(OFF_S >= SIZE * BM * 4, "the sums, over the rings");
    static_assert(CTAS == 2 || SMEM > 114 * 1024, "one CTA may take all of the tensor memory");
};

struct WideArgs {
    Q4View w[2];
    int act;
    int64_t M, N, groups;
    int32_t k_tiles, ntiles;
    void* y;
    int64_t y_stride;
    int* err;
    uint32_t spin_cap;
    bool stall;  // test only: the first copy of X is skipped
};

// kind::f16 instruction descriptor: D fp32, A and B fp16 (or bf16), K-major.
template <class T>
__host__ __device__ constexpr uint32_t idesc(int n)
{
    const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
    return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// Shared-memory matrix descriptor: K-major rows of 128 B swizzled by 128 B,
// 8-row atoms of 1 KB.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 |
           (uint64_t)2u << 61;
}

// Written for the whole warp with the issuing thread elected inside, so that
// the operands stay in uniform registers.
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accum)
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

// 32 consecutive tensor-memory columns of this thread's lane, there after
// tmem_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32])
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

__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

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

template <int REGS>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }
// A role's share: FROM registers a thread at launch, TO from here on.
template <int FROM, int TO>
__device__ __forceinline__ void take_registers()
{
    if constexpr (TO > FROM) more_registers<TO>();
    else if constexpr (TO < FROM) fewer_registers<TO>();
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bspx::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t at)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The whole warp waits; false if the wait ran out.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t cap)
{
    return __all_sync(FULL, bspx::mbar_wait_bounded(bar, parity, cap));
}

template <class T, int G, int BN, int MS>
__global__ void __launch_bounds__(Wide<G, BN, MS>::THREADS, Wide<G, BN, MS>::CTAS)
q4_wide_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ WideArgs a)
{
    using C = Wide<G, BN, MS>;
    constexpr int SA = C::SA, SB = C::SB, SC = C::SC, SS = C::SS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (bspx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const uint32_t rank = bspx::cluster_ctarank();
    const int64_t tile = blockIdx.x / ranks;
    const int64_t strip = tile / a.ntiles, n0 = tile % a.ntiles * BN;
    // this CTA's share of the columns, in blocks of 128
    const int units = a.k_tiles >> 1;
    const int k_begin = 2 * (int)((int64_t)units * rank / ranks);
    const int steps = 2 * (int)((int64_t)units * (rank + 1) / ranks) - k_begin;
    const uint32_t cap = a.spin_cap;

    uint64_t* a_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* a_empty = a_full + SA;
    uint64_t* b_full = a_empty + SA;
    uint64_t* b_empty = b_full + SB;
    uint64_t* c_full = b_empty + SB;
    uint64_t* c_empty = c_full + SC;
    uint64_t* s_full = c_empty + SC;
    uint64_t* s_empty = s_full + SS;
    uint64_t* d_full = s_empty + SS;
    uint64_t* d_empty = d_full + 2;
    uint64_t* drain = d_empty + 2;
    uint64_t* read = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(read + 1);

    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         bspx::smem_u32(tmem_slot)),
                     "r"(C::TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < SA; ++i) {
            bspx::mbar_init(a_full + i, C::DW);
            bspx::mbar_init(a_empty + i, 1);
        }
        for (int i = 0; i < SB; ++i) {
            bspx::mbar_init(b_full + i, 1);
            bspx::mbar_init(b_empty + i, 1);
        }
        for (int i = 0; i < SC; ++i) {
            bspx::mbar_init(c_full + i, 1);
            bspx::mbar_init(c_empty + i, C::DW);
        }
        for (int i = 0; i < SS; ++i) {
            bspx::mbar_init(s_full + i, 1);
            bspx::mbar_init(s_empty + i, C::PW);
        }
        for (int i = 0; i < 2; ++i) {
            bspx::mbar_init(d_full + i, 1);
            bspx::mbar_init(d_empty + i, C::PW);
        }
        bspx::mbar_init(drain, 1);
        bspx::mbar_init(read, C::PW);
        bspx::fence_mbar_init();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;
    bool failed = false;
    // (not before the tensor memory is this CTA's: a kernel that starts early
    // may take some, and then waits for this one)
    if (threadIdx.x == 0) launch_dependents();

    if (warp < 4) {
        take_registers<C::REGS, C::R_CONTROL>();
        if (warp == 0) {
            // ---------------- X
            wait_prior_grids();
            int i = 0;
            for (; i < steps; ++i) {
                const int s = i % SB;
                if (i >= SB && !wait(b_empty + s, (i / SB - 1) & 1, cap)) {
                    failed = true;
                    break;
                }
                if (lane == 0 && !(a.stall && i == 0)) {
                    bspx::mbar_arrive_expect_tx(b_full + s, (uint32_t)C::B_BYTES);
                    tma_load_2d(bspx::smem_u32(smem + C::OFF_B + s * C::B_BYTES), &map_x, (k_begin + i) * BK, (int)n0, b_full + s);
                }
                __syncwarp();
            }
            // no copy may land after the CTA is gone (the full cap, whatever `cap` is)
            for (int k = std::max(a.stall ? 1 : 0, i - SB); k < i; ++k) bspx::mbar_wait_bounded(b_full + k % SB, (k / SB) & 1);
        } else if (warp == 1) {
            // ---------------- products
            const int n = __shfl_sync(FULL, steps, 0);
            const uint32_t tm = __shfl_sync(FULL, tmem, 0);
            const uint64_t a_desc = smem_desc(bspx::smem_u32(smem + C::OFF_A)), b_desc = smem_desc(bspx::smem_u32(smem + C::OFF_B));
            constexpr uint32_t ID = idesc<T>(BN);
            constexpr int PARTS = G == 32 ? 2 : 1;            // groups of a step
            constexpr int STEPS = G == 128 ? 2 : 1;           // steps of a group
            constexpr int KS = BK / 16 / PARTS;               // products of a group in a step
            int sa = 0, sb = 0;                               // ring slots
            uint32_t pa = 0, pb = 0;
            // the next group's buffer is d; its last sums have been read when
            // phase pd of its barrier is over (a fresh barrier's phase 1 is)
            uint32_t buf = 0, pd = 1;
            for (int i = 0; i < n && !failed; i += STEPS) {
#pragma unroll
                for (int e = 0; e < STEPS; ++e) {
                    if (!wait(a_full + sa, pa, cap) || !wait(b_full + sb, pb, cap)) {
                        failed = true;
                        break;
                    }
                    const uint64_t ad = a_desc + (uint64_t)(sa * (MS * A_BYTES >> 4)), bd = b_desc + (uint64_t)(sb * (C::B_BYTES >> 4));
#pragma unroll
                    for (int x = 0; x < PARTS; ++x) {
                        if (e == 0) {
                            if (!wait(d_empty + buf, pd, cap)) {
                                failed = true;
                                break;
                            }
                            tc_after();
                        }
#pragma unroll
                        for (int k = 0; k < KS; ++k)
#pragma unroll
                            for (int m = 0; m < MS; ++m)
                                product(tm + buf * C::SIZE + m * BN, ad + (uint64_t)(m * (A_BYTES >> 4) + 2 * (x * KS + k)),
                                        bd + (uint64_t)(2 * (x * KS + k)), ID, e || k ? 1u : 0u);
                        if (e == STEPS - 1) {
                            commit(d_full + buf);
                            buf ^= 1u;
                            if (!buf) pd ^= 1u;
                        }
                    }
                    if (failed) break;
                    commit(a_empty + sa);
                    commit(b_empty + sb);
                    if (++sa == SA) { sa = 0; pa ^= 1u; }
                    if (++sb == SB) { sb = 0; pb ^= 1u; }
                }
            }
            // no product in flight and nobody reading when the tensor memory is
            // given back: with the full cap, and for readers that may be in
            // waits of their own before they say so
            __syncwarp();
            commit(drain);
            if (!wait(drain, 0, bspx::kSpinCap)) failed = true;
            bool done = false;
            for (int k = 0; k < 4 && !done; ++k) done = wait(read, 0, bspx::kSpinCap);
            if (!done) failed = true;
            tc_after();
            __syncwarp();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(C::TMEM) : "memory");
        } else if (warp == 3) {
            // ---------------- codes and zero points, and scales: they depend
            // on no kernel before this one
            const int64_t block = strip * units + (k_begin >> 1);  // of 128 columns
            const int n = steps >> 1;
            int u = 0, sc = 0, ss = 0;
            uint32_t pc = 0, ps = 0;
            for (; u < n; ++u) {
                if ((u >= SC && !wait(c_empty + sc, pc ^ 1u, cap)) || (u >= SS && !wait(s_empty + ss, ps ^ 1u, cap))) {
                    failed = true;
                    break;
                }
                if (lane == 0) {
                    uint8_t *to = smem + C::OFF_C + sc * C::C_BYTES, *to_s = smem + C::OFF_S + ss * C::S_BYTES;
                    uint32_t bytes = 0;
#pragma unroll
                    for (int m = 0; m < MS; ++m) bytes += 8192 + (a.w[m].zeros ? C::Z_BYTES : 0);
                    bspx::mbar_arrive_expect_tx(c_full + sc, bytes);
                    bspx::mbar_arrive_expect_tx(s_full + ss, C::S_BYTES);
#pragma unroll
                    for (int m = 0; m < MS; ++m) {
                        bspx::bulk_g2s(to + m * 8192, a.w[m].codes + (block + u) * 512, 8192, c_full + sc);
                        if (a.w[m].zeros)
                            bspx::bulk_g2s(to + MS * 8192 + m * C::Z_BYTES, a.w[m].zeros + (block + u) * C::Z_BYTES, C::Z_BYTES, c_full + sc);
                        bspx::bulk_g2s(to_s + m * (C::S_BYTES / MS), a.w[m].scales + (block + u) * (C::S_BYTES / MS / 4),
                                       C::S_BYTES / MS, s_full + ss);
                    }
                }
                __syncwarp();
                if (++sc == SC) { sc = 0; pc ^= 1u; }
                if (++ss == SS) { ss = 0; ps ^= 1u; }
            }
            for (int k = std::max(0, u - SC); k < u; ++k) bspx::mbar_wait_bounded(c_full + k % SC, (k / SC) & 1);
            for (int k = std::max(0, u - SS); k < u; ++k) bspx::mbar_wait_bounded(s_full + k % SS, (k / SS) & 1);
        }
        if (failed && lane == 0) atomicExch(a.err, (int)BSP_ERR_TIMEOUT);
        if (ranks > 1) {
            bspx::cluster_sync();
            bspx::cluster_sync();
        }
        return;
    }

    if (warp < 4 + C::DW) {
        take_registers<C::REGS, C::R_WIDEN>();
        // ---------------- codes -> A.  Warp w takes row tiles w, w + DW, ...
        // of the strips.  Lanes of odd rows store the upper half of their
        // columns first, so that the eight lanes of a store's phase reach
        // distinct banks.
        const int w = warp - 4, g = lane >> 2, t = lane & 3;
        constexpr int ZN = G == 32 ? 2 : 1;  // groups of a step
        const bool odd = g & 1;
        uint32_t from[C::TILES], zero[C::TILES], to[C::TILES];
        bool has_zeros[C::TILES];
#pragma unroll
        for (int x = 0; x < C::TILES; ++x) {
            const int rt = w + x * C::DW, m = rt / 8, r = rt % 8;
            has_zeros[x] = (m ? a.w[1] : a.w[0]).zeros != nullptr;
            from[x] = bspx::smem_u32(smem + C::OFF_C) + m * 8192 + r * 512 + lane * 16;
            zero[x] = bspx::smem_u32(smem + C::OFF_C) + MS * 8192 + m * C::Z_BYTES + r * 8 + g;
            to[x] = bspx::smem_u32(smem + C::OFF_A) + m * A_BYTES + r * 2048 + g * 128 + (((4 * (g & 1) + t) ^ g) << 4);
        }
        int sa = 0, sc = 0;
        uint32_t pa = 0, pc = 0;
        for (int u = 0; u < steps >> 1 && !failed; ++u) {
            if (!wait(c_full + sc, pc, cap)) {
                failed = true;
                break;
            }
            uint4 v[2][C::TILES];
            uint32_t z[2][C::TILES][ZN];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 0; x < C::TILES; ++x) {
                    v[e][x] = lds16(from[x] + sc * C::C_BYTES + e * 4096);
#pragma unroll
                    for (int y = 0; y < ZN; ++y)
                        z[e][x][y] = has_zeros[x] ? lds1(zero[x] + sc * C::C_BYTES + (e * BK / G + y) * 64) : 0x88u;
                }
            __syncwarp();
            if (lane == 0) bspx::mbar_arrive(c_empty + sc);
            if (++sc == SC) { sc = 0; pc ^= 1u; }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (2 * u + e >= SA && !wait(a_empty + sa, pa ^ 1u, cap)) {
                    failed = true;
                    break;
                }
#pragma unroll
                for (int x = 0; x < C::TILES; ++x) {
                    const uint4 q4 = v[e][x];
                    const uint32_t c[2][2] = {{odd ? q4.z : q4.x, odd ? q4.w : q4.y}, {odd ? q4.x : q4.z, odd ? q4.y : q4.w}};
                    const uint32_t at = to[x] + sa * (MS * A_BYTES);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t z0, z1, p[4], q[4];
                        Codes<T>::bias(ZN == 2 && (odd ? !h : h) ? z[e][x][ZN - 1] : z[e][x][0], z0, z1);
                        Codes<T>::widen(c[h][0], z0, z1, p);
                        Codes<T>::widen(c[h][1], z0, z1, q);
                        const uint32_t o = at ^ (h << 6);  // the other half: chunk ^ 4
                        sts16(o, p[0], p[2], q[0], q[2]);
                        sts16(o + 1024, p[1], p[3], q[1], q[3]);
                    }
                }
                bspx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) bspx::mbar_arrive(a_full + sa);
                if (++sa == SA) { sa = 0; pa ^= 1u; }
            }
        }
        if (failed && lane == 0) atomicExch(a.err, (int)BSP_ERR_TIMEOUT);
        if (ranks > 1) {
            bspx::cluster_sync();
            bspx::cluster_sync();
        }
        return;
    }

    take_registers<C::REGS, C::R_PROMOTE>();
    {
        // ---------------- sums of groups, scaled, into registers
        const int p = warp - 4 - C::DW, quad = warp & 3, row = 32 * quad + lane, c0 = (p >> 2) * C::COLS;
        const uint32_t scales = bspx::smem_u32(smem + C::OFF_S) + (row / 16 * 8 + row % 8) * 4 + (row >> 3 & 1) * 2;
        const float upper = row & 8 ? 1.f / Codes<T>::UPPER : 1.f;
        constexpr int PER = 128 / G;  // groups of a block
        uint64_t sum[MS][C::COLS / 2];
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
            for (int i = 0; i < C::COLS / 2; ++i) sum[m][i] = 0;
        const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16) + c0;
        int ss = 0, gi = 0;
        uint32_t ps = 0;
        for (int u = 0; u < steps >> 1 && !failed; ++u) {
            if (!wait(s_full + ss, ps, cap)) {
                failed = true;
                break;
            }
            float s[PER][MS];
#pragma unroll
            for (int y = 0; y < PER; ++y)
#pragma unroll
                for (int m = 0; m < MS; ++m)
                    s[y][m] = half_of<T>(lds2(scales + ss * C::S_BYTES + (m * PER + y) * 256), 0) * upper;
            __syncwarp();
            if (lane == 0) bspx::mbar_arrive(s_empty + ss);
            if (++ss == SS) { ss = 0; ps ^= 1u; }
#pragma unroll
            for (int y = 0; y < PER; ++y, ++gi) {
                if (!wait(d_full + (gi & 1), (gi >> 1) & 1, cap)) {
                    failed = true;
                    break;
                }
                tc_after();
#pragma unroll
                for (int m = 0; m < MS; ++m) {
                    const uint64_t f = pair(s[y][m], s[y][m]);
#pragma unroll
                    for (int c = 0; c < C::COLS; c += 32) {
                        uint32_t r[32];
                        tmem_ld32(at + (gi & 1) * C::SIZE + m * BN + c, r);
                        tmem_wait(r);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            sum[m][c / 2 + i] = fma2(f, pair(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), sum[m][c / 2 + i]);
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0) bspx::mbar_arrive(d_empty + (gi & 1));
            }
        }
        tc_before();
        __syncwarp();
        if (lane == 0) bspx::mbar_arrive(read);
        // ---------------- the sums to shared memory, [strip][column][row],
        // over the rings: every product is done, and every promoting warp
        // has its last scales
        asm volatile("bar.sync 1, %0;" ::"n"(C::PW * 32) : "memory");
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
            for (int i = 0; i < C::COLS / 2; ++i) {
                float v[2];
                unpair(sum[m][i], v[0], v[1]);
                part[(m * BN + c0 + 2 * i) * BM + row] = v[0];
                part[(m * BN + c0 + 2 * i + 1) * BM + row] = v[1];
            }
        if (ranks > 1) bspx::cluster_sync();
        else asm volatile("bar.sync 1, %0;" ::"n"(C::PW * 32) : "memory");
        wait_prior_grids();  // Y may still be read by the kernels before this one
        // a warp a column: four rows a lane
        const int first = BN * rank / ranks, last = (int)min((int64_t)(BN * (rank + 1) / ranks), a.N - n0);
        const int64_t m0 = strip * BM + 4 * lane;
        const bool whole = m0 + 4 <= a.M && a.y_stride % 4 == 0;
#pragma unroll 1
        for (int c = first + p; c < last && !failed; c += C::PW) {
            float4 v[MS];
#pragma unroll
            for (int m = 0; m < MS; ++m) {
                const uint32_t from = bspx::smem_u32(part + (m * BN + c) * BM + 4 * lane);
                v[m] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (uint32_t k = 0; k < ranks; ++k) {
                    float4 x;
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                                 : "r"(ranks > 1 ? bspx::mapa_shared(from, k) : from)
                                 : "memory");
                    v[m].x += x.x;
                    v[m].y += x.y;
                    v[m].z += x.z;
                    v[m].w += x.w;
                }
            }
            if (MS == 2) {
                v[0].x = activate(v[0].x, a.act) * v[MS - 1].x;
                v[0].y = activate(v[0].y, a.act) * v[MS - 1].y;
                v[0].z = activate(v[0].z, a.act) * v[MS - 1].z;
                v[0].w = activate(v[0].w, a.act) * v[MS - 1].w;
            }
            T* y = reinterpret_cast<T*>(a.y) + (n0 + c) * a.y_stride + m0;
            alignas(8) const T o[4] = {from_float<T>(v[0].x), from_float<T>(v[0].y), from_float<T>(v[0].z), from_float<T>(v[0].w)};
            if (whole) *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(o);
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m0 + e < a.M) y[e] = o[e];
        }
        if (ranks > 1) bspx::cluster_sync();  // others may still read this CTA's sums
    }
    if (failed && lane == 0) atomicExch(a.err, (int)BSP_ERR_TIMEOUT);
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

template <class T, int G, int BN, int MS>
bsp_status_t launch_wide(const Problem& p, int ranks, cudaStream_t s)
{
    using C = Wide<G, BN, MS>;
    static bsp_attr_once attr_once;
    if (!attr_once.run(p.device, [] {
            return cudaFuncSetAttribute(q4_wide_kernel<T, G, BN, MS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        }))
        return BSP_ERR_CUDA;
    const auto encode = encode_fn();
    if (!encode) return BSP_ERR_CUDA;
    CUtensorMap map;
    const cuuint64_t dims[2] = {(cuuint64_t)p.K, (cuuint64_t)p.N};
    const cuuint64_t strides[1] = {(cuuint64_t)p.x_stride * 2};
    const cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)BN};
    const cuuint32_t estr[2] = {1, 1};
    if (encode(&map, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void*>(p.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return BSP_ERR_INVALID_ARG;
    WideArgs a;
    a.w[0] = p.w;
    a.w[1] = p.up;
    a.act = p.act;
    a.M = p.M;
    a.N = p.N;
    a.groups = p.k_tiles * BK / G;
    a.k_tiles = (int32_t)p.k_tiles;
    a.ntiles = (int32_t)((p.N + BN - 1) / BN);
    a.y = p.y;
    a.y_stride = p.y_stride;
    a.err = p.err;
    a.spin_cap = bsp_spin_cap();
    a.stall = bsp_test_stall() != 0;
    const int64_t ctas = (p.M + BM - 1) / BM * a.ntiles * ranks;
    if (ctas > INT32_MAX) return BSP_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ranks;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q4_wide_kernel<T, G, BN, MS>, map, a) == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

// CTAs of a cluster that share a tile's columns: while the tiles leave half
// of the GPU's places idle and each keeps four blocks of 128 columns.
inline int split_of(const Problem& p, int64_t tiles, int ctas_an_sm)
{
    int r = 1;
    while (r < 8 && tiles * r * 2 <= (int64_t)p.num_sms * ctas_an_sm && p.k_tiles / 2 >= 4 * 2 * r) r *= 2;
    return r;
}

template <class T, int G>
bsp_status_t wide_by_shape(const Problem& p, cudaStream_t s)
{
    const int64_t strips = (p.M + BM - 1) / BM;
    auto go = [&](auto bn, auto ms) {
        constexpr int BN = decltype(bn)::value, MS = decltype(ms)::value;
        const int64_t tiles = strips * ((p.N + BN - 1) / BN);
        return launch_wide<T, G, BN, MS>(p, split_of(p, tiles, Wide<G, BN, MS>::CTAS), s);
    };
    using std::integral_constant;
    if (p.gated) {
        if (p.N <= 32) return go(integral_constant<int, 32>(), integral_constant<int, 2>());
        if (p.N <= 64) return go(integral_constant<int, 64>(), integral_constant<int, 2>());
        return go(integral_constant<int, 128>(), integral_constant<int, 2>());
    }
    if (p.N <= 32) return go(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (p.N <= 64) return go(integral_constant<int, 64>(), integral_constant<int, 1>());
    if (p.N <= 128) return go(integral_constant<int, 128>(), integral_constant<int, 1>());
    return go(integral_constant<int, 256>(), integral_constant<int, 1>());
}

template <class T>
bsp_status_t run_wide(const Problem& p, cudaStream_t s)
{
    if (p.K > INT32_MAX || p.N > INT32_MAX) return BSP_ERR_SHAPE;
    switch (p.group) {
    case 32: return wide_by_shape<T, 32>(p, s);
    case 64: return wide_by_shape<T, 64>(p, s);
    default: return wide_by_shape<T, 128>(p, s);
    }
}

}  // namespace
