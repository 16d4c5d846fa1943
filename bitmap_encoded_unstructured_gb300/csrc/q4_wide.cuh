// Products of 4-bit weights with many activation rows (prompts, batches of
// more than a few), and the gated form over two weights, on the
// 5th-generation tensor cores.
//
// A pair of CTAs takes 256 rows (two strips of W; the gated form: a strip of
// each weight) and BN rows of X, and walks the columns in blocks of 128:
//   A  codes less zero points as fp16 or bf16, exact small integers, made
//      by each CTA's widening warps from its own strip, in shared memory
//      (K-major, swizzled by 128 bytes: a lane's eight columns of a row are
//      one 16-byte chunk)
//   B  X by TMA, the same layout, half of the BN rows in each CTA
//   D  sums of one group of columns, in tensor memory, two to eight buffers; one
//      product (cta_group::2) works on both CTAs' rows
// Scales are applied to D: the promoting warps read a group's sums while
// the next group's products run, and add s D to fp32 sums in registers.  So no
// weight is rounded, whatever its scale; weights multiplied out and rounded to
// the type would leave an error of 1.3 times the output's own rounding (the
// gated form 1.55 times).
//
// Warps of a CTA: 0 loads X and 2 says when it is there, 1 issues the products
// (in the pair's first CTA), 3 loads codes and scales, DW widen, PW promote (a
// warp reaches the tensor-memory lanes 32 (w % 4) .. + 31, so a thread has one
// row).  The issuing warp sets the pace, not the tensor pipe: a wait costs it
// about 150 cycles though it is over, a product 75.  So a block has one
// barrier for all that its products read, from both CTAs.
// Where few tiles leave SMs idle, the pairs of a larger cluster share a
// tile's columns and add their parts in order through shared memory.
//
// What a block takes, and a tile at its ends (one wave, one pair a tile):
//   columns of Y    groups of 128    64         32          ends
//   64              480 ns           510        600         5 us
//   128             550              650        910         7
//   256             670              860        1370        9.5
// Large tiles of groups of 128 are bound by their products (540 of 670 ns;
// tensor pipe 66% busy), of 64 and 32 by the promoting warps (two and four
// passes over the sums a block), small tiles by a block's chain of waits.
// 1501 rows of 8192 x 28672: 490 us (1438 TFLOP/s, 0.76 of the library's bf16
// product); gated 2048 rows of 28672 x 8192: 1450 us (1327 TFLOP/s).
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
constexpr int BM = 128, BK = 128;      // rows of a strip, columns of a block
constexpr int A_HALF = BM * 64 * 2, A_BYTES = 2 * A_HALF;  // 64 columns of a strip; a block

// BN columns of Y, G columns of a group.  Registers of a thread by role, from
// REGS of each at launch (their sum over warpgroups is within the launch's),
// as the compiler needs them to spill nothing, or least.
template <int G, int BN, bool GATED>
struct Wide {
    static constexpr int DW = BN == 256 ? 4 : 8, PW = 8;
    static constexpr int WARPS = 4 + DW + PW, THREADS = 32 * WARPS;
    static constexpr int REGS = BN == 256 ? 128 : 96;
    static constexpr int R_CONTROL = BN >= 128 ? 40 : REGS;
    static constexpr int R_WIDEN = BN == 256 ? (GATED ? 120 : 136) : BN == 128 ? 104 : REGS;
    static constexpr int R_PROMOTE = BN == 256 ? (GATED ? 176 : 168) : BN == 128 ? 112 : REGS;
    static constexpr int TILES = 8 / DW;                  // row tiles of a widening warp
    static constexpr int COLS = BN / (PW / 4);            // columns of a promoting thread
    // rings: A with B, codes (with zero points), scales
    static constexpr int SR = BN >= 128 ? 3 : 4, SC = BN == 256 ? 3 : 6, SS = 8;
    // a buffer of D holds the sums of H groups of a block, BN columns
    // each; there are ND
    static constexpr int PER = 128 / G, H = PER < 256 / BN ? PER : 256 / BN;
    static constexpr int ND = 512 / (H * BN) < 8 ? 512 / (H * BN) : 8;
    static constexpr int B_HALF = BN / 2 * 64 * 2, B_BYTES = 2 * B_HALF;
    static constexpr int Z_BYTES = 128 / G * 64, C_BYTES = 8192 + Z_BYTES, S_BYTES = 128 / G * 256;
    static constexpr int OFF_B = SR * A_BYTES, OFF_C = OFF_B + SR * B_BYTES, OFF_S = OFF_C + SC * C_BYTES;
    static constexpr int OFF_BAR = OFF_S + SS * S_BYTES;
    static constexpr int NBAR = 3 * SR + 2 * (SC + SS + ND) + 2;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr uint32_t TMEM = ND * H * BN;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(OFF_S >= BN * BM * 4, "the sums, over the rings");
    static_assert(SMEM > 114 * 1024, "one CTA an SM: it may take all of the tensor memory");
};

struct WideArgs {
    Q4View w[2];
    int act;
    int64_t M, N, strips;
    int32_t k_tiles, ntiles;
    void* y;
    int64_t y_stride;
    int* err;
    uint32_t spin_cap;
    bool stall;  // test only: the first copy of X is skipped
};

// kind::f16 instruction descriptor: D fp32, A and B fp16 (or bf16), K-major,
// the 256 rows of both CTAs.
template <class T>
__host__ __device__ constexpr uint32_t idesc(int n)
{
    const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
    return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(2 * BM >> 4) << 24);
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
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}

// One arrival, when the products issued so far are done, on the barrier at
// this offset in each CTA of `mask` (by cluster rank).
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t mask)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            bspx::smem_u32(bar)),
        "h"((uint16_t)mask)
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

// (Volatile: a plain load may be moved behind the arrival that gives its slot
// back, and even behind the next wait.)
__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.volatile.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t at)
{
    uint16_t v;
    asm volatile("ld.volatile.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.volatile.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
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

// An arrival on a barrier of another CTA of the cluster (or this one's), by
// its shared-window address there.  It releases to this CTA only: what it
// tells of (a tile in this CTA's shared memory, behind a proxy fence; sums read from its tensor
// memory) is read by this SM's own tensor core.  A release to the cluster
// took some 1000 cycles.
__device__ __forceinline__ void arrive_at(uint32_t addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

template <class T, int G, int BN, bool GATED>
__global__ void __launch_bounds__(Wide<G, BN, GATED>::THREADS, 1)
q4_wide_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ WideArgs a)
{
    using C = Wide<G, BN, GATED>;
    static_assert(4 * C::R_CONTROL + C::DW * C::R_WIDEN + C::PW * C::R_PROMOTE <= C::WARPS * C::REGS,
                  "shares of the launch's registers");
    constexpr int SR = C::SR, SC = C::SC, SS = C::SS, ND = C::ND, PER = C::PER, H = C::H;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (bspx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const uint32_t rank = bspx::cluster_ctarank(), half = rank & 1u, lead = rank & ~1u;
    const uint32_t shares = ranks >> 1, share = rank >> 1;  // pairs that share the columns
    const int64_t tile = blockIdx.x / ranks;
    const int64_t strip = GATED ? tile / a.ntiles : tile / a.ntiles * 2 + half, n0 = tile % a.ntiles * BN;
    // (an odd last strip is read twice, and stored once)
    const int64_t strip_in = GATED || strip < a.strips ? strip : a.strips - 1;
    const Q4View& w = GATED && half ? a.w[1] : a.w[0];
    // this pair's share of the blocks of columns
    const int blocks_all = a.k_tiles >> 1;
    const int first = (int)((int64_t)blocks_all * share / shares);
    int blocks = (int)((int64_t)blocks_all * (share + 1) / shares) - first;
    const int64_t block0 = strip_in * blocks_all + first;
    const uint32_t cap = a.spin_cap;

    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // A and B of a block, in the first CTA
    uint64_t* x_full = full + SR;                                     // this CTA's half of B
    uint64_t* empty = x_full + SR;
    uint64_t* c_full = empty + SR;
    uint64_t* c_empty = c_full + SC;
    uint64_t* s_full = c_empty + SC;
    uint64_t* s_empty = s_full + SS;
    uint64_t* d_full = s_empty + SS;
    uint64_t* d_empty = d_full + ND;                                  // in the first CTA
    uint64_t* drain = d_empty + ND;
    uint64_t* read = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(read + 1);

    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         bspx::smem_u32(tmem_slot)),
                     "r"(C::TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < SR; ++i) {
            bspx::mbar_init(full + i, 2 * C::DW + 2);
            bspx::mbar_init(x_full + i, 1);
            bspx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < SC; ++i) {
            bspx::mbar_init(c_full + i, 1);
            bspx::mbar_init(c_empty + i, C::DW);
        }
        for (int i = 0; i < SS; ++i) {
            bspx::mbar_init(s_full + i, 1);
            bspx::mbar_init(s_empty + i, C::PW);
        }
        for (int i = 0; i < ND; ++i) {
            bspx::mbar_init(d_full + i, 1);
            bspx::mbar_init(d_empty + i, 2 * C::PW);
        }
        bspx::mbar_init(drain, 1);
        bspx::mbar_init(read, C::PW);
        bspx::fence_mbar_init();
    }
    tc_before();
    __syncthreads();
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    bool failed = false;
    uint32_t tmem = 0;
    // The pair meets before a warp reaches into the other CTA; the warps that
    // load, which do not, start at once.
    auto meet = [&]() {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        tc_after();
        tmem = *tmem_slot;
        // one product addresses both CTAs' tensor memory: they were given the same
        uint32_t other;
        const uint32_t at = bspx::mapa_shared(bspx::smem_u32(tmem_slot), rank ^ 1u);
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(at) : "memory");
        failed = other != tmem;
        if (failed) blocks = 0;
    };
    // The next kernel may start now that the tensor memory is this CTA's (one that
    // starts earlier may take some, and then waits for this kernel).
    if (threadIdx.x == 0) launch_dependents();
    // Every role waits for the kernels before this one ahead of its first
    // bounded wait that depends on X: a bounded wait counts only this kernel's
    // time.

    if (warp < 4) {
        take_registers<C::REGS, C::R_CONTROL>();
        if (warp == 0) {
            // ---------------- X: this CTA's half of the rows
            wait_prior_grids();
            int i = 0, s = 0;
            uint32_t ph = 0;
            for (; i < blocks; ++i) {
                if (i >= SR && !wait(empty + s, ph ^ 1u, cap)) {
                    failed = true;
                    break;
                }
                if (lane == 0 && !(a.stall && i == 0)) {
                    const uint32_t to = bspx::smem_u32(smem + C::OFF_B + s * C::B_BYTES);
                    bspx::mbar_arrive_expect_tx(x_full + s, (uint32_t)C::B_BYTES);
                    tma_load_2d(to, &map_x, (first + i) * BK, (int)(n0 + half * (BN / 2)), x_full + s);
                    tma_load_2d(to + C::B_HALF, &map_x, (first + i) * BK + 64, (int)(n0 + half * (BN / 2)), x_full + s);
                }
                __syncwarp();
                if (++s == SR) { s = 0; ph ^= 1u; }
            }
            // no copy may land after the CTA is gone (the full cap, whatever `cap` is)
            for (int k = std::max(a.stall ? 1 : 0, i - SR); k < i; ++k) bspx::mbar_wait_bounded(x_full + k % SR, (k / SR) & 1);
            const bool late = failed;
            meet();
            failed = failed || late;
        } else if (warp == 2) {
            // ---------------- tells the first CTA that this half of X is here
            meet();
            wait_prior_grids();
            int s = 0;
            uint32_t ph = 0;
            for (int i = 0; i < blocks; ++i) {
                if (!wait(x_full + s, ph, cap)) {
                    failed = true;
                    break;
                }
                if (lane == 0) arrive_at(bspx::mapa_shared(bspx::smem_u32(full + s), lead));
                __syncwarp();
                if (++s == SR) { s = 0; ph ^= 1u; }
            }
        } else if (warp == 1) {
            meet();
            wait_prior_grids();  // both CTAs: the second one's waits for the end of the products below count too
            if (!half) {
                // ---------------- products
                const int n = __shfl_sync(FULL, blocks, 0);
                const uint32_t tm = __shfl_sync(FULL, tmem, 0), both = __shfl_sync(FULL, 3u << lead, 0);
                const uint64_t a_desc = smem_desc(bspx::smem_u32(smem)), b_desc = smem_desc(bspx::smem_u32(smem + C::OFF_B));
                constexpr uint32_t ID = idesc<T>(BN);
                constexpr int KS = G / 16;                        // products of a group
                int s = 0;
                // the next groups' buffer is buf; its last sums have been read when
                // phase pd of its barrier is over (a fresh barrier's phase 1 is)
                uint32_t ph = 0, buf = 0, pd = 1;
                for (int i = 0; i < n && !failed; ++i) {
                    if (!wait(full + s, ph, cap)) {
                        failed = true;
                        break;
                    }
                    const uint64_t ad = a_desc + (uint64_t)(s * (A_BYTES >> 4)), bd = b_desc + (uint64_t)(s * (C::B_BYTES >> 4));
#pragma unroll
                    for (int x = 0; x < PER; ++x) {
                        if (x % H == 0) {
                            if (!wait(d_empty + buf, pd, cap)) {
                                failed = true;
                                break;
                            }
                            tc_after();
                        }
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            const int at = x * KS + k;            // of the block's eight
                            product(tm + (buf * H + x % H) * BN, ad + (uint64_t)((at >> 2) * (A_HALF >> 4) + (at & 3) * 2),
                                    bd + (uint64_t)((at >> 2) * (C::B_HALF >> 4) + (at & 3) * 2), ID, k ? 1u : 0u);
                        }
                        if (x == PER - 1) commit(empty + s, both);
                        if (x % H == H - 1) {
                            commit(d_full + buf, both);
                            if (++buf == ND) { buf = 0; pd ^= 1u; }
                        }
                    }
                    if (++s == SR) { s = 0; ph ^= 1u; }
                }
                __syncwarp();
                commit(drain, both);
            }
            // no product in flight and nobody reading when the tensor memory is
            // given back: with the full cap, and for those that may be in waits of
            // their own before they say so
            __syncwarp();
            bool done = false, idle = false;
            for (int k = 0; k < 4 && !idle; ++k) idle = wait(drain, 0, bspx::kSpinCap);
            for (int k = 0; k < 4 && !done; ++k) done = wait(read, 0, bspx::kSpinCap);
            if (!done || !idle) failed = true;
            tc_after();
            __syncwarp();
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM) : "memory");
        } else if (warp == 3) {
            // ---------------- codes and zero points, and scales: they depend
            // on no kernel before this one
            int u = 0, sc = 0, ss = 0;
            uint32_t pc = 0, ps = 0;
            for (; u < blocks; ++u) {
                if (u == SC) wait_prior_grids();
                if ((u >= SC && !wait(c_empty + sc, pc ^ 1u, cap)) || (u >= SS && !wait(s_empty + ss, ps ^ 1u, cap))) {
                    failed = true;
                    break;
                }
                if (lane == 0) {
                    uint8_t* to = smem + C::OFF_C + sc * C::C_BYTES;
                    bspx::mbar_arrive_expect_tx(c_full + sc, 8192 + (w.zeros ? C::Z_BYTES : 0));
                    bspx::bulk_g2s(to, w.codes + (block0 + u) * 512, 8192, c_full + sc);
                    if (w.zeros) bspx::bulk_g2s(to + 8192, w.zeros + (block0 + u) * C::Z_BYTES, C::Z_BYTES, c_full + sc);
                    bspx::mbar_arrive_expect_tx(s_full + ss, C::S_BYTES);
                    bspx::bulk_g2s(smem + C::OFF_S + ss * C::S_BYTES, w.scales + (block0 + u) * (C::S_BYTES / 4), C::S_BYTES,
                                   s_full + ss);
                }
                __syncwarp();
                if (++sc == SC) { sc = 0; pc ^= 1u; }
                if (++ss == SS) { ss = 0; ps ^= 1u; }
            }
            for (int k = std::max(0, u - SC); k < u; ++k) bspx::mbar_wait_bounded(c_full + k % SC, (k / SC) & 1);
            for (int k = std::max(0, u - SS); k < u; ++k) bspx::mbar_wait_bounded(s_full + k % SS, (k / SS) & 1);
            const bool late = failed;
            meet();
            failed = failed || late;
        }
        if (failed && lane == 0) atomicExch(a.err, (int)BSP_ERR_TIMEOUT);
        bspx::cluster_sync();
        bspx::cluster_sync();
        return;
    }

    if (warp < 4 + C::DW) {
        take_registers<C::REGS, C::R_WIDEN>();
        meet();
        // ---------------- codes -> A.  Warp w takes row tiles w, w + DW of the
        // strip.  Lanes of odd rows store the upper half of their columns
        // first, so that the eight lanes of a store's phase reach distinct
        // banks.
        const int w0 = warp - 4, g = lane >> 2, t = lane & 3;
        constexpr int ZN = G == 32 ? 4 : G == 64 ? 2 : 1;  // groups of a block
        const bool odd = g & 1, has_zeros = w.zeros != nullptr;
        const uint32_t from = bspx::smem_u32(smem + C::OFF_C) + w0 * 512 + lane * 16;
        const uint32_t zero = bspx::smem_u32(smem + C::OFF_C) + 8192 + w0 * 8 + g;
        const uint32_t to = bspx::smem_u32(smem) + w0 * 2048 + g * 128 + (((4 * (g & 1) + t) ^ g) << 4);
        const uint32_t told = bspx::mapa_shared(bspx::smem_u32(full), lead);
        int s = 0, sc = 0;
        uint32_t ph = 0, pc = 0;
        for (int u = 0; u < blocks; ++u) {
            // from block SC on codes come, and from block SR on slots fall free, only
            // once the kernels before this one are done (see the loads, and the products)
            if (u == (SC < SR ? SC : SR)) wait_prior_grids();
            if (!wait(c_full + sc, pc, cap)) {
                failed = true;
                break;
            }
            uint4 v[C::TILES][2];
            uint32_t z[C::TILES][ZN];
#pragma unroll
            for (int x = 0; x < C::TILES; ++x) {
#pragma unroll
                for (int e = 0; e < 2; ++e) v[x][e] = lds16(from + sc * C::C_BYTES + x * (C::DW * 512) + e * 4096);
#pragma unroll
                for (int y = 0; y < ZN; ++y)
                    z[x][y] = has_zeros ? lds1(zero + sc * C::C_BYTES + x * (C::DW * 8) + y * 64) : 0x88u;
            }
            if (u >= SR && !wait(empty + s, ph ^ 1u, cap)) {
                failed = true;
                break;
            }
#pragma unroll
            for (int x = 0; x < C::TILES; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 q4 = v[x][e];
                    const uint32_t c[2][2] = {{odd ? q4.z : q4.x, odd ? q4.w : q4.y}, {odd ? q4.x : q4.z, odd ? q4.y : q4.w}};
                    const uint32_t at = to + s * A_BYTES + e * A_HALF + x * (C::DW * 2048);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t z0, z1, p[4], q[4];
                        Codes<T>::bias(ZN == 4 ? ((odd ? !h : h) ? z[x][(2 * e + 1) % ZN] : z[x][2 * e % ZN]) : z[x][e % ZN],
                                       z0, z1);
                        Codes<T>::widen(c[h][0], z0, z1, p);
                        Codes<T>::widen(c[h][1], z0, z1, q);
                        const uint32_t o = at ^ (h << 6);  // the other half: chunk ^ 4
                        sts16(o, p[0], p[2], q[0], q[2]);
                        sts16(o + 1024, p[1], p[3], q[1], q[3]);
                    }
                }
            bspx::fence_proxy_async_smem();
            __syncwarp();
            // the codes' slot is given back here, behind the stores that need them:
            // an arrival right behind their loads went ahead of some lanes' (one
            // block in some thousands held codes of a later one)
            if (lane == 0) {
                arrive_at(told + s * 8);
                bspx::mbar_arrive(c_empty + sc);
            }
            if (++s == SR) { s = 0; ph ^= 1u; }
            if (++sc == SC) { sc = 0; pc ^= 1u; }
        }
        if (failed && lane == 0) atomicExch(a.err, (int)BSP_ERR_TIMEOUT);
        bspx::cluster_sync();
        bspx::cluster_sync();
        return;
    }

    take_registers<C::REGS, C::R_PROMOTE>();
    {
        meet();
        // ---------------- sums of groups, scaled, into registers
        const int p = warp - 4 - C::DW, quad = warp & 3, row = 32 * quad + lane, c0 = (p >> 2) * C::COLS;
        const uint32_t scales = bspx::smem_u32(smem + C::OFF_S) + (row / 16 * 8 + row % 8) * 4 + (row >> 3 & 1) * 2;
        const uint32_t told = bspx::mapa_shared(bspx::smem_u32(d_empty), lead);
        const float upper = row & 8 ? 1.f / Codes<T>::UPPER : 1.f;
        wait_prior_grids();
        float sum[C::COLS];
#pragma unroll
        for (int i = 0; i < C::COLS; ++i) sum[i] = 0.f;
        const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16) + c0;
        int ss = 0;
        uint32_t ps = 0, buf = 0, pd = 0;
        for (int u = 0; u < blocks && !failed; ++u) {
            if (!wait(s_full + ss, ps, cap)) {
                failed = true;
                break;
            }
            float f[PER];
#pragma unroll
            for (int y = 0; y < PER; ++y) f[y] = half_of<T>(lds2(scales + ss * C::S_BYTES + y * 256), 0) * upper;
#pragma unroll
            for (int y = 0; y < PER; ++y) {
                if (y % H == 0) {
                    if (!wait(d_full + buf, pd, cap)) {
                        failed = true;
                        break;
                    }
                    tc_after();
                }
#pragma unroll
                for (int c = 0; c < C::COLS; c += 32) {
                    uint32_t r[32];
                    tmem_ld32(at + (buf * H + y % H) * BN + c, r);
                    tmem_wait(r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[c + i] = fmaf(f[y], __uint_as_float(r[i]), sum[c + i]);
                }
                if (y % H == H - 1) {
                    tc_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(told + buf * 8);
                    if (++buf == ND) { buf = 0; pd ^= 1u; }
                }
            }
            if (lane == 0) bspx::mbar_arrive(s_empty + ss);  // (every lane has used its scales: see the codes)
            if (++ss == SS) { ss = 0; ps ^= 1u; }
        }
        tc_before();
        __syncwarp();
        if (lane == 0) bspx::mbar_arrive(read);
        constexpr float OUT = 1.f / Codes<T>::UNIT;
        const int64_t m = strip * BM + row;
        T* y = reinterpret_cast<T*>(a.y) + m;
        float* part = reinterpret_cast<float*>(smem);  // over the rings: every product is done
        if (shares == 1 && !GATED) {
            // ---------------- out as they are: a warp 32 rows of a column
            bspx::cluster_sync();
            if (!failed && m < a.M)
#pragma unroll
                for (int i = 0; i < C::COLS; ++i)
                    if (n0 + c0 + i < a.N) y[(n0 + c0 + i) * a.y_stride] = from_float<T>(sum[i] * OUT);
            bspx::cluster_sync();
        } else if (shares == 1) {
            // ---------------- gate and up meet: of every thread's columns the
            // first CTA finishes the first half, the second the other; what the
            // other CTA finishes goes to its shared memory
            constexpr int HALF = C::COLS / 2;
            float* own = part + (p >> 2) * (HALF * BM) + row;
            const uint32_t here = bspx::smem_u32(own), there = bspx::mapa_shared(here + BN / 2 * BM * 4, rank ^ 1u);
            const uint32_t to[2] = {half ? there : here, half ? here : there};
#pragma unroll
            for (int i = 0; i < C::COLS; ++i)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to[i / HALF] + i % HALF * BM * 4), "f"(sum[i]) : "memory");
            bspx::cluster_sync();
            const int64_t n1 = n0 + c0 + half * HALF;
            const int last = (int)min((int64_t)HALF, a.N - n1);
            const float* gate = own + (half ? BN / 2 * BM : 0);
            const float* up = own + (half ? 0 : BN / 2 * BM);
            if (!failed && m < a.M)
#pragma unroll 4
                for (int i = 0; i < last; ++i)
                    y[(n1 + i) * a.y_stride] = from_float<T>(activate(gate[i * BM] * OUT, a.act) * (up[i * BM] * OUT));
            bspx::cluster_sync();
        } else {
            // ---------------- parts to shared memory, [column][row], and their sums
            // from all CTAs that share the tile's columns
            asm volatile("bar.sync 1, %0;" ::"n"(C::PW * 32) : "memory");
#pragma unroll
            for (int i = 0; i < C::COLS; ++i) part[(c0 + i) * BM + row] = sum[i];
            bspx::cluster_sync();
            // a warp four columns at a time (another CTA's sums take some 1000 cycles
            // to come), four rows a lane.  Rows of one strip: its CTAs share its
            // columns.  Gated: all CTAs do.
            const int of = GATED ? ranks : shares, mine = GATED ? rank : share;
            const int from_col = BN * mine / of, to_col = (int)min((int64_t)(BN * (mine + 1) / of), a.N - n0);
            const int64_t m0 = strip * BM + 4 * lane;
            const bool whole = m0 + 4 <= a.M && a.y_stride % 4 == 0;
            auto total = [&](uint32_t side, int c0, float4 (&v)[4]) {  // of columns c0, c0 + PW, ...
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (uint32_t k = 0; k < shares; ++k) {
                    const uint32_t from = bspx::mapa_shared(bspx::smem_u32(part + c0 * BM + 4 * lane), 2 * k + side);
                    float4 x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(x[j].x), "=f"(x[j].y), "=f"(x[j].z), "=f"(x[j].w)
                                     : "r"(from + (c0 + j * C::PW < to_col ? j * C::PW * BM * 4 : 0))
                                     : "memory");
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j].x += x[j].x;
                        v[j].y += x[j].y;
                        v[j].z += x[j].z;
                        v[j].w += x[j].w;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = make_float4(v[j].x * OUT, v[j].y * OUT, v[j].z * OUT, v[j].w * OUT);
            };
#pragma unroll 1
            for (int c = from_col + p; c < to_col && !failed; c += 4 * C::PW) {
                float4 v[4], u[4];
                total(GATED ? 0 : half, c, v);
                if (GATED) total(1, c, u);
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    const int n = c + j * C::PW;
                    if (n >= to_col) break;
                    float4 z = v[0];
                    if (GATED)
                        z = make_float4(activate(z.x, a.act) * u[0].x, activate(z.y, a.act) * u[0].y,
                                        activate(z.z, a.act) * u[0].z, activate(z.w, a.act) * u[0].w);
                    T* y = reinterpret_cast<T*>(a.y) + (n0 + n) * a.y_stride + m0;
                    alignas(8) const T o[4] = {from_float<T>(z.x), from_float<T>(z.y), from_float<T>(z.z), from_float<T>(z.w)};
                    if (whole) *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(o);
                    else
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (m0 + e < a.M) y[e] = o[e];
#pragma unroll
                    for (int i = 0; i < 3; ++i) {  // the next one
                        v[i] = v[i + 1];
                        if (GATED) u[i] = u[i + 1];
                    }
                }
            }
            bspx::cluster_sync();  // others may still read this CTA's sums
        }
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

template <class T, int G, int BN, bool GATED>
bsp_status_t launch_wide(const Problem& p, int shares, cudaStream_t s)
{
    using C = Wide<G, BN, GATED>;
    static bsp_attr_once attr_once;
    if (!attr_once.run(p.device, [] {
            return cudaFuncSetAttribute(q4_wide_kernel<T, G, BN, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        }))
        return BSP_ERR_CUDA;
    const auto encode = encode_fn();
    if (!encode) return BSP_ERR_CUDA;
    CUtensorMap map;
    const cuuint64_t dims[2] = {(cuuint64_t)p.K, (cuuint64_t)p.N};
    const cuuint64_t strides[1] = {(cuuint64_t)p.x_stride * 2};
    const cuuint32_t box[2] = {64, BN / 2};
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
    a.strips = p.strips;
    a.k_tiles = (int32_t)p.k_tiles;
    a.ntiles = (int32_t)((p.N + BN - 1) / BN);
    a.y = p.y;
    a.y_stride = p.y_stride;
    a.err = p.err;
    a.spin_cap = bsp_spin_cap();
    a.stall = bsp_test_stall() != 0;
    const int64_t ctas = (GATED ? p.strips : (p.strips + 1) / 2) * a.ntiles * 2 * shares;
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
    at[1].val.clusterDim.x = 2 * shares;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q4_wide_kernel<T, G, BN, GATED>, map, a) == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

// Clusters of 2, 4, 6 and 8 CTAs, one CTA an SM, that fit the GPU at once.
template <class T, int G>
const int* clusters_at_once(int device, int num_sms)
{
    static std::mutex mu;
    static int most[64][4];
    if (device < 0 || device >= 64) return nullptr;
    std::lock_guard<std::mutex> g(mu);
    int* m = most[device];
    if (!m[0]) {
        auto* k = q4_wide_kernel<T, G, 256, false>;
        using C = Wide<G, 256, false>;
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return nullptr;
        for (int i = 3; i >= 0; --i) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2 * (i + 1));
            cfg.blockDim = dim3(C::THREADS);
            cfg.dynamicSmemBytes = C::SMEM;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = 2 * (i + 1);
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) return nullptr;
            m[i] = std::max(1, std::min(n, num_sms / (2 * (i + 1))));
        }
    }
    return m;
}

// The columns of Y a tile takes and the pairs that share its columns of W:
// the least of waves x (blocks of a pair x a block's time + what a tile takes
// at its ends), in tens of ns, measured one wave at a time on 19456 rows.
struct Plan {
    int bn, shares;
};
template <int G>
Plan plan_of(const Problem& p, const int* clusters)
{
    constexpr int BN[3] = {64, 128, 256};
    constexpr int BLOCK[3] = {G == 32 ? 60 : 48, G == 32 ? 92 : 55, G == 128 ? 67 : G == 64 ? 86 : 137};
    constexpr int ENDS[3] = {600, 790, 1060};
    const int64_t pairs = p.gated ? p.strips : (p.strips + 1) / 2, blocks = p.k_tiles / 2;
    Plan best = {256, 1};
    int64_t least = INT64_MAX;
    for (int i = 0; i < 3; ++i)
        for (int s = 1; s <= 4 && s <= blocks; ++s) {
            const int64_t tiles = pairs * ((p.N + BN[i] - 1) / BN[i]), waves = (tiles + clusters[s - 1] - 1) / clusters[s - 1];
            const int64_t cost = waves * ((blocks + s - 1) / s * BLOCK[i] + ENDS[i] + (s > 1 ? 100 : 0));
            if (cost < least) {
                least = cost;
                best = {BN[i], s};
            }
        }
    return best;
}

template <class T, int G>
bsp_status_t wide_by_shape(const Problem& p, cudaStream_t s)
{
    const int* clusters = clusters_at_once<T, G>(p.device, p.num_sms);
    if (!clusters) return BSP_ERR_CUDA;
    const Plan plan = plan_of<G>(p, clusters);
    auto go = [&](auto bn) {
        constexpr int BN = decltype(bn)::value;
        return p.gated ? launch_wide<T, G, BN, true>(p, plan.shares, s) : launch_wide<T, G, BN, false>(p, plan.shares, s);
    };
    using std::integral_constant;
    switch (plan.bn) {
    case 64: return go(integral_constant<int, 64>());
    case 128: return go(integral_constant<int, 128>());
    default: return go(integral_constant<int, 256>());
    }
}

template <class T>
bsp_status_t run_wide(const Problem& p, cudaStream_t s)
{
    switch (p.group) {
    case 32: return wide_by_shape<T, 32>(p, s);
    case 64: return wide_by_shape<T, 64>(p, s);
    default: return wide_by_shape<T, 128>(p, s);
    }
}

}  // namespace
