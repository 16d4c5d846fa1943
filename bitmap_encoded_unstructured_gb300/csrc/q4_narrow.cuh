// Products of 4-bit weights with up to 32 activation rows (decoding), and the
// gated form over two weights, on mma.sync.
//
// A warp takes RT row tiles (16 rows of W each) and a share of the columns;
// codes and scales run through a ring of its own in shared memory (cp.async:
// every lane reads back its own codes, so no barrier but the warp's).  Codes less zero points are small integers,
// exact in either type; they are multiplied as they are and the group's scale
// is applied to its fp32 sums, so no weight is rounded:
//   Y[n][m] += s sum_k (c - z) x
//   fp16: a masked nibble under the exponent of 1024 is 1024 + c, or 1024 +
//   16 c in the second nibble, which belongs to the tile's upper rows and so
//   to sums of their own; one subtraction of two values takes the rest away,
//   and the 16 comes off at the end.  bf16: the same with 2^-4 + 2^-11 c, for the
//   range of its sums (bsp_q4.cuh).
//   (A masked nibble alone, a subnormal, needs no subtraction, but tensor
//   cores align subnormals as if they had the smallest normal exponent: the sums
//   lose ten bits.)
// The warps of a CTA split the columns, and C CTAs of a cluster split them
// further where the row tiles alone do not fill the GPU; all parts are added in
// a fixed order.
//
// Nothing is saturated (DRAM 44%, issue slots 55%, logic pipe 56% with one row of 28672 x
// 8192; the same loads without the arithmetic run at 0.9 of a copy): a warp
// waits for its own chain of copy, widening and product, three or four
// CTAs of four warps an SM, and CTAs come in whole waves of 608 (32 rows of W
// a CTA; gated 16) or 456 (9 to 16 rows of X: 64 rows of W).  8192 columns, one row: 19456 rows of W (one wave)
// 18.5 us (0.66 of a copy), 28672 (1.47 waves) 27.0 (0.66), 38912 (two) 34.4
// (0.70).  Gated, 4096 columns: 9728 rows (one wave) 11.5 us, 11008 (1.13) 15.2.
// 16 rows, 5120 columns: 20480 rows of W (320 CTAs) 21.2 us, 29184 (456) 22.4.
// 17 to 32 rows: 8192 columns and 29184 rows of W 53.9 us with 32.  Short calls are latency:
// one row of 5120 x 5120 takes 7.2 us, of which the codes' bytes are 2.0.
#pragma once

#include "bsp_q4.cuh"

#include <algorithm>
#include <type_traits>

namespace {

using namespace bspq4;

constexpr int WARPS = 4, THREADS = WARPS * 32;

struct NarrowArgs {
    Q4View w[2];
    int act;
    int64_t M, K, groups;
    int32_t k_tiles, N;
    const void* x;
    int64_t x_stride;
    void* y;
    int64_t y_stride;
};

// A warp's ring: blocks of 128 columns of RT row tiles, with the scales and
// zero points of their groups.
template <int G, int RT, int NT>
struct Ring {
    static constexpr int PER = 128 / G;  // groups of a block
    static constexpr int S = RT * 1024, Z = S + PER * RT * 32;
    static constexpr int BYTES = (Z + PER * RT * 8 + 15) / 16 * 16;
    static constexpr int DEPTH = RT == 2 ? 6 : 4, ALL = WARPS * DEPTH * BYTES;
    static constexpr int CTAS = RT == 2 && NT == 1 ? 4 : 3;  // an SM
    static_assert(ALL >= WARPS * RT * 8 * NT * 17 * 4 + RT * 8 * NT * 16 * 4, "parts of the warps and their sum");
    static_assert(CTAS * (ALL + 1024) <= 227 * 1024, "shared memory");
};

template <int TO, int FROM>
__device__ __forceinline__ void cp16(uint32_t dst, const char* src)
{
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(TO), "n"(FROM) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const char* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}

// 16 bytes of activations.  Not through the read-only path: the kernel is
// resident while the kernel before it may still write them, and only loads
// behind griddepcontrol.wait see what it wrote (volatile asm keeps its place).
__device__ __forceinline__ uint4 ldg16(const char* at)
{
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
    return v;
}

// c += a b, or a b (FIRST).
template <class T, bool FIRST>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    const float z0 = FIRST ? 0.f : c[0], z1 = FIRST ? 0.f : c[1], z2 = FIRST ? 0.f : c[2], z3 = FIRST ? 0.f : c[3];
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
}

// What lanes of rows that are not there read as activations.
__device__ const uint4 kNothing[16] = {};

template <class T, int G, int NT, int RT, bool GATED, bool ZEROS>
__global__ void __launch_bounds__(THREADS, Ring<G, RT, NT>::CTAS) q4_narrow_kernel(const __grid_constant__ NarrowArgs a)
{
    using R = Ring<G, RT, NT>;
    constexpr int D = R::DEPTH, PER = R::PER;
    constexpr int TILES = GATED ? RT / 2 : RT;  // row tiles of Y
    constexpr int COLS = 8 * NT;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint32_t C, crank;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
    crank = bspx::cluster_ctarank();
    const int64_t tile0 = (int64_t)(blockIdx.x / C) * TILES, strip = tile0 / 8;
    const int rt0 = (int)(tile0 % 8);  // TILES divides 8: one strip
    const int n0 = blockIdx.y * COLS, n_here = min(COLS, a.N - n0);
    const uint32_t ring = bspx::smem_u32(smem) + warp * D * R::BYTES, ring_end = ring + D * R::BYTES;

    // this warp's blocks of 128 columns
    const int blocks = a.k_tiles >> 1, ranks = WARPS * C, rank = crank * WARPS + warp;
    const int first = (int)((int64_t)blocks * rank / ranks);
    const int count = (int)((int64_t)blocks * (rank + 1) / ranks) - first;

    // what this lane copies of a block, at the next block to copy
    const char *codes = nullptr, *codes_up = nullptr, *scales = nullptr, *zeros = nullptr;
    auto codes_of = [&](const Q4View& v) {
        return reinterpret_cast<const char*>(v.codes + (strip * a.k_tiles + 2 * first) * 256 + rt0 * 32 + lane);
    };
    codes = codes_of(a.w[0]);
    if (GATED) codes_up = codes_of(a.w[1]);
    const int64_t group0 = strip * a.groups + (int64_t)first * PER;
    if (lane < PER * RT * 2) {  // scales [group][row tile]: 32 bytes, two lanes
        const int p = lane / (RT * 2), r = lane / 2 % RT;
        const Q4View& v = GATED && r >= TILES ? a.w[1] : a.w[0];
        scales = reinterpret_cast<const char*>(v.scales + (group0 + p) * 64 + (rt0 + r % TILES) * 8) + lane % 2 * 16;
    }
    if (lane < PER * RT) {  // zero points: 8 bytes
        const int p = lane / RT, r = lane % RT;
        const uint8_t* z = (GATED && r >= TILES ? a.w[1] : a.w[0]).zeros;
        if (ZEROS && z) zeros = reinterpret_cast<const char*>(z + (group0 + p) * 64 + (rt0 + r % TILES) * 8);
    }
    const bool has_zeros[2] = {a.w[0].zeros != nullptr, GATED && a.w[1].zeros != nullptr};
    // activations go from L2 to registers, a block ahead: this lane's eight
    // columns of row 8 nt + g in each quarter of the block
    const char* x[NT];
    int step[NT];  // bytes between blocks; 0: the row is not there
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        step[i] = 8 * i + g < n_here ? 256 : 0;
        const int64_t at = (int64_t)(n0 + 8 * i + g) * a.x_stride + (int64_t)first * 128 + 8 * t;
        x[i] = step[i] ? reinterpret_cast<const char*>(a.x) + at * 2
                       : reinterpret_cast<const char*>(kNothing) + t * 16;
    }
    const int whole = (int)(a.K / 128) - first;       // blocks from here on that lie inside K
    const int left = (int)(a.K % 128) - 8 * t;        // of the block behind them: columns from this lane's first on
    uint4 b[NT][4];
    auto load_x = [&](int nt, int q) { b[nt][q] = ldg16(x[nt] + 64 * q); };
    auto load_last_x = [&](int nt, int q) {  // of a block in which K, a multiple of 8, ends
        b[nt][q] = make_uint4(0u, 0u, 0u, 0u);
        if (left > 32 * q) load_x(nt, q);
    };
    const int full = min(count, whole);  // blocks inside K

    auto copy_weights = [&](uint32_t slot) {
        const uint32_t to = slot + lane * 16;
        auto tile = [&](auto r) {
            constexpr int Q = decltype(r)::value;
            if constexpr (Q < RT) {
                cp16<Q * 512, Q % TILES * 512>(to, GATED && Q >= TILES ? codes_up : codes);
                cp16<RT * 512 + Q * 512, 4096 + Q % TILES * 512>(to, GATED && Q >= TILES ? codes_up : codes);
            }
        };
        tile(std::integral_constant<int, 0>());
        tile(std::integral_constant<int, 1>());
        tile(std::integral_constant<int, 2>());
        tile(std::integral_constant<int, 3>());
        if (lane < PER * RT * 2) cp16<R::S, 0>(to, scales);
        if (ZEROS && zeros) cp8(slot + R::Z + lane * 8, zeros);
        codes += 8192;
        if (GATED) codes_up += 8192;
        scales += PER * 256;
        if (ZEROS && zeros) zeros += PER * 64;
    };
    // weights do not depend on the kernels before this one
#pragma unroll
    for (int i = 0; i < D - 1; ++i) {
        if (i < count) copy_weights(ring + i * R::BYTES);
        cp_commit();
    }
    launch_dependents();
    wait_prior_grids();
    if (full > 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 4; ++q) load_x(nt, q);

    float out[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[r][nt][e] = 0.f;

    uint32_t slot = ring, to_slot = ring + (D - 1) * R::BYTES;  // to read; to fill: the one read last
    auto block = [&](int i, auto last) {
        constexpr bool LAST = decltype(last)::value;
        cp_wait<D - 2>();
        __syncwarp();  // every lane's copies of this block are there, and the slot of the last one is free
        if (i + D - 1 < count) copy_weights(to_slot);
        cp_commit();
        to_slot = slot;
        // the next block's activations take the place of this one's as they are
        // used (behind the last whole block: its own again)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[nt] += i + 1 < full ? step[nt] : 0;
        float acc[RT][NT][4];
        float s0[RT], s1[RT];
        uint32_t z0[RT], z1[RT];
        auto load_scales = [&](int p) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t pair = lds4(slot + R::S + (p * RT + r) * 32 + g * 4);
                s0[r] = half_of<T>(pair, 0);
                s1[r] = half_of<T>(pair, 1);
                const bool own = ZEROS && has_zeros[GATED && r >= TILES];
                Codes<T>::bias(own ? lds1(slot + R::Z + (p * RT + r) * 8 + g) : 0x88u, z0[r], z1[r]);
            }
        };
        auto flush = [&]() {  // the group's sums, scaled, into out
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) out[r][nt][e] = fmaf(e < 2 ? s0[r] : s1[r], acc[r][nt][e], out[r][nt][e]);
        };
        if (G == 128) load_scales(0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint4 w[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) w[r] = lds16(slot + e * (RT * 512) + r * 512 + lane * 16);
            if (G == 64) load_scales(e);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (G == 32) load_scales(2 * e + h);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        uint32_t av[4];
                        Codes<T>::widen(h ? (j ? w[r].w : w[r].z) : (j ? w[r].y : w[r].x), z0[r], z1[r], av);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4& q = b[nt][2 * e + h];
                            const uint32_t b0 = j ? q.z : q.x, b1 = j ? q.w : q.y;
                            if (j == 0 && (G == 32 || (h == 0 && (G == 64 || e == 0)))) mma<T, true>(acc[r][nt], av, b0, b1);
                            else mma<T, false>(acc[r][nt], av, b0, b1);
                        }
                    }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (!LAST) load_x(nt, 2 * e + h);
                if (G == 32) flush();
            }
            if (G == 64) flush();
        }
        if (G == 128) flush();
        slot += R::BYTES;
        if (slot == ring_end) slot = ring;
    };
    for (int i = 0; i < full; ++i) block(i, std::false_type());
    if (full < count) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (full > 0) x[nt] += step[nt];
#pragma unroll
            for (int q = 0; q < 4; ++q) load_last_x(nt, q);
        }
        block(full, std::true_type());
    }

    // ---- the warps' parts, then the cluster's, added in order
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* parts = reinterpret_cast<float*>(smem);          // [warp][row tile][column][17]
    float* sums = parts + WARPS * RT * COLS * 17;           // [row tile][column][16]
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                parts[((warp * RT + r) * COLS + 8 * nt + 2 * t + (e & 1)) * 17 + g + 8 * (e >> 1)] =
                    out[r][nt][e] * ((e < 2 ? 1.f : 1.f / Codes<T>::UPPER) / Codes<T>::UNIT);
    __syncthreads();
    for (int i = threadIdx.x; i < RT * COLS * 16; i += THREADS) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += parts[(w * RT * COLS + i / 16) * 17 + i % 16];
        sums[i] = v;
    }
    if (C > 1) bspx::cluster_sync();
    else __syncthreads();
    auto total = [&](int i) {
        if (C == 1) return sums[i];
        float v = 0.f;
        for (uint32_t c = 0; c < C; ++c) {
            float p;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(bspx::mapa_shared(bspx::smem_u32(sums + i), c)));
            v += p;
        }
        return v;
    };
    T* y = reinterpret_cast<T*>(a.y);
    for (int i = crank * THREADS + threadIdx.x; i < TILES * COLS * 16; i += THREADS * C) {
        const int row = i % (TILES * 16), n = i / (TILES * 16);
        const int64_t m = tile0 * 16 + row;
        if (m >= a.M || n >= n_here) continue;
        const int at = (row / 16 * COLS + n) * 16 + row % 16;
        float v = total(at);
        if (GATED) v = activate(v, a.act) * total(at + TILES * COLS * 16);
        y[(int64_t)(n0 + n) * a.y_stride + m] = from_float<T>(v);
    }
    if (C > 1) bspx::cluster_sync();  // others may still read this CTA's sums
}

template <class T, int G, int NT, int RT, bool GATED, bool ZEROS>
bsp_status_t launch_as(const Problem& p, cudaStream_t s)
{
    constexpr int SMEM = Ring<G, RT, NT>::ALL;
    static bsp_attr_once attr_once;
    if (!attr_once.run(p.device, [] {
            return cudaFuncSetAttribute(q4_narrow_kernel<T, G, NT, RT, GATED, ZEROS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        SMEM);
        }))
        return BSP_ERR_CUDA;
    NarrowArgs a;
    a.w[0] = p.w;
    a.w[1] = p.gated ? p.up : p.w;
    a.act = p.act;
    a.M = p.M;
    a.K = p.K;
    a.groups = p.k_tiles * 64 / G;
    a.k_tiles = (int32_t)p.k_tiles;
    a.N = (int32_t)p.N;
    a.x = p.x;
    a.x_stride = p.x_stride;
    a.y = p.y;
    a.y_stride = p.y_stride;
    constexpr int TILES = GATED ? RT / 2 : RT;
    const int64_t tiles = (p.M + 16 * TILES - 1) / (16 * TILES), blocks = (p.N + 8 * NT - 1) / (8 * NT);
    // a cluster splits the columns as far as its CTAs fit the GPU at once and
    // a warp keeps four blocks of columns (4864 x 4096, one row: 8.3 us in
    // clusters of four with two blocks a warp, 5.9 in pairs with four)
    const int64_t fit = (int64_t)Ring<G, RT, NT>::CTAS * p.num_sms / (tiles * blocks), keep = p.k_tiles / 2 / (4 * WARPS);
    const int c = (int)std::max<int64_t>(1, std::min<int64_t>({8, fit, keep}));
    if (tiles * c > INT32_MAX || blocks > 65535) return BSP_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * c), (unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = c;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q4_narrow_kernel<T, G, NT, RT, GATED, ZEROS>, a) == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

template <class T, int G, int NT, int RT, bool GATED>
bsp_status_t launch(const Problem& p, cudaStream_t s)
{
    return p.w.zeros || (GATED && p.up.zeros) ? launch_as<T, G, NT, RT, GATED, true>(p, s)
                                              : launch_as<T, G, NT, RT, GATED, false>(p, s);
}

template <class T, int G>
bsp_status_t by_shape(const Problem& p, cudaStream_t s)
{
    // activations are read once for every RT row tiles: two for up to 8
    // columns, four for up to 16 (and two again for up to 32, whose sums and
    // activations fill the registers)
    auto go = [&](auto gated) {
        constexpr bool GATED = decltype(gated)::value;
        if (p.N <= 8) return launch<T, G, 1, 2, GATED>(p, s);
        if (p.N <= 16) return launch<T, G, 2, 4, GATED>(p, s);
        return launch<T, G, 4, 2, GATED>(p, s);
    };
    return p.gated ? go(std::true_type()) : go(std::false_type());
}

template <class T>
bsp_status_t by_group(const Problem& p, cudaStream_t s)
{
    switch (p.group) {
    case 32: return by_shape<T, 32>(p, s);
    case 64: return by_shape<T, 64>(p, s);
    default: return by_shape<T, 128>(p, s);
    }
}

}  // namespace
