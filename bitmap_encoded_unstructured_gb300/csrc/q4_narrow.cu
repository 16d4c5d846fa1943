// Products of 4-bit weights with few activation rows (decoding), and the
// gated form over two weights, on mma.sync.
//
// A warp takes RT row tiles (16 rows of W each) and a share of the columns;
// codes, scales and activations run through a ring of its own in shared
// memory (cp.async: every lane reads back its own codes and activations, so
// no barrier but the warp's).  Codes less zero points are small integers,
// exact in either type; they are multiplied as they are and the group's scale
// is applied to its fp32 sums, so no weight is rounded:
//   Y[n][m] += s sum_k (c - z) x
//   fp16: a masked nibble under the exponent of 1024 is 1024 + c, or 1024 +
//   16 c in the second nibble, which belongs to the tile's upper rows and so
//   to sums of their own; one subtraction of two values takes the rest away,
//   and the 16 goes into the scale.  bf16: 128 + c.
//   (A masked nibble alone, a subnormal, needs no subtraction, but tensor
//   cores align subnormals as if they had the smallest normal exponent: the sums
//   lose ten bits.)
// The 8 warps of a CTA split the columns, and C CTAs of a cluster split them
// further where the row tiles alone do not fill the GPU; all parts are added in
// a fixed order.
#include "bsp_q4.cuh"

#include <algorithm>

namespace {

using namespace bspq4;

constexpr int WARPS = 8, THREADS = WARPS * 32;

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

template <int RT, int NT>
struct Slot {  // of a warp and a stage of 64 columns
    static constexpr int X = RT * 512, S = X + NT * 1024, Z = S + RT * 64, BYTES = Z + RT * 16;
};

template <int RT, int NT>
struct Ring {
    static constexpr int DEPTH = RT * NT == 2 ? 6 : 3;
    static constexpr int BYTES = WARPS * DEPTH * Slot<RT, NT>::BYTES;
    static_assert(BYTES >= WARPS * RT * 8 * NT * 17 * 4 + RT * 8 * NT * 16 * 4, "parts of the warps and their sum");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src)
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

template <class T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <class T, int G, int NT, int RT, bool GATED>
__global__ void __launch_bounds__(THREADS, 2) q4_narrow_kernel(const NarrowArgs a)
{
    using L = Slot<RT, NT>;
    using R = Ring<RT, NT>;
    constexpr int D = R::DEPTH;
    constexpr int TILES = GATED ? RT / 2 : RT;  // row tiles of Y
    constexpr int COLS = 8 * NT;
    constexpr int PER = 64 / G ? 64 / G : 1;    // groups of a stage (G = 128: one of two stages)
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint32_t C, crank;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
    crank = bspx::cluster_ctarank();
    const int64_t tile0 = (int64_t)(blockIdx.x / C) * TILES, strip = tile0 / 8;
    const int rt0 = (int)(tile0 % 8);  // TILES divides 8: one strip
    const int n0 = blockIdx.y * COLS, n_here = min(COLS, a.N - n0);
    const uint32_t ring = bspx::smem_u32(smem) + warp * D * L::BYTES;

    // this warp's columns: whole blocks of 128
    const int units = a.k_tiles >> 1, ranks = WARPS * C, rank = crank * WARPS + warp;
    const int k_begin = 2 * (int)((int64_t)units * rank / ranks);
    const int k_count = 2 * (int)((int64_t)units * (rank + 1) / ranks) - k_begin;

    auto of = [&](int r) { return GATED && r >= TILES ? a.w[1] : a.w[0]; };  // row tile r's weight
    const uint4* codes[RT];
    const uint8_t *meta = nullptr, *zero = nullptr;  // what this lane copies of the scales and zero points
#pragma unroll
    for (int r = 0; r < RT; ++r)
        codes[r] = of(r).codes + (strip * a.k_tiles + k_begin) * 256 + (rt0 + r % TILES) * 32 + lane;
    const int64_t group0 = strip * a.groups + (int64_t)k_begin * 64 / G;
    constexpr int CHUNKS = PER * 2;  // 16-byte pieces of a row tile's scales in a stage
    if (lane < RT * CHUNKS) {
        const int r = lane / CHUNKS, c = lane % CHUNKS;
        meta = reinterpret_cast<const uint8_t*>(of(r).scales + (group0 + c / 2) * 64 + (rt0 + r % TILES) * 8) + c % 2 * 16;
    }
    if (lane < RT * PER) {
        const int r = lane / PER;
        const uint8_t* z = of(r).zeros;
        if (z) zero = z + (group0 + lane % PER) * 64 + (rt0 + r % TILES) * 8;
    }
    const bool has_zeros[2] = {a.w[0].zeros != nullptr, GATED && a.w[1].zeros != nullptr};
    const char* xrow[NT];
    bool live[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        live[i] = 8 * i + g < n_here;
        xrow[i] = reinterpret_cast<const char*>(a.x) + (int64_t)(n0 + (live[i] ? 8 * i + g : 0)) * a.x_stride * 2;
    }

    auto copy_weights = [&](int i) {  // stage i of this warp
        const uint32_t slot = ring + (uint32_t)(i % D) * L::BYTES;
#pragma unroll
        for (int r = 0; r < RT; ++r) cp16(slot + r * 512 + lane * 16, codes[r] + (int64_t)i * 256, 16);
        if (G < 128 || !(i & 1)) {
            const int64_t at = (int64_t)(G == 128 ? i >> 1 : i) * PER * 64;
            if (lane < RT * CHUNKS) cp16(slot + L::S + lane / CHUNKS * 64 + lane % CHUNKS * 16, meta + at * 4, 16);
            if (lane < RT * PER && zero) cp8(slot + L::Z + lane / PER * 16 + lane % PER * 8, zero + at);
        }
    };
    auto copy_x = [&](int i) {
        const uint32_t slot = ring + (uint32_t)(i % D) * L::BYTES + L::X;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = (int64_t)(k_begin + i) * 64 + 32 * h + 8 * t;  // K is a multiple of 8
                if (live[nt]) cp16(slot + (2 * nt + h) * 512 + lane * 16, xrow[nt] + (k < a.K ? k * 2 : 0), k < a.K ? 16 : 0);
            }
    };

    // weights do not depend on the kernels before this one
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
        if (i < k_count) copy_weights(i);
    launch_dependents();
    wait_prior_grids();
#pragma unroll
    for (int i = 0; i < D - 1; ++i) {
        if (i < k_count) copy_x(i);
        cp_commit();
    }

    float out[RT][NT][4], acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[r][nt][e] = acc[r][nt][e] = 0.f;
    uint32_t scale[RT], z0[RT], z1[RT];

    auto load_scales = [&](uint32_t slot, int part) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            scale[r] = lds4(slot + L::S + r * 64 + part * 32 + g * 4);
            Codes<T>::bias(has_zeros[GATED ? r / TILES : 0] ? lds1(slot + L::Z + r * 16 + part * 8 + g) : 0x88u, z0[r],
                           z1[r]);
        }
    };
    auto flush = [&]() {  // the group's sums, scaled, into out
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float s0 = half_of<T>(scale[r], 0), s1 = half_of<T>(scale[r], 1) * (1.f / Codes<T>::UPPER);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    out[r][nt][e] = fmaf(e < 2 ? s0 : s1, acc[r][nt][e], out[r][nt][e]);
                    acc[r][nt][e] = 0.f;
                }
        }
    };

    for (int i0 = 0; i0 < k_count; i0 += 2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = i0 + e;
            cp_wait<D - 2>();
            __syncwarp();  // every lane's copies of this stage are there, and its slot of the last one is free
            if (i + D - 1 < k_count) {
                copy_weights(i + D - 1);
                copy_x(i + D - 1);
            }
            cp_commit();
            const uint32_t slot = ring + (uint32_t)(i % D) * L::BYTES;
            uint4 w[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) w[r] = lds16(slot + r * 512 + lane * 16);
            if (G == 64 || (G == 128 && e == 0)) load_scales(slot, 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 x[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    x[nt] = make_uint4(0u, 0u, 0u, 0u);
                    if (live[nt]) x[nt] = lds16(slot + L::X + (2 * nt + h) * 512 + lane * 16);
                }
                if (G == 32) load_scales(slot, h);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        uint32_t av[4];
                        Codes<T>::widen(h ? (j ? w[r].w : w[r].z) : (j ? w[r].y : w[r].x), z0[r], z1[r], av);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma<T>(acc[r][nt], av, j ? x[nt].z : x[nt].x, j ? x[nt].w : x[nt].y);
                    }
                }
                if (G == 32) flush();
            }
            if (G == 64 || (G == 128 && e == 1)) flush();
        }
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
                parts[((warp * RT + r) * COLS + 8 * nt + 2 * t + (e & 1)) * 17 + g + 8 * (e >> 1)] = out[r][nt][e];
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

template <class T, int G, int NT, int RT, bool GATED>
bsp_status_t launch(const Problem& p, cudaStream_t s)
{
    constexpr int SMEM = Ring<RT, NT>::BYTES;
    static bsp_attr_once attr_once;
    if (!attr_once.run(p.device, [] {
            return cudaFuncSetAttribute(q4_narrow_kernel<T, G, NT, RT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    // a cluster splits the columns until two CTAs an SM are there, or a warp
    // has less than two blocks of columns
    int c = 1;
    while (c < 8 && tiles * blocks * c < 2 * p.num_sms && p.k_tiles / 2 >= 2 * WARPS * c * 2) c *= 2;
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
    return cudaLaunchKernelEx(&cfg, q4_narrow_kernel<T, G, NT, RT, GATED>, a) == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

template <class T, int G>
bsp_status_t by_shape(const Problem& p, cudaStream_t s)
{
    // activations are read once for every RT row tiles: two for up to 8
    // columns, four for up to 16
    if (p.gated) return p.N <= 8 ? launch<T, G, 1, 2, true>(p, s) : launch<T, G, 2, 4, true>(p, s);
    return p.N <= 8 ? launch<T, G, 1, 2, false>(p, s) : launch<T, G, 2, 4, false>(p, s);
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

bsp_status_t bsp_run_q4_narrow(const Problem& p, cudaStream_t s)
{
    return p.dtype == BSP_FP16 ? by_group<__half>(p, s) : by_group<__nv_bfloat16>(p, s);
}
