// Internal declarations of the 4-bit weights (q4_weights.cu, q4_narrow.cuh,
// q4_wide.cuh): the handle, its layout and the products' arguments.
#pragma once

#include "bsp_internal.cuh"
#include "bsp_ptx.cuh"

#include <cuda_bf16.h>

#define BSP_Q4_MAGIC 0xB5B14B17u

// Layout.  W is padded to strips of 128 rows and blocks of 128 columns and cut
// into tiles of 16 rows x 64 columns of 512 bytes, 16 for each lane of a
// warp: [strip][columns / 64][row tile of the strip][lane].  Lane (g, t) =
// (lane / 4, lane % 4) holds rows g and g + 8 of the tile, columns 32 h + 8 t
// .. + 7 for h = 0, 1; its 32-bit word 2 h + j has columns k = 32 h + 8 t + 4 j
// and the three after it, one code a nibble:
//   nibble  0     1      2      3        4      5       6      7
//           g,k   g+8,k  g,k+2  g+8,k+2  g,k+1  g+8,k+1 g,k+3  g+8,k+3
// so that a mask leaves two neighbouring columns of one row in the two
// halves of a register: the A operand of mma.m16n8k16 with its columns
// renumbered (as the B operand's are), and eight columns of a row in 16
// bytes for a shared-memory tile.
//   scales  [strip][group][row tile][g] pairs (row g, row g + 8) of the dtype
//   zeros   [strip][group][row tile][g] bytes, row g in the low half, g + 8 above
// with group = columns / G.  A strip's block of 128 columns is one piece of
// memory in each of the three.  Rows past M have scales of 0.
struct Q4View {
    const uint4* codes;
    const uint32_t* scales;
    const uint8_t* zeros;  // null: 8 throughout
};

struct bsp_q4 {
    uint32_t magic;
    int device, num_sms;
    bsp_dtype_t dtype;  // of the scales, and of X and Y: BSP_FP16 or BSP_BF16
    int64_t M, K;
    int32_t group;      // 32, 64 or 128
    int64_t strips, k_tiles;  // of the padded grid; k_tiles is even
    uint4* codes;
    uint32_t* scales;
    uint8_t* zeros;
    int* err;  // as bsp_handle::err
    int64_t groups() const { return k_tiles * 64 / group; }  // of the padded grid
};

namespace bspq4 {

inline bool valid(const bsp_q4* h) { return h != nullptr && h->magic == BSP_Q4_MAGIC; }

// Everything a product reads and writes.  Two weights: the gated form.
struct Problem {
    Q4View w, up;
    bool gated;
    int act;  // bsp_act_t
    bsp_dtype_t dtype;
    int64_t M, K, strips, k_tiles;
    int32_t group;
    const void* x;
    int64_t x_stride, N;
    void* y;
    int64_t y_stride;
    int device, num_sms;
    int* err;
};

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

// The low (lo) or high half of a pair of the dtype as fp32.
template <class T>
__device__ __forceinline__ float half_of(uint32_t pair, int high)
{
    const uint16_t bits = (uint16_t)(high ? pair >> 16 : pair);
    return to_float(*reinterpret_cast<const T*>(&bits));
}

// Pairs of the dtype from a word of codes: UNIT (c - z) of rows g (a[0],
// a[2]), and UPPER times as much of rows g + 8; z0 and z1 are the pairs that
// bias() makes.  Outputs are divided by UNIT, a power of two: bf16 codes are
// that small so that a group's sum before its scale, at most 128 x 15 x 2^-11
// of the largest activation, is finite wherever the activations are.
template <class T>
struct Codes;
template <>
struct Codes<__half> {
    static constexpr float UNIT = 1.f, UPPER = 16.f;
    static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b)
    {
        const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&d);
    }
    static __device__ __forceinline__ void bias(uint32_t zeros, uint32_t& z0, uint32_t& z1)
    {
        z0 = (zeros & 15u) * 0x10001u | 0x64006400u;
        z1 = (zeros & 240u) * 0x10001u | 0x64006400u;
    }
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t z0, uint32_t z1, uint32_t (&a)[4])
    {
        const uint32_t v = w >> 8;
        a[0] = less((w & 0x000F000Fu) | 0x64006400u, z0);
        a[1] = less((w & 0x00F000F0u) | 0x64006400u, z1);
        a[2] = less((v & 0x000F000Fu) | 0x64006400u, z0);
        a[3] = less((v & 0x00F000F0u) | 0x64006400u, z1);
    }
};
template <>
struct Codes<__nv_bfloat16> {
    static constexpr float UNIT = 0x1p-11f, UPPER = 1.f;
    static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b)
    {
        const __nv_bfloat162 d =
            __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&d);
    }
    static __device__ __forceinline__ void bias(uint32_t zeros, uint32_t& z0, uint32_t& z1)
    {
        z0 = (zeros & 15u) * 0x10001u | 0x3D803D80u;
        z1 = (zeros >> 4) * 0x10001u | 0x3D803D80u;
    }
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t z0, uint32_t z1, uint32_t (&a)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = less(((w >> (4 * i)) & 0x000F000Fu) | 0x3D803D80u, i & 1 ? z1 : z0);
    }
};

__device__ __forceinline__ float activate(float g, int act)
{
    if (act == BSP_ACT_RELU) return g != g ? g : fmaxf(g, 0.f);  // a NaN stays one
    if (act == BSP_ACT_GELU) return 0.5f * g * erfcf(-0.70710678118654752f * g);
    // silu: g / (1 + exp(-y)) with y = g; gelu_tanh: the same with its own y,
    // 0.5 (1 + tanh(y / 2)) being 1 / (1 + exp(-y)).  From exp(-|y|): exp(-y) itself
    // would be infinite from y = -88.7 on, where the quotient is still far from 0 in bf16.
    const float y = act == BSP_ACT_SILU ? g : 1.59576912160573071f * (g + 0.044715f * g * g * g);
    const float e = __expf(-fabsf(y));
    return (y < 0.f ? g * e : g) / (1.f + e);
}

__device__ __forceinline__ void wait_prior_grids() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace bspq4

// Few rows of X (q4_narrow.cuh), and more (q4_wide.cuh), by type.  The narrow
// kernel takes 53.6 us for 32 rows of 28672 x 8192, 33.2 of 20480 x 5120, 16.3 of
// 11008 x 4096, 11.2 of 4096 x 4096 and 7.0 of 1024 x 4096, the wide one for 33
// rows 68.0, 40.0, 18.6, 9.8 and 6.5: it is ahead but for small weights.  With 33 the narrow
// one would read the codes twice.
constexpr int64_t BSP_Q4_NARROW_N = 32;
bsp_status_t bsp_run_q4_narrow_f16(const bspq4::Problem& p, cudaStream_t s);
bsp_status_t bsp_run_q4_narrow_bf16(const bspq4::Problem& p, cudaStream_t s);
bsp_status_t bsp_run_q4_wide_f16(const bspq4::Problem& p, cudaStream_t s);
bsp_status_t bsp_run_q4_wide_bf16(const bspq4::Problem& p, cudaStream_t s);
