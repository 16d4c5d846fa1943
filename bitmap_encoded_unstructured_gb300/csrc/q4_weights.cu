// 4-bit weights with group scales: quantising, the handle and its layout
// (bsp_q4.cuh), and the entry points of their products.
#include "bsp_overlap.h"
#include "bsp_q4.cuh"

#include <cmath>
#include <new>

namespace {

using namespace bspq4;

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// ---------------------------------------------------------------- encoding

// One warp a group of a row: the scale (and zero point), and its codes two
// to a byte.  A lane takes columns 2 lane and 2 lane + 1 of every 64.
template <class T>
__global__ void q4_quantise_kernel(const T* W, int64_t M, int64_t K, int32_t G, int64_t groups, uint8_t* codes,
                                   T* scales, uint8_t* zeros)
{
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (item >= M * groups) return;
    const int64_t m = item / groups, gr = item % groups, k0 = gr * G;
    const int cols = (int)min((int64_t)G, K - k0);
    float w[2][2];
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = 64 * i + 2 * lane + e;
            float v = c < cols ? to_float(W[m * K + k0 + c]) : 0.f;
            w[i][e] = v;
            if (isfinite(v)) {
                lo = fminf(lo, v);
                hi = fmaxf(hi, v);
            }
        }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, d));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, d));
    }
    // (hi - lo itself may pass the range of fp32)
    const float want = zeros ? __fsub_rn(__fdiv_rn(hi, 15.f), __fdiv_rn(lo, 15.f)) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
    const T rounded = from_float<T>(want);
    const float s = to_float(rounded);
    float z = 8.f;
    if (zeros) z = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 8.f;
    if (lane == 0) {
        scales[item] = rounded;
        if (zeros) zeros[item] = (uint8_t)z;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = 64 * i + 2 * lane;
        if (c >= cols) continue;
        uint32_t byte = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float q = z;
            if (s > 0.f && w[i][e] == w[i][e]) q = fminf(fmaxf(rintf(__fdiv_rn(w[i][e], s)) + z, 0.f), 15.f);
            byte |= (uint32_t)q << (4 * e);
        }
        codes[(m * K + k0 + c) >> 1] = (uint8_t)byte;
    }
}

// ------------------------------------------------------------------ layout

// Eight codes of row m from column k on (a multiple of 8), column k in the
// lowest nibble; 8s outside the matrix.
__device__ __forceinline__ uint32_t eight(const uint8_t* codes, int64_t M, int64_t K, int64_t m, int64_t k)
{
    return m < M && k < K ? *reinterpret_cast<const uint32_t*>(codes + ((m * K + k) >> 1)) : 0x88888888u;
}

__device__ __forceinline__ uint32_t nibble(uint32_t w, int i) { return (w >> (4 * i)) & 15u; }

// The first row and column of lane i of the layout.
struct Place {
    int64_t m, k;
};
__device__ __forceinline__ Place place_of(int64_t i, int64_t k_tiles)
{
    const int lane = (int)(i & 31), rt = (int)(i >> 5 & 7);
    const int64_t tile = i >> 8;  // strip, columns / 64
    return {tile / k_tiles * 128 + rt * 16 + (lane >> 2), tile % k_tiles * 64 + 8 * (lane & 3)};
}
// The first row of pair i of the scales, and its group.
__device__ __forceinline__ Place pair_of(int64_t i, int64_t groups)
{
    return {(i >> 6) / groups * 128 + (i >> 3 & 7) * 16 + (i & 7), (i >> 6) % groups};
}

// A thread a lane of a tile.
__global__ void q4_pack_kernel(const uint8_t* codes, int64_t M, int64_t K, int64_t k_tiles, int64_t n, uint4* out)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t m = place_of(i, k_tiles).m, k = place_of(i, k_tiles).k;
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = eight(codes, M, K, m, k + 32 * h), b = eight(codes, M, K, m + 8, k + 32 * h);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[2 * h + j] = nibble(a, 4 * j) | nibble(b, 4 * j) << 4 | nibble(a, 4 * j + 2) << 8 |
                           nibble(b, 4 * j + 2) << 12 | nibble(a, 4 * j + 1) << 16 | nibble(b, 4 * j + 1) << 20 |
                           nibble(a, 4 * j + 3) << 24 | nibble(b, 4 * j + 3) << 28;
    }
    out[i] = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight codes of row g (upper = 0) or g + 8 in the plain order, from words
// 2 h and 2 h + 1.
__device__ __forceinline__ uint32_t plain(uint32_t w0, uint32_t w1, int upper)
{
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t w = (j ? w1 : w0) >> (4 * upper);
        v |= (nibble(w, 0) | nibble(w, 4) << 4 | nibble(w, 2) << 8 | nibble(w, 6) << 12) << (16 * j);
    }
    return v;
}

__global__ void q4_unpack_kernel(const uint4* in, int64_t M, int64_t K, int64_t k_tiles, int64_t n, uint8_t* codes)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t m = place_of(i, k_tiles).m, k = place_of(i, k_tiles).k;
    const uint4 w = in[i];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (m + 8 * u < M && k + 32 * h < K)
                *reinterpret_cast<uint32_t*>(codes + (((m + 8 * u) * K + k + 32 * h) >> 1)) =
                    h ? plain(w.z, w.w, u) : plain(w.x, w.y, u);
}

// Scales and zero points between the plain form [M][plain_groups] and the
// layout [strip][groups][row tile][8] of pairs (row g, row g + 8); a thread a pair.
__global__ void q4_pack_scales_kernel(const uint16_t* scales, const uint8_t* zeros, int64_t M, int64_t plain_groups,
                                      int64_t groups, int64_t n, uint32_t* out, uint8_t* zeros_out, int* bad)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t m = pair_of(i, groups).m, gr = pair_of(i, groups).k;
    uint32_t s = 0, z = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const bool in = m + 8 * u < M && gr < plain_groups;
        const int64_t at = (m + 8 * u) * plain_groups + gr;
        if (in) s |= (uint32_t)scales[at] << (16 * u);
        const uint32_t zero = in && zeros ? zeros[at] : 8u;
        if (zero > 15u) *bad = 1;
        z |= (zero & 15u) << (4 * u);
    }
    out[i] = s;
    if (zeros_out) zeros_out[i] = (uint8_t)z;
}

__global__ void q4_unpack_scales_kernel(const uint32_t* in, const uint8_t* zeros_in, int64_t M, int64_t plain_groups,
                                        int64_t groups, int64_t n, uint16_t* scales, uint8_t* zeros)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t m = pair_of(i, groups).m, gr = pair_of(i, groups).k;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (m + 8 * u >= M || gr >= plain_groups) continue;
        const int64_t at = (m + 8 * u) * plain_groups + gr;
        if (scales) scales[at] = (uint16_t)(in[i] >> (16 * u));
        if (zeros) zeros[at] = zeros_in ? (zeros_in[i] >> (4 * u)) & 15 : 8;
    }
}

template <class T>
__global__ void q4_decode_kernel(Q4View v, int64_t M, int64_t K, int32_t G, int64_t k_tiles, int64_t n, T* W)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t m = place_of(i, k_tiles).m, k = place_of(i, k_tiles).k;
    const uint4 w = v.codes[i];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (k + 32 * h >= K) continue;
        const int64_t at = (m / 128 * (k_tiles * 64 / G) + (k + 32 * h) / G) * 64 + m % 128 / 16 * 8 + m % 8;
        const uint32_t pair = v.scales[at], zero = v.zeros ? v.zeros[at] : 0x88u;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (m + 8 * u >= M) continue;
            const uint32_t c = h ? plain(w.z, w.w, u) : plain(w.x, w.y, u);
            const float s = half_of<T>(pair, u), z = (float)((zero >> (4 * u)) & 15u);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const T p[2] = {from_float<T>(s * ((float)nibble(c, 2 * e) - z)),
                                from_float<T>(s * ((float)nibble(c, 2 * e + 1) - z))};
                o[e] = *reinterpret_cast<const uint16_t*>(p) | (uint32_t)*reinterpret_cast<const uint16_t*>(p + 1) << 16;
            }
            *reinterpret_cast<uint4*>(W + (m + 8 * u) * K + k + 32 * h) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ------------------------------------------------------------------ handle

constexpr int BLOCK = 256;
// Blocks for n threads (the sizes that the checks let through fit a grid).
unsigned blocks_for(int64_t n, int per = BLOCK) { return (unsigned)((n + per - 1) / per); }

void free_q4(bsp_q4* h)
{
    if (!h) return;
    cudaFree(h->codes);
    cudaFree(h->scales);
    cudaFree(h->zeros);
    cudaFree(h->err);
    h->magic = 0;
    delete h;
}

bsp_status_t check_shape(bsp_dtype_t dtype, int64_t M, int64_t K, int32_t group)
{
    if (dtype != BSP_FP16 && dtype != BSP_BF16) return BSP_ERR_DTYPE;
    if (M < 1 || M > INT32_MAX || K < 1 || K > INT32_MAX || K % 8) return BSP_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return BSP_ERR_SHAPE;
    // a thread a lane of a tile, and a warp a group
    if ((M + 127) / 128 * ((K + 127) / 128) > (int64_t)1 << 24) return BSP_ERR_SHAPE;
    return BSP_OK;
}

// Temporary device memory of a call that synchronises.
struct Temp {
    void* p = nullptr;
    ~Temp() { cudaFree(p); }
    bool get(size_t n) { return bsp_malloc(&p, n ? n : 1) == cudaSuccess; }
};

// A handle from plain device arrays; synchronises s.
bsp_status_t build(bsp_dtype_t dtype, int64_t M, int64_t K, int32_t group, const uint8_t* codes, const void* scales,
                   const uint8_t* zeros, cudaStream_t s, bsp_q4** out)
{
    bsp_q4* h = new (std::nothrow) bsp_q4{};
    if (!h) return BSP_ERR_OOM;
    h->magic = BSP_Q4_MAGIC;
    h->dtype = dtype;
    h->M = M;
    h->K = K;
    h->group = group;
    h->strips = (M + 127) / 128;
    h->k_tiles = (K + 127) / 128 * 2;
    const int64_t lanes = h->strips * h->k_tiles * 256, pairs = h->strips * h->groups() * 64;
    bsp_status_t st = BSP_OK;
    int bad = 0;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess)
        st = BSP_ERR_CUDA;
    else if (bsp_malloc(&h->codes, lanes * 16) != cudaSuccess || bsp_malloc(&h->scales, pairs * 4) != cudaSuccess ||
             (zeros && bsp_malloc(&h->zeros, pairs) != cudaSuccess) || bsp_malloc(&h->err, sizeof(int)) != cudaSuccess)
        st = BSP_ERR_OOM;
    else {
        q4_pack_kernel<<<blocks_for(lanes), BLOCK, 0, s>>>(codes, M, K, h->k_tiles, lanes, h->codes);
        if (cudaMemsetAsync(h->err, 0, sizeof(int), s) != cudaSuccess) st = BSP_ERR_CUDA;
        q4_pack_scales_kernel<<<blocks_for(pairs), BLOCK, 0, s>>>((const uint16_t*)scales, zeros, M,
                                                                  (K + group - 1) / group, h->groups(), pairs,
                                                                  h->scales, h->zeros, h->err);
        if (cudaGetLastError() != cudaSuccess ||
            cudaMemcpyAsync(&bad, h->err, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
            cudaMemsetAsync(h->err, 0, sizeof(int), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
            st = BSP_ERR_CUDA;
    }
    if (st == BSP_OK && bad) st = BSP_ERR_INVALID_ARG;
    if (st != BSP_OK) {
        cudaStreamSynchronize(s);  // nothing may still write what is freed
        free_q4(h);
        return st;
    }
    *out = h;
    return BSP_OK;
}

// Checks of a product's activations and outputs, before any CUDA call.
bsp_status_t check_rows(const bsp_q4* h, const void* X, int64_t x_stride, int64_t N, const void* Y, int64_t y_stride)
{
    if (N < 0 || N > INT32_MAX || (N && (!X || !Y))) return BSP_ERR_INVALID_ARG;
    if (N > 1 && (x_stride < h->K || x_stride % 8 || y_stride < h->M)) return BSP_ERR_SHAPE;
    if (N > 1 && (x_stride > INT64_MAX / 4 / N || y_stride > INT64_MAX / 4 / N)) return BSP_ERR_SHAPE;
    if (!aligned(X, 16) || !aligned(Y, 16)) return BSP_ERR_ALIGN;
    if (bspo::meet({X, N, 2 * h->K, 2 * x_stride}, {Y, N, 2 * h->M, 2 * y_stride})) return BSP_ERR_INVALID_ARG;
    return BSP_OK;
}

Q4View view(const bsp_q4* h) { return {h->codes, h->scales, h->zeros}; }

bsp_status_t run(const bsp_q4* h, const bsp_q4* up, const void* X, int64_t x_stride, int64_t N, int act, void* Y,
                 int64_t y_stride, cudaStream_t s)
{
    if (N == 0) return BSP_OK;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    Problem p = {};
    p.w = view(h);
    p.up = up ? view(up) : p.w;
    p.gated = up != nullptr;
    p.act = act;
    p.dtype = h->dtype;
    p.M = h->M;
    p.K = h->K;
    p.strips = h->strips;
    p.k_tiles = h->k_tiles;
    p.group = h->group;
    p.x = X;
    p.x_stride = N > 1 ? x_stride : h->K;
    p.N = N;
    p.y = Y;
    p.y_stride = N > 1 ? y_stride : h->M;
    p.device = h->device;
    p.num_sms = h->num_sms;
    p.err = h->err;
    const bool f16 = p.dtype == BSP_FP16;
    if (N <= BSP_Q4_NARROW_N) return f16 ? bsp_run_q4_narrow_f16(p, s) : bsp_run_q4_narrow_bf16(p, s);
    return f16 ? bsp_run_q4_wide_f16(p, s) : bsp_run_q4_wide_bf16(p, s);
}

}  // namespace

extern "C" {

bsp_status_t bsp_q4_encode(const void* W, bsp_dtype_t dtype, int64_t M, int64_t K, int32_t group, int zeros,
                           bsp_stream_t stream, bsp_q4_t* out)
{
    if (!out) return BSP_ERR_INVALID_ARG;
    *out = nullptr;
    if (!W || (zeros != 0 && zeros != 1)) return BSP_ERR_INVALID_ARG;
    if (const bsp_status_t st = check_shape(dtype, M, K, group); st != BSP_OK) return st;
    if (!aligned(W, 16)) return BSP_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t groups = (K + group - 1) / group, items = M * groups;
    Temp codes, scales, zp;
    if (!codes.get(M * K / 2) || !scales.get(items * 2) || !zp.get(zeros ? items : 0)) return BSP_ERR_OOM;
    uint8_t* z = zeros ? (uint8_t*)zp.p : nullptr;
    const unsigned blocks = blocks_for(items, BLOCK / 32);
    if (dtype == BSP_FP16)
        q4_quantise_kernel<__half><<<blocks, BLOCK, 0, s>>>((const __half*)W, M, K, group, groups, (uint8_t*)codes.p,
                                                            (__half*)scales.p, z);
    else
        q4_quantise_kernel<__nv_bfloat16><<<blocks, BLOCK, 0, s>>>((const __nv_bfloat16*)W, M, K, group, groups,
                                                                   (uint8_t*)codes.p, (__nv_bfloat16*)scales.p, z);
    if (cudaGetLastError() != cudaSuccess) return BSP_ERR_CUDA;
    return build(dtype, M, K, group, (uint8_t*)codes.p, scales.p, z, s, out);
}

bsp_status_t bsp_q4_import(const uint8_t* codes, const void* scales, const uint8_t* zeros, bsp_dtype_t dtype,
                           int64_t M, int64_t K, int32_t group, bsp_stream_t stream, bsp_q4_t* out)
{
    if (!out) return BSP_ERR_INVALID_ARG;
    *out = nullptr;
    if (!codes || !scales) return BSP_ERR_INVALID_ARG;
    if (const bsp_status_t st = check_shape(dtype, M, K, group); st != BSP_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t items = M * ((K + group - 1) / group);
    Temp c, sc, z;
    if (!c.get(M * K / 2) || !sc.get(items * 2) || !z.get(zeros ? items : 0)) return BSP_ERR_OOM;
    if (cudaMemcpyAsync(c.p, codes, M * K / 2, cudaMemcpyDefault, s) != cudaSuccess ||
        cudaMemcpyAsync(sc.p, scales, items * 2, cudaMemcpyDefault, s) != cudaSuccess ||
        (zeros && cudaMemcpyAsync(z.p, zeros, items, cudaMemcpyDefault, s) != cudaSuccess)) {
        cudaStreamSynchronize(s);
        return BSP_ERR_CUDA;
    }
    return build(dtype, M, K, group, (uint8_t*)c.p, sc.p, zeros ? (uint8_t*)z.p : nullptr, s, out);
}

bsp_status_t bsp_q4_export(bsp_q4_t h, uint8_t* codes, void* scales, uint8_t* zeros, bsp_stream_t stream)
{
    if (!valid(h)) return BSP_ERR_INVALID_ARG;
    if (!aligned(codes, 4) || !aligned(scales, 2)) return BSP_ERR_ALIGN;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t lanes = h->strips * h->k_tiles * 256, pairs = h->strips * h->groups() * 64;
    if (codes) q4_unpack_kernel<<<blocks_for(lanes), BLOCK, 0, s>>>(h->codes, h->M, h->K, h->k_tiles, lanes, codes);
    if (scales || zeros)
        q4_unpack_scales_kernel<<<blocks_for(pairs), BLOCK, 0, s>>>(h->scales, h->zeros, h->M,
                                                                    (h->K + h->group - 1) / h->group, h->groups(),
                                                                    pairs, (uint16_t*)scales, zeros);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

bsp_status_t bsp_q4_decode(bsp_q4_t h, void* W, bsp_stream_t stream)
{
    if (!valid(h) || !W) return BSP_ERR_INVALID_ARG;
    if (!aligned(W, 16)) return BSP_ERR_ALIGN;
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t lanes = h->strips * h->k_tiles * 256;
    if (h->dtype == BSP_FP16)
        q4_decode_kernel<<<blocks_for(lanes), BLOCK, 0, s>>>(view(h), h->M, h->K, h->group, h->k_tiles, lanes, (__half*)W);
    else
        q4_decode_kernel<<<blocks_for(lanes), BLOCK, 0, s>>>(view(h), h->M, h->K, h->group, h->k_tiles, lanes,
                                                             (__nv_bfloat16*)W);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

bsp_status_t bsp_q4_info(bsp_q4_t h, bsp_q4_info_t* out)
{
    if (!valid(h) || !out) return BSP_ERR_INVALID_ARG;
    *out = {h->M, h->K, (int32_t)h->dtype, h->group, h->zeros ? 1 : 0, h->device, (h->K + h->group - 1) / h->group};
    return BSP_OK;
}

bsp_status_t bsp_q4_storage_bytes(bsp_q4_t h, uint64_t* bytes)
{
    if (!valid(h) || !bytes) return BSP_ERR_INVALID_ARG;
    const uint64_t n = (uint64_t)h->M * (uint64_t)((h->K + h->group - 1) / h->group);
    *bytes = ((uint64_t)h->M * (uint64_t)h->K + 1) / 2 + 2 * n + (h->zeros ? (n + 1) / 2 : 0);
    return BSP_OK;
}

bsp_status_t bsp_q4_check(bsp_q4_t h, bsp_stream_t stream)
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

bsp_status_t bsp_q4_destroy(bsp_q4_t h)
{
    if (!valid(h)) return BSP_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    cudaDeviceSynchronize();
    free_q4(h);
    return BSP_OK;
}

bsp_status_t bsp_q4_mm(bsp_q4_t h, const void* X, int64_t x_stride, int64_t N, void* Y, int64_t y_stride,
                       bsp_stream_t stream)
{
    if (!valid(h)) return BSP_ERR_INVALID_ARG;
    if (const bsp_status_t st = check_rows(h, X, x_stride, N, Y, y_stride); st != BSP_OK) return st;
    return run(h, nullptr, X, x_stride, N, 0, Y, y_stride, (cudaStream_t)stream);
}

bsp_status_t bsp_q4_gated(bsp_q4_t gate, bsp_q4_t up, const void* X, int64_t x_stride, int64_t N, bsp_act_t act,
                          void* Y, int64_t y_stride, bsp_stream_t stream)
{
    if (!valid(gate) || !valid(up) || act < BSP_ACT_SILU || act > BSP_ACT_RELU) return BSP_ERR_INVALID_ARG;
    if (gate->dtype != up->dtype) return BSP_ERR_DTYPE;
    if (gate->M != up->M || gate->K != up->K || gate->group != up->group) return BSP_ERR_SHAPE;
    if (gate->device != up->device) return BSP_ERR_INVALID_ARG;
    if (const bsp_status_t st = check_rows(gate, X, x_stride, N, Y, y_stride); st != BSP_OK) return st;
    return run(gate, up, X, x_stride, N, act, Y, y_stride, (cudaStream_t)stream);
}

}  // extern "C"
