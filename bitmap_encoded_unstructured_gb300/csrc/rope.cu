// Rotary positions with one or several axes: query and key rows turned by
// their positions, in one launch.
//
// A pair's angle is positions[axis] * freq.  Far positions lose an angle held
// in fp32 (at 10^6 its last bit is 0.06 radians), so the handle keeps each
// frequency in turns as a 64-bit fraction, F = freq / (2 pi) 2^64 mod 2^64 to
// the nearest: position * F in 64-bit integers drops whole turns exactly, and
// read as signed it is the angle in 2^-64 turns, rounded once to fp32 (so
// that a small angle keeps its relative accuracy).  Error: position 2^-65
// turns, and the one rounding.
//
// A block makes the cosines and sines of its rows once, in shared memory,
// and then passes over the heads: a thread takes VEC pairs (two 16-byte
// pieces at VEC = 8, of 8 and 8 values half a rotation apart, or of 16
// neighbours).  8101 rows of 64 + 8 heads of 128 with three axes take 51 to 55 us
// (5.4 TB/s, 0.80 of a copy, 81% of the warps resident and waiting for
// memory); one row, or 256 of 32 + 4 heads, are bound by the launch.
#include "bsp_overlap.h"
#include "bsp_q4.cuh"

#include <algorithm>
#include <cmath>
#include <new>

#define BSP_ROPE_MAGIC 0xB5B10709u

struct bsp_rope {
    uint32_t magic;
    int device, num_sms;
    int32_t dim, rot, axes, interleaved;
    float scale;
    uint64_t* turns;  // device [rot / 2]
    uint8_t* axis;    // device [rot / 2]
};

namespace {

using bspq4::from_float;
using bspq4::to_float;

constexpr int MOST_ROWS = 8;  // of a block
constexpr int THREADS = 256;

struct Rows {
    const char* in;
    char* out;
    int64_t in_row, in_head, out_row, out_head;  // bytes
    int32_t heads;
    bool moves;  // the output is not the input
    bool clear;  // rows that are not there become zeros
};

struct RopeArgs {
    Rows x[2];
    const int32_t* positions;
    int64_t axis_stride, rows;
    const uint64_t* turns;
    const uint8_t* axis;
    int32_t dim, half, axes, block_rows;
    float scale, sign;
};

template <int BYTES>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };

template <class T, int N>
struct __align__(N * sizeof(T)) Pack {
    T v[N];
};

template <class T, int N>
__device__ __forceinline__ Pack<T, N> load(const char* p)
{
    using W = typename Word<N * sizeof(T)>::type;
    const W w = *reinterpret_cast<const W*>(p);
    return *reinterpret_cast<const Pack<T, N>*>(&w);
}
template <class T, int N>
__device__ __forceinline__ void store(char* p, const Pack<T, N>& x)
{
    using W = typename Word<N * sizeof(T)>::type;
    *reinterpret_cast<W*>(p) = *reinterpret_cast<const W*>(&x);
}

template <class T, int N>
__device__ __forceinline__ void clear(char* p)
{
    using W = typename Word<N * sizeof(T)>::type;
    *reinterpret_cast<W*>(p) = W{};
}

// threadIdx.x: the piece of a head (VEC pairs, or behind them the tail's
// values); threadIdx.y: heads of the block's rows in turn.
template <class T, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_kernel(const RopeArgs a)
{
    extern __shared__ __align__(16) float4 table[];  // [row][VEC / 2][pieces]: two (cos, sin) each
    __shared__ bool there[MOST_ROWS];
    const int pieces = a.half / VEC, tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    const int64_t row0 = (int64_t)blockIdx.x * a.block_rows;
    const int rows = (int)min((int64_t)a.block_rows, a.rows - row0);
    bspq4::launch_dependents();
    bspq4::wait_prior_grids();
    if (tid < rows) {
        bool ok = true;
        for (int x = 0; x < a.axes; ++x) ok = ok && a.positions[x * a.axis_stride + row0 + tid] >= 0;
        there[tid] = ok;
    }
    for (int i = tid; i < rows * a.half; i += threads) {
        const int r = i / a.half, p = i - r * a.half;
        const uint32_t pos = (uint32_t)a.positions[(a.axes > 1 ? a.axis[p] : 0) * a.axis_stride + row0 + r];
        const int64_t turn = (int64_t)((uint64_t)pos * a.turns[p]);
        float s, c;
        sincospif((float)turn * 0x1p-63f, &s, &c);
        reinterpret_cast<float2*>(table)[((r * (VEC / 2) + p % VEC / 2) * pieces + p / VEC) * 2 + (p & 1)] =
            make_float2(c * a.scale, s * a.scale * a.sign);
    }
    __syncthreads();
    const int all = a.x[0].heads + a.x[1].heads;
    // this block's heads of each row
    const int h0 = (int)((int64_t)all * blockIdx.y / gridDim.y), heads = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y) - h0;
    const int piece = threadIdx.x;
    int r = 0, h = threadIdx.y;
    for (;; h += blockDim.y) {
        while (h >= heads && r < rows) {
            h -= heads;
            ++r;
        }
        if (r >= rows) return;
        const bool key = h0 + h >= a.x[0].heads;
        const Rows& x = a.x[key];
        if (!there[r] && !x.clear) continue;
        const int hd = h0 + h - (key ? a.x[0].heads : 0);
        const char* in = x.in + (row0 + r) * x.in_row + hd * x.in_head;
        char* out = x.out + (row0 + r) * x.out_row + hd * x.out_head;
        if (piece >= pieces) {  // the values that do not turn
            const int64_t at = (2 * a.half + (piece - pieces) * 8) * (int64_t)sizeof(T);
            if (!there[r]) clear<T, 8>(out + at);
            else if (x.moves) store<T, 8>(out + at, load<T, 8>(in + at));
            continue;
        }
        const int64_t at0 = (INTERLEAVED ? 2 : 1) * piece * VEC * (int64_t)sizeof(T);
        const int64_t at1 = at0 + (INTERLEAVED ? VEC : a.half) * (int64_t)sizeof(T);
        if (!there[r]) {
            clear<T, VEC>(out + at0);
            clear<T, VEC>(out + at1);
            continue;
        }
        Pack<T, VEC> u = load<T, VEC>(in + at0), v = load<T, VEC>(in + at1);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float4 t = table[(r * (VEC / 2) + i) * pieces + piece];
            auto turn = [](T& x, T& y, float c, float s) {
                const float p = to_float(x), q = to_float(y);
                x = from_float<T>(fmaf(p, c, -(q * s)));
                y = from_float<T>(fmaf(q, c, p * s));
            };
            if (INTERLEAVED) {
                Pack<T, VEC>& w = i < VEC / 4 ? u : v;
                const int e = 4 * i % VEC;
                turn(w.v[e], w.v[e + 1], t.x, t.y);
                turn(w.v[e + 2], w.v[e + 3], t.z, t.w);
            } else {
                turn(u.v[2 * i], v.v[2 * i], t.x, t.y);
                turn(u.v[2 * i + 1], v.v[2 * i + 1], t.z, t.w);
            }
        }
        store(out + at0, u);
        store(out + at1, v);
    }
}

bool valid(const bsp_rope* h) { return h != nullptr && h->magic == BSP_ROPE_MAGIC; }
bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

void free_rope(bsp_rope* h)
{
    if (!h) return;
    cudaFree(h->turns);
    cudaFree(h->axis);
    h->magic = 0;
    delete h;
}

// freq / (2 pi) 2^64 mod 2^64, to the nearest: the quotient as an unevaluated
// sum of two doubles (1 / (2 pi) has two terms), whose whole turns drop out.
uint64_t turns_of(double freq)
{
    if (freq < 0) return 0 - turns_of(-freq);
    const double inv = 0x1.45f306dc9c883p-3, inv_rest = -0x1.6b01ec5417056p-57;
    const double t = freq * inv, rest = std::fma(freq, inv, -t) + freq * inv_rest;
    const double part = std::ldexp(t - std::floor(t), 64), whole = std::floor(part);  // exact
    return (uint64_t)whole + (uint64_t)std::llrint(part - whole + std::ldexp(rest, 64));
}

// A row tensor's memory as strided pieces: by rows where heads lie inside
// them, by heads where rows do, else as one.
bspo::Rows extent(const void* at, int64_t rows, int64_t heads, int64_t dim, int64_t row, int64_t head)
{
    const int64_t by_row = (heads - 1) * (heads > 1 ? head : 0) + dim, by_head = (rows - 1) * (rows > 1 ? row : 0) + dim;
    if (rows < 2 || row >= by_row) return {at, rows, 2 * by_row, 2 * row};
    if (heads < 2 || head >= by_head) return {at, heads, 2 * by_head, 2 * head};
    return {at, 1, 2 * (by_row + (rows - 1) * row), 0};
}

bsp_status_t check_rows(const bsp_rope* h, const bsp_rope_rows_t& x, int64_t rows)
{
    if (x.heads < 0) return BSP_ERR_SHAPE;
    if (!x.heads || !rows) return BSP_OK;
    if (!x.in || !x.out) return BSP_ERR_INVALID_ARG;
    const int64_t most = INT64_MAX / 8;
    if (rows > 1 && (x.in_row < 0 || x.in_row % 8 || x.out_row < h->dim || x.out_row % 8 || x.in_row > most / rows ||
                     x.out_row > most / rows))
        return BSP_ERR_SHAPE;
    if (x.heads > 1 && (x.in_head < 0 || x.in_head % 8 || x.out_head < h->dim || x.out_head % 8 ||
                        x.in_head > most / x.heads || x.out_head > most / x.heads))
        return BSP_ERR_SHAPE;
    if (rows > 1 && x.heads > 1 && x.out_row < (x.heads - 1) * x.out_head + h->dim &&
        x.out_head < (rows - 1) * x.out_row + h->dim)
        return BSP_ERR_SHAPE;
    if (!aligned(x.in, 16) || !aligned(x.out, 16)) return BSP_ERR_ALIGN;
    return BSP_OK;
}

bool same(const bsp_rope_rows_t& x, int64_t rows)
{
    return x.in == x.out && (rows < 2 || x.in_row == x.out_row) && (x.heads < 2 || x.in_head == x.out_head);
}

template <class T>
bsp_status_t launch(const bsp_rope* h, const RopeArgs& a0, cudaStream_t s)
{
    RopeArgs a = a0;
    const int vec = a.half % 8 == 0 ? 8 : 4, pieces = a.half / vec + (a.dim - 2 * a.half) / 8;
    const int per = std::max(1, THREADS / pieces), heads = a.x[0].heads + a.x[1].heads;
    // rows share a block's cosines where there are eight blocks an SM without
    // more; heads are split where there are not
    const int64_t want = 8 * (int64_t)h->num_sms;
    a.block_rows = (int32_t)std::min<int64_t>(MOST_ROWS, std::max<int64_t>(1, a.rows / want));
    const int64_t blocks = (a.rows + a.block_rows - 1) / a.block_rows;
    const int64_t split = std::min<int64_t>((heads + per - 1) / per, std::max<int64_t>(1, want / blocks));
    if (blocks > INT32_MAX || split > 65535) return BSP_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)split);
    cfg.blockDim = dim3((unsigned)pieces, (unsigned)per);
    cfg.dynamicSmemBytes = (size_t)a.block_rows * a.half * 8;
    cfg.stream = s;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    auto k = h->interleaved ? (vec == 8 ? rope_kernel<T, 8, true> : rope_kernel<T, 4, true>)
                            : (vec == 8 ? rope_kernel<T, 8, false> : rope_kernel<T, 4, false>);
    return cudaLaunchKernelEx(&cfg, k, a) == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

}  // namespace

extern "C" {

bsp_status_t bsp_rope_create(const bsp_rope_desc_t* d, bsp_stream_t stream, bsp_rope_t* out)
{
    if (!out) return BSP_ERR_INVALID_ARG;
    *out = nullptr;
    if (!d || !d->freq) return BSP_ERR_INVALID_ARG;
    if (d->dim < 8 || d->dim > 1024 || d->dim % 8 || d->rot < 8 || d->rot > d->dim || d->rot % 8 || d->axes < 1 ||
        d->axes > 8)
        return BSP_ERR_SHAPE;
    if ((d->interleaved != 0 && d->interleaved != 1) || !std::isfinite(d->scale)) return BSP_ERR_INVALID_ARG;
    const int half = d->rot / 2;
    uint64_t turns[512];
    uint8_t axis[512];
    for (int i = 0; i < half; ++i) {
        if (!(std::fabs(d->freq[i]) <= 65536.0)) return BSP_ERR_INVALID_ARG;
        turns[i] = turns_of(d->freq[i]);
        axis[i] = d->axis ? d->axis[i] : 0;
        if (axis[i] >= d->axes) return BSP_ERR_INVALID_ARG;
    }
    bsp_rope* h = new (std::nothrow) bsp_rope{};
    if (!h) return BSP_ERR_OOM;
    h->magic = BSP_ROPE_MAGIC;
    h->dim = d->dim;
    h->rot = d->rot;
    h->axes = d->axes;
    h->interleaved = d->interleaved;
    h->scale = d->scale;
    cudaStream_t s = (cudaStream_t)stream;
    bsp_status_t st = BSP_OK;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess)
        st = BSP_ERR_CUDA;
    else if (bsp_malloc(&h->turns, half * sizeof(uint64_t)) != cudaSuccess || bsp_malloc(&h->axis, half) != cudaSuccess)
        st = BSP_ERR_OOM;
    else if (cudaMemcpyAsync(h->turns, turns, half * sizeof(uint64_t), cudaMemcpyHostToDevice, s) != cudaSuccess ||
             cudaMemcpyAsync(h->axis, axis, half, cudaMemcpyHostToDevice, s) != cudaSuccess ||
             cudaStreamSynchronize(s) != cudaSuccess)
        st = BSP_ERR_CUDA;
    if (st != BSP_OK) {
        free_rope(h);
        return st;
    }
    *out = h;
    return BSP_OK;
}

bsp_status_t bsp_rope_destroy(bsp_rope_t h)
{
    if (!valid(h)) return BSP_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    cudaDeviceSynchronize();
    free_rope(h);
    return BSP_OK;
}

bsp_status_t bsp_rope_apply(bsp_rope_t h, const bsp_rope_rows_t* q, const bsp_rope_rows_t* k, bsp_dtype_t dtype,
                            int64_t rows, const int32_t* positions, int64_t axis_stride, int inverse,
                            bsp_stream_t stream)
{
    if (!valid(h) || (inverse != 0 && inverse != 1)) return BSP_ERR_INVALID_ARG;
    if (dtype != BSP_FP16 && dtype != BSP_BF16) return BSP_ERR_DTYPE;
    if (rows < 0 || rows > INT32_MAX || (rows && !positions)) return BSP_ERR_INVALID_ARG;
    if (h->axes > 1 && (axis_stride < rows || axis_stride > INT64_MAX / 64)) return BSP_ERR_SHAPE;
    const bsp_rope_rows_t none = {};
    const bsp_rope_rows_t x[2] = {q ? *q : none, k ? *k : none};
    for (int i = 0; i < 2; ++i)
        if (const bsp_status_t st = check_rows(h, x[i], rows); st != BSP_OK) return st;
    if (!aligned(positions, 4)) return BSP_ERR_ALIGN;
    if (!rows || (int64_t)x[0].heads + x[1].heads == 0) return BSP_OK;
    if ((int64_t)x[0].heads + x[1].heads > INT32_MAX) return BSP_ERR_SHAPE;
    // what is written: its own input element for element, or apart from it;
    // apart from everything else
    for (int i = 0; i < 2; ++i) {
        if (!x[i].heads) continue;
        const bspo::Rows w = extent(x[i].out, rows, x[i].heads, h->dim, x[i].out_row, x[i].out_head);
        if (bspo::meet(w, {positions, h->axes, 4 * rows, 4 * axis_stride})) return BSP_ERR_INVALID_ARG;
        for (int j = 0; j < 2; ++j) {
            if (!x[j].heads) continue;
            if (!(i == j && same(x[i], rows)) &&
                bspo::meet(w, extent(x[j].in, rows, x[j].heads, h->dim, x[j].in_row, x[j].in_head)))
                return BSP_ERR_INVALID_ARG;
            if (i < j && bspo::meet(w, extent(x[j].out, rows, x[j].heads, h->dim, x[j].out_row, x[j].out_head)))
                return BSP_ERR_INVALID_ARG;
        }
    }
    DeviceGuard g(h->device);
    if (!g.ok) return BSP_ERR_CUDA;
    RopeArgs a = {};
    for (int i = 0; i < 2; ++i)
        a.x[i] = {(const char*)x[i].in, (char*)x[i].out,         2 * x[i].in_row, 2 * x[i].in_head, 2 * x[i].out_row,
                  2 * x[i].out_head,    x[i].heads,              !same(x[i], rows),  x[i].clear == 1};
    a.positions = positions;
    a.axis_stride = h->axes > 1 ? axis_stride : 0;
    a.rows = rows;
    a.turns = h->turns;
    a.axis = h->axis;
    a.dim = h->dim;
    a.half = h->rot / 2;
    a.axes = h->axes;
    a.scale = h->scale;
    a.sign = inverse ? -1.f : 1.f;
    return dtype == BSP_FP16 ? launch<__half>(h, a, (cudaStream_t)stream) : launch<__nv_bfloat16>(h, a, (cudaStream_t)stream);
}

}  // extern "C"
