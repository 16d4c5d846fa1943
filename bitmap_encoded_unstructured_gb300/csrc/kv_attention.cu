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
// drafts): bound by the bytes of the codes.  The CTAs share the cached rows
// of all requests evenly ("units" of UNIT rows of one KV head, in order of
// request, head and row group), so that neither ragged lengths nor few
// requests leave SMs idle; a segment (request, head, row group) cut between
// CTAs is joined by the last of them to arrive, in order.
//
// Inside a CTA each warp streams 32 rows of every unit through a ring of
// its own (TMA boxes of the paged codes, no block-wide barrier in the loop)
// and works on them alone:
//   S^T[row][query] = codes_K . q     mma m16n8k16, A = codes as exact fp16
//   O^T[dim][query] += codes_V^T . W  W = p * V scale
// Codes become fp16 by a byte permute under the exponent of 1024 and one
// subtraction (1024 + 128 + c - 1152, exact).  The dims a thread multiplies
// are chosen so that its operands are whole 16-byte chunks: the k index of a
// product may be permuted freely as long as both sides agree.
constexpr int DEC_WARPS = 4;
constexpr int SUB = 32;                  // rows of a unit that one warp takes
constexpr int UNIT = DEC_WARPS * SUB;
constexpr int PART_FLOATS = 4352;        // of one partial result: queries x (dims + 3), at most

template <int DP, int NT>
struct DecCfg {
    static constexpr int BOX = DP < 128 ? DP : 128;    // bytes of a smem row
    static constexpr int REGIONS = DP / BOX;
    static constexpr int HALF = SUB * DP;              // K (or V) codes of a stage
    static constexpr int STAGE = 2 * HALF;
    static constexpr int STAGES = DP == 64 ? 4 : 3;
    static constexpr int RING = DEC_WARPS * STAGES * STAGE;
    static constexpr int Q = 8 * NT;                   // query rows of a segment
    static constexpr int OPAD = DP + 4;                // floats of a row of the joining buffer
    static constexpr int OFF_STAT = RING;              // m, l, mw of each warp
    static constexpr int OFF_BAR = OFF_STAT + DEC_WARPS * Q * 3 * 4;
    static constexpr int SMEM = OFF_BAR + DEC_WARPS * STAGES * 8 + 64 + 1024;
    static_assert(DEC_WARPS * Q * OPAD * 4 <= RING, "joining buffer in the idle ring");
    static_assert(Q * (DP + 3) <= PART_FLOATS, "partial result");
};

struct DecodeArgs {
    AttnArgs a;
    float* parts;
    int* arrivals;
    int* err;
    uint32_t spin_cap;
    int32_t most_rows;  // requests with more query rows than this (per KV head) are not this kernel's
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
// (lo rounded down to whole sub-tiles), in units; row groups of Q queries.
struct Share {
    Request r;
    int seen, lo, units, groups;  // first cached row that a query sees, and the sub-tile it starts in
};

template <int Q>
__device__ __forceinline__ Share share_of(const DecodeArgs& d, int b)
{
    const AttnArgs& a = d.a;
    Share s;
    s.r = request_of(a.s, a.c.page_shift, b);
    const int64_t rows = (int64_t)s.r.n * a.group;
    if (rows > d.most_rows) s.r.n = 0;
    const int first = s.r.len - s.r.n;
    s.seen = a.window ? max(0, first - a.window + 1) : 0;
    s.lo = s.seen & ~(SUB - 1);
    s.groups = s.r.n ? (int)((rows + Q - 1) / Q) : 0;
    s.units = max(1, (s.r.len - s.lo + UNIT - 1) / UNIT);  // at least one: it writes the zeros of rows that see nothing
    return s;
}

template <class T, int DP, int NT>
__global__ void __launch_bounds__(DEC_WARPS * 32, 2)
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
    int* note = reinterpret_cast<int*>(smem + C::OFF_BAR + DEC_WARPS * C::STAGES * 8);
    uint8_t* ring = smem + warp * C::STAGES * C::STAGE;

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

    // this CTA's range of units: each thread sums a run of requests, and the
    // one whose run holds the first unit says where it is
    __shared__ int64_t scan[DEC_WARPS];
    const int per = (B + DEC_WARPS * 32 - 1) / (DEC_WARPS * 32);
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) {
        const Share s = share_of<Q>(d, b);
        sum += (int64_t)s.units * s.groups * H;
    }
    int64_t upto = sum;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int64_t o = __shfl_up_sync(FULL, upto, i);
        if (lane >= i) upto += o;
    }
    if (lane == 31) scan[warp] = upto;
    if (lane < C::STAGES) bspx::mbar_init(full + lane, 1);
    bspx::fence_mbar_init();
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < DEC_WARPS; ++w) {
        if (w < warp) upto += scan[w];
        total += scan[w];
    }
    const int64_t P = min((int64_t)gridDim.x, total);  // CTAs that have work
    if ((int64_t)blockIdx.x >= P) return;
    const int64_t u0 = total * blockIdx.x / P, u1 = total * (blockIdx.x + 1) / P;
    if (upto - sum <= u0 && u0 < upto) {
        int64_t at = upto - sum;
        for (int b = b0; b < b1; ++b) {
            const Share s = share_of<Q>(d, b);
            const int64_t n = (int64_t)s.units * s.groups * H;
            if (u0 < at + n) {
                note[0] = b;
                *reinterpret_cast<int64_t*>(note + 2) = u0 - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    int b = note[0];
    int64_t off = *reinterpret_cast<int64_t*>(note + 2);  // unit within the request
    uint32_t stage = 0, phase = 0;
    uint32_t fill = 0;                                    // stage of the next load
    bool failed = false;

    for (int64_t u = u0; u < u1;) {
        Share s = share_of<Q>(d, b);
        while (off >= (int64_t)s.units * s.groups * H) {  // next request with work
            off -= (int64_t)s.units * s.groups * H;
            s = share_of<Q>(d, ++b);
        }
        const int64_t seg = off / s.units;
        const int t0 = (int)(off - seg * s.units), n_units = (int)min((int64_t)(s.units - t0), u1 - u);
        const int h = (int)(seg / s.groups), rg = (int)(seg - (int64_t)h * s.groups);
        const int first = s.r.len - s.r.n, rows = s.r.n * a.group;
        const int32_t* table = a.s.table + (int64_t)b * a.s.table_stride;
        const int tok0 = s.lo + t0 * UNIT + warp * SUB;  // this warp's first row; the next ones are UNIT apart

        // queries: a thread's chunks of its row, the scale of its columns' logits
        uint32_t qf[NT][CH][8];
        float qs[NT][2];
        int pos[NT][2];  // positions of the columns' queries
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = rg * Q + nt * 8 + g;
            float top = 0.f, x[CH][16];
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int ch = DP == 64 ? c : 8 * (j >> 1) + 2 * c + (j & 1);
                if (r < rows && ch * 16 < a.c.dim) {
                    const T* q = (const T*)a.q + (int64_t)(s.r.r0 + r / a.group) * a.q_row +
                                 (int64_t)(h * a.group + r % a.group) * a.q_head + ch * 16;
                    const uint4 v0 = *reinterpret_cast<const uint4*>(q), v1 = *reinterpret_cast<const uint4*>(q + 8);
                    const T* e0 = reinterpret_cast<const T*>(&v0);
                    const T* e1 = reinterpret_cast<const T*>(&v1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[j][e] = to_float(e0[e]);
                        x[j][8 + e] = to_float(e1[e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[j][e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[j][e]));
            }
            // bfloat16 rows are brought into fp16's range by a power of two
            // (exact but for values 2^-24 below the row's largest)
            float unit = 1.f;
            if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
                const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
                unit = __uint_as_float(e << 23);
                const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
                for (int j = 0; j < CH; ++j)
#pragma unroll
                    for (int e2 = 0; e2 < 16; ++e2) x[j][e2] *= inv;
            }
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) qf[nt][j][e] = h2bits(__floats2half2_rn(x[j][2 * e], x[j][2 * e + 1]));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qs[nt][e] = __shfl_sync(FULL, unit, (2 * c + e) * 4) * (a.scale * 1.4426950408889634f);
                pos[nt][e] = first + (rg * Q + nt * 8 + 2 * c + e) / a.group;
            }
        }

        float acc[MT][NT][4];
        float m[NT][2], mw[NT][2], l[NT][2], lift[NT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = mw[nt][e] = NONE;
                l[nt][e] = 0.f;
                lift[nt][e] = LIFT;
            }

        // pages and scales of this warp's next 32 sub-tiles, one per lane
        // (two pages where a page holds 16 rows); -1: nothing to see there
        int pg[2], npg[2];
        float ks[2], vs[2];
        auto pages_from = [&](int k, int (&p)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = tok0 + (k + lane) * UNIT + 16 * i;
                p[i] = -1;
                if (k + lane < n_units && tok < s.r.len && ((tok >> sh) + 1) << sh > s.seen) {
                    const int v = table[tok >> sh];
                    if (v >= 0 && v < a.c.pages) p[i] = v;
                }
            }
        };
        auto issue = [&](int k, int p0, int p1) {  // loads of sub-tile k into the next free stage
            if (lane == 0) {
                uint8_t* st = ring + fill * C::STAGE;
                const bool two = sh == 4;
                const uint32_t bytes = two ? ((p0 >= 0) + (p1 >= 0)) * 32u * DP : (p0 >= 0 ? 64u * DP : 0u);
                if (bytes) bspx::mbar_arrive_expect_tx(full + fill, bytes);
                else bspx::mbar_arrive(full + fill);
                const int row = (tok0 + k * UNIT) & ((1 << sh) - 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int p = i ? p1 : p0;
                    if (p < 0 || (i && !two)) continue;
#pragma unroll
                    for (int rgn = 0; rgn < C::REGIONS; ++rgn) {
                        uint8_t* to = st + rgn * SUB * C::BOX + i * 16 * C::BOX;
                        tma_load_4d(to, &map_k, rgn * 128, two ? 0 : row, h, p, full + fill);
                        tma_load_4d(to + C::HALF, &map_v, rgn * 128, two ? 0 : row, h, p, full + fill);
                    }
                }
            }
            __syncwarp();
            if (++fill == C::STAGES) fill = 0;
        };
        pages_from(0, pg);
        pages_from(32, npg);
        auto scales = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ks[i] = vs[i] = 0.f;
                if (pg[i] >= 0) {
                    ks[i] = a.c.k_scale[(int64_t)pg[i] * a.c.scale_stride + h];
                    vs[i] = a.c.v_scale[(int64_t)pg[i] * a.c.scale_stride + h];
                }
            }
        };
        int issued = 0;
        auto issue_next = [&](int k) {  // k: the sub-tile being worked on
            const int w = issued - (k & ~31);
            const int p0 = __shfl_sync(FULL, w < 32 ? pg[0] : npg[0], w & 31);
            const int p1 = __shfl_sync(FULL, w < 32 ? pg[1] : npg[1], w & 31);
            issue(issued, p0, p1);
            ++issued;
        };
        while (issued < n_units && issued < C::STAGES) issue_next(0);
        scales();

        for (int k = 0; k < n_units; ++k) {
            if (k && (k & 31) == 0) {
                pg[0] = npg[0];
                pg[1] = npg[1];
                pages_from(k + 32, npg);
                scales();
            }
            const int tok = tok0 + k * UNIT;
            const int p0 = __shfl_sync(FULL, pg[0], k & 31), p1 = __shfl_sync(FULL, pg[1], k & 31);
            float kscale[2], vscale[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                kscale[i] = __shfl_sync(FULL, ks[i], k & 31);
                vscale[i] = __shfl_sync(FULL, vs[i], k & 31);
            }
            if (!bspx::mbar_wait_bounded(full + stage, phase, failed ? 1u : d.spin_cap)) failed = true;
            failed = __any_sync(FULL, failed);
            const uint8_t* kt = ring + stage * C::STAGE;
            const uint8_t* vt = kt + C::HALF;
            if (p0 >= 0 || p1 >= 0) {
                // S^T
                float sc[2][NT][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[i][nt][e] = 0.f;
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        const int ch = DP == 64 ? c : 2 * c + (j & 1);
                        const int r0 = 16 * i + g, r1 = r0 + 8;
                        const int sw0 = DP == 64 ? (r0 >> 1) & 3 : r0 & 7, sw1 = DP == 64 ? (r1 >> 1) & 3 : r1 & 7;
                        const uint8_t* reg = kt + (j >> 1) * SUB * C::BOX;
                        const uint4 w0 = *reinterpret_cast<const uint4*>(reg + r0 * C::BOX + ((ch ^ sw0) << 4));
                        const uint4 w1 = *reinterpret_cast<const uint4*>(reg + r1 * C::BOX + ((ch ^ sw1) << 4));
                        const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t y0 = x0[w] ^ 0x80808080u, y1 = x1[w] ^ 0x80808080u;
                            const uint32_t a0 = widen(y0, 0x4140), a2 = widen(y0, 0x4342);
                            const uint32_t a1 = widen(y1, 0x4140), a3 = widen(y1, 0x4342);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(sc[i][nt], a0, a1, a2, a3, qf[nt][j][2 * w], qf[nt][j][2 * w + 1]);
                        }
                    }
                }
                // logits (in powers of two), masked where a query does not see the row
                const bool edge = tok + SUB - 1 > first || (a.window && tok <= s.r.len - 1 - a.window) || p0 < 0 ||
                                  (sh == 4 && p1 < 0);
                float lv[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool there = sh == 4 ? (i ? p1 : p0) >= 0 : p0 >= 0;
                    lv[i] = vscale[i] != 0.f ? __log2f(fabsf(vscale[i])) : NONE;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = sc[i][nt][e] * (kscale[i] * qs[nt][e & 1]);
                            if (edge) {
                                const int j = tok + 16 * i + g + (e >> 1) * 8, p = pos[nt][e & 1];
                                if (!there || j > p || (a.window && j <= p - a.window)) x = -INFINITY;
                            }
                            sc[i][nt][e] = x;
                        }
                }
                // running maxima, allowed to lag
                bool lag = false;
                float hi[NT][2][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) hi[nt][e][i] = fmaxf(sc[i][nt][e], sc[i][nt][e + 2]);
                        lag |= fmaxf(hi[nt][e][0], hi[nt][e][1]) > m[nt][e] + LAZY;
                        lag |= fmaxf(hi[nt][e][0] + lv[0], hi[nt][e][1] + lv[1]) > mw[nt][e] + LAZY;
                    }
                if (__any_sync(FULL, lag)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float t = fmaxf(hi[nt][e][0], hi[nt][e][1]);
                            float tw = fmaxf(hi[nt][e][0] + lv[0], hi[nt][e][1] + lv[1]);
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) {
                                t = fmaxf(t, __shfl_xor_sync(FULL, t, x));
                                tw = fmaxf(tw, __shfl_xor_sync(FULL, tw, x));
                            }
                            t = fmaxf(t, m[nt][e]);
                            tw = fmaxf(tw, mw[nt][e]);
                            l[nt][e] *= ex2(m[nt][e] - t);
                            const float back = ex2(mw[nt][e] - tw);
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                acc[i][nt][e] *= back;
                                acc[i][nt][e + 2] *= back;
                            }
                            m[nt][e] = t;
                            mw[nt][e] = tw;
                            lift[nt][e] = ex2(fminf(t - tw, 120.f)) * LIFT;
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
                        for (int e = 0; e < 4; ++e) {
                            p[e] = ex2(sc[i][nt][e] - m[nt][e & 1]);
                            l[nt][e & 1] += p[e];
                            p[e] *= lift[nt][e & 1] * vscale[i];
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
                                    mma16816(acc[rgn * 8 + 2 * w + half][nt], a0, a1, a2, a3, wf[i][nt][0],
                                             wf[i][nt][1]);
                            }
                    }
                }
            }
            __syncwarp();  // the stage is read: it may be filled again
            if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            if (issued < n_units) issue_next(k);
        }

        // the warps' sums meet in shared memory (the ring is idle)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(FULL, l[nt][e], x);
                if (g == 0) {
                    float* st = stat + warp * 3 * Q + nt * 8 + 2 * c + e;
                    st[0] = m[nt][e];
                    st[Q] = l[nt][e];
                    st[2 * Q] = mw[nt][e];
                }
            }
        __syncthreads();
        float* join = reinterpret_cast<float*>(smem);  // [warp][Q][OPAD]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int qr = nt * 8 + 2 * c + e;
                float top = NONE;
#pragma unroll
                for (int w = 0; w < DEC_WARPS; ++w) top = fmaxf(top, stat[w * 3 * Q + 2 * Q + qr]);
                const float f = ex2(mw[nt][e] - top) * (1.f / LIFT);
                float* o = join + (warp * Q + qr) * C::OPAD;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int dim = DP == 64 ? g * 8 + 2 * i : (i >> 3) * 128 + g * 16 + 2 * (i & 7);
                    *reinterpret_cast<float2*>(o + dim) = make_float2(acc[i][nt][e] * f, acc[i][nt][e + 2] * f);
                }
            }
        __syncthreads();
        const int64_t seg_u0 = u - t0;                         // first unit of the segment, of all
        const int64_t c0 = ((seg_u0 + 1) * P - 1) / total, c1 = ((seg_u0 + s.units) * P - 1) / total;  // its CTAs
        const bool whole = c0 == c1;
        float* part = d.parts + (2 * (int64_t)blockIdx.x + (t0 ? 0 : 1)) * PART_FLOATS;  // begun earlier, or here
        for (int i = tid; i < Q * (DP / 4); i += DEC_WARPS * 32) {
            const int qr = i / (DP / 4), dim = i % (DP / 4) * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = NONE, lsum = 0.f, topw = NONE;
#pragma unroll
            for (int w = 0; w < DEC_WARPS; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(join + (w * Q + qr) * C::OPAD + dim);
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
                top = fmaxf(top, stat[w * 3 * Q + qr]);
                topw = fmaxf(topw, stat[w * 3 * Q + 2 * Q + qr]);
            }
#pragma unroll
            for (int w = 0; w < DEC_WARPS; ++w) lsum += stat[w * 3 * Q + Q + qr] * ex2(stat[w * 3 * Q + qr] - top);
            if (!whole) {
                *reinterpret_cast<float4*>(part + qr * DP + dim) = o;
                if (dim == 0) {
                    part[Q * DP + qr] = top;
                    part[Q * DP + Q + qr] = lsum;
                    part[Q * DP + 2 * Q + qr] = topw;
                }
                continue;
            }
            const int r = rg * Q + qr;
            if (r < rows) {
                const int64_t row = s.r.r0 + r / a.group, head = h * a.group + r % a.group;
                const float f = lsum > 0.f ? ex2(topw - top) / lsum : 0.f;
                if (dim < a.c.dim) {
                    alignas(8) T y[4] = {from_float<T>(o.x * f), from_float<T>(o.y * f), from_float<T>(o.z * f),
                                         from_float<T>(o.w * f)};
                    *reinterpret_cast<uint2*>((T*)a.out + row * a.o_row + head * a.o_head + dim) =
                        *reinterpret_cast<const uint2*>(y);
                }
                if (a.lse && dim == 0)
                    a.lse[row * a.heads + head] =
                        lsum > 0.f ? (top + __log2f(lsum)) * 0.6931471805599453f : -INFINITY;
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = atomicAdd(d.arrivals + c0, 1);
                note[1] = n == (int)(c1 - c0);
                if (note[1]) d.arrivals[c0] = 0;
            }
            __syncthreads();
            if (note[1]) {  // the last part is here: join them all, in order
                __threadfence();
                for (int i = tid; i < Q * (DP / 4); i += DEC_WARPS * 32) {
                    const int qr = i / (DP / 4), dim = i % (DP / 4) * 4;
                    const int r = rg * Q + qr;
                    if (r >= rows) continue;
                    float top = NONE, topw = NONE;
                    for (int64_t x = c0; x <= c1; ++x) {
                        const float* st = d.parts + (2 * x + (x == c0 ? 1 : 0)) * PART_FLOATS + Q * DP + qr;
                        top = fmaxf(top, __ldcg(st));
                        topw = fmaxf(topw, __ldcg(st + 2 * Q));
                    }
                    float lsum = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int64_t x = c0; x <= c1; ++x) {
                        const float* from = d.parts + (2 * x + (x == c0 ? 1 : 0)) * PART_FLOATS;
                        const float* st = from + Q * DP + qr;
                        lsum += __ldcg(st + Q) * ex2(__ldcg(st) - top);
                        const float f = ex2(__ldcg(st + 2 * Q) - topw);
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(from + qr * DP + dim));
                        o.x += y.x * f;
                        o.y += y.y * f;
                        o.z += y.z * f;
                        o.w += y.w * f;
                    }
                    const int64_t row = s.r.r0 + r / a.group, head = h * a.group + r % a.group;
                    const float f = lsum > 0.f ? ex2(topw - top) / lsum : 0.f;
                    if (dim < a.c.dim) {
                        alignas(8) T y[4] = {from_float<T>(o.x * f), from_float<T>(o.y * f), from_float<T>(o.z * f),
                                             from_float<T>(o.w * f)};
                        *reinterpret_cast<uint2*>((T*)a.out + row * a.o_row + head * a.o_head + dim) =
                            *reinterpret_cast<const uint2*>(y);
                    }
                    if (a.lse && dim == 0)
                        a.lse[row * a.heads + head] =
                            lsum > 0.f ? (top + __log2f(lsum)) * 0.6931471805599453f : -INFINITY;
                }
            }
        }
        // the joining buffer is the ring again: its next loads (async proxy)
        // come after these reads and writes
        bspx::fence_proxy_async_smem();
        __syncthreads();
        u += n_units;
        off += n_units;
    }
    if (failed && lane == 0) atomicExch(d.err, (int)BSP_ERR_TIMEOUT);
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

constexpr int DECODE_CTAS_PER_SM = 3;  // at most

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
    const int grid = h->num_sms * std::clamp(per_sm[dev], 1, DECODE_CTAS_PER_SM);
    kv_decode_kernel<T, DP, NT><<<grid, DEC_WARPS * 32, C::SMEM, s>>>(h->map_k, h->map_v, d);
    return cudaGetLastError() == cudaSuccess ? BSP_OK : BSP_ERR_CUDA;
}

template <class T>
bsp_status_t run_decode(const bsp_kv* h, const DecodeArgs& d, int nt, cudaStream_t s)
{
    if (d.a.c.dim <= 64)
        return nt == 1 ? launch_decode<T, 64, 1>(h, d, s) : nt == 2 ? launch_decode<T, 64, 2>(h, d, s)
                                                                   : launch_decode<T, 64, 4>(h, d, s);
    if (d.a.c.dim <= 128)
        return nt == 1 ? launch_decode<T, 128, 1>(h, d, s) : nt == 2 ? launch_decode<T, 128, 2>(h, d, s)
                                                                    : launch_decode<T, 128, 4>(h, d, s);
    return nt == 1 ? launch_decode<T, 256, 1>(h, d, s) : launch_decode<T, 256, 2>(h, d, s);
}

template <class T>
bsp_status_t run(const bsp_kv* h, const AttnArgs& a, int64_t max_new, cudaStream_t s)
{
    const int64_t most = max_new * a.group;
    // Query blocks of 8, 16 or 32 rows: the smallest that holds the largest
    // request.  Requests with more rows are the prompt kernel's, whose row
    // tiles have 128 rows and whose dims end at 128.
    const int few = a.c.dim > 128 ? INT32_MAX : 32;
    const int nt = most <= 8 ? 1 : most <= 16 ? 2 : 4;
    const DecodeArgs d = {a, h->parts, h->arrivals, h->err, bsp_spin_cap(), few};
    if (const bsp_status_t st = run_decode<T>(h, d, nt, s)) return st;
    if (most <= few || !a.s.batch) return BSP_OK;
    return bsp_run_kv_prompt(h, a, std::is_same<T, __half>::value ? BSP_FP16 : BSP_BF16, few, s);
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
    h->decode_ctas = h->num_sms * DECODE_CTAS_PER_SM;
    if (cudaMalloc(&h->parts, (size_t)2 * h->decode_ctas * PART_FLOATS * sizeof(float)) != cudaSuccess ||
        cudaMalloc(&h->arrivals, (size_t)h->decode_ctas * sizeof(int)) != cudaSuccess)
        return BSP_ERR_OOM;
    if (cudaMemsetAsync(h->arrivals, 0, (size_t)h->decode_ctas * sizeof(int), s) != cudaSuccess) return BSP_ERR_CUDA;
    return BSP_OK;
}

void attention_free(bsp_kv* h)
{
    cudaFree(h->parts);
    cudaFree(h->arrivals);
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
