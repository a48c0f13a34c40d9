// q8_quant.cu -- quantization of matrices to 8-bit blocks, in row order, in
// transposed order, or both from one read.
//
// Bounded by memory: an element is read once (2 or 4 bytes) and written once
// or twice (1 byte each), so a 128 x 128 tile lives in one CTA's registers:
// 256 threads, each eight consecutive rows by eight columns (bfloat16 stays
// packed in pairs: maxima take one instruction a pair, and half the registers
// let twice the tiles be in flight).  Row maxima meet in the 16 lanes that
// share a row, column maxima in shared memory.  Eight consecutive rows in a
// thread make eight consecutive bytes of the transposed tile, which is
// exchanged through 16 KB of shared memory and written as whole 128-byte rows.
#include "q8.cuh"

namespace dion {
namespace {

using namespace q8;

constexpr int kThreads = 256;
constexpr int kTile = 128;

struct QuantParams {
    Q8QuantArgs a;
    int tiles_c;
    bool wf32;
};

// The transposed tile: row c (a column of x) is 16 granules of 8 bytes;
// granule g (rows 8 g .. 8 g + 7 of x) sits at g ^ (c / 8 % 16), so the 16 lanes
// that write the same g for columns 8 l + i fall on 16 different granules.
__device__ __forceinline__ int t_granule(int c, int g) { return c * 16 + (g ^ ((c >> 3) & 15)); }

// A thread's 8 x 8 values, pairs (2 i, 2 i + 1) of a row together.
template <bool PACKED, bool NORM> struct Frag;
template <> struct Frag<true, false> {   // bfloat16 as stored
    uint32_t v[8][4];
    __device__ __forceinline__ float2 get(int j, int i) const { return unpack2(v[j][i]); }
    __device__ __forceinline__ void set(int j, int i, float2 f) { v[j][i] = pack2(f); }   // f holds bfloat16 values
    typedef uint32_t Max;                // largest magnitudes of a pair's two columns
    __device__ __forceinline__ static Max zero() { return 0u; }
    __device__ __forceinline__ void take(Max& m, int j, int i) const
    {
        const uint32_t a = v[j][i] & 0x7fff7fffu;
        const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&a));
        m = *reinterpret_cast<const uint32_t*>(&r);
    }
    __device__ __forceinline__ static uint2 bits(Max m) { return make_uint2(m << 16, m & 0xffff0000u); }
    __device__ __forceinline__ static Max of_bits(uint32_t a, uint32_t b) { return (a >> 16) | b; }
    __device__ __forceinline__ static Max max16(Max m)    // over lanes l and l + 16
    {
        const Max o = __shfl_xor_sync(0xffffffffu, m, 16);
        const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&o));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
};
struct PairMax {                         // of float32 values
    typedef float2 Max;
    __device__ __forceinline__ static Max zero() { return make_float2(0.f, 0.f); }
    __device__ __forceinline__ static void larger(Max& m, float2 v)
    {
        m.x = fmaxf(m.x, fabsf(v.x));
        m.y = fmaxf(m.y, fabsf(v.y));
    }
    __device__ __forceinline__ static uint2 bits(Max m) { return make_uint2(__float_as_uint(m.x), __float_as_uint(m.y)); }
    __device__ __forceinline__ static Max of_bits(uint32_t a, uint32_t b)
    {
        return make_float2(__uint_as_float(a), __uint_as_float(b));
    }
    __device__ __forceinline__ static Max max16(Max m)
    {
        return make_float2(fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, 16)), fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, 16)));
    }
};
template <bool NORM> struct Frag<false, NORM> : PairMax {
    float2 v[8][4];
    __device__ __forceinline__ float2 get(int j, int i) const { return v[j][i]; }
    __device__ __forceinline__ void set(int j, int i, float2 f) { v[j][i] = f; }
    __device__ __forceinline__ void take(Max& m, int j, int i) const { larger(m, v[j][i]); }
    __device__ __forceinline__ void norm(int j, float rs, const float2 (&w)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = mul2(mul2(v[j][i], make_float2(rs, rs)), w[i]);
    }
};
// bfloat16 as stored, times the row's and the columns' factors wherever it is
// read: two products each time cost less than the occupancy of 64 registers
// (again() keeps the compiler from holding on to the products).
template <> struct Frag<true, true> : PairMax {
    uint32_t v[8][4];
    float rs[8];
    float2 w[4];
    __device__ __forceinline__ float2 get(int j, int i) const
    {
        return mul2(mul2(unpack2(v[j][i]), make_float2(rs[j], rs[j])), w[i]);
    }
    // the value as read from memory; later only to make products NaN
    __device__ __forceinline__ void set(int j, int i, float2 f) { v[j][i] = pack2(f); }
    __device__ __forceinline__ void take(Max& m, int j, int i) const { larger(m, get(j, i)); }
    __device__ __forceinline__ void norm(int j, float r, const float2 (&f)[4])
    {
        rs[j] = r;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = f[i];
    }
    __device__ __forceinline__ void again()
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) asm volatile("" : "+r"(v[j][i]));
    }
};

// Maxima over the 16 lanes of a half-warp of eight values each: in three
// rounds a lane hands on half of the values it still holds (8 shuffles, where
// eight separate maxima take 32).  Returns that of value l / 2.
__device__ __forceinline__ uint32_t max16_of8(const uint32_t (&v)[8], int l)
{
    uint32_t a[4], b[2];
    const bool h8 = l & 8, h4 = l & 4, h2 = l & 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = max(h8 ? v[j + 4] : v[j], __shfl_xor_sync(0xffffffffu, h8 ? v[j] : v[j + 4], 8));
#pragma unroll
    for (int j = 0; j < 2; ++j) b[j] = max(h4 ? a[j + 2] : a[j], __shfl_xor_sync(0xffffffffu, h4 ? a[j] : a[j + 2], 4));
    uint32_t c = max(h2 ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, h2 ? b[0] : b[1], 2));
    return max(c, __shfl_xor_sync(0xffffffffu, c, 1));
}

// SHIFT: rows of x that do not start on 16-byte boundaries.
template <typename T, int FMT, bool ROWS, bool COLS, bool SQUARE, bool SHIFT, bool NORM>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : NORM ? 3 : ROWS && COLS ? 3 : 4) q8_quant_kernel(const QuantParams p)
{
    constexpr bool PACKED = sizeof(T) == 2;
    typedef Frag<PACKED, NORM> F;
    __shared__ uint2 tile[COLS ? kTile * 16 : 1];
    __shared__ typename F::Max colmax[(COLS || SQUARE) ? kThreads / 32 : 1][kTile / 2];
    __shared__ float colinv[kTile];
    const Q8QuantArgs& a = p.a;
    allow_next();
    wait_previous();
    const int tr = blockIdx.x / p.tiles_c, tc = blockIdx.x % p.tiles_c, b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
    const int g = warp * 2 + half;                    // row granule of this half-warp
    const int r0 = tr * kTile + 8 * g, c0 = tc * kTile;
    const T* x = reinterpret_cast<const T*>(a.x) + (long long)b * a.sx;

    F f;
    Raw8<T> u[8];
    if (r0 + 8 <= a.rows && c0 + kTile <= a.cols && !SHIFT) {
        const T* src = x + (long long)r0 * a.ldx + c0 + 8 * l;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < (int)(sizeof(T) / 2); ++i) u[j].u[i] = reinterpret_cast<const uint4*>(src + j * a.ldx)[i];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (r0 + j < a.rows) {
                u[j] = load_raw8<SHIFT>(x + (long long)(r0 + j) * a.ldx, c0, a.cols, l);
            } else {
#pragma unroll
                for (int i = 0; i < (int)(sizeof(T) / 2); ++i) u[j].u[i] = make_uint4(0, 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (PACKED) {
            f.v[j][0] = u[j].u[0].x;
            f.v[j][1] = u[j].u[0].y;
            f.v[j][2] = u[j].u[0].z;
            f.v[j][3] = u[j].u[0].w;
        } else {
            unpack8(u[j], f.v[j]);
        }
    }
    if constexpr (NORM) {
        float2 w[4];
        if (p.wf32) unpack8(load_raw8<true>(reinterpret_cast<const float*>(a.weight), c0, a.cols, l), w);
        else unpack8(load_raw8<true>(reinterpret_cast<const bf16*>(a.weight), c0, a.cols, l), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f.norm(j, r0 + j < a.rows ? a.rstd[r0 + j] : 0.f, w);
    }
    // largest magnitudes along this thread's rows and columns
    uint32_t rm[8], all = 0;
    typename F::Max cm[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) cm[i] = F::zero();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        typename F::Max m = F::zero();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.take(m, j, i);
            if (COLS && !SQUARE) f.take(cm[i], j, i);
        }
        const uint2 mb = F::bits(m);
        rm[j] = max(mb.x, mb.y);
        all = max(all, rm[j]);
    }
    if constexpr (PACKED && NORM) f.again();
    if (all >= kInfBits) {                            // rare: infinities become NaN; neither counts
        all = 0;
        uint32_t c8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c8[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            rm[j] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = f.get(j, i);
                const uint32_t u = finite_mag_bits(v.x), w = finite_mag_bits(v.y);
                rm[j] = max(rm[j], max(u, w));
                c8[2 * i] = max(c8[2 * i], u);
                c8[2 * i + 1] = max(c8[2 * i + 1], w);
                if constexpr (PACKED && NORM) {
                    const uint32_t nx = u == 0 && mag_bits(v.x) >= kInfBits ? 0x7fffu : 0u;
                    const uint32_t ny = w == 0 && mag_bits(v.y) >= kInfBits ? 0x7fff0000u : 0u;
                    f.v[j][i] |= nx | ny;            // the factor's NaN makes the product NaN
                } else {
                    f.set(j, i, make_float2(inf_to_nan(v.x), inf_to_nan(v.y)));
                }
            }
            all = max(all, rm[j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) cm[i] = F::of_bits(c8[2 * i], c8[2 * i + 1]);
    }
    if constexpr (PACKED && NORM) f.again();
    float sq_inv = 1.f;
    if (SQUARE) {
        uint32_t* wm = reinterpret_cast<uint32_t*>(colmax);
        all = max16(all);
        all = max(all, __shfl_xor_sync(0xffffffffu, all, 16));
        if (lane == 0) wm[warp] = all;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) all = max(all, wm[w]);
        const uint32_t byte = scale_byte<FMT>(all);
        sq_inv = inv_scale(byte);
        if (threadIdx.x == 0) {
            if (ROWS) a.s[(long long)b * a.ss + (long long)tr * a.lds + tc] = (uint8_t)byte;
            if (COLS) a.st[(long long)b * a.sst + (long long)tc * a.ldst + tr] = (uint8_t)byte;
        }
    } else if (COLS) {
        // column maxima: both halves of the warp, then the eight warps; pair i of lane l at [4 l + i]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cm[i] = F::max16(cm[i]);
            if (half == 0) colmax[warp][4 * l + i] = cm[i];
        }
        __syncthreads();
        if (threadIdx.x < kTile / 2) {
            uint32_t m0 = 0, m1 = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                const uint2 m = F::bits(colmax[w][threadIdx.x]);
                m0 = max(m0, m.x);
                m1 = max(m1, m.y);
            }
            const int i = threadIdx.x & 3, lc = threadIdx.x >> 2;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = 8 * lc + 2 * i + e;
                const uint32_t sb = scale_byte<FMT>(e ? m1 : m0);
                colinv[c] = inv_scale(sb);
                if (c0 + c < a.cols) a.st[(long long)b * a.sst + (long long)(c0 + c) * a.ldst + tr] = (uint8_t)sb;
            }
        }
        __syncthreads();
    }
    if (ROWS) {
        uint8_t* q = a.q + (long long)b * a.sq + (long long)r0 * a.ldq;
        float inv = sq_inv;
        if (!SQUARE) {
            const uint32_t byte = scale_byte<FMT>(max16_of8(rm, l));      // of row l / 2 of the eight
            inv = inv_scale(byte);
            if (!(l & 1) && r0 + (l >> 1) < a.rows)
                a.s[(long long)b * a.ss + (long long)(r0 + (l >> 1)) * a.lds + tc] = (uint8_t)byte;
        }
        const bool in = c0 + 8 * l + 8 <= a.cols;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = SQUARE ? inv : __shfl_sync(0xffffffffu, inv, (lane & 16) + 2 * j);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = mul2(f.get(j, i), make_float2(s, s));
                w[i] = cvt2<FMT>(v.x, v.y);
            }
            if (r0 + j >= a.rows) continue;
            if (in) {
                *reinterpret_cast<uint2*>(q + j * a.ldq + c0 + 8 * l) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = c0 + 8 * l + i;
                    if (c < a.cols) q[j * a.ldq + c] = (uint8_t)(w[i >> 1] >> (8 * (i & 1)));
                }
            }
        }
    }
    if constexpr (PACKED && NORM && ROWS && COLS) f.again();
    if (COLS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ca = 8 * l + 2 * i, cb = ca + 1;
            const float2 inv = SQUARE ? make_float2(sq_inv, sq_inv) : make_float2(colinv[ca], colinv[cb]);
            uint32_t wa[4], wb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = mul2(f.get(2 * j, i), inv), v = mul2(f.get(2 * j + 1, i), inv);
                wa[j] = cvt2<FMT>(u.x, v.x);
                wb[j] = cvt2<FMT>(u.y, v.y);
            }
            tile[t_granule(ca, g)] = make_uint2(wa[0] | (wa[1] << 16), wa[2] | (wa[3] << 16));
            tile[t_granule(cb, g)] = make_uint2(wb[0] | (wb[1] << 16), wb[2] | (wb[3] << 16));
        }
        __syncthreads();
        uint8_t* qt = a.qt + (long long)b * a.sqt;
        // eight threads a row of the transposed tile, 16 bytes (two granules) each
        const int ch = threadIdx.x & 7;
        const int rbase = tr * kTile + 16 * ch;
#pragma unroll
        for (int k = 0; k < kTile / (kThreads / 8); ++k) {
            const int c = (threadIdx.x >> 3) + k * (kThreads / 8);
            if (c0 + c >= a.cols) break;
            const uint2 lo = tile[t_granule(c, 2 * ch)], hi = tile[t_granule(c, 2 * ch + 1)];
            uint8_t* o = qt + (long long)(c0 + c) * a.ldqt + rbase;
            if (rbase + 16 <= a.rows) {
                *reinterpret_cast<uint4*>(o) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (rbase + e < a.rows) o[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
            }
        }
    }
}

template <typename T, int FMT, bool ROWS, bool COLS, bool SQUARE, bool SHIFT>
cudaError_t go(const QuantParams& p, cudaStream_t st)
{
    const dim3 grid((unsigned)(cdiv(p.a.rows, kTile) * p.tiles_c), (unsigned)p.a.batch);
    if (p.a.rstd)
        return launch_overlapped("q8_quantize_norm", q8_quant_kernel<T, FMT, ROWS, COLS, SQUARE, SHIFT, true>, grid,
                      dim3(kThreads), 0, st, p);
    return launch_overlapped("q8_quantize", q8_quant_kernel<T, FMT, ROWS, COLS, SQUARE, SHIFT, false>, grid, dim3(kThreads), 0,
                  st, p);
}

template <typename T, int FMT, bool SHIFT>
cudaError_t pick(const QuantParams& p, cudaStream_t st)
{
    const bool rows = p.a.q != nullptr, cols = p.a.qt != nullptr;
    if (p.a.square) {
        if (rows && cols) return go<T, FMT, true, true, true, SHIFT>(p, st);
        return rows ? go<T, FMT, true, false, true, SHIFT>(p, st) : go<T, FMT, false, true, true, SHIFT>(p, st);
    }
    if (rows && cols) return go<T, FMT, true, true, false, SHIFT>(p, st);
    return rows ? go<T, FMT, true, false, false, SHIFT>(p, st) : go<T, FMT, false, true, false, SHIFT>(p, st);
}

template <typename T>
cudaError_t typed(const QuantParams& p, dion_q8_format fmt, cudaStream_t st)
{
    const size_t e = sizeof(T);
    const bool shift = (uintptr_t)p.a.x % 16 || (p.a.ldx * e) % 16 || (p.a.batch > 1 && (p.a.sx * e) % 16);
    if (fmt == DION_E4M3) return shift ? pick<T, DION_E4M3, true>(p, st) : pick<T, DION_E4M3, false>(p, st);
    return shift ? pick<T, DION_E5M2, true>(p, st) : pick<T, DION_E5M2, false>(p, st);
}

}  // namespace

cudaError_t q8_quantize(const Q8QuantArgs& a, dion_dtype dt, dion_q8_format fmt, cudaStream_t st)
{
    if (a.batch == 0 || a.rows == 0 || a.cols == 0) return cudaSuccess;
    const QuantParams p{a, (int)cdiv(a.cols, kTile), a.wdt == DION_F32};
    return dt == DION_F32 ? typed<float>(p, fmt, st) : typed<bf16>(p, fmt, st);
}

}  // namespace dion
