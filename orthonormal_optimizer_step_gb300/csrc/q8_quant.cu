// q8_quant.cu -- quantization of matrices to 8-bit blocks, in row order, in
// transposed order, or both from one read.
//
// Bounded by memory: an element is read once (2 or 4 bytes) and written once
// or twice (1 byte each), so a 128 x 128 tile lives in one CTA's registers:
// 256 threads, each eight consecutive rows by eight columns.  Row maxima meet
// in the 16 lanes that share a row, column maxima in shared memory.  Eight
// consecutive rows in a thread make eight consecutive bytes of the transposed
// tile, which is exchanged through 16 KB of shared memory and written as whole
// 128-byte rows.
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

template <typename T, int FMT, bool ROWS, bool COLS, bool SQUARE, bool VEC, bool NORM>
__global__ void __launch_bounds__(kThreads) q8_quant_kernel(const QuantParams p)
{
    __shared__ uint2 tile[COLS ? kTile * 16 : 1];
    __shared__ uint32_t colmax[(COLS || SQUARE) ? kThreads / 32 : 1][kTile];
    __shared__ uint8_t colscale[kTile];
    const Q8QuantArgs& a = p.a;
    const int tr = blockIdx.x / p.tiles_c, tc = blockIdx.x % p.tiles_c, b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
    const int g = warp * 2 + half;                    // row granule of this half-warp
    const int r0 = tr * kTile + 8 * g, c0 = tc * kTile;
    const T* x = reinterpret_cast<const T*>(a.x) + (long long)b * a.sx;

    float f[8][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (r0 + j < a.rows) {
            load8<VEC>(x + (long long)(r0 + j) * a.ldx, c0, a.cols, l, f[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[j][i] = 0.f;
        }
    }
    if (NORM) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + elem<VEC>(l, i);
            w[i] = c >= a.cols ? 0.f : p.wf32 ? reinterpret_cast<const float*>(a.weight)[c]
                                              : to_f(reinterpret_cast<const bf16*>(a.weight)[c]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float rs = r0 + j < a.rows ? a.rstd[r0 + j] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[j][i] = __fmul_rn(__fmul_rn(f[j][i], rs), w[i]);
        }
    }
    // largest magnitudes, along this thread's rows and columns
    uint32_t rm[8], cm[8], all = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        rm[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) rm[j] = max(rm[j], mag_bits(f[j][i]));
        all = max(all, rm[j]);
    }
    if (all >= kInfBits) {                            // rare: infinities become NaN and do not count
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            rm[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[j][i] = inf_to_nan(f[j][i]);
                rm[j] = max(rm[j], finite_mag_bits(f[j][i]));
            }
        }
        all = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) all = max(all, rm[j]);
    }
    uint32_t sq_byte = 127;
    if (SQUARE) {
        all = max16(all);
        all = max(all, __shfl_xor_sync(0xffffffffu, all, 16));
        if (lane == 0) colmax[0][warp] = all;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) all = max(all, colmax[0][w]);
        sq_byte = scale_byte<FMT>(all);
        if (threadIdx.x == 0) {
            if (ROWS) a.s[(long long)b * a.ss + (long long)tr * a.lds + tc] = (uint8_t)sq_byte;
            if (COLS) a.st[(long long)b * a.sst + (long long)tc * a.ldst + tr] = (uint8_t)sq_byte;
        }
    } else if (COLS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cm[i] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) cm[i] = max(cm[i], finite_mag_bits(f[j][i]));
            cm[i] = max(cm[i], __shfl_xor_sync(0xffffffffu, cm[i], 16));
            if (half == 0) colmax[warp][elem<VEC>(l, i)] = cm[i];
        }
        __syncthreads();
        if (threadIdx.x < kTile) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) m = max(m, colmax[w][threadIdx.x]);
            const uint32_t sb = scale_byte<FMT>(m);
            colscale[threadIdx.x] = (uint8_t)sb;
            if (c0 + (int)threadIdx.x < a.cols)
                a.st[(long long)b * a.sst + (long long)(c0 + threadIdx.x) * a.ldst + tr] = (uint8_t)sb;
        }
        __syncthreads();
    }
    if (ROWS) {
        uint8_t* q = a.q + (long long)b * a.sq;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t byte = sq_byte;
            if (!SQUARE) {
                byte = scale_byte<FMT>(max16(rm[j]));
                if (l == 0 && r0 + j < a.rows)
                    a.s[(long long)b * a.ss + (long long)(r0 + j) * a.lds + tc] = (uint8_t)byte;
            }
            if (r0 + j < a.rows)
                store_q8<VEC, FMT>(q + (long long)(r0 + j) * a.ldq, c0, a.cols, l, f[j], inv_scale(byte));
        }
    }
    if (COLS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = elem<VEC>(l, i);
            const float inv = inv_scale(SQUARE ? sq_byte : (uint32_t)colscale[c]);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = cvt2<FMT>(f[2 * j][i] * inv, f[2 * j + 1][i] * inv);
            tile[t_granule(c, g)] = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        }
        __syncthreads();
        uint8_t* qt = a.qt + (long long)b * a.sqt;
        // eight threads a row of the transposed tile, 16 bytes (two granules) each
        const int ch = threadIdx.x & 7;
        const int rbase = tr * kTile + 16 * ch;
        for (int c = threadIdx.x >> 3; c < kTile && c0 + c < a.cols; c += kThreads / 8) {
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

template <typename T, int FMT, bool ROWS, bool COLS, bool SQUARE, bool VEC>
cudaError_t go(const QuantParams& p, cudaStream_t st)
{
    const dim3 grid((unsigned)(cdiv(p.a.rows, kTile) * p.tiles_c), (unsigned)p.a.batch);
    if (p.a.rstd)
        return launch("q8_quantize_norm", q8_quant_kernel<T, FMT, ROWS, COLS, SQUARE, VEC, true>, grid,
                      dim3(kThreads), 0, st, p);
    return launch("q8_quantize", q8_quant_kernel<T, FMT, ROWS, COLS, SQUARE, VEC, false>, grid, dim3(kThreads), 0,
                  st, p);
}

template <typename T, int FMT, bool VEC>
cudaError_t pick(const QuantParams& p, cudaStream_t st)
{
    const bool rows = p.a.q != nullptr, cols = p.a.qt != nullptr;
    if (p.a.square) {
        if (rows && cols) return go<T, FMT, true, true, true, VEC>(p, st);
        return rows ? go<T, FMT, true, false, true, VEC>(p, st) : go<T, FMT, false, true, true, VEC>(p, st);
    }
    if (rows && cols) return go<T, FMT, true, true, false, VEC>(p, st);
    return rows ? go<T, FMT, true, false, false, VEC>(p, st) : go<T, FMT, false, true, false, VEC>(p, st);
}

template <typename T>
cudaError_t typed(const QuantParams& p, dion_q8_format fmt, cudaStream_t st)
{
    const size_t e = sizeof(T);
    const bool vec = ((uintptr_t)p.a.x % 16 == 0) && (p.a.ldx * e) % 16 == 0 && (p.a.batch == 1 || (p.a.sx * e) % 16 == 0);
    if (fmt == DION_E4M3) return vec ? pick<T, DION_E4M3, true>(p, st) : pick<T, DION_E4M3, false>(p, st);
    return vec ? pick<T, DION_E5M2, true>(p, st) : pick<T, DION_E5M2, false>(p, st);
}

}  // namespace

cudaError_t q8_quantize(const Q8QuantArgs& a, dion_dtype dt, dion_q8_format fmt, cudaStream_t st)
{
    if (a.batch == 0 || a.rows == 0 || a.cols == 0) return cudaSuccess;
    const QuantParams p{a, (int)cdiv(a.cols, kTile), a.wdt == DION_F32};
    return dt == DION_F32 ? typed<float>(p, fmt, st) : typed<bf16>(p, fmt, st);
}

}  // namespace dion
