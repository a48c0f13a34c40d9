// q8_norm.cu -- root-mean-square norm with the residual's addition and 8-bit
// output, and its gradient.
//
// Forward: bounded by memory.  One CTA holds a row in registers (one read of x
// and the residual, one write of h and of the bytes), so the sum of squares,
// the scaling and the block maxima all work on the values of that one read.
#include "q8.cuh"

namespace dion {

int num_sms();

namespace {

using namespace q8;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the CTA; every thread gets it.  red: one float per warp, free for
// reuse only after the caller's next barrier.
__device__ __forceinline__ float cta_sum(float v, float* red)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? red[lane] : 0.f);
}

struct NormParams {
    Q8NormArgs a;
    bool wf32;
};

template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int c0, int cols, int l, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = c0 + elem<VEC>(l, i);
        f[i] = c >= cols ? 0.f : f32 ? reinterpret_cast<const float*>(w)[c] : to_f(reinterpret_cast<const bf16*>(w)[c]);
    }
}

// One 128-value block of y per half-warp: scale, bytes.
template <int FMT, bool VEC>
__device__ __forceinline__ void emit_block(const Q8NormArgs& a, long long row, int c0, int l, float (&y)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, mag_bits(y[i]));
    if (m >= kInfBits) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = inf_to_nan(y[i]);
            m = max(m, finite_mag_bits(y[i]));
        }
    }
    const uint32_t byte = scale_byte<FMT>(max16(m));
    if (c0 >= a.cols) return;
    if (l == 0) a.s[row * a.lds + (c0 >> 7)] = (uint8_t)byte;
    store_q8<VEC, FMT>(a.q + row * a.ldq, c0, a.cols, l, y, inv_scale(byte));
}

// NV blocks per half-warp: block index = half-warp index + k * (half-warps).
template <typename T, int FMT, bool VEC, int NV>
__global__ void __launch_bounds__(1024) norm_q8_kernel(const NormParams p)
{
    __shared__ float red[32];
    const Q8NormArgs& a = p.a;
    const long long row = blockIdx.x;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    float f[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) load8<VEC>(x, (hw + k * nhw) * 128, a.cols, l, f[k]);
    if (a.res) {
        const T* r = reinterpret_cast<const T*>(a.res) + row * a.ldr;
        T* h = reinterpret_cast<T*>(a.h) + row * a.ldh;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float g[8];
            load8<VEC>(r, (hw + k * nhw) * 128, a.cols, l, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[k][i] = to_f(from_f<T>(f[k][i] + g[i]));
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) store8<VEC>(h, (hw + k * nhw) * 128, a.cols, l, f[k]);
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[k][i], f[k][i], ss);
    const float rstd = 1.f / sqrtf(cta_sum(ss, red) / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c0 = (hw + k * nhw) * 128;
        float w[8];
        load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[k][i] = __fmul_rn(__fmul_rn(f[k][i], rstd), w[i]);
        emit_block<FMT, VEC>(a, row, c0, l, f[k]);
    }
}

// Rows longer than the registers hold: the same steps over the row twice, the
// second time from h (or x), which the first pass left in L2.
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(1024) norm_q8_long_kernel(const NormParams p)
{
    __shared__ float red[32];
    const Q8NormArgs& a = p.a;
    const long long row = blockIdx.x;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* src = a.res ? reinterpret_cast<const T*>(a.h) + row * a.ldh : x;
    float ss = 0.f;
    for (int c0 = hw * 128; c0 < a.cols; c0 += nhw * 128) {
        float f[8];
        load8<VEC>(x, c0, a.cols, l, f);
        if (a.res) {
            float g[8];
            load8<VEC>(reinterpret_cast<const T*>(a.res) + row * a.ldr, c0, a.cols, l, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = to_f(from_f<T>(f[i] + g[i]));
            store8<VEC>(reinterpret_cast<T*>(a.h) + row * a.ldh, c0, a.cols, l, f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
    }
    const float rstd = 1.f / sqrtf(cta_sum(ss, red) / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    // a thread reads back the very elements that it wrote; whole warps stay
    // in the loop together (the block maximum is exchanged between lanes)
    for (int base = 0; base < a.cols; base += nhw * 128) {
        const int c0 = base + hw * 128;
        float f[8], w[8];
        load8<VEC>(src, c0, a.cols, l, f);
        load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(__fmul_rn(f[i], rstd), w[i]);
        emit_block<FMT, VEC>(a, row, c0, l, f);
    }
}

template <typename T, int FMT, bool VEC>
cudaError_t norm_go(const NormParams& p, cudaStream_t st)
{
    const int blocks = (int)cdiv(p.a.cols, 128);
    const dim3 grid((unsigned)p.a.rows);
    // two half-warps a warp, as many blocks a half-warp as it takes
    if (blocks <= 16)
        return launch("rms_norm_q8", norm_q8_kernel<T, FMT, VEC, 1>, grid, dim3((unsigned)cdiv(blocks, 2) * 32), 0, st, p);
    if (blocks <= 128)
        return launch("rms_norm_q8", norm_q8_kernel<T, FMT, VEC, 2>, grid, dim3((unsigned)cdiv(blocks, 4) * 32), 0, st, p);
    if (blocks <= 256)
        return launch("rms_norm_q8", norm_q8_kernel<T, FMT, VEC, 4>, grid, dim3((unsigned)cdiv(blocks, 8) * 32), 0, st, p);
    return launch("rms_norm_q8_long", norm_q8_long_kernel<T, FMT, VEC>, grid, dim3(1024), 0, st, p);
}

template <typename T>
cudaError_t norm_typed(const NormParams& p, dion_q8_format fmt, cudaStream_t st)
{
    const size_t e = sizeof(T);
    const Q8NormArgs& a = p.a;
    bool vec = (uintptr_t)a.x % 16 == 0 && (a.ldx * e) % 16 == 0;
    if (a.res)
        vec = vec && (uintptr_t)a.res % 16 == 0 && (a.ldr * e) % 16 == 0 && (uintptr_t)a.h % 16 == 0 && (a.ldh * e) % 16 == 0;
    if (fmt == DION_E4M3) return vec ? norm_go<T, DION_E4M3, true>(p, st) : norm_go<T, DION_E4M3, false>(p, st);
    return vec ? norm_go<T, DION_E5M2, true>(p, st) : norm_go<T, DION_E5M2, false>(p, st);
}

// ------------------------------------------------------------------ gradient
struct BwdParams {
    NormBwdArgs a;
    bool wf32;
};

// Each CTA walks rows blockIdx.x, + gridDim.x, ...; a thread owns NV chunks of
// eight columns and keeps their sums of dy * xhat in registers until the end,
// when they go to the CTA's row of the workspace.
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const BwdParams p)
{
    __shared__ float red[2][32];
    const NormBwdArgs& a = p.a;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    float dw[NV][8], w[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_weight<VEC>(a.w, p.wf32, (hw + k * nhw) * 128, a.cols, l, w[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = 0.f;
    }
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        float g[NV][8], xh[NV][8], d[NV][8];
        const float rstd = a.rstd[row];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            load8<VEC>(reinterpret_cast<const T*>(a.dy) + row * a.lddy, (hw + k * nhw) * 128, a.cols, l, g[k]);
            load8<VEC>(reinterpret_cast<const T*>(a.h) + row * a.ldh, (hw + k * nhw) * 128, a.cols, l, xh[k]);
        }
        if (a.dh) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                load8<VEC>(reinterpret_cast<const T*>(a.dh) + row * a.lddh, (hw + k * nhw) * 128, a.cols, l, d[k]);
        }
        float c = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[k][i] *= rstd;
                dw[k][i] = fmaf(g[k][i], xh[k][i], dw[k][i]);
                g[k][i] *= w[k][i];
                c = fmaf(g[k][i], xh[k][i], c);
            }
        c = cta_sum(c, red[flip]) / (float)a.cols;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[k][i] = rstd * fmaf(-c, xh[k][i], g[k][i]);
                if (a.dh) g[k][i] += d[k][i];
            }
            store8<VEC>(reinterpret_cast<T*>(a.dx) + row * a.lddx, (hw + k * nhw) * 128, a.cols, l, g[k]);
        }
    }
    float* part = a.part + (long long)blockIdx.x * a.cols;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = (hw + k * nhw) * 128 + elem<VEC>(l, i);
            if (c < a.cols) part[c] = dw[k][i];
        }
}

// Rows longer than the registers hold: one row at a time, and the sums of
// dy * xhat in the CTA's row of the workspace instead of in registers.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const BwdParams p)
{
    __shared__ float red[2][32];
    const NormBwdArgs& a = p.a;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    float* part = a.part + (long long)blockIdx.x * a.cols;
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const float rstd = a.rstd[row];
        const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.lddy;
        const T* h = reinterpret_cast<const T*>(a.h) + row * a.ldh;
        float sum = 0.f;
        for (int c0 = hw * 128; c0 < a.cols; c0 += nhw * 128) {
            float g[8], xh[8], w[8];
            load8<VEC>(dy, c0, a.cols, l, g);
            load8<VEC>(h, c0, a.cols, l, xh);
            load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(g[i] * w[i], xh[i] * rstd, sum);
        }
        const float c = cta_sum(sum, red[flip]) / (float)a.cols;
        for (int c0 = hw * 128; c0 < a.cols; c0 += nhw * 128) {
            float g[8], xh[8], w[8], d[8];
            load8<VEC>(dy, c0, a.cols, l, g);
            load8<VEC>(h, c0, a.cols, l, xh);
            load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
            if (a.dh) load8<VEC>(reinterpret_cast<const T*>(a.dh) + row * a.lddh, c0, a.cols, l, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = c0 + elem<VEC>(l, i);
                xh[i] *= rstd;
                if (col < a.cols) part[col] = fmaf(g[i], xh[i], row == blockIdx.x ? 0.f : part[col]);
                g[i] = rstd * fmaf(-c, xh[i], g[i] * w[i]);
                if (a.dh) g[i] += d[i];
            }
            store8<VEC>(reinterpret_cast<T*>(a.dx) + row * a.lddx, c0, a.cols, l, g);
        }
    }
}

// dw = sum of the workspace's rows, in their order: 32 columns a CTA, 32
// threads down each, joined in shared memory.
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float* part, int groups, int cols, float* dw)
{
    __shared__ float t[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float s = 0.f;
    if (c < cols)
        for (int r = y; r < groups; r += 32) s += part[(long long)r * cols + c];
    t[y][x] = s;
    __syncthreads();
    const float v = warp_sum(t[x][y]);
    if (x == 0 && blockIdx.x * 32 + y < cols) dw[blockIdx.x * 32 + y] = v;
}

// Row groups of the gradient kernel: CTAs that fill the SMs.
int bwd_groups(int rows, int cols)
{
    const int blocks = (int)cdiv(cols, 128);
    const int per_sm = blocks <= 16 ? 8 : blocks <= 64 ? 2 : 1;
    const long long g = (long long)num_sms() * per_sm;
    return (int)(rows < g ? rows : g);
}

template <typename T, bool VEC>
cudaError_t bwd_go(const BwdParams& p, cudaStream_t st)
{
    const int blocks = (int)cdiv(p.a.cols, 128), groups = bwd_groups(p.a.rows, p.a.cols);
    const dim3 grid((unsigned)groups);
    cudaError_t e;
    if (blocks <= 16)
        e = launch("rms_norm_backward", norm_bwd_kernel<T, VEC, 1>, grid, dim3((unsigned)cdiv(blocks, 2) * 32), 0, st, p);
    else if (blocks <= 128)
        e = launch("rms_norm_backward", norm_bwd_kernel<T, VEC, 2>, grid, dim3((unsigned)cdiv(blocks, 4) * 32), 0, st, p);
    else
        e = launch("rms_norm_backward_long", norm_bwd_long_kernel<T, VEC>, grid, dim3(1024), 0, st, p);
    if (e != cudaSuccess) return e;
    return launch("rms_norm_backward_sum", norm_bwd_sum_kernel, dim3((unsigned)cdiv(p.a.cols, 32)), dim3(1024), 0, st,
                  (const float*)p.a.part, groups, p.a.cols, p.a.dw);
}

template <typename T>
cudaError_t bwd_typed(const BwdParams& p, cudaStream_t st)
{
    const size_t e = sizeof(T);
    const NormBwdArgs& a = p.a;
    bool vec = (uintptr_t)a.dy % 16 == 0 && (a.lddy * e) % 16 == 0 && (uintptr_t)a.h % 16 == 0 && (a.ldh * e) % 16 == 0 &&
               (uintptr_t)a.dx % 16 == 0 && (a.lddx * e) % 16 == 0;
    if (a.dh) vec = vec && (uintptr_t)a.dh % 16 == 0 && (a.lddh * e) % 16 == 0;
    return vec ? bwd_go<T, true>(p, st) : bwd_go<T, false>(p, st);
}

}  // namespace

cudaError_t rms_norm_q8(const Q8NormArgs& a, dion_dtype dt, dion_q8_format fmt, cudaStream_t st)
{
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const NormParams p{a, a.wdt == DION_F32};
    return dt == DION_F32 ? norm_typed<float>(p, fmt, st) : norm_typed<bf16>(p, fmt, st);
}

size_t norm_backward_workspace(int rows, int cols)
{
    return (size_t)bwd_groups(rows, cols) * (size_t)cols * sizeof(float);
}

cudaError_t rms_norm_backward(const NormBwdArgs& a, dion_dtype dt, cudaStream_t st)
{
    if (a.cols == 0) return cudaSuccess;
    if (a.rows == 0) return cudaMemsetAsync(a.dw, 0, (size_t)a.cols * sizeof(float), st);
    const BwdParams p{a, a.wdt == DION_F32};
    return dt == DION_F32 ? bwd_typed<float>(p, st) : bwd_typed<bf16>(p, st);
}

}  // namespace dion
