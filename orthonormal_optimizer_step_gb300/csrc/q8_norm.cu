// q8_norm.cu -- root-mean-square norm with the residual's addition and 8-bit
// output, and its gradient.
//
// Both are bounded by memory: a row's values are read once into registers, the
// sums, the scaling and the block maxima all work on them there, and each
// output is written once.  Two forms of each kernel:
//   - one row a CTA (few rows, or rows that are not aligned for wide accesses);
//   - streaming: as many CTAs as run at once walk the rows, and every thread
//     copies its own chunks of the next rows into shared memory
//     asynchronously (cp.async; a thread reads back only what it copied, so the
//     ring needs no barrier), which keeps loads in flight while a row waits
//     for its sum.
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
    if (nw == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? red[lane] : 0.f);
}

template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int c0, int cols, int l, float2 (&f)[4])
{
    if (f32) load8<VEC>(reinterpret_cast<const float*>(w), c0, cols, l, f);
    else load8<VEC>(reinterpret_cast<const bf16*>(w), c0, cols, l, f);
}

__device__ __forceinline__ float sum_squares(const float2 (&f)[4], float ss)
{
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) t = fma2(f[i], f[i], t);
    return ss + (t.x + t.y);
}

struct NormParams {
    Q8NormArgs a;
    bool wf32;
};

// One 128-value block of y = f * rstd * w per half-warp: scale and bytes.
template <int FMT, bool VEC>
__device__ __forceinline__ void emit_block(const Q8NormArgs& a, long long row, int c0, int l, float2 (&f)[4], float rstd,
                                           const float2 (&w)[4])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = mul2(mul2(f[i], make_float2(rstd, rstd)), w[i]);
        m = fmaxf(m, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));       // NaN does not count
    }
    uint32_t mb = __float_as_uint(m);
    if (mb >= kInfBits) {                                        // rare: nor does an infinity, which becomes NaN
        mb = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = make_float2(inf_to_nan(f[i].x), inf_to_nan(f[i].y));
            mb = max(mb, max(finite_mag_bits(f[i].x), finite_mag_bits(f[i].y)));
        }
    }
    const uint32_t byte = scale_byte<FMT>(max16(mb));
    if (c0 >= a.cols) return;
    if (l == 0) a.s[row * a.lds + (c0 >> 7)] = (uint8_t)byte;
    store_q8<VEC, FMT>(a.q + row * a.ldq, c0, a.cols, l, f, inv_scale(byte));
}

// h = x + residual, rounded to T, of one chunk
template <typename T>
__device__ __forceinline__ void add_rounded(float2 (&f)[4], const float2 (&g)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = add2(f[i], g[i]);
        if (sizeof(T) == 2) f[i] = unpack2(pack2(f[i]));
    }
}

// One row a CTA, NV blocks per half-warp: block = half-warp + k * half-warps.
template <typename T, int FMT, bool VEC, int NV>
__global__ void __launch_bounds__(1024) norm_q8_kernel(const NormParams p)
{
    __shared__ float red[32];
    const Q8NormArgs& a = p.a;
    const long long row = blockIdx.x;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    float2 f[NV][4], w[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k) load8<VEC>(x, (hw + k * nhw) * 128, a.cols, l, f[k]);
    if (a.res) {
        const T* r = reinterpret_cast<const T*>(a.res) + row * a.ldr;
        T* h = reinterpret_cast<T*>(a.h) + row * a.ldh;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            load8<VEC>(r, (hw + k * nhw) * 128, a.cols, l, w[k]);
            add_rounded<T>(f[k], w[k]);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) store8<VEC>(h, (hw + k * nhw) * 128, a.cols, l, f[k]);
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_weight<VEC>(a.w, p.wf32, (hw + k * nhw) * 128, a.cols, l, w[k]);
        ss = sum_squares(f[k], ss);
    }
    const float rstd = 1.f / sqrtf(cta_sum(ss, red) / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) emit_block<FMT, VEC>(a, row, (hw + k * nhw) * 128, l, f[k], rstd, w[k]);
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
        float2 f[4];
        load8<VEC>(x, c0, a.cols, l, f);
        if (a.res) {
            float2 g[4];
            load8<VEC>(reinterpret_cast<const T*>(a.res) + row * a.ldr, c0, a.cols, l, g);
            add_rounded<T>(f, g);
            store8<VEC>(reinterpret_cast<T*>(a.h) + row * a.ldh, c0, a.cols, l, f);
        }
        ss = sum_squares(f, ss);
    }
    const float rstd = 1.f / sqrtf(cta_sum(ss, red) / (float)a.cols + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    // a thread reads back the very elements that it wrote; whole warps stay
    // in the loop together (the block maximum is exchanged between lanes)
    for (int base = 0; base < a.cols; base += nhw * 128) {
        const int c0 = base + hw * 128;
        float2 f[4], w[4];
        load8<VEC>(src, c0, a.cols, l, f);
        load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
        emit_block<FMT, VEC>(a, row, c0, l, f, rstd, w);
    }
}

// -------------------------------------------------- streaming over many rows
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's ring of S rows: NIN inputs, NV chunks of eight columns each
// (block and lane as above), stored as [slot][input][chunk][word][thread].
template <typename T, int NIN, int NV, int S>
struct Ring {
    static constexpr int W = sizeof(T) / 2;
    uint4* mine;
    __device__ __forceinline__ uint4* at(int slot, int in, int k, int w) const
    {
        return mine + (((slot * NIN + in) * NV + k) * W + w) * blockDim.x;
    }
    __device__ __forceinline__ void fetch(int slot, int in, int k, const T* src) const
    {
#pragma unroll
        for (int w = 0; w < W; ++w)
            copy_async((uint32_t)__cvta_generic_to_shared(at(slot, in, k, w)), reinterpret_cast<const uint4*>(src) + w);
    }
    __device__ __forceinline__ void read(int slot, int in, int k, float2 (&f)[4]) const
    {
        Raw8<T> r;
#pragma unroll
        for (int w = 0; w < W; ++w) r.u[w] = *at(slot, in, k, w);
        unpack8(r, f);
    }
    static size_t bytes(int threads) { return (size_t)S * NIN * NV * W * threads * 16; }
};

// cols is a multiple of 8: a thread's chunk lies in the row or past it.
template <typename T, int FMT, bool RES, int NV, int S>
__global__ void __launch_bounds__(1024) norm_q8_stream_kernel(const NormParams p)
{
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][32];
    const Q8NormArgs& a = p.a;
    const Ring<T, RES ? 2 : 1, NV, S> ring{ring_smem + threadIdx.x};
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    const T* x = reinterpret_cast<const T*>(a.x);
    const T* r = reinterpret_cast<const T*>(a.res);
    float2 w[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k) load_weight<true>(a.w, p.wf32, (hw + k * nhw) * 128, a.cols, l, w[k]);
    auto issue = [&](long long row, int slot) {
        if (row < a.rows) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (hw + k * nhw) * 128 + 8 * l;
                if (c >= a.cols) continue;
                ring.fetch(slot, 0, k, x + row * a.ldx + c);
                if (RES) ring.fetch(slot, 1, k, r + row * a.ldr + c);
            }
        }
        copy_commit();
    };
    long long ahead = blockIdx.x;
#pragma unroll
    for (int s = 0; s < S - 1; ++s, ahead += gridDim.x) issue(ahead, s);
    int slot = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, ahead += gridDim.x) {
        issue(ahead, slot ? slot - 1 : S - 1);
        copy_wait<S - 1>();
        float2 f[NV][4];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c0 = (hw + k * nhw) * 128;
            if (c0 + 8 * l < a.cols) {
                ring.read(slot, 0, k, f[k]);
                if (RES) {
                    float2 g[4];
                    ring.read(slot, 1, k, g);
                    add_rounded<T>(f[k], g);
                    store8<true>(reinterpret_cast<T*>(a.h) + row * a.ldh, c0, a.cols, l, f[k]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) f[k][i] = make_float2(0.f, 0.f);
            }
            ss = sum_squares(f[k], ss);
        }
        const float rstd = 1.f / sqrtf(cta_sum(ss, red[slot & 1]) / (float)a.cols + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) emit_block<FMT, true>(a, row, (hw + k * nhw) * 128, l, f[k], rstd, w[k]);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
}

// Threads of a streaming CTA (one chunk a thread up to 8192 columns, two up to
// 16384), CTAs of it on an SM, and whether the ring leaves room for them.
constexpr int kStages = 4;
int stream_threads(int cols) { return (int)cdiv(cols, cols <= 8192 ? 256 : 512) * 32; }
int stream_ctas(int cols)
{
    const int t = stream_threads(cols);
    return t >= 1024 ? 1 : 1024 / t < 16 ? 1024 / t : 16;
}
constexpr size_t kRingRoom = 200 * 1024;        // of an SM's shared memory, for all its CTAs

template <typename T, int FMT, bool RES, int NV>
cudaError_t norm_stream(const NormParams& p, cudaStream_t st)
{
    typedef Ring<T, RES ? 2 : 1, NV, kStages> R;
    const int threads = stream_threads(p.a.cols);
    static std::atomic<unsigned long long> attr{0};
    const cudaError_t e = smem_attr_once((const void*)norm_q8_stream_kernel<T, FMT, RES, NV, kStages>, (int)kRingRoom, attr);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)num_sms() * stream_ctas(p.a.cols);
    return launch("rms_norm_q8_stream", norm_q8_stream_kernel<T, FMT, RES, NV, kStages>,
                  dim3((unsigned)(p.a.rows < grid ? p.a.rows : grid)), dim3((unsigned)threads), R::bytes(threads), st, p);
}

template <typename T, int FMT, bool VEC>
cudaError_t norm_go(const NormParams& p, cudaStream_t st)
{
    const int cols = p.a.cols, blocks = (int)cdiv(cols, 128);
    // Streaming pays once every CTA has several rows to prefetch.
    if (VEC && cols % 8 == 0 && cols <= 16384 && p.a.rows > 2ll * num_sms() * stream_ctas(cols)) {
        const size_t ring = (size_t)kStages * (p.a.res ? 2 : 1) * cdiv(cols, 128) * 128 * sizeof(T) * stream_ctas(cols);
        if (ring <= kRingRoom) {
            if (cols <= 8192) return p.a.res ? norm_stream<T, FMT, true, 1>(p, st) : norm_stream<T, FMT, false, 1>(p, st);
            return p.a.res ? norm_stream<T, FMT, true, 2>(p, st) : norm_stream<T, FMT, false, 2>(p, st);
        }
    }
    const dim3 grid((unsigned)p.a.rows);
    // two half-warps a warp, as many blocks a half-warp as it takes
    if (blocks <= 16)
        return launch("rms_norm_q8", norm_q8_kernel<T, FMT, VEC, 1>, grid, dim3((unsigned)cdiv(blocks, 2) * 32), 0, st, p);
    if (blocks <= 128)
        return launch("rms_norm_q8", norm_q8_kernel<T, FMT, VEC, 2>, grid, dim3((unsigned)cdiv(blocks, 4) * 32), 0, st, p);
    return launch("rms_norm_q8_long", norm_q8_long_kernel<T, FMT, VEC>, grid, dim3(1024), 0, st, p);
}

template <typename T>
cudaError_t norm_typed(const NormParams& p, dion_q8_format fmt, cudaStream_t st)
{
    const size_t e = sizeof(T);
    const Q8NormArgs& a = p.a;
    bool vec = (uintptr_t)a.x % 16 == 0 && (a.ldx * e) % 16 == 0 && (uintptr_t)a.w % 16 == 0;
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

// First half of a row's gradient, one chunk: xhat, the share of dw, and the
// share of the row's sum of g * xhat.  g: dy, then dy * w.
__device__ __forceinline__ float bwd_sums(float2 (&g)[4], float2 (&xh)[4], const float2 (&w)[4], float rstd,
                                          float2 (&dw)[4], float c)
{
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        xh[i] = mul2(xh[i], make_float2(rstd, rstd));
        dw[i] = fma2(g[i], xh[i], dw[i]);
        g[i] = mul2(g[i], w[i]);
        t = fma2(g[i], xh[i], t);
    }
    return c + (t.x + t.y);
}
// Second half: dx (without dh) into g.
__device__ __forceinline__ void bwd_dx(float2 (&g)[4], const float2 (&xh)[4], float rstd, float c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = mul2(make_float2(rstd, rstd), fma2(make_float2(-c, -c), xh[i], g[i]));
}

template <bool VEC, int NV>
__device__ __forceinline__ void store_part(float* part, int cols, int l, int hw, int nhw, const float2 (&dw)[NV][4])
{
#pragma unroll
    for (int k = 0; k < NV; ++k) store8<VEC>(part, (hw + k * nhw) * 128, cols, l, dw[k]);
}

// Each CTA walks rows blockIdx.x, + gridDim.x, ...; a thread owns NV chunks of
// eight columns and keeps their sums of dy * xhat in registers until the end,
// when they go to the CTA's row of the workspace.
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const BwdParams p)
{
    __shared__ float red[2][32];
    const NormBwdArgs& a = p.a;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    float2 dw[NV][4], w[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_weight<VEC>(a.w, p.wf32, (hw + k * nhw) * 128, a.cols, l, w[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[k][i] = make_float2(0.f, 0.f);
    }
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        float2 g[NV][4], xh[NV][4], d[NV][4];
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
        for (int k = 0; k < NV; ++k) c = bwd_sums(g[k], xh[k], w[k], rstd, dw[k], c);
        c = cta_sum(c, red[flip]) / (float)a.cols;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            bwd_dx(g[k], xh[k], rstd, c);
            if (a.dh) {
#pragma unroll
                for (int i = 0; i < 4; ++i) g[k][i] = add2(g[k][i], d[k][i]);
            }
            store8<VEC>(reinterpret_cast<T*>(a.dx) + row * a.lddx, (hw + k * nhw) * 128, a.cols, l, g[k]);
        }
    }
    store_part<VEC, NV>(a.part + (long long)blockIdx.x * a.cols, a.cols, l, hw, nhw, dw);
}

// The same with the rows' inputs prefetched into shared memory.
template <typename T, bool DH, int NV, int S>
__global__ void __launch_bounds__(1024) norm_bwd_stream_kernel(const BwdParams p)
{
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][32];
    const NormBwdArgs& a = p.a;
    const Ring<T, DH ? 3 : 2, NV, S> ring{ring_smem + threadIdx.x};
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    float2 dw[NV][4], w[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_weight<true>(a.w, p.wf32, (hw + k * nhw) * 128, a.cols, l, w[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[k][i] = make_float2(0.f, 0.f);
    }
    auto issue = [&](long long row, int slot) {
        if (row < a.rows) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (hw + k * nhw) * 128 + 8 * l;
                if (c >= a.cols) continue;
                ring.fetch(slot, 0, k, reinterpret_cast<const T*>(a.dy) + row * a.lddy + c);
                ring.fetch(slot, 1, k, reinterpret_cast<const T*>(a.h) + row * a.ldh + c);
                if (DH) ring.fetch(slot, 2, k, reinterpret_cast<const T*>(a.dh) + row * a.lddh + c);
            }
        }
        copy_commit();
    };
    long long ahead = blockIdx.x;
#pragma unroll
    for (int s = 0; s < S - 1; ++s, ahead += gridDim.x) issue(ahead, s);
    float rstd = blockIdx.x < a.rows ? a.rstd[blockIdx.x] : 0.f;
    int slot = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, ahead += gridDim.x) {
        issue(ahead, slot ? slot - 1 : S - 1);
        const float rstd_next = row + gridDim.x < a.rows ? a.rstd[row + gridDim.x] : 0.f;
        copy_wait<S - 1>();
        float2 g[NV][4], xh[NV][4];
        float c = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if ((hw + k * nhw) * 128 + 8 * l < a.cols) {
                ring.read(slot, 0, k, g[k]);
                ring.read(slot, 1, k, xh[k]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) g[k][i] = xh[k][i] = make_float2(0.f, 0.f);
            }
            c = bwd_sums(g[k], xh[k], w[k], rstd, dw[k], c);
        }
        c = cta_sum(c, red[slot & 1]) / (float)a.cols;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c0 = (hw + k * nhw) * 128;
            if (c0 + 8 * l >= a.cols) continue;
            bwd_dx(g[k], xh[k], rstd, c);
            if (DH) {
                float2 d[4];
                ring.read(slot, 2, k, d);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[k][i] = add2(g[k][i], d[i]);
            }
            store8<true>(reinterpret_cast<T*>(a.dx) + row * a.lddx, c0, a.cols, l, g[k]);
        }
        rstd = rstd_next;
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    store_part<true, NV>(a.part + (long long)blockIdx.x * a.cols, a.cols, l, hw, nhw, dw);
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
        float2 g[4], xh[4], w[4], d[4], dw[4] = {};
        for (int c0 = hw * 128; c0 < a.cols; c0 += nhw * 128) {
            load8<VEC>(dy, c0, a.cols, l, g);
            load8<VEC>(h, c0, a.cols, l, xh);
            load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
            sum = bwd_sums(g, xh, w, rstd, dw, sum);
        }
        const float c = cta_sum(sum, red[flip]) / (float)a.cols;
        for (int c0 = hw * 128; c0 < a.cols; c0 += nhw * 128) {
            load8<VEC>(dy, c0, a.cols, l, g);
            load8<VEC>(h, c0, a.cols, l, xh);
            load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
            if (row == blockIdx.x) {
#pragma unroll
                for (int i = 0; i < 4; ++i) dw[i] = make_float2(0.f, 0.f);
            } else {
                load8<VEC>(part, c0, a.cols, l, dw);
            }
            if (a.dh) load8<VEC>(reinterpret_cast<const T*>(a.dh) + row * a.lddh, c0, a.cols, l, d);
            bwd_sums(g, xh, w, rstd, dw, 0.f);
            store8<VEC>(part, c0, a.cols, l, dw);
            bwd_dx(g, xh, rstd, c);
            if (a.dh) {
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = add2(g[i], d[i]);
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
    if (c < cols) {
#pragma unroll 8
        for (int r = y; r < groups; r += 32) s += part[(long long)r * cols + c];
    }
    t[y][x] = s;
    __syncthreads();
    const float v = warp_sum(t[x][y]);
    if (x == 0 && blockIdx.x * 32 + y < cols) dw[blockIdx.x * 32 + y] = v;
}

// Row groups of the gradient kernel: CTAs that fill the SMs.
int bwd_groups(int rows, int cols)
{
    const long long g = (long long)num_sms() * stream_ctas(cols);
    return (int)(rows < g ? rows : g);
}

template <typename T, bool DH, int NV>
cudaError_t bwd_stream(const BwdParams& p, cudaStream_t st)
{
    typedef Ring<T, DH ? 3 : 2, NV, kStages> R;
    const int threads = stream_threads(p.a.cols);
    static std::atomic<unsigned long long> attr{0};
    const cudaError_t e = smem_attr_once((const void*)norm_bwd_stream_kernel<T, DH, NV, kStages>, (int)kRingRoom, attr);
    if (e != cudaSuccess) return e;
    return launch("rms_norm_backward_stream", norm_bwd_stream_kernel<T, DH, NV, kStages>,
                  dim3((unsigned)bwd_groups(p.a.rows, p.a.cols)), dim3((unsigned)threads), R::bytes(threads), st, p);
}

template <typename T, bool VEC>
cudaError_t bwd_rows(const BwdParams& p, cudaStream_t st)
{
    const int cols = p.a.cols, blocks = (int)cdiv(cols, 128), groups = bwd_groups(p.a.rows, cols);
    if (VEC && cols % 8 == 0 && cols <= 16384 && p.a.rows > 2ll * num_sms() * stream_ctas(cols)) {
        const size_t ring = (size_t)kStages * (p.a.dh ? 3 : 2) * cdiv(cols, 128) * 128 * sizeof(T) * stream_ctas(cols);
        if (ring <= kRingRoom) {
            if (cols <= 8192) return p.a.dh ? bwd_stream<T, true, 1>(p, st) : bwd_stream<T, false, 1>(p, st);
            return p.a.dh ? bwd_stream<T, true, 2>(p, st) : bwd_stream<T, false, 2>(p, st);
        }
    }
    const dim3 grid((unsigned)groups);
    if (blocks <= 64)
        return launch("rms_norm_backward", norm_bwd_kernel<T, VEC, 1>, grid, dim3((unsigned)cdiv(blocks, 2) * 32), 0, st, p);
    if (blocks <= 128)
        return launch("rms_norm_backward", norm_bwd_kernel<T, VEC, 2>, grid, dim3((unsigned)cdiv(blocks, 4) * 32), 0, st, p);
    return launch("rms_norm_backward_long", norm_bwd_long_kernel<T, VEC>, grid, dim3(1024), 0, st, p);
}

template <typename T>
cudaError_t bwd_typed(const BwdParams& p, cudaStream_t st)
{
    const size_t e = sizeof(T);
    const NormBwdArgs& a = p.a;
    // (the workspace is 256-byte aligned, but its rows of cols floats are 16-byte aligned only if cols % 4 == 0)
    bool vec = (uintptr_t)a.dy % 16 == 0 && (a.lddy * e) % 16 == 0 && (uintptr_t)a.h % 16 == 0 && (a.ldh * e) % 16 == 0 &&
               (uintptr_t)a.dx % 16 == 0 && (a.lddx * e) % 16 == 0 && (uintptr_t)a.w % 16 == 0 && a.cols % 4 == 0;
    if (a.dh) vec = vec && (uintptr_t)a.dh % 16 == 0 && (a.lddh * e) % 16 == 0;
    const cudaError_t err = vec ? bwd_rows<T, true>(p, st) : bwd_rows<T, false>(p, st);
    if (err != cudaSuccess) return err;
    return launch("rms_norm_backward_sum", norm_bwd_sum_kernel, dim3((unsigned)cdiv(a.cols, 32)), dim3(1024), 0, st,
                  (const float*)a.part, bwd_groups(a.rows, a.cols), a.cols, a.dw);
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
