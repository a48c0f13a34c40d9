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

// a / n, within a rounding, for the n whose 1 / n is given: every thread of a
// row forms its mean and root, so their instructions count.
__device__ __forceinline__ float div_by(float a, float n, float inv_n)
{
    const float q = a * inv_n, r = fmaf(fmaf(-q, n, a), inv_n, q);
    return fabsf(q) < __int_as_float(0x7f800000) ? r : q;
}
// 1 / sqrt(v), one Newton step from the hardware's approximation (v = 0 or
// infinite: the approximation itself).
__device__ __forceinline__ float inv_sqrt(float v)
{
    const float r = rsqrtf(v), e = fmaf(-v * r, r, 1.f);
    return isfinite(e) ? fmaf(0.5f * r, e, r) : r;
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
    float inv_cols;
};

// One 128-value block of y = f * rstd * w per half-warp: scale and bytes of
// the row at q and s.
template <int FMT, bool VEC>
__device__ __forceinline__ void emit_block(uint8_t* q, uint8_t* s, int cols, int c0, int l, float2 (&f)[4], float rstd,
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
    if (c0 >= cols) return;
    if (l == 0) s[c0 >> 7] = (uint8_t)byte;
    store_q8<VEC, FMT>(q, c0, cols, l, f, inv_scale(byte));
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
    allow_next();
    wait_previous();
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
    const float rstd = inv_sqrt(div_by(cta_sum(ss, red), (float)a.cols, p.inv_cols) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) 
        emit_block<FMT, VEC>(a.q + row * a.ldq, a.s + row * a.lds, a.cols, (hw + k * nhw) * 128, l, f[k], rstd, w[k]);
}

// Rows longer than the registers hold: the same steps over the row twice, the
// second time from h (or x), which the first pass left in L2.
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(1024) norm_q8_long_kernel(const NormParams p)
{
    __shared__ float red[32];
    const Q8NormArgs& a = p.a;
    allow_next();
    wait_previous();
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
    const float rstd = inv_sqrt(div_by(cta_sum(ss, red), (float)a.cols, p.inv_cols) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    // a thread reads back the very elements that it wrote; whole warps stay
    // in the loop together (the block maximum is exchanged between lanes)
    for (int base = 0; base < a.cols; base += nhw * 128) {
        const int c0 = base + hw * 128;
        float2 f[4], w[4];
        load8<VEC>(src, c0, a.cols, l, f);
        load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
        emit_block<FMT, VEC>(a.q + row * a.ldq, a.s + row * a.lds, a.cols, c0, l, f, rstd, w);
    }
}

// -------------------------------------------------- streaming over many rows
// Rows in flight.
constexpr int kNormStages = 3;
// Rows over 8192: two in flight, and the weights from memory instead of beside them.
constexpr int bwd_stages(int nv) { return nv > 2 ? 2 : 3; }
constexpr int bwd_own(int nv) { return nv > 2 ? 0 : 4; }
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
    static __host__ __device__ size_t bytes(int threads) { return (size_t)S * NIN * NV * W * threads * 16; }
};

// Steps of one row in elements, and of a grid of rows.
template <typename T>
struct RowPtr {
    const T* p;
    long long step;
    __device__ __forceinline__ RowPtr(const void* base, long long ld, int c)
        : p(reinterpret_cast<const T*>(base) + blockIdx.x * ld + c), step(gridDim.x * ld) {}
};

// cols is a multiple of 8: a thread's chunk lies in the row or past it.  Bound
// by instructions before by memory (70 % of the issue slots with one chunk a
// thread and the row's mean and root by division): hence two chunks a thread,
// which share a row's sum, and pointers that step from row to row.
template <typename T, int FMT, bool RES, int NV, int S>
__global__ void __launch_bounds__(512, NV <= 2 ? 2 : 1) norm_q8_stream_kernel(const NormParams p)
{
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][32];
    const Q8NormArgs& a = p.a;
    allow_next();
    wait_previous();
    const Ring<T, RES ? 2 : 1, NV, S> ring{ring_smem + threadIdx.x};
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    const int cols = a.cols, c = hw * 128 + 8 * l, kstep = nhw * 128;     // chunk k at c + k * kstep
    RowPtr<T> x(a.x, a.ldx, c), r(a.res, a.ldr, c);
    T* h = reinterpret_cast<T*>(a.h) + blockIdx.x * a.ldh;
    uint8_t* q = a.q + blockIdx.x * a.ldq;
    uint8_t* sc = a.s + blockIdx.x * a.lds;
    const long long hstep = gridDim.x * a.ldh, qstep = gridDim.x * a.ldq, sstep = gridDim.x * a.lds;
    float2 w[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k) load_weight<true>(a.w, p.wf32, hw * 128 + k * kstep, cols, l, w[k]);
    auto issue = [&](int row, int slot) {
        if (row < a.rows) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (c + k * kstep >= cols) continue;
                ring.fetch(slot, 0, k, x.p + k * kstep);
                if (RES) ring.fetch(slot, 1, k, r.p + k * kstep);
            }
        }
        x.p += x.step;
        r.p += r.step;
        copy_commit();
    };
    const int grid = gridDim.x;
    long long ahead = blockIdx.x;
#pragma unroll
    for (int s = 0; s < S - 1; ++s, ahead += grid) issue((int)min(ahead, (long long)a.rows), s);
    int slot = 0, flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += grid, ahead += grid) {
        issue((int)min(ahead, (long long)a.rows), slot ? slot - 1 : S - 1);
        copy_wait<S - 1>();
        float2 f[NV][4];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (c + k * kstep < cols) {
                ring.read(slot, 0, k, f[k]);
                if (RES) {
                    float2 g[4];
                    ring.read(slot, 1, k, g);
                    add_rounded<T>(f[k], g);
                    store8<true>(h, hw * 128 + k * kstep, cols, l, f[k]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) f[k][i] = make_float2(0.f, 0.f);
            }
            ss = sum_squares(f[k], ss);
        }
        const float rstd = inv_sqrt(div_by(cta_sum(ss, red[flip]), (float)cols, p.inv_cols) + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) emit_block<FMT, true>(q, sc, cols, hw * 128 + k * kstep, l, f[k], rstd, w[k]);
        h += hstep;
        q += qstep;
        sc += sstep;
        slot = slot + 1 == S ? 0 : slot + 1;
        flip ^= 1;
    }
}

// Streaming launches: chunks a thread, threads of a CTA, CTAs of it on an SM
// (by `room` threads of the kernel's registers and by shared memory: ring_col
// bytes a column in each row in flight, own_col more); ctas = 0: no room.
constexpr size_t kRingRoom = 208 * 1024;        // of an SM's shared memory
struct StreamPlan {
    int nv, threads, ctas;
    size_t smem;
};
int stream_chunks(int cols) { return cols <= 1024 ? 1 : cols <= 8192 ? 2 : 4; }
StreamPlan stream_plan(int cols, int stages, int ring_col, int own_col, int room)
{
    StreamPlan s{};
    s.nv = stream_chunks(cols);
    if (cols > 16384) return s;
    s.threads = (int)cdiv(cols, 256 * s.nv) * 32;
    s.smem = (size_t)(stages * ring_col + own_col) * s.nv * s.threads * 8;
    const int by_regs = (s.nv > 2 ? 512 : room) / s.threads, by_smem = (int)(kRingRoom / (s.smem + 1280));
    s.ctas = by_regs < by_smem ? by_regs : by_smem;
    if (s.ctas > 16) s.ctas = 16;
    if (s.ctas < 1 && by_smem >= 1) s.ctas = 1;
    return s;
}
// It pays once every CTA has several rows to prefetch, and for bfloat16 only:
// a float32 row's own loads keep memory busy, and two of its CTAs' rings fill
// an SM (8192 x 4096 float32: norm 65 us a row a CTA, 99 streamed; gradient 85
// and 138; bfloat16: 61 and 42, gradient 58 and 46).
bool stream_pays(const StreamPlan& s, int rows) { return s.ctas > 0 && rows > 2ll * num_sms() * s.ctas; }

template <typename T, int FMT, bool RES, int NV>
cudaError_t norm_stream(const NormParams& p, const StreamPlan& s, cudaStream_t st)
{
    static std::atomic<unsigned long long> attr{0};
    const cudaError_t e = smem_attr_once((const void*)norm_q8_stream_kernel<T, FMT, RES, NV, kNormStages>, (int)kRingRoom, attr);
    if (e != cudaSuccess) return e;
    return launch_overlapped("rms_norm_q8_stream", norm_q8_stream_kernel<T, FMT, RES, NV, kNormStages>, dim3((unsigned)(num_sms() * s.ctas)),
                  dim3((unsigned)s.threads), s.smem, st, p);
}

template <typename T, int FMT, bool RES>
cudaError_t norm_stream_nv(const NormParams& p, const StreamPlan& s, cudaStream_t st)
{
    if (s.nv == 1) return norm_stream<T, FMT, RES, 1>(p, s, st);
    return s.nv == 2 ? norm_stream<T, FMT, RES, 2>(p, s, st) : norm_stream<T, FMT, RES, 4>(p, s, st);
}

template <typename T, int FMT, bool VEC>
cudaError_t norm_go(const NormParams& p, cudaStream_t st)
{
    const int cols = p.a.cols, blocks = (int)cdiv(cols, 128);
    if constexpr (VEC && sizeof(T) == 2) {
        const StreamPlan s = stream_plan(cols, kNormStages, (p.a.res ? 2 : 1) * (int)sizeof(T), 0, 1024);
        if (cols % 8 == 0 && stream_pays(s, p.a.rows))
            return p.a.res ? norm_stream_nv<T, FMT, true>(p, s, st) : norm_stream_nv<T, FMT, false>(p, s, st);
    }
    const dim3 grid((unsigned)p.a.rows);
    // two half-warps a warp, as many blocks a half-warp as it takes
    if (blocks <= 16)
        return launch_overlapped("rms_norm_q8", norm_q8_kernel<T, FMT, VEC, 1>, grid, dim3((unsigned)cdiv(blocks, 2) * 32), 0, st, p);
    if (blocks <= 128)
        return launch_overlapped("rms_norm_q8", norm_q8_kernel<T, FMT, VEC, 2>, grid, dim3((unsigned)cdiv(blocks, 4) * 32), 0, st, p);
    return launch_overlapped("rms_norm_q8_long", norm_q8_long_kernel<T, FMT, VEC>, grid, dim3(1024), 0, st, p);
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
    float inv_cols;
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
// NV = 4 (rows over 8192): weights and dh are read where they are used.
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) norm_bwd_kernel(const BwdParams p)
{
    __shared__ float red[2][32];
    const NormBwdArgs& a = p.a;
    allow_next();
    wait_previous();
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    float2 dw[NV][4], w[4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[k][i] = make_float2(0.f, 0.f);
    if (NV == 1) load_weight<VEC>(a.w, p.wf32, hw * 128, a.cols, l, w);
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        float2 g[NV][4], xh[NV][4], d[4];
        const T* dh = reinterpret_cast<const T*>(a.dh) + row * a.lddh;
        const float rstd = a.rstd[row];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            load8<VEC>(reinterpret_cast<const T*>(a.dy) + row * a.lddy, (hw + k * nhw) * 128, a.cols, l, g[k]);
            load8<VEC>(reinterpret_cast<const T*>(a.h) + row * a.ldh, (hw + k * nhw) * 128, a.cols, l, xh[k]);
        }
        if (NV == 1 && a.dh) load8<VEC>(dh, hw * 128, a.cols, l, d);
        float c = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (NV > 1) load_weight<VEC>(a.w, p.wf32, (hw + k * nhw) * 128, a.cols, l, w);
            c = bwd_sums(g[k], xh[k], w, rstd, dw[k], c);
        }
        c = div_by(cta_sum(c, red[flip]), (float)a.cols, p.inv_cols);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            bwd_dx(g[k], xh[k], rstd, c);
            if (a.dh) {
                if (NV > 1) load8<VEC>(dh, (hw + k * nhw) * 128, a.cols, l, d);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[k][i] = add2(g[k][i], d[i]);
            }
            store8<VEC>(reinterpret_cast<T*>(a.dx) + row * a.lddx, (hw + k * nhw) * 128, a.cols, l, g[k]);
        }
    }
    store_part<VEC, NV>(a.part + (long long)blockIdx.x * a.cols, a.cols, l, hw, nhw, dw);
}

// The same with the rows' inputs prefetched into shared memory, where the
// thread's weights are as well (in registers they would cost the occupancy
// that the two chunks a thread leave).
template <typename T, bool DH, int NV, int S>
__global__ void __maxnreg__(NV <= 2 ? 80 : 128) norm_bwd_stream_kernel(const BwdParams p)
{
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][32];
    const NormBwdArgs& a = p.a;
    allow_next();
    wait_previous();
    const Ring<T, DH ? 3 : 2, NV, S> ring{ring_smem + threadIdx.x};
    float4* wmine = reinterpret_cast<float4*>(ring_smem + (Ring<T, DH ? 3 : 2, NV, S>::bytes(blockDim.x)) / 16) + threadIdx.x;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4, nhw = blockDim.x >> 4;
    const int cols = a.cols, c = hw * 128 + 8 * l, kstep = nhw * 128;
    RowPtr<T> dy(a.dy, a.lddy, c), h(a.h, a.ldh, c), dh(a.dh, a.lddh, c);
    T* dx = reinterpret_cast<T*>(a.dx) + blockIdx.x * a.lddx;
    const long long dxstep = gridDim.x * a.lddx;
    float2 dw[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (bwd_own(NV)) {
            float2 w[4];
            load_weight<true>(a.w, p.wf32, hw * 128 + k * kstep, cols, l, w);
            wmine[2 * k * blockDim.x] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
            wmine[(2 * k + 1) * blockDim.x] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[k][i] = make_float2(0.f, 0.f);
    }
    auto issue = [&](int row, int slot) {
        if (row < a.rows) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (c + k * kstep >= cols) continue;
                ring.fetch(slot, 0, k, dy.p + k * kstep);
                ring.fetch(slot, 1, k, h.p + k * kstep);
                if (DH) ring.fetch(slot, 2, k, dh.p + k * kstep);
            }
        }
        dy.p += dy.step;
        h.p += h.step;
        if (DH) dh.p += dh.step;
        copy_commit();
    };
    const int grid = gridDim.x;
    long long ahead = blockIdx.x;
#pragma unroll
    for (int s = 0; s < S - 1; ++s, ahead += grid) issue((int)min(ahead, (long long)a.rows), s);
    float rstd = blockIdx.x < a.rows ? a.rstd[blockIdx.x] : 0.f;
    int slot = 0, flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += grid, ahead += grid) {
        issue((int)min(ahead, (long long)a.rows), slot ? slot - 1 : S - 1);
        const float rstd_next = row + grid < a.rows ? a.rstd[row + grid] : 0.f;
        copy_wait<S - 1>();
        float2 g[NV][4], xh[NV][4];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (c + k * kstep < cols) {
                ring.read(slot, 0, k, g[k]);
                ring.read(slot, 1, k, xh[k]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) g[k][i] = xh[k][i] = make_float2(0.f, 0.f);
            }
            float2 w[4];
            if (bwd_own(NV)) {
                const float4 u = wmine[2 * k * blockDim.x], v = wmine[(2 * k + 1) * blockDim.x];
                w[0] = make_float2(u.x, u.y);
                w[1] = make_float2(u.z, u.w);
                w[2] = make_float2(v.x, v.y);
                w[3] = make_float2(v.z, v.w);
            } else {
                load_weight<true>(a.w, p.wf32, hw * 128 + k * kstep, cols, l, w);
            }
            sum = bwd_sums(g[k], xh[k], w, rstd, dw[k], sum);
        }
        const float mean = div_by(cta_sum(sum, red[flip]), (float)cols, p.inv_cols);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (c + k * kstep >= cols) continue;
            bwd_dx(g[k], xh[k], rstd, mean);
            if (DH) {
                float2 d[4];
                ring.read(slot, 2, k, d);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[k][i] = add2(g[k][i], d[i]);
            }
            store8<true>(dx, hw * 128 + k * kstep, cols, l, g[k]);
        }
        dx += dxstep;
        rstd = rstd_next;
        slot = slot + 1 == S ? 0 : slot + 1;
        flip ^= 1;
    }
    store_part<true, NV>(a.part + (long long)blockIdx.x * cols, cols, l, hw, nhw, dw);
}

// Small problems in one launch and without a workspace (dx must not lie over dy
// or h): dw needs no row's sum, so CTAs of their own form it, W columns each
// with the CTA's threads down the rows, beside one CTA a row for dx.  They read
// dy and h a second time, from L2.  A call of 100 x 768 takes 14 us, 22 with a
// workspace and the join; 64 x 4096 on the GPU 2.5 and 4.4.
template <typename T, bool VEC, int W>
__global__ void __launch_bounds__(1024) norm_bwd_small_kernel(const BwdParams p)
{
    __shared__ float red[32];
    __shared__ float t[W][33];
    const NormBwdArgs& a = p.a;
    allow_next();
    wait_previous();
    if (blockIdx.x < a.rows) {
        const long long row = blockIdx.x;
        const int l = threadIdx.x & 15, c0 = (threadIdx.x >> 4) * 128;
        float2 g[4], xh[4], w[4], d[4], dw[4] = {};
        const float rstd = a.rstd[row];
        load8<VEC>(reinterpret_cast<const T*>(a.dy) + row * a.lddy, c0, a.cols, l, g);
        load8<VEC>(reinterpret_cast<const T*>(a.h) + row * a.ldh, c0, a.cols, l, xh);
        load_weight<VEC>(a.w, p.wf32, c0, a.cols, l, w);
        if (a.dh) load8<VEC>(reinterpret_cast<const T*>(a.dh) + row * a.lddh, c0, a.cols, l, d);
        const float c = div_by(cta_sum(bwd_sums(g, xh, w, rstd, dw, 0.f), red), (float)a.cols, p.inv_cols);
        bwd_dx(g, xh, rstd, c);
        if (a.dh) {
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = add2(g[i], d[i]);
        }
        store8<VEC>(reinterpret_cast<T*>(a.dx) + row * a.lddx, c0, a.cols, l, g);
        return;
    }
    const int c1 = (blockIdx.x - a.rows) * W, x = threadIdx.x % W, y = threadIdx.x / W, lanes = blockDim.x / W;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    float s = 0.f;
    if (c1 + x < a.cols) {
        const T* dy = reinterpret_cast<const T*>(a.dy) + c1 + x;
        const T* h = reinterpret_cast<const T*>(a.h) + c1 + x;
#pragma unroll 8
        for (int r = y; r < a.rows; r += lanes) s = fmaf(to_f(dy[r * a.lddy]), __fmul_rn(to_f(h[r * a.ldh]), a.rstd[r]), s);
    }
#pragma unroll
    for (int o = W; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane < W) t[x][warp] = s;
    __syncthreads();
    for (int c = warp; c < W; c += nw) {
        const float v = warp_sum(lane < nw ? t[c][lane] : 0.f);
        if (lane == 0 && c1 + c < a.cols) a.dw[c1 + c] = v;
    }
}

// Rows longer than the registers hold: one row at a time, and the sums of
// dy * xhat in the CTA's row of the workspace instead of in registers.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const BwdParams p)
{
    __shared__ float red[2][32];
    const NormBwdArgs& a = p.a;
    allow_next();
    wait_previous();
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
        const float c = div_by(cta_sum(sum, red[flip]), (float)a.cols, p.inv_cols);
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

// dw = sum of the workspace's rows, always in the same order: W columns a CTA,
// 1024 / W threads down each, joined in the warps and then in shared memory.
// Eight columns (a sector of each row) make enough CTAs of few columns: 16384 x
// 256, 2432 groups, takes 8.9 us with the gradient, 12.2 with 32 columns a CTA;
// 8192 x 4096 47.8 and 45.8.
template <int W>
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float* part, int groups, int cols, float* dw)
{
    __shared__ float t[W][33];
    allow_next();
    wait_previous();
    const int x = threadIdx.x % W, y = threadIdx.x / W, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * W + x;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int r = y; r < groups; r += 1024 / W) s += part[(long long)r * cols + c];
    }
#pragma unroll
    for (int o = W; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane < W) t[x][warp] = s;
    __syncthreads();
    if (warp >= W) return;
    const float v = warp_sum(t[warp][lane]);
    if (lane == 0 && blockIdx.x * W + warp < cols) dw[blockIdx.x * W + warp] = v;
}

// The gradient kernel that keeps one row at a time: threads of a CTA, and row
// groups (the CTAs that run at once, each with a row of the workspace). The
// streaming kernel makes no more of them.
int bwd_threads(int cols)
{
    const int blocks = (int)cdiv(cols, 128);
    return blocks <= 64 ? (int)cdiv(blocks, 2) * 32 : blocks <= 128 ? (int)cdiv(blocks, 8) * 32 : 1024;
}
int bwd_ctas(int cols)
{
    const int n = 1024 / bwd_threads(cols);
    return n < 16 ? n : 16;
}
int bwd_groups(int rows, int cols)
{
    const long long g = (long long)num_sms() * bwd_ctas(cols);
    return (int)(rows < g ? rows : g);
}

template <typename T, bool DH, int NV>
cudaError_t bwd_stream(const BwdParams& p, const StreamPlan& s, cudaStream_t st)
{
    static std::atomic<unsigned long long> attr{0};
    const cudaError_t e = smem_attr_once((const void*)norm_bwd_stream_kernel<T, DH, NV, bwd_stages(NV)>, (int)kRingRoom, attr);
    if (e != cudaSuccess) return e;
    return launch_overlapped("rms_norm_backward_stream", norm_bwd_stream_kernel<T, DH, NV, bwd_stages(NV)>, dim3((unsigned)(num_sms() * s.ctas)),
                  dim3((unsigned)s.threads), s.smem, st, p);
}

template <typename T, bool DH>
cudaError_t bwd_stream_nv(const BwdParams& p, const StreamPlan& s, cudaStream_t st)
{
    if (s.nv == 1) return bwd_stream<T, DH, 1>(p, s, st);
    return s.nv == 2 ? bwd_stream<T, DH, 2>(p, s, st) : bwd_stream<T, DH, 4>(p, s, st);
}

template <typename T, bool VEC>
cudaError_t bwd_small(const BwdParams& p, cudaStream_t st)
{
    const int t = bwd_threads(p.a.cols);
    const dim3 block((unsigned)(t > 512 ? t : 512));
    if (p.a.cols < 1024)
        return launch_overlapped("rms_norm_backward_small", norm_bwd_small_kernel<T, VEC, 8>,
                                 dim3((unsigned)(p.a.rows + cdiv(p.a.cols, 8))), block, 0, st, p);
    return launch_overlapped("rms_norm_backward_small", norm_bwd_small_kernel<T, VEC, 32>,
                             dim3((unsigned)(p.a.rows + cdiv(p.a.cols, 32))), block, 0, st, p);
}

// Launches the gradient over the rows; groups: the rows of the workspace it fills.
template <typename T, bool VEC>
cudaError_t bwd_rows(const BwdParams& p, int& groups, cudaStream_t st)
{
    const int cols = p.a.cols, blocks = (int)cdiv(cols, 128);
    if constexpr (VEC && sizeof(T) == 2) {
        const int nv = stream_chunks(cols);
        StreamPlan s = stream_plan(cols, bwd_stages(nv), (p.a.dh ? 3 : 2) * (int)sizeof(T), bwd_own(nv), 768);
        if (s.ctas > bwd_ctas(cols)) s.ctas = bwd_ctas(cols);
        if (cols % 8 == 0 && stream_pays(s, p.a.rows)) {
            groups = num_sms() * s.ctas;
            return p.a.dh ? bwd_stream_nv<T, true>(p, s, st) : bwd_stream_nv<T, false>(p, s, st);
        }
    }
    groups = bwd_groups(p.a.rows, cols);
    const dim3 grid((unsigned)groups), block((unsigned)bwd_threads(cols));
    if (blocks <= 64) return launch_overlapped("rms_norm_backward", norm_bwd_kernel<T, VEC, 1>, grid, block, 0, st, p);
    if (blocks <= 128) return launch_overlapped("rms_norm_backward", norm_bwd_kernel<T, VEC, 4>, grid, block, 0, st, p);
    return launch_overlapped("rms_norm_backward_long", norm_bwd_long_kernel<T, VEC>, grid, block, 0, st, p);
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
    if (!a.part) return vec ? bwd_small<T, true>(p, st) : bwd_small<T, false>(p, st);
    int groups = 0;
    const cudaError_t err = vec ? bwd_rows<T, true>(p, groups, st) : bwd_rows<T, false>(p, groups, st);
    if (err != cudaSuccess) return err;
    if (a.cols < 1024)
        return launch_overlapped("rms_norm_backward_sum", norm_bwd_sum_kernel<8>, dim3((unsigned)cdiv(a.cols, 8)), dim3(1024), 0, st,
                      (const float*)a.part, groups, a.cols, a.dw);
    return launch_overlapped("rms_norm_backward_sum", norm_bwd_sum_kernel<32>, dim3((unsigned)cdiv(a.cols, 32)), dim3(1024), 0, st,
                  (const float*)a.part, groups, a.cols, a.dw);
}

}  // namespace

cudaError_t rms_norm_q8(const Q8NormArgs& a, dion_dtype dt, dion_q8_format fmt, cudaStream_t st)
{
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const NormParams p{a, a.wdt == DION_F32, 1.f / (float)a.cols};
    return dt == DION_F32 ? norm_typed<float>(p, fmt, st) : norm_typed<bf16>(p, fmt, st);
}

bool norm_backward_small(int rows, int cols)
{
    return cols <= 8192 && rows <= 2048 && (long long)rows * cols <= 1 << 21;
}

size_t norm_backward_workspace(int rows, int cols)
{
    return (size_t)bwd_groups(rows, cols) * (size_t)cols * sizeof(float);
}

cudaError_t rms_norm_backward(const NormBwdArgs& a, dion_dtype dt, cudaStream_t st)
{
    if (a.cols == 0) return cudaSuccess;
    if (a.rows == 0) return cudaMemsetAsync(a.dw, 0, (size_t)a.cols * sizeof(float), st);
    const BwdParams p{a, a.wdt == DION_F32, 1.f / (float)a.cols};
    return dt == DION_F32 ? bwd_typed<float>(p, st) : bwd_typed<bf16>(p, st);
}

}  // namespace dion
