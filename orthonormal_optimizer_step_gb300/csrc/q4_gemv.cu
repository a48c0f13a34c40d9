// q4_gemv.cu -- y = x W^T for a few rows of x and 4-bit weights with group
// scales.
//
// The time is that of reading the weights once, so everything else has to fit
// beside the loads: a lane reads 16 bytes (32 weights) of two rows and needs
// about 1.5 instructions a weight.  The products run on the tensor cores as
// mma.m16n8k16 (16 rows of W against 8 columns, the columns being x's rows): a
// weight q + 8 becomes the bfloat16 128 + (q + 8) by one shift and one logic
// operation, a packed subtraction leaves q, exactly, and products of it with
// bfloat16 x are exact in the float32 accumulator.  The held layout puts a
// lane's operands of eight such products into its 16 bytes and keeps each
// product inside one group, whose scale then multiplies the accumulated sum.
// x float32 goes in as three bfloat16 terms in columns of their own, 8-bit rows
// as the bfloat16 they are exactly.
//
// A CTA takes 64 rows of W, a warp 16 of them.  Where these are too few CTAs to
// fill the GPU, a cluster of up to eight splits the contraction and joins
// through distributed shared memory, in the order of the shares.
#include <algorithm>

#include "q4.cuh"

namespace dion {

int num_sms();

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kRows = 16 * kWarps;
constexpr int kBatch = 4;                    // chunks that a warp loads together, while it works on as many

struct MatParams {
    int m, n, k;
    int tokens, terms;                       // rows of x a pass, columns each of them takes
    int chunks, per, panel;                  // of the contraction; a share's; those whose x is held at once
    dion_x_type xt;
    const void* x; long long ldx;
    const uint8_t* sx; long long ldsx;
    int x_wide;                              // x's rows start on 16-byte boundaries
    const uint8_t* q; long long ldq;
    const bf16* s; long long lds;
    int groups, s_wide;                      // scale rows start on boundaries of a batch's scales
    void* y; long long ldy; int y_f32;
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pairs (columns 2 i, 2 i + 1) of a held word as bfloat16.
template <int I>
__device__ __forceinline__ uint32_t weights2(uint32_t w)
{
    uint32_t v = ((w >> (4 * I)) & 0x000f000fu) | 0x43004300u, r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x43084308u));   // 128 + 8
    return r;
}

// Weights are read once: they pass L1 by.
__device__ __forceinline__ uint4 load_once(const uint8_t* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float load_remote(const float* p, uint32_t rank)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// 2^(byte - 127), NaN for byte 255.
__device__ __forceinline__ float power_of(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7fc00000u) : byte ? __uint_as_float(byte << 23) : 0x1p-127f;
}

// Eight columns of x from col on as bfloat16 (three terms of float32), zeros past k.
__device__ __forceinline__ void load_x(const MatParams& p, int row, int col, uint4 (&out)[3])
{
    float2 f[4];
    const bool whole = p.x_wide && col + 8 <= p.k;
    if (p.xt == DION_X_BF16) {
        const bf16* r = (const bf16*)p.x + row * p.ldx + col;
        if (whole) {
            out[0] = *reinterpret_cast<const uint4*>(r);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(col + 2 * i < p.k ? to_f(r[2 * i]) : 0.f, col + 2 * i + 1 < p.k ? to_f(r[2 * i + 1]) : 0.f);
    } else if (p.xt == DION_X_F32) {
        const float* r = (const float*)p.x + row * p.ldx + col;
        if (whole) {
            q8::Raw8<float> v;
            v.u[0] = reinterpret_cast<const uint4*>(r)[0];
            v.u[1] = reinterpret_cast<const uint4*>(r)[1];
            q8::unpack8(v, f);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = make_float2(col + 2 * i < p.k ? r[2 * i] : 0.f, col + 2 * i + 1 < p.k ? r[2 * i + 1] : 0.f);
        }
    } else {
        const uint8_t* r = (const uint8_t*)p.x + row * p.ldx + col;
        uint32_t w[2] = {0, 0};
        if (col + 8 <= p.k) {                // (8-bit rows are aligned)
            const uint2 v = *reinterpret_cast<const uint2*>(r);
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < p.k) w[i >> 2] |= (uint32_t)r[i] << (8 * (i & 3));
        }
        const float s = col < p.k ? power_of(p.sx[row * p.ldsx + col / 128]) : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint16_t b = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            uint32_t h;
            if (p.xt == DION_X_E4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
            else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(b));
            float2 v;
            asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
                : "=f"(v.x), "=f"(v.y)
                : "r"(h));
            f[i] = q8::mul2(v, make_float2(s, s));
        }
    }
    q8::Raw8<bf16> t;
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        q8::pack8(t, f);
        out[e] = t.u[0];
        if (p.terms == 1) break;
        float2 h[4];
        q8::unpack8(t, h);
        // what the term leaves (an infinity or NaN leaves nothing)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i].x = q8::mag_bits(h[i].x) < q8::kInfBits ? f[i].x - h[i].x : 0.f;
            f[i].y = q8::mag_bits(h[i].y) < q8::kInfBits ? f[i].y - h[i].y : 0.f;
        }
    }
}

// What a warp loads together: weights of rows g and g + 8 and their scales.
template <int GROUP>
struct Batch {
    static constexpr int S = 128 / GROUP;    // scales of a chunk
    uint4 w[kBatch][2];
    uint32_t s[2][kBatch * S / 2];           // two scales a word
};

template <int GROUP>
__device__ __forceinline__ void load_batch(const MatParams& p, Batch<GROUP>& b, const uint8_t* const (&q)[2],
                                           const bf16* const (&s)[2], int c, int end)
{
    constexpr int S = 128 / GROUP;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
        if (c + u < end) {
            b.w[u][0] = load_once(q[0] + 64ll * (c + u));
            b.w[u][1] = load_once(q[1] + 64ll * (c + u));
        }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const bf16* at = s[r] + (long long)c * S;
        if (p.s_wide && (c + kBatch) * S <= p.groups) {
            if constexpr (S == 1) {
                const uint2 v = *reinterpret_cast<const uint2*>(at);
                b.s[r][0] = v.x;
                b.s[r][1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < S / 2; ++i) {
                    const uint4 v = reinterpret_cast<const uint4*>(at)[i];
                    b.s[r][4 * i] = v.x;
                    b.s[r][4 * i + 1] = v.y;
                    b.s[r][4 * i + 2] = v.z;
                    b.s[r][4 * i + 3] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kBatch * S / 2; ++i) {
                const uint16_t* u = reinterpret_cast<const uint16_t*>(at) + 2 * i;
                const int left = p.groups - c * S - 2 * i;
                b.s[r][i] = (left > 0 ? u[0] : 0u) | (left > 1 ? (uint32_t)u[1] << 16 : 0u);
            }
        }
    }
}

template <int MB, int GROUP>
__device__ __forceinline__ void chunk_products(const Batch<GROUP>& b, int u, const uint8_t* xs, int xpitch, const bool (&has)[MB],
                                               float (&acc)[MB][4])
{
    constexpr int S = 128 / GROUP;
    float sum[MB][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w0 = j == 0 ? b.w[u][0].x : j == 1 ? b.w[u][0].y : j == 2 ? b.w[u][0].z : b.w[u][0].w;
        const uint32_t w1 = j == 0 ? b.w[u][1].x : j == 1 ? b.w[u][1].y : j == 2 ? b.w[u][1].z : b.w[u][1].w;
        const uint32_t a0[4] = {weights2<0>(w0), weights2<1>(w0), weights2<2>(w0), weights2<3>(w0)};
        const uint32_t a1[4] = {weights2<0>(w1), weights2<1>(w1), weights2<2>(w1), weights2<3>(w1)};
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            if (j * 32 % GROUP == 0) sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.f;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (has[i]) x = *reinterpret_cast<const uint4*>(xs + 8 * i * xpitch + 64 * j);
            mma(sum[i], a0[0], a1[0], a0[1], a1[1], x.x, x.y);
            mma(sum[i], a0[2], a1[2], a0[3], a1[3], x.z, x.w);
            if ((j + 1) * 32 % GROUP == 0) {
                const int e = u * S + j * 32 / GROUP;
                const uint32_t v0 = b.s[0][e / 2], v1 = b.s[1][e / 2];
                const float s0 = __uint_as_float(e & 1 ? v0 & 0xffff0000u : v0 << 16);
                const float s1 = __uint_as_float(e & 1 ? v1 & 0xffff0000u : v1 << 16);
                acc[i][0] = fmaf(s0, sum[i][0], acc[i][0]);
                acc[i][1] = fmaf(s0, sum[i][1], acc[i][1]);
                acc[i][2] = fmaf(s1, sum[i][2], acc[i][2]);
                acc[i][3] = fmaf(s1, sum[i][3], acc[i][3]);
            }
        }
    }
}

template <int MB, int GROUP>
__global__ void __launch_bounds__(kThreads) q4_matmul_kernel(const MatParams p, const int shares)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int share = shares > 1 ? (int)cluster_rank() : 0;
    const int row0 = (int)(blockIdx.x / shares) * kRows, token0 = blockIdx.y * p.tokens;
    const int tokens = min(p.tokens, p.m - token0), cols = tokens * p.terms;
    const int xpitch = 256 * p.panel + 64;   // bytes; eight rows' 16-byte words then meet no bank twice
    float* sums = (float*)(smem + p.tokens * p.terms * xpitch);   // [column][row of W]
    const int c0 = share * p.per, c1 = min(c0 + p.per, p.chunks);
    const bool active = row0 + 16 * warp < p.n;
    const int r0 = min(row0 + 16 * warp + g, p.n - 1), r1 = min(row0 + 16 * warp + g + 8, p.n - 1);
    const uint8_t* const q[2] = {p.q + r0 * p.ldq + 16 * t, p.q + r1 * p.ldq + 16 * t};
    const bf16* const s[2] = {p.s + r0 * p.lds, p.s + r1 * p.lds};
    bool has[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) has[i] = 8 * i + g < cols;
    float acc[MB][4] = {};
    wait_previous();
    allow_next();
    for (int pc = c0; pc < c1; pc += p.panel) {
        const int pe = min(pc + p.panel, c1);
        Batch<GROUP> b[2];
        if (active) load_batch(p, b[0], q, s, pc, pe);
        if (pc > c0) __syncthreads();        // the last panel's x has been read
        const int units = 16 * (pe - pc);    // of eight columns
        for (int i = threadIdx.x; i < tokens * units; i += kThreads) {
            const int row = i / units, u = i - row * units;
            uint4 v[3];
            load_x(p, token0 + row, 128 * pc + 8 * u, v);
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < p.terms) *reinterpret_cast<uint4*>(smem + (row * p.terms + e) * xpitch + 16 * u) = v[e];
        }
        __syncthreads();
        if (active) {
            const uint8_t* xs = smem + g * xpitch + 16 * t;
#pragma unroll 1
            for (int c = pc; c < pe; c += 2 * kBatch) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = c + h * kBatch;
                    if (at >= pe) break;
                    if (at + kBatch < pe) load_batch(p, b[h ^ 1], q, s, at + kBatch, pe);
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        if (at + u >= pe) break;
                        chunk_products<MB, GROUP>(b[h], u, xs + 256 * (at + u - pc), xpitch, has, acc);
                    }
                }
            }
        }
    }
    if (active) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = 8 * i + 2 * t + (e & 1);
                if (col < cols) sums[col * kRows + 16 * warp + g + 8 * (e >> 1)] = acc[i][e];
            }
    }
    if (shares > 1) cluster_sync();
    else __syncthreads();
    for (int i = share * kThreads + threadIdx.x; i < tokens * kRows; i += shares * kThreads) {
        const int row = i / kRows, r = i % kRows;
        if (row0 + r >= p.n) continue;
        float v = 0.f;
        for (int e = 0; e < p.terms; ++e) {
            const float* at = sums + (row * p.terms + e) * kRows + r;
            if (shares == 1) v += *at;
            else
                for (int h = 0; h < shares; ++h) v += load_remote(at, h);
        }
        const long long o = (token0 + row) * p.ldy + row0 + r;
        if (p.y_f32) ((float*)p.y)[o] = v;
        else ((bf16*)p.y)[o] = __float2bfloat16_rn(v);
    }
    if (shares > 1) cluster_sync();          // the others have read this CTA's sums
}

// Shares of the contraction (CTAs of a cluster): as many as it takes for three
// CTAs an SM, each with whole batches of chunks.
int shares_of(long long row_blocks, int chunks, int& per)
{
    int s = (int)std::min<long long>(8, cdiv(3ll * num_sms(), row_blocks));
    s = std::max(1, std::min(s, (int)cdiv(chunks, kBatch)));
    per = (int)(cdiv(cdiv(chunks, s), kBatch) * kBatch);
    return (int)cdiv(chunks, per);
}

constexpr int kPanelBytes = 65536;           // of x held at once

template <int MB, int GROUP>
cudaError_t go(MatParams& p, int shares, cudaStream_t st)
{
    static std::atomic<unsigned long long> attr{0};
    const int cols = p.tokens * p.terms;
    const size_t smem = (size_t)cols * (256 * p.panel + 64) + (size_t)cols * kRows * sizeof(float);
    cudaError_t e = smem_attr_once((const void*)q4_matmul_kernel<MB, GROUP>, 2 * kPanelBytes, attr);
    if (e != cudaSuccess) return e;
    return launch_cluster("q4_matmul", q4_matmul_kernel<MB, GROUP>,
                          dim3((unsigned)(cdiv(p.n, kRows) * shares), (unsigned)cdiv(p.m, p.tokens)), dim3(kThreads), shares, smem, st, p,
                          shares);
}

template <int GROUP>
cudaError_t pick(MatParams& p, cudaStream_t st)
{
    const int shares = shares_of(cdiv(p.n, kRows), p.chunks, p.per);
    const int cols = p.tokens * p.terms;
    p.panel = std::min(p.per, std::max(kBatch, kPanelBytes / (256 * cols) / kBatch * kBatch));
    if (cols <= 8) return go<1, GROUP>(p, shares, st);
    if (cols <= 16) return go<2, GROUP>(p, shares, st);
    return go<4, GROUP>(p, shares, st);
}

}  // namespace

cudaError_t q4_matmul(const Q4MatArgs& a, cudaStream_t st)
{
    if (a.m == 0 || a.w.rows == 0) return cudaSuccess;
    if (a.w.cols == 0) {
        const size_t e = a.ydt == DION_F32 ? 4 : 2;
        return cudaMemset2DAsync(a.y, (size_t)a.ldy * e, 0, (size_t)a.w.rows * e, (size_t)a.m, st);
    }
    MatParams p{};
    p.m = a.m; p.n = a.w.rows; p.k = a.w.cols;
    p.terms = a.xt == DION_X_F32 ? 3 : 1;
    p.tokens = std::min(a.m, 32 / p.terms);
    p.chunks = (int)cdiv(p.k, 128);
    p.xt = a.xt; p.x = a.x; p.ldx = a.ldx; p.sx = a.sx; p.ldsx = a.ldsx;
    p.x_wide = (uintptr_t)a.x % 16 == 0 && a.ldx * (a.xt == DION_X_F32 ? 4 : 2) % 16 == 0;
    p.q = a.w.q; p.ldq = a.w.ldq;
    p.s = a.w.s; p.lds = a.w.lds;
    p.groups = (int)cdiv(p.k, a.w.group);
    const int wide = std::min(16, 8 * 128 / a.w.group);            // bytes of a batch's scales that are loaded at once
    p.s_wide = (uintptr_t)a.w.s % wide == 0 && a.w.lds * 2 % wide == 0;
    p.y = a.y; p.ldy = a.ldy; p.y_f32 = a.ydt == DION_F32;
    return a.w.group == 32 ? pick<32>(p, st) : a.w.group == 64 ? pick<64>(p, st) : pick<128>(p, st);
}

}  // namespace dion
