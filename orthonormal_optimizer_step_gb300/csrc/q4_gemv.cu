// q4_gemv.cu -- y = x W^T for a few rows of x and 4-bit weights with group
// scales.
//
// The time is that of reading the weights once, so everything else has to fit
// beside the loads: a lane reads 16 bytes (32 weights) of two rows and has about
// 1.9 instructions a weight if the memory is not to wait.  The products run on
// the tensor cores as mma.m16n8k16 (16 rows of W against 8 columns, the columns
// being x's rows): a weight q + 8 becomes the float16 1024 + (q + 8) or, four bits
// higher, 1024 + 16 (q + 8) by one logic operation, and a packed addition or
// multiply-add leaves q, exactly: 9 instructions for eight weights (bfloat16, whose
// mantissa has no room for the higher place, takes 11).  The held layout puts a
// lane's operands of eight such products into its 16 bytes and keeps each product
// inside one group, whose scale then multiplies the accumulated sum.
//
// x enters as float16 times a power of two for each row and 128 columns, its
// largest value there in [2^14, 2^15): bfloat16 exactly (down to 2^-31 of that
// largest value, within 2^-39 of it below), 8-bit rows exactly with the scale that
// they have, and float32 as two terms (within 2^-24, and 2^-39 of the largest) in
// columns of their own.  Products of such operands are exact in the float32
// accumulator.
//
// Tiles are 16 rows of W.  Weights and scales go to shared memory by
// asynchronous copies, each lane its own 16 bytes, two batches of four chunks
// (8 KB a warp) ahead through all of a warp's tiles: no register waits for them
// and no barrier hands them over.  The eight warps of a CTA share a tile's
// contraction or take tiles of their own, and the CTAs of a cluster share it too
// where the tiles are few or x is too large for one CTA's shared memory; sums
// are joined in the order of the shares, through distributed shared memory
// between CTAs.
//
// Measured: 1 x 53248 x 16384 in 77 us, 5.8 TB/s (0.86 of a copy's rate); 1 x 4096
// x 4096 in 4.9, of which its weights' time is 1.3 and a launch's start, x and a
// tile's latency the rest; 16 x 4096 x 14336 of 8-bit rows in 17.5 (weights 4.7):
// each CTA converts its 57000 values of x, and joins.
#include <algorithm>

#include "q4.cuh"

namespace dion {

int num_sms();

namespace {

constexpr int kUnit = 4;                     // shares of the contraction are multiples of these chunks

// How a kernel of 8 MB columns is laid out.
template <int MB>
struct Cfg {
    static constexpr int WARPS = MB == 2 ? 12 : 8, THREADS = 32 * WARPS;
    static constexpr int CTAS = MB == 1 ? 2 : 1;                   // an SM
    static constexpr int BATCH = MB == 1 ? 4 : 2;                  // chunks that a warp copies together
    static constexpr int AHEAD = 2;          // batches in flight
};

constexpr int kMostShared = 225 * 1024;       // bytes of a CTA

struct MatParams {
    int m, n, k;
    int tokens, terms;                       // rows of x a pass, columns each of them takes
    int chunks, per;                         // of the contraction; a CTA's share of them
    int split;                               // warps that share a tile
    int blocks, held;                        // blocks of warps / split tiles; those whose sums wait for a join
    dion_x_type xt;
    const void* x; long long ldx;
    const uint8_t* sx; long long ldsx;
    int x_wide;                              // x's rows start on 16-byte boundaries
    const uint8_t* q; long long ldq;
    const bf16* s; long long lds;
    int groups, s_wide;               // scale rows start on 4-byte boundaries
    void* y; long long ldy; int y_f32;
};

// d = A B, or d + A B.
template <bool ADD>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (ADD)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Pairs (columns 0 and 1, 2 and 3) of the low bytes of a held word's halves as float16.
__device__ __forceinline__ void weights4(uint32_t w, uint32_t& p0, uint32_t& p1)
{
    uint32_t a, b;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(a) : "r"(w), "r"(0x000f000fu), "r"(0x64006400u));   // (w & mask) | 1024
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(b) : "r"(w), "r"(0x00f000f0u), "r"(0x64006400u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p0) : "r"(a), "r"(0x64086408u));                          // 1024 + 8
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p1) : "r"(b), "r"(0x2c002c00u), "r"(0xd480d480u));    // / 16, - (64 + 8)
}

// Asynchronous copies to shared memory (weights are read once and pass L1 by).
__device__ __forceinline__ void copy16(uint32_t to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the last `LEFT` groups are here.
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

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

// x comes in two steps, a thread doing both for its units of eight columns:
// copied as it is to the place of its float16 (8, 16 or, in two terms' places, 32
// bytes), then converted there.  All copies are issued before the first weights:
// behind the weights in flight a load of x takes as long as they do (8 rows of
// 14336x4096 took 4 us longer than one).
template <int XT, int THREADS>
__device__ __forceinline__ void copy_x(const MatParams& p, int token0, int tokens, int c0, int c1, uint8_t* xs, int xpitch,
                                       uint32_t magic)
{
    constexpr int TERMS = XT == DION_X_F32 ? 2 : 1, BYTES = XT == DION_X_F32 ? 32 : XT == DION_X_BF16 ? 16 : 8;
    const int units = 16 * (c1 - c0), all = tokens * units;
    for (int i = threadIdx.x; i < all; i += THREADS) {
        const int row = (int)__umulhi(i, magic), u = i - row * units, col = 128 * c0 + 8 * u, left = p.k - col;
        uint8_t* to = xs + row * TERMS * xpitch + 16 * u;
        const uint8_t* from = (const uint8_t*)p.x + ((token0 + row) * p.ldx + col) * (BYTES / 8);
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(to);
        if (left >= 8 && (BYTES == 8 || p.x_wide)) {               // (8-bit rows are aligned)
            if (BYTES == 8) {
                copy8(d, from);
            } else {
                copy16(d, from);
                if (BYTES == 32) copy16(d + xpitch, from + 16);
            }
        } else {                                                   // zeros past k
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint8_t* at = to + (BYTES == 32 ? (e >> 2) * xpitch + 4 * (e & 3) : BYTES / 8 * e);
                if (BYTES == 32) *reinterpret_cast<uint32_t*>(at) = e < left ? reinterpret_cast<const uint32_t*>(from)[e] : 0u;
                else if (BYTES == 16) *reinterpret_cast<uint16_t*>(at) = e < left ? reinterpret_cast<const uint16_t*>(from)[e] : 0;
                else *at = e < left ? from[e] : 0;
            }
        }
    }
}

__device__ __forceinline__ uint32_t half2_of(float2 v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
    return r;
}
__device__ __forceinline__ float2 floats_of(uint32_t h)
{
    float2 v;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "r"(h));
    return v;
}

// A unit of plain x to float16, in place; returns the power of two that it is to
// be multiplied by.  The 16 lanes of a half-warp hold a row's 128 columns.
template <int XT>
__device__ __forceinline__ float convert_x(uint8_t* at, int pitch)
{
    float2 f[4];
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    if constexpr (XT == DION_X_BF16) {
        f[0] = q8::unpack2(v.x);
        f[1] = q8::unpack2(v.y);
        f[2] = q8::unpack2(v.z);
        f[3] = q8::unpack2(v.w);
    } else {
        q8::Raw8<float> r;
        r.u[0] = v;
        r.u[1] = *reinterpret_cast<const uint4*>(at + pitch);
        q8::unpack8(r, f);
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) amax = max(amax, max(q8::finite_mag_bits(f[i].x), q8::finite_mag_bits(f[i].y)));
    const uint32_t half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = max(amax, __shfl_xor_sync(half, amax, o));
    // 2^-e takes amax into [2^14, 2^15); below 2^-112 it stays 2^126, which takes float32's least numbers to 2^-23
    const uint32_t e = max(amax >> 23, 15u);                       // biased: e - 14 + 127 is e's
    const float down = __uint_as_float((268u - e) << 23), up = __uint_as_float((e - 14u) << 23);
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 w = q8::mul2(f[i], make_float2(down, down));
        h[i] = half2_of(w);
        if (XT == DION_X_F32) {
            const float2 a = floats_of(h[i]);
            // what the first term leaves (an infinity or NaN leaves nothing)
            l[i] = half2_of(make_float2(q8::mag_bits(a.x) < q8::kInfBits ? w.x - a.x : 0.f,
                                        q8::mag_bits(a.y) < q8::kInfBits ? w.y - a.y : 0.f));
        }
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
    if (XT == DION_X_F32) *reinterpret_cast<uint4*>(at + pitch) = make_uint4(l[0], l[1], l[2], l[3]);
    return up;
}
// A unit of 8-bit x.
template <int XT>
__device__ __forceinline__ void widen_x(uint8_t* at)
{
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t b = (uint16_t)((i < 2 ? v.x : v.y) >> (16 * (i & 1)));
        if (XT == DION_X_E4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[i]) : "h"(b));
        else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h[i]) : "h"(b));
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
}

// What copy_x brought, converted by the threads that copied it; powers: [chunk][column].
template <int XT, int THREADS>
__device__ __forceinline__ void convert_all(int tokens, int c0, int c1, uint8_t* xs, int xpitch, float* powers, int columns,
                                            uint32_t magic)
{
    constexpr int TERMS = XT == DION_X_F32 ? 2 : 1;
    const int units = 16 * (c1 - c0), all = tokens * units;
#pragma unroll 2
    for (int i = threadIdx.x; i < all; i += THREADS) {             // (whole half-warps)
        const int row = (int)__umulhi(i, magic), u = i - row * units;
        uint8_t* at = xs + row * TERMS * xpitch + 16 * u;
        if constexpr (XT == DION_X_F32 || XT == DION_X_BF16) {
            const float up = convert_x<XT>(at, xpitch);
            if (u % 16 < TERMS) powers[u / 16 * columns + row * TERMS + u % 16] = up;
        } else {
            widen_x<XT>(at);
        }
    }
}

// A batch in shared memory: [chunk][row g or g + 8][lane] 16 bytes of weights,
// then [row of the tile] the batch's scales.
template <int GROUP, int BATCH>
struct Batch {
    static constexpr int S = 128 / GROUP;                          // scales of a chunk
    static constexpr int ROW = BATCH * S * 2;                     // bytes of a row's scales
    // a row's distance: eight rows' scales then lie in different banks
    static constexpr int PITCH = ROW + (GROUP == 32 ? 8 : 4);
    static constexpr int WEIGHTS = BATCH * 1024, BYTES = WEIGHTS + 16 * PITCH;
    static_assert(BYTES % 16 == 0 && ROW % 4 == 0, "whole words");
};

// Where a warp copies from next: its lanes' places in rows g and g + 8 of a tile.
struct Place {
    const uint8_t* q[2];
    const bf16* s[2];
};
// to: the batch's place; c: its first chunk, of which those before `end` exist.
template <int GROUP, int BATCH>
__device__ __forceinline__ void copy_batch(const MatParams& p, uint8_t* to, const Place& at, int c, int end, int lane)
{
    using B = Batch<GROUP, BATCH>;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t w = (uint32_t)__cvta_generic_to_shared(to) + 16 * lane;
    const bool whole = c + BATCH <= end;
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
        if (whole || c + u < end) {
            copy16(w + 1024 * u, at.q[0] + 64 * u);
            copy16(w + 1024 * u + 512, at.q[1] + 64 * u);
        }
    uint8_t* s = to + B::WEIGHTS + g * B::PITCH;
    constexpr int WORDS = B::ROW / 4;                              // of two scales: 1 to 8
    if (p.s_wide && (c + BATCH) * B::S <= p.groups) {
#pragma unroll
        for (int i = 0; i < (WORDS + 3) / 4; ++i)
            if (WORDS >= 4 || t < WORDS) {
                const uint32_t d = (uint32_t)__cvta_generic_to_shared(s) + 4 * t + 16 * i;
                copy4(d, (const uint8_t*)at.s[0] + 4 * t + 16 * i);
                copy4(d + 8 * B::PITCH, (const uint8_t*)at.s[1] + 4 * t + 16 * i);
            }
    } else {
#pragma unroll
        for (int i = 0; i < (WORDS + 3) / 4; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int e = 2 * t + 8 * i, left = p.groups - c * B::S - e;
                const uint16_t* u = reinterpret_cast<const uint16_t*>(at.s[r]) + e;
                const uint32_t v = (left > 0 ? u[0] : 0u) | (left > 1 ? (uint32_t)u[1] << 16 : 0u);
                if (WORDS >= 4 || t < WORDS) *reinterpret_cast<uint32_t*>(s + 8 * r * B::PITCH + 2 * e) = v;
            }
    }
}

// acc += the products of a chunk.  w: the lane's 16 bytes of row g, those of row g + 8 512 bytes on; s: row g's
// scales of the chunk, row g + 8's eight rows on; xs: the lane's place in the chunk, columns: of its columns,
// powers: in its powers of two.
template <int MB, int GROUP, class B>
__device__ __forceinline__ void chunk_products(const uint8_t* w, const uint8_t* s, const uint8_t* xs, const int (&columns)[MB],
                                               const float* powers, float (&acc)[MB][4])
{
    const uint4 q0 = *reinterpret_cast<const uint4*>(w), q1 = *reinterpret_cast<const uint4*>(w + 512);
    uint32_t sw[2][(B::S + 1) / 2];                                // two scales a word
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint8_t* at = s + 8 * r * B::PITCH;
        if constexpr (B::S == 1) sw[r][0] = *reinterpret_cast<const uint16_t*>(at);
        else if constexpr (B::S == 2) sw[r][0] = *reinterpret_cast<const uint32_t*>(at);
        else {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            sw[r][0] = v.x;
            sw[r][1] = v.y;
        }
    }
    float sum[MB][4], scaled[MB][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w0 = j == 0 ? q0.x : j == 1 ? q0.y : j == 2 ? q0.z : q0.w;
        const uint32_t w1 = j == 0 ? q1.x : j == 1 ? q1.y : j == 2 ? q1.z : q1.w;
        uint32_t a[2][4];                    // rows g and g + 8, columns 0 1 and 2 3; then 4 5 and 6 7
        weights4(w0, a[0][0], a[0][2]);
        weights4(w1, a[0][1], a[0][3]);
        weights4(w0 >> 8, a[1][0], a[1][2]);
        weights4(w1 >> 8, a[1][1], a[1][3]);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(xs + columns[i] + 64 * j);
            if (j * 32 % GROUP == 0) mma<false>(sum[i], a[0], x.x, x.y);
            else mma<true>(sum[i], a[0], x.x, x.y);
            mma<true>(sum[i], a[1], x.z, x.w);
            if ((j + 1) * 32 % GROUP == 0) {
                constexpr int PER = GROUP / 32;
                const int e = j / PER;
                const uint32_t v0 = sw[0][e / 2], v1 = sw[1][e / 2];
                const float s0 = __uint_as_float(e & 1 ? v0 & 0xffff0000u : v0 << 16);
                const float s1 = __uint_as_float(e & 1 ? v1 & 0xffff0000u : v1 << 16);
                if (j * 32 < GROUP) {
                    scaled[i][0] = s0 * sum[i][0];
                    scaled[i][1] = s0 * sum[i][1];
                    scaled[i][2] = s1 * sum[i][2];
                    scaled[i][3] = s1 * sum[i][3];
                } else {
                    scaled[i][0] = fmaf(s0, sum[i][0], scaled[i][0]);
                    scaled[i][1] = fmaf(s0, sum[i][1], scaled[i][1]);
                    scaled[i][2] = fmaf(s1, sum[i][2], scaled[i][2]);
                    scaled[i][3] = fmaf(s1, sum[i][3], scaled[i][3]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const float2 up = *reinterpret_cast<const float2*>(powers + 8 * i);
        acc[i][0] = fmaf(up.x, scaled[i][0], acc[i][0]);
        acc[i][1] = fmaf(up.y, scaled[i][1], acc[i][1]);
        acc[i][2] = fmaf(up.x, scaled[i][2], acc[i][2]);
        acc[i][3] = fmaf(up.y, scaled[i][3], acc[i][3]);
    }
}

// Sums of a cluster's held blocks, to y: CTA `share` adds its part of them.
template <int THREADS>
__device__ __forceinline__ void join(const MatParams& p, const float* hold, int first, int step, int count, int shares, int share,
                                     int token0, int tokens)
{
    const int tiles = THREADS / 32 / p.split, cols = p.tokens * p.terms;
    cluster_sync();
    for (int i = share * THREADS + threadIdx.x; i < count * tiles * tokens * 16; i += shares * THREADS) {
        const int r = i & 15, token = i / 16 % tokens, tile = i / 16 / tokens;      // tile: of all held ones
        const int row = ((first + tile / tiles * step) * tiles + tile % tiles) * 16 + r;
        if (row >= p.n) continue;
        float v = 0.f;
        for (int e = 0; e < p.terms; ++e)
            for (int h = 0; h < shares; ++h) v += load_remote(hold + (tile * cols + token * p.terms + e) * 16 + r, h);
        const long long o = (token0 + token) * p.ldy + row;
        if (p.y_f32) ((float*)p.y)[o] = v;
        else ((bf16*)p.y)[o] = __float2bfloat16_rn(v);
    }
    cluster_sync();                          // the others have read this CTA's sums
}

template <int MB, int GROUP>
__global__ void __launch_bounds__(Cfg<MB>::THREADS, Cfg<MB>::CTAS) q4_matmul_kernel(const MatParams p, const int shares)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int share = shares > 1 ? (int)cluster_rank() : 0;
    const int first = blockIdx.x / shares, step = gridDim.x / shares, token0 = blockIdx.y * p.tokens;
    const int tokens = min(p.tokens, p.m - token0), cols = tokens * p.terms, most = p.tokens * p.terms;
    const int xpitch = 256 * p.per + 64;     // bytes; eight rows' 16-byte words then meet no bank twice
    constexpr int kWarps = Cfg<MB>::WARPS, kBatch = Cfg<MB>::BATCH, kAhead = Cfg<MB>::AHEAD, kThreads = Cfg<MB>::THREADS;
    using B = Batch<GROUP, kBatch>;
    uint8_t* ring = smem + warp * (kAhead * B::BYTES);           // [batch in flight], this warp's
    uint8_t* xall = smem + kWarps * kAhead * B::BYTES;           // [column][xpitch]
    float* powers = (float*)(xall + most * xpitch);              // [chunk][8 MB columns]
    float* parts = powers + p.per * 8 * MB;                      // [2][warp][column][16]: a warp's sums of a tile
    float* hold = parts + 2 * kWarps * most * 16;                // [held][tile of the block][column][16]
    const int c0 = share * p.per, c1 = min(c0 + p.per, p.chunks);
    // this warp's tile of a block, and its share of the CTA's chunks in whole batches (it may have none)
    const int tiles = kWarps / p.split, mine = warp / p.split, part = warp % p.split;
    const int each = (c1 - c0 + p.split * kBatch - 1) / (p.split * kBatch) * kBatch;
    const int w0 = min(c0 + part * each, c1), w1 = min(w0 + each, c1);
    const int batches = max(1, (w1 - w0 + kBatch - 1) / kBatch);
    // this lane's columns (past the last one, that one again: nothing reads their sums)
    int columns[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) columns[i] = min(8 * i + g, cols - 1) * xpitch;
    wait_previous();
    allow_next();

    int lb = first, li = 0;                  // block and batch that are copied next
    Place at;
    auto copy_next = [&](int slot) {
        if (lb < p.blocks) {
            if (li == 0) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = min(16 * (lb * tiles + mine) + g + 8 * r, p.n - 1);
                    at.q[r] = p.q + row * p.ldq + 64ll * w0 + 16 * t;
                    at.s[r] = p.s + row * p.lds + (long long)w0 * B::S;
                }
            }
            copy_batch<GROUP, kBatch>(p, ring + slot * B::BYTES, at, w0 + li * kBatch, w1, lane);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                at.q[r] += 64 * kBatch;
                at.s[r] += kBatch * B::S;
            }
            if (++li == batches) {
                li = 0;
                lb += step;
            }
        }
        copies_end();                        // (an empty group keeps the count)
    };
    const uint32_t magic = 0xffffffffu / (16 * (c1 - c0)) + 1;     // quotients by a row's units as products: exact below 2^32 / units
    if (p.xt == DION_X_BF16) copy_x<DION_X_BF16, kThreads>(p, token0, tokens, c0, c1, xall, xpitch, magic);
    else if (p.xt == DION_X_F32) copy_x<DION_X_F32, kThreads>(p, token0, tokens, c0, c1, xall, xpitch, magic);
    else {
        copy_x<DION_X_E4M3, kThreads>(p, token0, tokens, c0, c1, xall, xpitch, magic);
        for (int i = threadIdx.x; i < tokens * (c1 - c0); i += kThreads) {
            const int row = i / (c1 - c0), c = i - row * (c1 - c0);
            powers[c * 8 * MB + row] = power_of(p.sx[(token0 + row) * p.ldsx + c0 + c]);
        }
    }
    copies_end();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) copy_next(i);
    copies_wait<kAhead>();                   // x is here
    if (p.xt == DION_X_BF16) convert_all<DION_X_BF16, kThreads>(tokens, c0, c1, xall, xpitch, powers, 8 * MB, magic);
    else if (p.xt == DION_X_F32) convert_all<DION_X_F32, kThreads>(tokens, c0, c1, xall, xpitch, powers, 8 * MB, magic);
    else if (p.xt == DION_X_E4M3) convert_all<DION_X_E4M3, kThreads>(tokens, c0, c1, xall, xpitch, powers, 8 * MB, magic);
    else convert_all<DION_X_E5M2, kThreads>(tokens, c0, c1, xall, xpitch, powers, 8 * MB, magic);
    __syncthreads();

    const uint8_t* xs = xall + 16 * t + 256 * (w0 - c0);
    const float* ups = powers + (w0 - c0) * 8 * MB + 2 * t;
    float acc[MB][4] = {};
    int cb = first, ci = 0, turn = 0, held = 0, slot = 0;
    while (cb < p.blocks) {
        copies_wait<kAhead - 1>();
        __syncwarp();                        // the other lanes' scales
        const uint8_t* wq = ring + slot * B::BYTES + 16 * lane;
        const uint8_t* ws = ring + slot * B::BYTES + B::WEIGHTS + g * B::PITCH;
        const int c = ci * kBatch;
        if (w0 + c + kBatch <= w1) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                chunk_products<MB, GROUP, B>(wq + 1024 * u, ws + 2 * B::S * u, xs + 256 * (c + u), columns, ups + (c + u) * 8 * MB, acc);
        } else {
#pragma unroll 1
            for (int u = 0; w0 + c + u < w1; ++u)
                chunk_products<MB, GROUP, B>(wq + 1024 * u, ws + 2 * B::S * u, xs + 256 * (c + u), columns, ups + (c + u) * 8 * MB, acc);
        }
        __syncwarp();                        // all lanes have read the scales
        copy_next(slot);
        slot = slot + 1 == kAhead ? 0 : slot + 1;
        if (++ci == batches) {
            // the tile's end: the sums of the warps that share it
            float* to = parts + ((turn * kWarps + warp) * most) * 16;
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = 8 * i + 2 * t + (e & 1);
                    if (col < cols) to[col * 16 + g + 8 * (e >> 1)] = acc[i][e];
                    acc[i][e] = 0.f;
                }
            if (p.split == 1) __syncwarp();
            else asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "r"(32 * p.split) : "memory");
            const float* from = parts + ((turn * kWarps + mine * p.split) * most) * 16;
            const int row0 = (cb * tiles + mine) * 16;
            if (shares == 1) {
                for (int i = part * 32 + lane; i < tokens * 16; i += 32 * p.split) {
                    const int r = i & 15, token = i >> 4;
                    float v = 0.f;
                    for (int e = 0; e < p.terms; ++e)
                        for (int w = 0; w < p.split; ++w) v += from[(w * most + token * p.terms + e) * 16 + r];
                    if (row0 + r < p.n) {
                        const long long o = (token0 + token) * p.ldy + row0 + r;
                        if (p.y_f32) ((float*)p.y)[o] = v;
                        else ((bf16*)p.y)[o] = __float2bfloat16_rn(v);
                    }
                }
            } else {
                float* kept = hold + (held * tiles + mine) * most * 16;
                for (int i = part * 32 + lane; i < cols * 16; i += 32 * p.split) {
                    float v = 0.f;
                    for (int w = 0; w < p.split; ++w) v += from[w * most * 16 + i];
                    kept[i] = v;
                }
                if (++held == p.held || cb + step >= p.blocks) {
                    join<kThreads>(p, hold, cb - (held - 1) * step, step, held, shares, share, token0, tokens);
                    held = 0;
                }
            }
            // (two turns: who writes a turn's sums again has passed the other's barrier, so all have read them)
            turn ^= 1;
            ci = 0;
            cb += step;
        }
    }
}

// CTAs of a cluster of `shares` that run at once (whole clusters lie in a group of SMs).
int clusters_at_once(int shares)
{
    constexpr int at_once[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    return std::max(1, at_once[shares] * num_sms() / 152);
}

// CTAs an SM, for their shared memory.
template <class C>
int ctas_of(size_t bytes) { return std::min(C::CTAS, (int)(228 * 1024 / (bytes + 1024))); }

// Chunks of a CTA's share of `chunks` where s CTAs share them; 0: one of them would have none.
constexpr int share_of(int chunks, int s)
{
    const int per = ((chunks + s - 1) / s + kUnit - 1) / kUnit * kUnit;
    return s > 1 && (chunks + per - 1) / per != s ? 0 : per;
}
// Bytes of a CTA's sums that wait for a join: a block's at least.
template <int MB>
constexpr size_t hold_bytes() { return std::max(16384, Cfg<MB>::WARPS * 8 * MB * 64); }
// Shared memory of a CTA: the batches in flight, x, its powers of two, and the warps' sums.
template <int MB, int GROUP>
constexpr size_t shared_bytes(int cols, int per, int s)
{
    using C = Cfg<MB>;
    return (size_t)C::WARPS * C::AHEAD * Batch<GROUP, C::BATCH>::BYTES + (size_t)cols * (256 * per + 64 + 128 * C::WARPS) + 32 * MB * per +
           (s > 1 ? hold_bytes<MB>() : 0);
}
template <int MB, int GROUP>
constexpr bool fits(int cols, int chunks)
{
    for (int s = 1; s <= 8; ++s)
        if (const int per = share_of(chunks, s); per && shared_bytes<MB, GROUP>(cols, per, s) <= kMostShared) return true;
    return false;
}
// What the header says of the weights' being read again.
constexpr int kLongestOfAllColumns = 16384;
template <int GROUP>
constexpr bool all_columns_fit()
{
    for (int c = 1; c <= kLongestOfAllColumns / 128; ++c)
        if (!fits<4, GROUP>(32, c)) return false;
    return !fits<4, GROUP>(32, kLongestOfAllColumns / 128 + 1);
}
static_assert(all_columns_fit<32>() && all_columns_fit<64>() && all_columns_fit<128>(), "longest rows of which 32 columns are one pass");

// How the work is cut, for p.tokens rows a pass: CTAs that share the contraction
// (returned; 0: x does not fit), warps that share a tile, and a CTA's shared
// memory.  The cut with the least estimate of an SM's time is taken, in the time
// that its warps need for a chunk each (about 0.2 us): its blocks one after the
// other (one of two CTAs an SM that runs alone takes 1.3 of its time beside the
// other, not half of two), whose warps work on whole batches and need two chunks'
// time for a tile's end; x, 0.55 for a thread's unit of eight columns; a join, 7.
// us with every number of warps that share a tile, from all down to one, and the
// estimates:
//   1 x 53248 x 16384 (g128)   79.9  76.3  84.2 106.3     405  393  405  438
//   1 x  4096 x 14336          12.5  10.8  16.8  29.0      44   43   79  152
//   1 x 53248 x  4096          25.9  24.1  24.2  29.7     134  115  110  114
//   1 x 32768 x  1024          11.7   8.8   7.6   7.2      85   44   25   21
//   16 x 4096 x 14336 (q8, 4 shares)  22.3 19.4 17.5 22.8  65   49   41   47
template <int MB, int GROUP>
int cut(MatParams& p, size_t& smem)
{
    using C = Cfg<MB>;
    constexpr size_t hold = hold_bytes<MB>();
    const int tiles = (int)cdiv(p.n, 16), cols = p.tokens * p.terms;
    float least = 0.f;
    int best = 0;
    for (int s = 1; s <= 8 && (best == 0 || cdiv(p.chunks, s) >= C::BATCH); ++s) {
        const int per = share_of(p.chunks, s);
        const size_t bytes = shared_bytes<MB, GROUP>(cols, per, s);
        if (!per || bytes > kMostShared) continue;
        const int at_once = clusters_at_once(s), per_sm = ctas_of<C>(bytes);
        const float x = 0.55f * 16 / C::THREADS * p.tokens * per, join = s > 1 ? 7.f : 0.f;
        for (int split = C::WARPS; split; split /= 2) {
            const int blocks = (int)cdiv(tiles, C::WARPS / split), rest = blocks % (per_sm * at_once);
            const float full = (float)(blocks / (per_sm * at_once) * per_sm);
            const float rounds = full + (rest == 0 ? 0.f : rest > at_once ? 2.f : per_sm == 2 ? 1.3f : 1.f);
            const float t = rounds * (float)(cdiv(per, split * C::BATCH) * C::BATCH + 2) + (blocks > at_once ? per_sm : 1) * x + join;
            if (best && t >= least) continue;
            least = t;
            best = s;
            p.per = per;
            p.split = split;
            p.blocks = blocks;
            const int block = C::WARPS / split * cols * 64;
            p.held = std::max(1, (int)hold / block);
            smem = bytes;
        }
        if (best == s && (long long)tiles * C::BATCH > 8ll * C::WARPS * at_once) break;    // tiles enough: no more shares
    }
    return best;
}

template <int MB, int GROUP>
cudaError_t go(MatParams& p, cudaStream_t st)
{
    using C = Cfg<MB>;
    static std::atomic<unsigned long long> attr{0};
    cudaError_t e = smem_attr_once((const void*)q4_matmul_kernel<MB, GROUP>, kMostShared, attr);
    if (e != cudaSuccess) return e;
    size_t smem = 0;
    int shares = cut<MB, GROUP>(p, smem);
    for (; !shares && p.tokens > 1; shares = cut<MB, GROUP>(p, smem)) --p.tokens;     // (fewer rows a pass)
    if (!shares) return cudaErrorInvalidValue;
    const int clusters = std::min(p.blocks, ctas_of<C>(smem) * clusters_at_once(shares));
    return launch_cluster("q4_matmul", q4_matmul_kernel<MB, GROUP>, dim3((unsigned)(clusters * shares), (unsigned)cdiv(p.m, p.tokens)),
                          dim3(C::THREADS), shares, smem, st, p, shares);
}

template <int GROUP>
cudaError_t pick(MatParams& p, cudaStream_t st)
{
    const int cols = p.tokens * p.terms;
    if (cols <= 8) return go<1, GROUP>(p, st);
    if (cols <= 16) return go<2, GROUP>(p, st);
    return go<4, GROUP>(p, st);
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
    p.terms = a.xt == DION_X_F32 ? 2 : 1;
    p.chunks = (int)cdiv(p.k, 128);
    p.xt = a.xt; p.x = a.x; p.ldx = a.ldx; p.sx = a.sx; p.ldsx = a.ldsx;
    p.x_wide = (uintptr_t)a.x % 16 == 0 && a.ldx * (a.xt == DION_X_F32 ? 4 : 2) % 16 == 0;
    p.q = a.w.q; p.ldq = a.w.ldq;
    p.s = a.w.s; p.lds = a.w.lds;
    p.groups = (int)cdiv(p.k, a.w.group);
    p.s_wide = (uintptr_t)a.w.s % 4 == 0 && a.w.lds % 2 == 0;
    p.y = a.y; p.ldy = a.ldy; p.y_f32 = a.ydt == DION_F32;
    p.tokens = std::min(p.m, 32 / p.terms);
    return a.w.group == 32 ? pick<32>(p, st) : a.w.group == 64 ? pick<64>(p, st) : pick<128>(p, st);
}

}  // namespace dion
