// q4_quant.cu -- weights to 4 bits with group scales and back.
//
// Half a warp takes one 128-column chunk of a row: lane l its columns 8 l ..
// 8 l + 7, which are one 32-bit word of the held chunk, so the reads and the
// 64-byte write of a chunk are contiguous and a group is 4, 8 or 16 lanes.
#include "q4.cuh"

namespace dion {
namespace {

using namespace q8;

constexpr int kThreads = 256, kHalves = kThreads / 16;
constexpr int kUnits = 4;          // chunks of a half-warp, loaded together

// Place of lane l's word (columns 8 l ..) in its chunk.
__device__ __forceinline__ int word_of(int l) { return 4 * (l & 3) + (l >> 2); }

template <typename T, int GROUP>
__global__ void __launch_bounds__(kThreads)
    q4_quantize_kernel(const Q4Side w, const T* x, const long long ldx, const bool aligned, const uint32_t chunks,
                       const uint32_t units)
{
    wait_previous();
    allow_next();
    const int l = threadIdx.x & 15, half = threadIdx.x >> 4;
    Raw8<T> raw[kUnits];
    uint32_t row[kUnits], chunk[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint32_t unit = min((blockIdx.x * kUnits + u) * kHalves + half, units - 1);   // (the last one again)
        row[u] = unit / chunks;
        chunk[u] = unit - row[u] * chunks;
        const T* r = x + row[u] * ldx;
        raw[u] = aligned ? load_raw8<false>(r, 128 * (int)chunk[u], w.cols, l) : load_raw8<true>(r, 128 * (int)chunk[u], w.cols, l);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        float2 f[4];
        unpack8(raw[u], f);
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = max(amax, max(mag_bits(f[i].x), mag_bits(f[i].y)));
#pragma unroll
        for (int o = GROUP / 16; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const bool finite = amax < kInfBits;
        const bf16 s = finite ? from_f<bf16>(__fdiv_rn(__uint_as_float(amax), 7.f)) : from_f<bf16>(__uint_as_float(0x7fc00000u));
        const float by = to_f(s);
        uint32_t word;
        if (finite && by >= 0x1p-100f) {
            // Quotients by the scale's reciprocal and Markstein's correction, whose remainder is exact: the division's
            // own results, ties among them.  1.5 * 2^23 + 8 rounds them to whole numbers, plus eight, in the low bits
            // (a scale is bf16(amax / 7), so they lie in -7 .. 7).
            const float inv = __frcp_rn(by);
            word = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = mul2(f[i], make_float2(inv, inv));
                const float2 rest = fma2(make_float2(-v.x, -v.y), make_float2(by, by), f[i]);
                const float2 w = fma2(rest, make_float2(inv, inv), v);
                const float2 q = add2(w, make_float2(12582920.f, 12582920.f));
                // columns 2 i and 2 i + 1: four bits of each half
                word += __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x5410) << (4 * i);
            }
        } else {
            word = 0x88888888u;
            if (finite && by > 0.f) {
                word = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = __fdiv_rn(i & 1 ? f[i >> 1].y : f[i >> 1].x, by);
                    const int q = min(max(__float2int_rn(v), -8), 7) + 8;
                    word |= (uint32_t)q << (4 * (i >> 1) + 16 * (i & 1));
                }
            }
        }
        const int col = 128 * (int)chunk[u] + 8 * l;
        if ((blockIdx.x * kUnits + u) * kHalves + half < units) {
            reinterpret_cast<uint32_t*>(w.q + row[u] * w.ldq)[16 * chunk[u] + word_of(l)] = word;
            if (l % (GROUP / 8) == 0 && col < w.cols) w.s[row[u] * w.lds + col / GROUP] = s;
        }
    }
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(kThreads)
    q4_dequantize_kernel(const Q4Side w, T* y, const long long ldy, const bool aligned, const uint32_t chunks,
                         const uint32_t units)
{
    wait_previous();
    allow_next();
    const int l = threadIdx.x & 15, half = threadIdx.x >> 4;
    uint32_t row[kUnits], chunk[kUnits], word[kUnits];
    float s[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint32_t unit = min((blockIdx.x * kUnits + u) * kHalves + half, units - 1);
        row[u] = unit / chunks;
        chunk[u] = unit - row[u] * chunks;
        const int col = 128 * (int)chunk[u] + 8 * l;
        word[u] = reinterpret_cast<const uint32_t*>(w.q + row[u] * w.ldq)[16 * chunk[u] + word_of(l)];
        s[u] = col < w.cols ? to_f(w.s[row[u] * w.lds + col / GROUP]) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if ((blockIdx.x * kUnits + u) * kHalves + half >= units) break;
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // four bits in a float's low ones are 2^23 + q + 8
            const uint32_t w = (word[u] >> (4 * i)) & 0x000f000fu;
            const float2 q = add2(make_float2(__uint_as_float(w & 15u | 0x4b000000u), __uint_as_float(w >> 16 | 0x4b000000u)),
                                  make_float2(-8388616.f, -8388616.f));
            f[i] = mul2(q, make_float2(s[u], s[u]));
        }
        T* r = y + row[u] * ldy;
        const int c0 = 128 * (int)chunk[u];
        if (aligned && c0 + 8 * l + 8 <= w.cols) {
            store8<true>(r, c0, w.cols, l, f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + 8 * l + i < w.cols) r[c0 + 8 * l + i] = from_f<T>(i & 1 ? f[i >> 1].y : f[i >> 1].x);
        }
    }
}

template <typename T>
bool rows_aligned(const void* p, long long ld) { return (uintptr_t)p % 16 == 0 && ld * sizeof(T) % 16 == 0; }

template <typename T, int GROUP>
cudaError_t quantize(const Q4Side& w, const void* x, long long ldx, cudaStream_t st)
{
    const long long chunks = cdiv(w.cols, 128), units = chunks * w.rows;
    return launch_overlapped("q4_quantize", q4_quantize_kernel<T, GROUP>, dim3((unsigned)cdiv(units, kHalves * kUnits)),
                             dim3(kThreads), 0, st, w, (const T*)x, ldx, rows_aligned<T>(x, ldx), (uint32_t)chunks, (uint32_t)units);
}
template <typename T, int GROUP>
cudaError_t dequantize(const Q4Side& w, void* y, long long ldy, cudaStream_t st)
{
    const long long chunks = cdiv(w.cols, 128), units = chunks * w.rows;
    return launch_overlapped("q4_dequantize", q4_dequantize_kernel<T, GROUP>, dim3((unsigned)cdiv(units, kHalves * kUnits)),
                             dim3(kThreads), 0, st, w, (T*)y, ldy, rows_aligned<T>(y, ldy), (uint32_t)chunks, (uint32_t)units);
}

}  // namespace

cudaError_t q4_quantize(const Q4Side& w, dion_dtype dt, const void* x, long long ldx, cudaStream_t st)
{
    if (dt == DION_F32)
        return w.group == 32 ? quantize<float, 32>(w, x, ldx, st) : w.group == 64 ? quantize<float, 64>(w, x, ldx, st)
                                                                                  : quantize<float, 128>(w, x, ldx, st);
    return w.group == 32 ? quantize<bf16, 32>(w, x, ldx, st) : w.group == 64 ? quantize<bf16, 64>(w, x, ldx, st)
                                                                             : quantize<bf16, 128>(w, x, ldx, st);
}

cudaError_t q4_dequantize(const Q4Side& w, dion_dtype dt, void* y, long long ldy, cudaStream_t st)
{
    if (dt == DION_F32)
        return w.group == 32 ? dequantize<float, 32>(w, y, ldy, st) : w.group == 64 ? dequantize<float, 64>(w, y, ldy, st)
                                                                                    : dequantize<float, 128>(w, y, ldy, st);
    return w.group == 32 ? dequantize<bf16, 32>(w, y, ldy, st) : w.group == 64 ? dequantize<bf16, 64>(w, y, ldy, st)
                                                                               : dequantize<bf16, 128>(w, y, ldy, st);
}

}  // namespace dion
