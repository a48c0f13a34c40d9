// q4_quant.cu -- weights to 4 bits with group scales and back.
//
// Half a warp takes one 128-column chunk of a row: lane l its columns 8 l ..
// 8 l + 7, which are one 32-bit word of the held chunk, so the reads and the
// 64-byte write of a chunk are contiguous and a group is 4, 8 or 16 lanes.
//
// 14336 x 4096 bfloat16 values take 34 us (147 MB move, 22 us at a copy's rate:
// 15 instructions a value fill 73 % of the issue slots) and 23 to 25 us back.
#include "q4.cuh"

namespace dion {
namespace {

using namespace q8;

constexpr int kThreads = 128, kHalves = kThreads / 16;
constexpr int kUnits = 4;          // chunks of a half-warp, loaded together

// Place of lane l's word (columns 8 l ..) in its chunk.
__device__ __forceinline__ int word_of(int l) { return 4 * (l & 3) + (l >> 2); }

// Rows' chunks, numbered through the matrix.
struct Units {
    uint32_t count, chunks;            // all, and of a row
    uint32_t magic;                    // a number's row by a product, or 0: by a division
    __device__ __forceinline__ void at(uint32_t unit, uint32_t& row, uint32_t& chunk) const
    {
        row = magic ? __umulhi(unit, magic) : unit / chunks;
        chunk = unit - row * chunks;
    }
};

// Magnitude bits of the largest of a lane's eight values, as float32's: infinities and NaN are the largest.
__device__ __forceinline__ uint32_t amax_bits(const Raw8<bf16>& r, const float2 (&)[4])
{
    const uint4 u = r.u[0];
    const uint32_t m = 0x7fff7fffu, a = __vimax3_u16x2(u.x & m, u.y & m, __vmaxu2(u.z & m, u.w & m));
    return max(a << 16, a & 0xffff0000u);
}
__device__ __forceinline__ uint32_t amax_bits(const Raw8<float>&, const float2 (&f)[4])
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = max(a, max(mag_bits(f[i].x), mag_bits(f[i].y)));
    return a;
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(kThreads)
    q4_quantize_kernel(const Q4Side w, const T* x, const long long ldx, const bool aligned, const Units units)
{
    wait_previous();
    allow_next();
    const int l = threadIdx.x & 15, half = threadIdx.x >> 4;
    Raw8<T> raw[kUnits];
    uint32_t row[kUnits], chunk[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        units.at(min((blockIdx.x * kUnits + u) * kHalves + half, units.count - 1), row[u], chunk[u]);     // (the last one again)
        const T* r = x + row[u] * ldx;
        raw[u] = aligned ? load_raw8<false>(r, 128 * (int)chunk[u], w.cols, l) : load_raw8<true>(r, 128 * (int)chunk[u], w.cols, l);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        float2 f[4];
        unpack8(raw[u], f);
        uint32_t amax = amax_bits(raw[u], f);
#pragma unroll
        for (int o = GROUP / 16; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const bool finite = amax < kInfBits;
        // Quotients are products with a reciprocal and a correction from their remainder, which is formed exactly
        // (Markstein's): the division's own results, ties among them, down to where remainders would be subnormal.
        float by = __uint_as_float(amax);
        if (by >= 0x1p-90f) {
            const float q = __fmul_rn(by, 1.f / 7.f);
            by = __fmaf_rn(__fmaf_rn(q, -7.f, by), 1.f / 7.f, q);
        } else {
            by = __fdiv_rn(by, 7.f);
        }
        const bf16 s = from_f<bf16>(finite ? by : __uint_as_float(0x7fc00000u));
        by = to_f(s);
        uint32_t word;
        if (finite && by >= 0x1p-100f) {
            // 1.5 * 2^23 + 8 rounds to whole numbers, plus eight, in the low bits (a scale is bf16(amax / 7), so they
            // lie in -7 .. 7).
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(by));
            word = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = mul2(f[i], make_float2(inv, inv));
                const float2 rest = fma2(v, make_float2(-by, -by), f[i]);
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
        if ((blockIdx.x * kUnits + u) * kHalves + half < units.count) {
            reinterpret_cast<uint32_t*>(w.q + row[u] * w.ldq)[16 * chunk[u] + word_of(l)] = word;
            if (l % (GROUP / 8) == 0 && col < w.cols) w.s[row[u] * w.lds + col / GROUP] = s;
        }
    }
}

// A word's values times their group's scale, each rounded once.  bfloat16: 128 + q + 8 from the bits, less 136,
// exactly, and one product of bfloat16 numbers.
__device__ __forceinline__ void values_of(uint32_t word, uint32_t s, Raw8<bf16>& r)
{
    uint32_t v[4];
    const uint32_t s2 = s | (s << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(((word >> (4 * i)) & 0x000f000fu) | 0x43004300u), "r"(0x43084308u));
        asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(s2));
    }
    r.u[0] = make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void values_of(uint32_t word, uint32_t s, Raw8<float>& r)
{
    float2 f[4];
    const float scale = __uint_as_float(s << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // four bits in a float's low ones are 2^23 + q + 8
        const uint32_t w = (word >> (4 * i)) & 0x000f000fu;
        const float2 q = add2(make_float2(__uint_as_float((w & 15u) | 0x4b000000u), __uint_as_float((w >> 16) | 0x4b000000u)),
                              make_float2(-8388616.f, -8388616.f));
        f[i] = mul2(q, make_float2(scale, scale));
    }
    pack8(r, f);
}

// A lane's eight values to a row whose address is a multiple of their bytes.  float32 in one store of 32 bytes: as two
// of 16, each leaves half of every 32-byte sector to the other (14336x4096 56 us, so 42).
__device__ __forceinline__ void store_row(bf16* to, const Raw8<bf16>& v) { *reinterpret_cast<uint4*>(to) = v.u[0]; }
__device__ __forceinline__ void store_row(float* to, const Raw8<float>& v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v.u[0].x), "r"(v.u[0].y), "r"(v.u[0].z),
                 "r"(v.u[0].w), "r"(v.u[1].x), "r"(v.u[1].y), "r"(v.u[1].z), "r"(v.u[1].w)
                 : "memory");
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(kThreads)
    q4_dequantize_kernel(const Q4Side w, T* y, const long long ldy, const bool aligned, const Units units)
{
    wait_previous();
    allow_next();
    const int l = threadIdx.x & 15, half = threadIdx.x >> 4;
    uint32_t row[kUnits], chunk[kUnits], word[kUnits], s[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        units.at(min((blockIdx.x * kUnits + u) * kHalves + half, units.count - 1), row[u], chunk[u]);
        const int col = 128 * (int)chunk[u] + 8 * l;
        word[u] = reinterpret_cast<const uint32_t*>(w.q + row[u] * w.ldq)[16 * chunk[u] + word_of(l)];
        s[u] = col < w.cols ? reinterpret_cast<const uint16_t*>(w.s)[row[u] * w.lds + col / GROUP] : 0u;
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if ((blockIdx.x * kUnits + u) * kHalves + half >= units.count) break;
        Raw8<T> v;
        values_of(word[u], s[u], v);
        const int col = 128 * (int)chunk[u] + 8 * l;
        T* to = y + row[u] * ldy + col;
        if (aligned && col + 8 <= w.cols) {
            store_row(to, v);
        } else {
            float2 f[4];
            unpack8(v, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < w.cols) to[i] = from_f<T>(i & 1 ? f[i >> 1].y : f[i >> 1].x);
        }
    }
}

template <typename T>
bool rows_aligned(const void* p, long long ld, size_t a = 16) { return (uintptr_t)p % a == 0 && ld * sizeof(T) % a == 0; }

Units units_of(const Q4Side& w)
{
    Units u;
    u.chunks = (uint32_t)cdiv(w.cols, 128);
    u.count = u.chunks * (uint32_t)w.rows;
    // ceil(2^32 / chunks): exact for numbers below 2^32 / chunks
    u.magic = u.chunks > 1 && (uint64_t)u.count * u.chunks < 1ull << 32 ? (uint32_t)(((1ull << 32) + u.chunks - 1) / u.chunks) : 0;
    return u;
}

template <typename T, int GROUP>
cudaError_t quantize(const Q4Side& w, const void* x, long long ldx, cudaStream_t st)
{
    const Units u = units_of(w);
    return launch_overlapped("q4_quantize", q4_quantize_kernel<T, GROUP>, dim3((unsigned)cdiv(u.count, kHalves * kUnits)),
                             dim3(kThreads), 0, st, w, (const T*)x, ldx, rows_aligned<T>(x, ldx), u);
}
template <typename T, int GROUP>
cudaError_t dequantize(const Q4Side& w, void* y, long long ldy, cudaStream_t st)
{
    const Units u = units_of(w);
    return launch_overlapped("q4_dequantize", q4_dequantize_kernel<T, GROUP>, dim3((unsigned)cdiv(u.count, kHalves * kUnits)),
                             dim3(kThreads), 0, st, w, (T*)y, ldy, rows_aligned<T>(y, ldy, 8 * sizeof(T)), u);
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
