// q8.cuh -- block quantization to 8-bit floating point: the scale of a block
// from its largest magnitude, the conversion of scaled values, and the
// chunks of eight values that the norm and quantization kernels move.
//
// A block's scale is 2^e, the smallest power of two with amax <= MAX * 2^e.
// Both formats have MAX = 1.75 * 2^x (448 = 1.75 * 2^8, 57344 = 1.75 * 2^15),
// so for amax = 1.f * 2^p: e = p - x, plus one if 1.f > 1.75.  On the float's
// bits that is one addition that carries into the exponent when the mantissa
// exceeds that of 1.75 (0x600000).  Dividing by a power of two is exact, so a
// value is rounded once, in the conversion.
#pragma once

#include "common.cuh"
#include "../../include/dion_q8.h"

namespace dion {
namespace q8 {

constexpr uint32_t kInfBits = 0x7f800000u;

// Scale byte (e + 127) of a block whose largest finite magnitude has the given bits.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits)
{
    constexpr int X = FMT == DION_E4M3 ? 8 : 15;
    const int e = (int)((amax_bits + 0x1fffffu) >> 23) - X;   // biased by 127
    return amax_bits == 0 ? 127u : (uint32_t)max(e, 0);
}

// 2^-(byte - 127) as a float: byte lies in [0, 247], so the result is normal.
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two scaled values to two bytes, a in the low one.
template <int FMT>
__device__ __forceinline__ uint32_t cvt2(float a, float b)
{
    uint16_t r;
    if (FMT == DION_E4M3)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Pairs of float32 in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
          "l"(*reinterpret_cast<const uint64_t*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}
// Two bfloat16 in a word (the first in the low half) to float32.
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 v)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Magnitude for a block's maximum: infinities and NaN do not count.
__device__ __forceinline__ uint32_t finite_mag_bits(float v)
{
    const uint32_t b = mag_bits(v);
    return b >= kInfBits ? 0u : b;
}

// An infinity would saturate to the format's largest value; it becomes NaN instead.
__device__ __forceinline__ float inf_to_nan(float v)
{
    return mag_bits(v) == kInfBits ? __uint_as_float(0x7fffffffu) : v;
}

// Maximum over the 16 lanes of a half-warp.
__device__ __forceinline__ uint32_t max16(uint32_t v)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The half-warp's 16 lanes hold one 128-value block, eight values a lane.
// VEC: lane l holds values 8 l .. 8 l + 7 (one wide access); otherwise values
// l, l + 16, .. (rows whose base or pitch is not a multiple of 16 bytes:
// neighbouring lanes then still touch neighbouring elements).
template <bool VEC>
__device__ __forceinline__ int elem(int l, int i)
{
    return VEC ? 8 * l + i : l + 16 * i;
}



// Eight values as four pairs; raw: as stored (one or two 16-byte words).
template <typename T> struct Raw8 { uint4 u[sizeof(T) / 2]; };
__device__ __forceinline__ void unpack8(const Raw8<bf16>& r, float2 (&f)[4])
{
    f[0] = unpack2(r.u[0].x);
    f[1] = unpack2(r.u[0].y);
    f[2] = unpack2(r.u[0].z);
    f[3] = unpack2(r.u[0].w);
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float2 (&f)[4])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[2 * i] = make_float2(__uint_as_float(r.u[i].x), __uint_as_float(r.u[i].y));
        f[2 * i + 1] = make_float2(__uint_as_float(r.u[i].z), __uint_as_float(r.u[i].w));
    }
}
__device__ __forceinline__ void pack8(Raw8<bf16>& r, const float2 (&f)[4])
{
    r.u[0] = make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
__device__ __forceinline__ void pack8(Raw8<float>& r, const float2 (&f)[4])
{
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r.u[i] = make_uint4(__float_as_uint(f[2 * i].x), __float_as_uint(f[2 * i].y), __float_as_uint(f[2 * i + 1].x),
                            __float_as_uint(f[2 * i + 1].y));
}

// Eight consecutive values at any address: the 16-byte words that hold them
// (none that holds no byte of them is read), shifted into place.
template <typename T>
__device__ __forceinline__ Raw8<T> load_shifted(const T* p)
{
    constexpr int W = sizeof(T) * 2;                    // 32-bit words of the values
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint4* b = reinterpret_cast<const uint4*>(a & ~(uintptr_t)15);
    const uint32_t m = (uint32_t)a & 15u;
    uint32_t w[W + 4];
#pragma unroll
    for (int i = 0; i <= W / 4; ++i) {
        const uint4 u = i < W / 4 || m ? b[i] : make_uint4(0, 0, 0, 0);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < W + 2; ++i) w[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < W + 1; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
    if (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = m & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    }
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < W / 4; ++i) r.u[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    return r;
}
// A lane's eight consecutive values of the block at column c0 of a row that may
// start anywhere; zeros past the row.
template <bool SHIFT, typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* row, int c0, int cols, int l)
{
    const T* p = row + c0 + 8 * l;
    Raw8<T> r;
    if (c0 + 8 * l + 8 <= cols) {
        if (SHIFT) return load_shifted(p);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(c0 + 8 * l + 2 * i < cols ? to_f(p[2 * i]) : 0.f,
                               c0 + 8 * l + 2 * i + 1 < cols ? to_f(p[2 * i + 1]) : 0.f);
        pack8(r, f);
    }
    return r;
}

// A lane's eight values of the block at column c0 of a row; zeros past the row.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int c0, int cols, int l, float2 (&f)[4])
{
    if (VEC && c0 + 8 * l + 8 <= cols) {
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.u[i] = reinterpret_cast<const uint4*>(row + c0 + 8 * l)[i];
        unpack8(r, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int a = c0 + elem<VEC>(l, 2 * i), b = c0 + elem<VEC>(l, 2 * i + 1);
            f[i] = make_float2(a < cols ? to_f(row[a]) : 0.f, b < cols ? to_f(row[b]) : 0.f);
        }
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int c0, int cols, int l, const float2 (&f)[4])
{
    if (VEC && c0 + 8 * l + 8 <= cols) {
        Raw8<T> r;
        pack8(r, f);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(row + c0 + 8 * l)[i] = r.u[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int a = c0 + elem<VEC>(l, 2 * i), b = c0 + elem<VEC>(l, 2 * i + 1);
            if (a < cols) row[a] = from_f<T>(f[i].x);
            if (b < cols) row[b] = from_f<T>(f[i].y);
        }
    }
}

// Eight values of a lane, scaled and converted, to a row of 8-bit values
// (16-byte aligned rows, so a lane's eight bytes are 8-byte aligned).
template <bool VEC, int FMT>
__device__ __forceinline__ void store_q8(uint8_t* row, int c0, int cols, int l, const float2 (&f)[4], float inv)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = mul2(f[i], make_float2(inv, inv));
        w[i] = cvt2<FMT>(v.x, v.y);
    }
    if (VEC && c0 + 8 * l + 8 <= cols) {
        *reinterpret_cast<uint2*>(row + c0 + 8 * l) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + elem<VEC>(l, i);
            if (c < cols) row[c] = (uint8_t)(w[i >> 1] >> (8 * (i & 1)));
        }
    }
}

}  // namespace q8

// Host side: argument bundles of the q8 entry points, checked by q8_api.cu.
struct Q8QuantArgs {
    int batch, rows, cols;
    const void* x; long long ldx, sx;
    const float* rstd; const void* weight; dion_dtype wdt;
    int square;
    uint8_t* q; long long ldq, sq;
    uint8_t* s; long long lds, ss;
    uint8_t* qt; long long ldqt, sqt;
    uint8_t* st; long long ldst, sst;
};
cudaError_t q8_quantize(const Q8QuantArgs& a, dion_dtype dt, dion_q8_format fmt, cudaStream_t stream);

struct Q8NormArgs {
    int rows, cols;
    const void* x; long long ldx;
    const void* res; long long ldr;
    const void* w; dion_dtype wdt;
    float eps;
    void* h; long long ldh;
    uint8_t* q; long long ldq;
    uint8_t* s; long long lds;
    float* rstd;
};
cudaError_t rms_norm_q8(const Q8NormArgs& a, dion_dtype dt, dion_q8_format fmt, cudaStream_t stream);

struct NormBwdArgs {
    int rows, cols;
    const void* dy; long long lddy;
    const void* h; long long ldh;
    const float* rstd;
    const void* w; dion_dtype wdt;
    const void* dh; long long lddh;
    void* dx; long long lddx;
    float* dw;
    float* part;                // workspace: row groups x cols partial sums of dw; null: a small problem's one launch
};
size_t norm_backward_workspace(int rows, int cols);
bool norm_backward_small(int rows, int cols);    // needs no workspace if dx is apart from dy and h
cudaError_t rms_norm_backward(const NormBwdArgs& a, dion_dtype dt, cudaStream_t stream);

// One operand of the product: rows of 8-bit values, their format and scales.
struct Q8Side {
    int rows;
    const uint8_t* q; long long ld; dion_q8_format fmt;
    const uint8_t* s; long long lds; int square;
};
struct Q8MatArgs {
    int k;
    Q8Side a, b;
    void* c; long long ldc; dion_dtype cdt;
    int* status;
};
cudaError_t q8_matmul(const Q8MatArgs& a, cudaStream_t stream);

}  // namespace dion
