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



template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int c0, int cols, int l, float (&f)[8])
{
    if (VEC && c0 + 8 * l + 8 <= cols) {
        const T* p = row + c0 + 8 * l;
        if (sizeof(T) == 2) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + elem<VEC>(l, i);
            f[i] = c < cols ? to_f(row[c]) : 0.f;
        }
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int c0, int cols, int l, const float (&f)[8])
{
    if (VEC && c0 + 8 * l + 8 <= cols) {
        T* p = row + c0 + 8 * l;
        if (sizeof(T) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + elem<VEC>(l, i);
            if (c < cols) row[c] = from_f<T>(f[i]);
        }
    }
}

// Eight values of a lane, scaled and converted, to a row of 8-bit values
// (16-byte aligned rows, so a lane's eight bytes are 8-byte aligned).
template <bool VEC, int FMT>
__device__ __forceinline__ void store_q8(uint8_t* row, int c0, int cols, int l, const float (&f)[8], float inv)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cvt2<FMT>(f[2 * i] * inv, f[2 * i + 1] * inv);
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
    float* part;                // workspace: row groups x cols partial sums of dw
};
size_t norm_backward_workspace(int rows, int cols);
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
