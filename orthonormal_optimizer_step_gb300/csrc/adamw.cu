// adamw.cu -- AdamW over many tensors in one launch, and the norm of many
// gradients (include/dion_adamw.h).
//
// The list travels in the kernel's parameters (up to 32 KB), so a call moves
// nothing to the device first and can be captured.  Tensors are cut into chunks
// of 2048 values, eight consecutive ones a thread, numbered through the list; a
// CTA finds its first chunk's tensor by bisection over the first chunk of each.
// A warp's 256 values are one block of an 8-bit state, so a block's largest
// magnitude is one reduction over the warp.
//
// Memory bounds the step with float32 states: 67 million values take 217 us with
// bfloat16 parameters and gradients, 274 with float32 ones, 0.99 to 1.01 of the
// time of a copy of as many bytes.  With 8-bit states and bfloat16 the arithmetic
// of a value (decoding, roots, dither, encoding) fills three quarters of the issue
// slots: 133 us for 67 million, 0.75 of the copy's rate (float32 parameters 0.99).
// Where all first moments are dithered (1 - beta1 below 3/32), 262 million take 510
// us instead of 485.
// The norm of 436 MB takes 69 us (0.92).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "q8.cuh"
#include "../../include/dion_adamw.h"

namespace dion {

int num_sms();

namespace {

using namespace q8;

constexpr int kThreads = 256, kPer = 8, kChunk = kThreads * kPer;
static_assert(32 * kPer == DION_ADAMW_BLOCK, "a warp holds one block of an 8-bit state");
constexpr int kBlockLog = 8;
static_assert(1 << kBlockLog == DION_ADAMW_BLOCK, "blocks by shifts");

enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2, kState8 = 4, kWide = 8, kWhole = 16 };   // 16-byte accesses; float32 values in 32 bytes

struct Entry {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    bf16* copy;
    long long n;
    float lr_factor, decay_factor;
    uint32_t index, flags;
};

template <int CAP>
struct Table {
    int count;
    uint32_t chunks;
    uint32_t first[CAP];           // number of each tensor's first chunk
    Entry e[CAP];
};
constexpr int kSmall = 32, kLarge = 384;
static_assert(sizeof(Table<kLarge>) <= 32764 - 256, "kernel parameters");

// Constants of a step, each formed in float64 and rounded once.
struct Constants {
    float b1, c1, b2, c2;          // c = 1 - b
    float rate, root, eps, decay;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), eps, lr * weight_decay
    uint32_t key;                  // of the dither
    float one;                     // 1, where the compiler does not see it (add_apart)
};

// A hash of a 32-bit word: two rounds of shift, exclusive or and product.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x = (x ^ (x >> 16)) * 0x9E3779B1u;
    x = (x ^ (x >> 15)) * 0x85EBCA6Bu;
    return x ^ (x >> 16);
}

__host__ __device__ inline Constants constants(double lr, double b1, double b2, double eps, double wd, long long step,
                                               uint32_t seed)
{
    Constants c;
    c.b1 = (float)b1;
    c.c1 = (float)(1.0 - b1);
    c.b2 = (float)b2;
    c.c2 = (float)(1.0 - b2);
    c.rate = (float)(lr / (1.0 - pow(b1, (double)step)));
    c.root = (float)(1.0 / sqrt(1.0 - pow(b2, (double)step)));
    // (reciprocals take subnormal numbers for zero, and nothing times their infinity is no number)
    c.eps = eps > 0 ? fmaxf((float)eps, 0x1p-126f) : (float)eps;
    c.decay = (float)(lr * wd);
    c.key = mix(seed * 0x632BE5ABu + (uint32_t)step);
    c.one = 1.f;
    return c;
}

// Tensor of chunk c: the last one whose first chunk is at or before it.
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& t, uint32_t c)
{
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Eight consecutive values from p on, of which the first `k` exist.
template <typename T>
__device__ __forceinline__ void load_values(const T* p, bool wide, int k, float2 (&f)[4])
{
    if (wide && k >= 8) {
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
        unpack8(r, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(2 * i < k ? to_f(p[2 * i]) : 0.f, 2 * i + 1 < k ? to_f(p[2 * i + 1]) : 0.f);
    }
}
template <typename T>
__device__ __forceinline__ void store_values(T* p, bool wide, int k, const float2 (&f)[4], bool whole = false)
{
    if (sizeof(T) == 4 && whole && k >= 8) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0].x), "f"(f[0].y), "f"(f[1].x),
                     "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x), "f"(f[3].y)
                     : "memory");
    } else if (wide && k >= 8) {
        Raw8<T> r;
        pack8(r, f);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = r.u[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (2 * i < k) p[2 * i] = from_f<T>(f[i].x);
            if (2 * i + 1 < k) p[2 * i + 1] = from_f<T>(f[i].y);
        }
    }
}
__device__ __forceinline__ uint2 load_bytes(const uint8_t* p, bool wide, int k)
{
    if (wide && k >= 8) return *reinterpret_cast<const uint2*>(p);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < k) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_bytes(uint8_t* p, bool wide, int k, const uint32_t (&w)[2])
{
    if (wide && k >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < k) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// Two E4M3 bytes (the first in the low one) to float32.
__device__ __forceinline__ float2 e4m3_pair(uint32_t w)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    float2 f;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.f32.f16 %0, lo;\n\t"
        "cvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}
__device__ __forceinline__ void e4m3_values(uint2 b, float scale, float2 (&f)[4])
{
    const float2 s = make_float2(scale, scale);
    f[0] = mul2(e4m3_pair(b.x & 0xffffu), s);
    f[1] = mul2(e4m3_pair(b.x >> 16), s);
    f[2] = mul2(e4m3_pair(b.y & 0xffffu), s);
    f[3] = mul2(e4m3_pair(b.y >> 16), s);
}

// The scales of a block's two states from their largest finite magnitudes, and the
// scales' reciprocals.  The division is a product with the reciprocal of 448 and
// Markstein's correction, whose remainder is exact, so that the quotient is rounded
// once; below 2^-100 only the bound counts.  The reciprocal's correction is the
// same, and rounds once but for a scale whose mantissa is all ones (a unit off).
__device__ __forceinline__ void block_scales(float2 amax, float2& scale, float2& inverse)
{
    const float2 by = make_float2(1.f / 448.f, 1.f / 448.f);
    const float2 q = mul2(amax, by);
    const float2 r = fma2(fma2(q, make_float2(-448.f, -448.f), amax), by, q);
    scale = make_float2(fmaxf(r.x, 0x1p-100f), fmaxf(r.y, 0x1p-100f));
    float2 y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(scale.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(scale.y));
    inverse = fma2(fma2(make_float2(-scale.x, -scale.y), y, make_float2(1.f, 1.f)), y, y);
}

// Each element's dither is mix((at + j) ^ key) with at a multiple of eight, so
// that (at + j) ^ key = x ^ j and mix's first shift is the same for all eight:
// the upper 20 bits for the root, the lower 12 and a half for the first moment.
struct Dither {
    uint32_t y;
    __device__ __forceinline__ Dither(long long at, uint32_t key)
    {
        const uint32_t x = (uint32_t)at ^ key ^ (uint32_t)(at >> 32);
        y = x ^ (x >> 16);
    }
    __device__ __forceinline__ uint32_t hash(int j) const
    {
        uint32_t w = (y ^ (uint32_t)j) * 0x9E3779B1u;
        w = (w ^ (w >> 15)) * 0x85EBCA6Bu;
        return w ^ (w >> 16);
    }
    __device__ __forceinline__ uint32_t operator()(int j) const { return hash(j) >> 12; }
    __device__ __forceinline__ uint32_t first(int j) const { return (hash(j) & 0xfffu) << 8 | 0x80u; }
};

// E4M3 bytes of x = r / scale >= 0 (finite), rounded up where the dither
// carries; 0 where an r above zero might have to be raised.  Times 2^-120 a
// float's exponent is that of E4M3 (biases 127 and 7), its subnormals being
// among the float's, and the 20 mantissa bits below E4M3's three are the place
// between two values.  x may exceed 448 by a rounding and is held to 448's code,
// 126.  Four values are 7 instructions beside the additions: upper halves in
// pairs, their minima, and the bytes at bit 4 of each.
__device__ __forceinline__ uint32_t dithered4(float2 a, float2 b, const Dither& dither, int j)
{
    const uint32_t lo = __byte_perm(__float_as_uint(a.x) + dither(j), __float_as_uint(a.y) + dither(j + 1), 0x7632);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x) + dither(j + 2), __float_as_uint(b.y) + dither(j + 3), 0x7632);
    return __byte_perm(__vminu2(lo, 0x07ef07efu) >> 4, __vminu2(hi, 0x07ef07efu) >> 4, 0x6420);
}

// The same with signs: the bytes' upper bits are those of the halves.
__device__ __forceinline__ uint32_t dithered4_signed(float2 a, float2 b, const Dither& dither, int j)
{
    const uint32_t lo = __byte_perm(__float_as_uint(a.x) + dither.first(j), __float_as_uint(a.y) + dither.first(j + 1), 0x7632);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x) + dither.first(j + 2), __float_as_uint(b.y) + dither.first(j + 3), 0x7632);
    const uint32_t l = (__vminu2(lo & 0x7fff7fffu, 0x07ef07efu) >> 4 & 0x007f007fu) | (lo >> 8 & 0x00800080u);
    const uint32_t h = (__vminu2(hi & 0x7fff7fffu, 0x07ef07efu) >> 4 & 0x007f007fu) | (hi >> 8 & 0x00800080u);
    return __byte_perm(l, h, 0x6420);
}

// What a thread holds of a chunk: eight values of each, of which k exist (the
// others are zero).
struct Values {
    float2 p[4], g[4], m[4], v[4];
};

// a + b, rounded by itself.  In packed form the compiler joins an addition with
// the product before it, explicit rounding or not (measured: a quarter of the
// sums had the bits of a fused operation); a multiply-add with a one that it does
// not know cannot be joined.
__device__ __forceinline__ float2 add_apart(float2 a, float2 b, float one) { return fma2(a, make_float2(one, one), b); }

// Moments after the step.  Each operation is rounded once (none is fused with
// another), so that the bits of 8-bit states follow from the formula alone.
__device__ __forceinline__ void moments(Values& x, const Constants& c, float f)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 g = mul2(x.g[j], make_float2(f, f));
        x.m[j] = add_apart(mul2(x.m[j], make_float2(c.b1, c.b1)), mul2(g, make_float2(c.c1, c.c1)), c.one);
        x.v[j] = add_apart(mul2(x.v[j], make_float2(c.b2, c.b2)), mul2(mul2(g, g), make_float2(c.c2, c.c2)), c.one);
    }
}

// The parameters after the step, for r = sqrt(v) times a power of two and root
// divided by it.  The update carries the errors of an approximate root and
// reciprocal, 2^-23 of it each.  exact (float32 parameters): the decay is subtracted
// with the update, p + (u - decay p), since beside one it would be rounded to a
// multiple of 2^-24 (lr * weight_decay of 1e-7 decays by 1.2e-7 then, 2e-8 not at
// all, every value in every step); in bfloat16 that is lost in the parameter's own
// rounding.  An infinite parameter stays.
__device__ __forceinline__ void parameters(Values& x, const float2 (&r)[4], float root, float eps, float rate, float decay, bool exact)
{
    const float keep = 1.f - decay;
    float most = 0.f;
    if (exact)
#pragma unroll
        for (int j = 0; j < 4; ++j) most = fmaxf(most, fmaxf(fabsf(x.p[j].x), fabsf(x.p[j].y)));
    const bool finite = most < __uint_as_float(kInfBits);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 d = fma2(r[j], make_float2(root, root), make_float2(eps, eps));
        float2 i;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i.x) : "f"(d.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i.y) : "f"(d.y));
        const float2 u = mul2(mul2(x.m[j], make_float2(-rate, -rate)), i);
        if (!exact) {
            x.p[j] = fma2(x.p[j], make_float2(keep, keep), u);
            continue;
        }
        float2 p = add2(x.p[j], fma2(x.p[j], make_float2(-decay, -decay), u));
        if (!finite) {
            if (mag_bits(x.p[j].x) == kInfBits) p.x = fmaf(x.p[j].x, keep, u.x);
            if (mag_bits(x.p[j].y) == kInfBits) p.y = fmaf(x.p[j].y, keep, u.y);
        }
        x.p[j] = p;
    }
}

__device__ __forceinline__ uint32_t max3(uint32_t a, uint32_t b, uint32_t c) { return max(max(a, b), c); }

// 2^32 sqrt(v) for 0 <= v < 2^63: Newton's step on s = w / sqrt(w), w = 2^64 v, with
// the residual w - s^2 formed exactly, from a reciprocal root within 2^-22.  The
// result is off the real root by 2^-43 of it before its one rounding, so it is the
// nearest float32 but for a few v in a million (whose root lies that close to
// half-way between two).  A third of the instructions of the function that has no
// such exceptions; w is a normal number for subnormal v too, which the reciprocal
// root would need three more for.
constexpr float kRootScale = 0x1p32f;
constexpr uint32_t kRootBits = 0x5f000000;           // of 2^63
__device__ __forceinline__ float2 roots(float2 v)
{
    const float2 w = mul2(v, make_float2(0x1p64f, 0x1p64f));
    float2 y;                                        // (of zero: finite, and the product with it zero)
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(fmaxf(w.x, 0x1p-90f)));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(fmaxf(w.y, 0x1p-90f)));
    const float2 s = mul2(w, y);
    const float2 residual = fma2(make_float2(-s.x, -s.y), s, w);
    return fma2(residual, mul2(y, make_float2(0.5f, 0.5f)), s);
}

// Where a first moment is rounded by its dither.  Rounded to nearest, a value that a
// step changes by less than half the format's distance there stays what it was, in
// every step: one whose gradient has stopped would never reach zero, while its root
// goes on falling to the least code, and the parameter would move for ever.  The
// next value down is a ninth to a sixteenth away, so
//  - with 1 - beta1 >= 3/32 the decay alone takes every value from 2^-6 on to
//    another one.  Below, all distances are 2^-9, and a value is dithered where the
//    gradient's part is at most that (with a larger part nearest rounding does move
//    it).  Nearest rounding elsewhere has half the error.
//  - with less all values are dithered (ALL).
constexpr float kNearest = 3.f / 32.f;               // least 1 - beta1

// Of a thread's eight bytes of first moments, those below 2^-6 (0x08) of values that are not zero, one bit each.  (In a
// block of zeros, a row of an embedding that no token used, mi is zero.)
__device__ __forceinline__ uint32_t small_codes(const uint32_t (&w)[2], const float2 (&m)[4], float mi)
{
    uint32_t mask = 0;
    if ((((w[0] & 0x78787878u) + 0x78787878u) & ((w[1] & 0x78787878u) + 0x78787878u) & 0x80808080u) != 0x80808080u && mi != 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!(w[j >> 2] >> (8 * (j & 3)) & 0x78u) && (j & 1 ? m[j >> 1].y : m[j >> 1].x) != 0.f) mask |= 1u << j;
    }
    return mask;
}
// Their dithered codes.  Few threads come here and the others' registers are scarce, so what the moments were made of
// is read again (262 million bfloat16 values 485 us; kept in registers, 490 to 497): g, the old bytes m and scale (none is
// overwritten yet); mi: the new scale's reciprocal.
template <typename G>
__device__ __forceinline__ void dither_small(uint32_t mask, const G* g, const uint8_t* m, const float* scale, const Constants& c, float f,
                                             float mi, const Dither& dither, uint32_t (&mw)[2])
{
    do {
        const int j = __ffs(mask) - 1, at = 8 * (j & 3);
        mask &= mask - 1;
        const float part = __fmul_rn(__fmul_rn(to_f(g[j]), f), c.c1);
        const float v = __fadd_rn(__fmul_rn(__fmul_rn(e4m3_pair(m[j]).x, *scale), c.b1), part);
        if (fabsf(part * mi) <= 0x1p-9f) {
            const uint32_t code = (__float_as_uint(fabsf(v * mi) * 0x1p-120f) + dither.first(j)) >> 20;
            const uint32_t w = ((j < 4 ? mw[0] : mw[1]) & ~(0x7fu << at)) | code << at;
            if (j < 4) mw[0] = w;
            else mw[1] = w;
        }
    } while (mask);
}

// The roots of second moments v, times kRootScale, and the 8-bit states of a warp's block of 256; mi: the reciprocal of
// the first moments' scale.
template <bool ALL>
__device__ __forceinline__ void encode(const float2 (&m)[4], const float2 (&v)[4], float2 (&r)[4], const Dither& dither, float& ms,
                                       float& mi, float& rs, uint32_t (&mw)[2], uint32_t (&rw)[2])
{
    // infinities reach the maxima, and a v that is NaN; a NaN of m does not, and has its own byte in the conversion (a
    // dithered one has none, so it counts there)
    float mmax = 0.f;
    uint32_t vmax = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (ALL) {
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(mmax) : "f"(fabsf(m[j].x)));
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(mmax) : "f"(fabsf(m[j].y)));
        } else {
            mmax = fmaxf(mmax, fmaxf(fabsf(m[j].x), fabsf(m[j].y)));
        }
        vmax = max3(vmax, __float_as_uint(v[j].x), __float_as_uint(v[j].y));
    }
    uint32_t mbits = __reduce_max_sync(0xffffffffu, __float_as_uint(mmax));
    vmax = __reduce_max_sync(0xffffffffu, vmax);
    float rmax;
    const bool plain = mbits < kInfBits && vmax < kRootBits;       // the same in all lanes
    if (plain) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = roots(v[j]);
        rmax = roots(make_float2(__uint_as_float(vmax), 0.f)).x;
    } else {
        uint32_t rbits = mbits = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = make_float2(__fsqrt_rn(v[j].x) * kRootScale, __fsqrt_rn(v[j].y) * kRootScale);
            mbits = max3(mbits, finite_mag_bits(m[j].x), finite_mag_bits(m[j].y));
            rbits = max3(rbits, finite_mag_bits(r[j].x), finite_mag_bits(r[j].y));
        }
        mbits = __reduce_max_sync(0xffffffffu, mbits);
        rmax = __uint_as_float(__reduce_max_sync(0xffffffffu, rbits));
    }
    float2 scale, inverse;
    block_scales(make_float2(__uint_as_float(mbits), rmax * (1.f / kRootScale)), scale, inverse);
    ms = scale.x;
    rs = scale.y;
    mi = mbits ? inverse.x : 0.f;
    const float ri = inverse.y * (1.f / kRootScale);
    uint32_t least = 0xffffffffu;
    float2 x[4], y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = mul2(m[j], make_float2(mi, mi));
        if (ALL) {
            y[j] = mul2(y[j], make_float2(0x1p-120f, 0x1p-120f));
        } else {
            const uint32_t w = plain ? cvt2<DION_E4M3>(y[j].x, y[j].y) : cvt2<DION_E4M3>(inf_to_nan(y[j].x), inf_to_nan(y[j].y));
            mw[j >> 1] = j & 1 ? mw[j >> 1] | (w << 16) : w;
        }
        x[j] = mul2(mul2(r[j], make_float2(ri, ri)), make_float2(0x1p-120f, 0x1p-120f));
        least = min(min(least, __float_as_uint(x[j].x)), __float_as_uint(x[j].y));
    }
    if (ALL) {
        mw[0] = dithered4_signed(y[0], y[1], dither, 0);
        mw[1] = dithered4_signed(y[2], y[3], dither, 4);
    }
    rw[0] = dithered4(x[0], x[1], dither, 0);
    rw[1] = dithered4(x[2], x[3], dither, 4);
    if (least < 1u << 20) {                          // below E4M3's least value, 2^-9: may have become zero
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if ((j & 1 ? r[j >> 1].y : r[j >> 1].x) > 0.f && !(rw[j >> 2] >> (8 * (j & 3)) & 0xffu)) rw[j >> 2] |= 1u << (8 * (j & 3));
    }
    if (!plain) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (mag_bits(j & 1 ? r[j >> 1].y : r[j >> 1].x) >= kInfBits) rw[j >> 2] |= 0x7fu << (8 * (j & 3));
            if (ALL && mag_bits(j & 1 ? m[j >> 1].y : m[j >> 1].x) >= kInfBits) mw[j >> 2] |= 0x7fu << (8 * (j & 3));
        }
    }
}

// A step with 8-bit states on what a thread holds; encodes them into mw and rw, with the block's new scales in ms and rs.
template <bool ALL>
__device__ __forceinline__ void step8(Values& x, uint2 mb, uint2 rb, float& ms, float& mi, float& rs, const Constants& c, float f,
                                          float rate, float decay, bool exact, const Dither& dither, uint32_t (&mw)[2],
                                          uint32_t (&rw)[2])
{
    float2 r[4];
    e4m3_values(mb, ms, x.m);
    e4m3_values(rb, rs, x.v);
#pragma unroll
    for (int j = 0; j < 4; ++j) x.v[j] = mul2(x.v[j], x.v[j]);
    moments(x, c, f);
    encode<ALL>(x.m, x.v, r, dither, ms, mi, rs, mw, rw);
    parameters(x, r, c.root * (1.f / kRootScale), c.eps, rate, decay, exact);
}

// A step with float32 states.
__device__ __forceinline__ void step32(Values& x, const Constants& c, float f, float rate, float decay, bool exact)
{
    float2 r[4];
    moments(x, c, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        asm("sqrt.approx.f32 %0, %1;" : "=f"(r[j].x) : "f"(x.v[j].x));
        asm("sqrt.approx.f32 %0, %1;" : "=f"(r[j].y) : "f"(x.v[j].y));
    }
    parameters(x, r, c.root, c.eps, rate, decay, exact);
}

// Whole chunks of a tensor with aligned addresses come through shared memory, each
// warp copying what it will read itself, 16 bytes a lane side by side, so that two
// chunks are in flight and no register waits for them.  The instructions around a
// chunk's eight values a thread count (81 a value with the general loop's branches
// and addresses took 655 us for 262 million bfloat16 values with 8-bit states), so
// types are fixed and addresses are kept.
constexpr int kAhead = 2;
struct Stage {
    // a warp's values in the memory's order, from the start of its 1 KB whatever their type: warps go on to the next
    // tensor, whose types may be others, without waiting for each other
    uint4 value[2][kThreads / 32][64];               // [p | g]
    uint4 state[2][kThreads / 32][64];               // [m | v]
    float scale[2][kThreads / 32];                   // [m | r]
};
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(to);
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(from), "n"(BYTES) : "memory");
}
// A lane's eight values' words of a warp's, copied side by side: word i of lane l is word 32 i + l there.
template <int W>
__device__ __forceinline__ void fetch_words(uint4* to, const uint4* from)
{
#pragma unroll
    for (int i = 0; i < W; ++i) copy_async<16>(to + 32 * i, from + 32 * i);
}
template <typename T>
__device__ __forceinline__ void read_words(const uint4* from, float2 (&f)[4])
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.u[i] = from[i];
    unpack8(r, f);
}
template <typename P, typename G, bool EIGHT, bool ALL = false>
__device__ __forceinline__ void whole_chunks(const Entry& e, long long at, int left, uint32_t step, const Constants& c, float f, float rate,
                                             float decay, uint32_t key, Stage* stages)
{
    using S = typename std::conditional<EIGHT, uint8_t, float>::type;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // (scales' and words' addresses are formed anew: kept, they spill, 262 million bfloat16 values with 8-bit states 491 us
    // and 67 million float32 ones 172 instead of 485 and 160)
    P* p = (P*)e.p + at;
    const G* g = (const G*)e.g + at;                 // (this thread's eight values; as are the next)
    S* m = (S*)e.m + at;
    S* v = (S*)e.v + at;
    bf16* copy = sizeof(P) == 4 && e.copy ? e.copy + at : nullptr;
    constexpr int PW = sizeof(P) / 2, GW = sizeof(G) / 2;          // words of a thread
    auto fetch = [&](Stage& to, int d) {             // chunk d from there
        if (d < left) {
            const long long ahead = (long long)d * step;
            fetch_words<PW>(&to.value[0][warp][lane], (const uint4*)(p + ahead) - (PW - 1) * lane);
            fetch_words<GW>(&to.value[1][warp][lane], (const uint4*)(g + ahead) - (GW - 1) * lane);
            if constexpr (EIGHT) {
                copy_async<8>((uint2*)to.state[0][warp] + lane, m + ahead);
                copy_async<8>((uint2*)to.state[1][warp] + lane, v + ahead);
                if (lane < 2) copy_async<4>(&to.scale[lane][warp], (lane ? e.vs : e.ms) + ((at + ahead) >> kBlockLog));
            } else {
                fetch_words<2>(&to.state[0][warp][lane], (const uint4*)(m + ahead) - lane);
                fetch_words<2>(&to.state[1][warp][lane], (const uint4*)(v + ahead) - lane);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");       // (an empty group keeps the count)
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(stages[i], i);
#pragma unroll 1
    while (left > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (left <= 0) break;
            Stage& from = stages[i];
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            __syncwarp();                            // the other lanes' copies
            Values x;
            read_words<P>(&from.value[0][warp][lane * PW], x.p);
            read_words<G>(&from.value[1][warp][lane * GW], x.g);
            uint2 mb, rb;
            float s0, s1;
            if constexpr (EIGHT) {
                mb = ((const uint2*)from.state[0][warp])[lane], rb = ((const uint2*)from.state[1][warp])[lane];
                s0 = from.scale[0][warp], s1 = from.scale[1][warp];
            } else {
                read_words<float>(&from.state[0][warp][lane * 2], x.m);
                read_words<float>(&from.state[1][warp][lane * 2], x.v);
            }
            __syncwarp();                            // all lanes have read theirs
            fetch(from, kAhead);
            if constexpr (EIGHT) {
                uint32_t mw[2], rw[2];
                float mi;
                const Dither dither(at, key);
                step8<ALL>(x, mb, rb, s0, mi, s1, c, f, rate, decay, sizeof(P) == 4, dither, mw, rw);
                store_values(p, true, 8, x.p);
                *reinterpret_cast<uint2*>(v) = make_uint2(rw[0], rw[1]);
                if (!ALL) {
                    if (const uint32_t mask = small_codes(mw, x.m, mi)) dither_small(mask, g, m, e.ms + (at >> kBlockLog), c, f, mi, dither, mw);
                    __syncwarp();                    // all lanes have read the old scale
                }
                *reinterpret_cast<uint2*>(m) = make_uint2(mw[0], mw[1]);
                if (lane == 0) {
                    e.ms[at >> kBlockLog] = s0;
                    e.vs[at >> kBlockLog] = s1;
                }
            } else {
                step32(x, c, f, rate, decay, sizeof(P) == 4);
                store_values(p, true, 8, x.p, true);
                store_values(m, true, 8, x.m, true);
                store_values(v, true, 8, x.v, true);
            }
            if (sizeof(P) == 4 && copy) {
                store_values(copy, true, 8, x.p);
                copy += step;
            }
            at += step;
            p += step;
            g += step;
            m += step;
            v += step;
            --left;
        }
    }
}

constexpr int kStepCtas = 3;                         // an SM
constexpr int kStepShared = kAhead * sizeof(Stage);
static_assert(kStepCtas * (kStepShared + 1024) <= 228 * 1024, "shared memory of an SM");

// Which states the tensors of a list have.
enum : int { kAll32 = 1, kAll8 = 2, kMixed = 3 };

// (with DEV the constants are read from memory; as parameters they take no registers: 262 million bfloat16 values with
// 8-bit states 485 us instead of 491)
template <int CAP, int KIND, bool DEV>
__global__ void __launch_bounds__(kThreads, kStepCtas)
    adamw_kernel(const __grid_constant__ Table<CAP> t, const __grid_constant__ Constants given, const Constants* dev, const float* scale)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Stage* stages = reinterpret_cast<Stage*>(smem);
    wait_previous();
    allow_next();
    const float f = scale ? *scale : 1.f;
    if (f != f) return;
    Constants read;
    if (DEV) read = *dev;
    const Constants& c = DEV ? read : given;
    const int lane = threadIdx.x & 31;
    const uint32_t step = gridDim.x;
    for (uint32_t chunk = blockIdx.x; chunk < t.chunks;) {
        const int i = tensor_of(t, chunk);
        const Entry& e = t.e[i];
        const uint32_t first = t.first[i], stop = i + 1 < t.count ? t.first[i + 1] : t.chunks;
        const uint32_t flags = e.flags;
        const bool wide = flags & kWide;
        const float rate = c.rate * e.lr_factor, decay = c.decay * e.lr_factor * e.decay_factor;
        const uint32_t key = mix(c.key ^ e.index);
        const bool eight = KIND == kMixed ? flags & kState8 : KIND == kAll8;
        if (flags & (eight ? kWide : kWhole)) {
            const uint32_t full = (uint32_t)(e.n / kChunk), own = chunk - first;
            const int whole = own < full ? (int)((full - own + step - 1) / step) : 0;      // chunks of this CTA
            if (whole > 0) {
                const long long at = (long long)own * kChunk + threadIdx.x * kPer;
                const uint32_t by = step * kChunk;     // (the grid is some thousand CTAs)
                if (KIND != kAll8 && !eight) {
                    if (flags & kParamBf16) {
                        if (flags & kGradBf16) whole_chunks<bf16, bf16, false>(e, at, whole, by, c, f, rate, decay, key, stages);
                        else whole_chunks<bf16, float, false>(e, at, whole, by, c, f, rate, decay, key, stages);
                    } else {
                        if (flags & kGradBf16) whole_chunks<float, bf16, false>(e, at, whole, by, c, f, rate, decay, key, stages);
                        else whole_chunks<float, float, false>(e, at, whole, by, c, f, rate, decay, key, stages);
                    }
                }
                if (KIND != kAll32 && eight) {
                    const bool all = c.c1 < kNearest;
                    if (flags & kParamBf16) {
                        if (flags & kGradBf16) all ? whole_chunks<bf16, bf16, true, true>(e, at, whole, by, c, f, rate, decay, key, stages)
                                                   : whole_chunks<bf16, bf16, true>(e, at, whole, by, c, f, rate, decay, key, stages);
                        else all ? whole_chunks<bf16, float, true, true>(e, at, whole, by, c, f, rate, decay, key, stages)
                                 : whole_chunks<bf16, float, true>(e, at, whole, by, c, f, rate, decay, key, stages);
                    } else {
                        if (flags & kGradBf16) all ? whole_chunks<float, bf16, true, true>(e, at, whole, by, c, f, rate, decay, key, stages)
                                                   : whole_chunks<float, bf16, true>(e, at, whole, by, c, f, rate, decay, key, stages);
                        else all ? whole_chunks<float, float, true, true>(e, at, whole, by, c, f, rate, decay, key, stages)
                                 : whole_chunks<float, float, true>(e, at, whole, by, c, f, rate, decay, key, stages);
                    }
                }
                chunk += whole * step;
            }
        }
        for (; chunk < stop; chunk += step) {
            const long long at = (long long)(chunk - first) * kChunk + threadIdx.x * kPer;
            const long long left = e.n - at;
            // (of the last chunk whole warps may have nothing; a warp stays together)
            if (left + lane * kPer <= 0) continue;
            const int k = (int)max(0ll, min(left, 8ll));
            Values x;
            if (flags & kParamBf16) load_values((const bf16*)e.p + at, wide, k, x.p);
            else load_values((const float*)e.p + at, wide, k, x.p);
            if (flags & kGradBf16) load_values((const bf16*)e.g + at, wide, k, x.g);
            else load_values((const float*)e.g + at, wide, k, x.g);
            if (eight) {
                const long long block = at / DION_ADAMW_BLOCK;
                const uint2 mb = load_bytes((const uint8_t*)e.m + at, wide, k), rb = load_bytes((const uint8_t*)e.v + at, wide, k);
                float ms = e.ms[block], rs = e.vs[block];
                uint32_t mw[2], rw[2];
                float mi;
                const Dither dither(at, key);
                const uint8_t* bytes = (const uint8_t*)e.m + at;
                if (c.c1 < kNearest) {
                    step8<true>(x, mb, rb, ms, mi, rs, c, f, rate, decay, !(flags & kParamBf16), dither, mw, rw);
                } else {
                    step8<false>(x, mb, rb, ms, mi, rs, c, f, rate, decay, !(flags & kParamBf16), dither, mw, rw);
                    const uint32_t mask = small_codes(mw, x.m, mi);
                    if (mask && flags & kGradBf16) dither_small(mask, (const bf16*)e.g + at, bytes, e.ms + block, c, f, mi, dither, mw);
                    else if (mask) dither_small(mask, (const float*)e.g + at, bytes, e.ms + block, c, f, mi, dither, mw);
                }
                __syncwarp();                        // all lanes have read the block's scales
                if (lane == 0) {
                    e.ms[block] = ms;
                    e.vs[block] = rs;
                }
                store_bytes((uint8_t*)e.m + at, wide, k, mw);
                store_bytes((uint8_t*)e.v + at, wide, k, rw);
            } else {
                load_values((const float*)e.m + at, wide, k, x.m);
                load_values((const float*)e.v + at, wide, k, x.v);
                step32(x, c, f, rate, decay, !(flags & kParamBf16));
                store_values((float*)e.m + at, wide, k, x.m);
                store_values((float*)e.v + at, wide, k, x.v);
            }
            if (flags & kParamBf16) {
                store_values((bf16*)e.p + at, wide, k, x.p);
            } else {
                store_values((float*)e.p + at, wide, k, x.p);
                if (e.copy) store_values(e.copy + at, wide, k, x.p);
            }
        }
    }
}

// The constants of a step whose numbers are on the device, and its count.
__global__ void adamw_constants_kernel(const double* hyper, long long* step, uint32_t seed, const float* scale,
                                       Constants* out)
{
    wait_previous();
    allow_next();
    if (scale && *scale != *scale) return;          // a skipped step does not count
    const long long t = *step + 1;
    *out = constants(hyper[0], hyper[1], hyper[2], hyper[3], hyper[4], t, seed);
    *step = t;
}

// ------------------------------------------------------------- gradient norm
// Squares of a thread's eight values of each of N chunks, all loaded first.
template <int N, typename T>
__device__ __forceinline__ float squares(const T* g)
{
    Raw8<T> raw[N];
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) raw[u].u[i] = reinterpret_cast<const uint4*>(g + u * kChunk)[i];
    float2 acc[2] = {};
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float2 x[4];
        unpack8(raw[u], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j & 1] = fma2(x[j], x[j], acc[j & 1]);
    }
    return (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
}

// Sum of the squares of chunks `chunk` .. `end` - 1, in thread 0.
template <int CAP>
__device__ __forceinline__ double sum_squares(const Table<CAP>& t, uint32_t chunk, uint32_t end, double (&sums)[kThreads / 32])
{
    constexpr int N = 4;                             // chunks of float32 in flight, twice as many of bfloat16
    double sum = 0;                                  // of 64 float32 squares at a time
    for (int i = tensor_of(t, chunk); chunk < end; ++i) {
        const Entry& e = t.e[i];
        const uint32_t stop = i + 1 < t.count ? min(end, t.first[i + 1]) : end;
        const uint32_t flags = e.flags;
        long long at = (long long)(chunk - t.first[i]) * kChunk + threadIdx.x * kPer;
        while (chunk < stop) {
            if ((flags & kWide) && chunk + 2 * N <= stop && at + (2 * N - 1) * kChunk + (kThreads - threadIdx.x) * kPer <= e.n) {
                float part;
                if (flags & kGradBf16) {
                    part = squares<2 * N>((const bf16*)e.g + at);
                } else {
                    part = squares<N>((const float*)e.g + at);
                    part += squares<N>((const float*)e.g + at + N * kChunk);
                }
                sum += (double)part;
                chunk += 2 * N;
                at += 2 * N * kChunk;
            } else {
                const int k = (int)max(0ll, min(e.n - at, 8ll));
                float2 g[4], acc = make_float2(0.f, 0.f);
                if (flags & kGradBf16) load_values((const bf16*)e.g + at, flags & kWide, k, g);
                else load_values((const float*)e.g + at, flags & kWide, k, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc = fma2(g[j], g[j], acc);
                sum += (double)(acc.x + acc.y);
                ++chunk;
                at += kChunk;
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kThreads / 32; ++w) sum += sums[w];
    return sum;
}

__device__ __forceinline__ void write_norm(double sum, double max_norm, float* out)
{
    const double norm = sqrt(sum);
    out[0] = (float)norm;
    out[1] = isfinite(norm) ? (float)fmin(1.0, max_norm / (norm + 1e-6)) : __int_as_float(0x7fffffff);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ Table<CAP> t, double* part)
{
    __shared__ double sums[kThreads / 32];
    wait_previous();
    allow_next();
    const double sum = sum_squares(t, (uint32_t)((uint64_t)t.chunks * blockIdx.x / gridDim.x),
                                   (uint32_t)((uint64_t)t.chunks * (blockIdx.x + 1) / gridDim.x), sums);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) grad_norm_join_kernel(const double* part, int parts, double max_norm, float* out)
{
    __shared__ double sums[kThreads / 32];
    wait_previous();
    allow_next();
    double sum = 0;
    for (int i = threadIdx.x; i < parts; i += kThreads) sum += part[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) sum += sums[w];
        write_norm(sum, max_norm, out);
    }
}

// Few values: one cluster's CTAs, joined through distributed shared memory, so
// that a call is one launch and has no workspace.  Lists of few values have many
// small tensors, so 256 threads take single chunks, four of them together, whose
// tensors are told by a table.
constexpr int kFewThreads = 1024, kFewChunks = 512, kMedium = 256;
struct TensorOf {
    uint16_t chunk[kFewChunks];
};
template <int CAP>
__global__ void __launch_bounds__(kFewThreads)
    grad_norm_small_kernel(const __grid_constant__ Table<CAP> t, const __grid_constant__ TensorOf of, const double max_norm, float* out)
{
    constexpr uint32_t N = 4;
    const uint32_t groups = gridDim.x * (kFewThreads / kThreads);      // (the grid is the cluster)
    __shared__ double sums[kFewThreads / 32];
    __shared__ double mine;
    wait_previous();
    allow_next();
    double sum = 0;
    for (uint32_t c = blockIdx.x * (kFewThreads / kThreads) + threadIdx.x / kThreads; c < t.chunks; c += N * groups) {
        // 16-byte words first, as they are (anything done to one would wait for it before the next is asked for);
        // of a chunk without them, its squares
        uint4 raw[N][2];
        bool half[N];
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (uint32_t u = 0; u < N; ++u) {
            const uint32_t chunk = c + u * groups;
            const int i = of.chunk[min(chunk, (uint32_t)kFewChunks - 1)];
            const Entry& e = t.e[i];
            const long long at = ((long long)chunk - t.first[i]) * kChunk + threadIdx.x % kThreads * kPer;
            const int k = chunk < t.chunks ? (int)max(0ll, min(e.n - at, 8ll)) : 0;
            raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            half[u] = e.flags & kGradBf16;
            if (k == 8 && (e.flags & kWide)) {
                const uint4* w = (const uint4*)((const uint8_t*)e.g + at * (half[u] ? 2 : 4));
                raw[u][0] = w[0];
                if (!half[u]) raw[u][1] = w[1];
            } else if (k > 0) {
                float2 g[4];
                if (half[u]) load_values((const bf16*)e.g + at, false, k, g);
                else load_values((const float*)e.g + at, false, k, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc = fma2(g[j], g[j], acc);
            }
        }
#pragma unroll
        for (uint32_t u = 0; u < N; ++u) {
            float2 g[4];
            if (half[u]) {
                Raw8<bf16> r;
                r.u[0] = raw[u][0];
                unpack8(r, g);
            } else {
                Raw8<float> r;
                r.u[0] = raw[u][0];
                r.u[1] = raw[u][1];
                unpack8(r, g);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) acc = fma2(g[j], g[j], acc);
        }
        sum += (double)(acc.x + acc.y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        sum = sums[threadIdx.x];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (threadIdx.x == 0) mine = sum;
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        for (int r = 1; r < (int)gridDim.x; ++r) {
            uint32_t a;
            double v;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(&mine)), "r"(r));
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(a) : "memory");
            sum += v;
        }
        write_norm(sum, max_norm, out);
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");      // its sums have been read
}
static_assert(kFewThreads == 32 * 32, "one warp joins a CTA's warps");

// ---------------------------------------------------------------------- host
size_t bytes_of(dion_dtype t) { return t == DION_F32 ? 4 : 2; }
bool type_ok(dion_dtype t) { return t == DION_F32 || t == DION_BF16; }
bool at_least(const void* p, size_t a) { return p && (uintptr_t)p % a == 0; }

constexpr long long kMostValues = 1ll << 38;

bool grad_ok(const dion_adamw_tensor& t) { return type_ok(t.g_type) && at_least(t.g, bytes_of(t.g_type)); }

bool tensor_ok(const dion_adamw_tensor& t)
{
    if (!grad_ok(t) || !type_ok(t.p_type) || !at_least(t.p, bytes_of(t.p_type))) return false;
    if (!t.m || !t.v || !t.m_scale != !t.v_scale) return false;
    if (t.m_scale ? !at_least(t.m_scale, 4) || !at_least(t.v_scale, 4) : !at_least(t.m, 4) || !at_least(t.v, 4)) return false;
    if (t.copy && (t.p_type != DION_F32 || (uintptr_t)t.copy % 2)) return false;
    return std::isfinite(t.lr_factor) && std::isfinite(t.decay_factor);
}

// Checks a list; `full`: also what a step reads beside the gradients.
dion_status list_ok(int count, const dion_adamw_tensor* tensors, bool full)
{
    if (count < 0 || (count > 0 && !tensors)) return DION_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const dion_adamw_tensor& t = tensors[i];
        if (t.n < 0) return DION_ERR_INVALID_ARG;
        if (t.n > 0 && !(full ? tensor_ok(t) : grad_ok(t))) return DION_ERR_INVALID_ARG;
        if (t.n > kMostValues) return DION_ERR_UNSUPPORTED;
    }
    return DION_OK;
}

// Fills a table with tensors from `i` on; returns the next one's number.
template <int CAP>
int fill(Table<CAP>& t, int i, int count, const dion_adamw_tensor* tensors, bool full)
{
    t.count = 0;
    t.chunks = 0;
    for (; i < count && t.count < CAP; ++i) {
        const dion_adamw_tensor& s = tensors[i];
        if (s.n == 0) continue;
        const uint32_t chunks = (uint32_t)cdiv(s.n, kChunk);
        if (t.chunks + (uint64_t)chunks > 0x7fffffffu) break;      // (the next launch takes it)
        Entry& e = t.e[t.count];
        e.g = s.g;
        e.n = s.n;
        e.flags = s.g_type == DION_BF16 ? (uint32_t)kGradBf16 : 0u;
        uintptr_t all = (uintptr_t)s.g;
        if (full) {
            e.p = s.p;
            e.m = s.m;
            e.v = s.v;
            e.ms = s.m_scale;
            e.vs = s.v_scale;
            e.copy = (bf16*)s.copy;
            e.lr_factor = s.lr_factor;
            e.decay_factor = s.decay_factor;
            e.index = (uint32_t)i;
            e.flags |= (s.p_type == DION_BF16 ? kParamBf16 : 0u) | (s.m_scale ? kState8 : 0u);
            // eight 8-bit states are 8 bytes
            all |= (uintptr_t)s.p | (uintptr_t)s.copy | ((uintptr_t)s.m | (uintptr_t)s.v) << (s.m_scale ? 1 : 0);
        }
        if (all % 16 == 0) e.flags |= kWide;
        if (all % 32 == 0) e.flags |= kWhole;
        t.first[t.count++] = t.chunks;
        t.chunks += chunks;
    }
    return i;
}

template <int CAP, int KIND, bool DEV>
cudaError_t step_table_as(const Table<CAP>& t, const Constants& c, const Constants* dev, const float* scale, cudaStream_t st)
{
    static std::atomic<unsigned long long> attr{0};
    const cudaError_t e = smem_attr_once((const void*)adamw_kernel<CAP, KIND, DEV>, kStepShared, attr);
    if (e != cudaSuccess) return e;
    // Eight times what runs at once, taking chunks in turn: the CTAs at work then read and write side by side, and none
    // ends much later than the others.  262 million bfloat16 values with 8-bit states, before other steps: 501 us, 24 times 525, once 539;
    // with contiguous ranges for each CTA 575.
    const unsigned ctas = (unsigned)std::min<long long>(t.chunks, 8ll * kStepCtas * num_sms());
    return launch_overlapped("adamw", adamw_kernel<CAP, KIND, DEV>, dim3(ctas), dim3(kThreads), kStepShared, st, t, c, dev, scale);
}

template <int CAP, int KIND>
cudaError_t step_table(const Table<CAP>& t, const Constants& c, const Constants* dev, const float* scale, cudaStream_t st)
{
    return dev ? step_table_as<CAP, KIND, true>(t, c, dev, scale, st) : step_table_as<CAP, KIND, false>(t, c, dev, scale, st);
}

template <int CAP>
cudaError_t step_some(int& i, int count, const dion_adamw_tensor* tensors, const Constants& c, const Constants* dev,
                      const float* scale, cudaStream_t st)
{
    Table<CAP> t;
    i = fill(t, i, count, tensors, true);
    if (t.chunks == 0) return cudaSuccess;
    int kind = 0;
    for (int k = 0; k < t.count; ++k) kind |= t.e[k].flags & kState8 ? kAll8 : kAll32;
    // A kernel of one kind of states has the registers for it: 262 million bfloat16 values with 8-bit states 485 us, in the mixed
    // one 495.
    return kind == kAll32 ? step_table<CAP, kAll32>(t, c, dev, scale, st) : kind == kAll8 ? step_table<CAP, kAll8>(t, c, dev, scale, st)
                                                                                          : step_table<CAP, kMixed>(t, c, dev, scale, st);
}

dion_status step_all(int count, const dion_adamw_tensor* tensors, const Constants& c, const Constants* dev,
                     const float* scale, cudaStream_t st)
{
    for (int i = 0; i < count;)
        DION_TRY(count - i <= kSmall ? step_some<kSmall>(i, count, tensors, c, dev, scale, st)
                                     : step_some<kLarge>(i, count, tensors, c, dev, scale, st));
    return DION_OK;
}

template <int CAP>
cudaError_t norm_some(int& i, int count, const dion_adamw_tensor* tensors, double* part, int most, int& parts,
                      cudaStream_t st)
{
    Table<CAP> t;
    i = fill(t, i, count, tensors, false);
    if (t.chunks == 0) return cudaSuccess;
    const int grid = (int)std::min<long long>(t.chunks < 2048 ? t.chunks : cdiv(t.chunks, 16), most);
    double* at = part + parts;
    parts += grid;
    return launch_overlapped("grad_norm", grad_norm_kernel<CAP>, dim3((unsigned)grid), dim3(kThreads), 0, st, t, at);
}

// Partial sums of a launch, one a CTA.  436 MB of bfloat16: 8 CTAs an SM 77 us, 6 69, 4 73, 2 98, 32 94.
int norm_ctas() { return 6 * num_sms(); }
// Launches of a list: by tensors, and by the chunks that a table counts (a
// tensor of kMostValues has 2^27, so one takes 15 at least).
long long norm_launches(int count) { return cdiv(count, kLarge) + cdiv(count, 15); }

// Lists whose norm is one launch without a workspace: 867000 float32 values in 63
// tensors take 9 us on the GPU so and 7 in two launches, but a call, host
// included, takes 9 against 16.
bool few_values(int count, const dion_adamw_tensor* tensors)
{
    if (count > kMedium) return false;
    long long chunks = 0;
    for (int i = 0; i < count && chunks <= kFewChunks; ++i) chunks += cdiv(tensors[i].n, kChunk);
    return chunks <= kFewChunks;
}
// CTAs of that launch's cluster: 16 where the device has room for such a cluster (asked once a device; beyond eight is
// not portable), else 8, which take 11 us for the 867000 values.
template <int CAP>
int norm_cluster()
{
    static std::atomic<unsigned long long> known{0}, wide{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev > 63) return 8;
    const unsigned long long bit = 1ull << dev;
    if (!(known.load(std::memory_order_acquire) & bit)) {
        const auto kernel = grad_norm_small_kernel<CAP>;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 16;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kFewThreads);
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&clusters, (const void*)kernel, &cfg) == cudaSuccess && clusters > 0)
            wide.fetch_or(bit, std::memory_order_acq_rel);
        else
            cudaGetLastError();
        known.fetch_or(bit, std::memory_order_acq_rel);
    }
    return wide.load(std::memory_order_acquire) & bit ? 16 : 8;
}
template <int CAP>
cudaError_t norm_few(int count, const dion_adamw_tensor* tensors, double max_norm, float* out, cudaStream_t st)
{
    Table<CAP> t;
    TensorOf of;
    fill(t, 0, count, tensors, false);
    for (int i = 0; i < t.count; ++i)
        for (uint32_t c = t.first[i]; c < (i + 1 < t.count ? t.first[i + 1] : t.chunks); ++c) of.chunk[c] = (uint16_t)i;
    for (uint32_t c = t.chunks; c < kFewChunks; ++c) of.chunk[c] = 0;
    if (t.count == 0) {                              // (an entry is read for chunks that do not exist as well)
        t.first[0] = 0;
        t.e[0] = Entry{};
    }
    const int cluster = norm_cluster<CAP>();
    return launch_cluster("grad_norm_small", grad_norm_small_kernel<CAP>, dim3((unsigned)cluster), dim3(kFewThreads), cluster, 0, st, t, of,
                          max_norm, out);
}

bool hyper_ok(double lr, double b1, double b2, double eps, double wd)
{
    return std::isfinite(lr) && std::isfinite(wd) && std::isfinite(eps) && eps >= 0 && b1 >= 0 && b1 < 1 && b2 >= 0 && b2 < 1;
}

}  // namespace
}  // namespace dion

using namespace dion;

extern "C" dion_status dion_adamw_step(int count, const dion_adamw_tensor* tensors, double lr, double beta1, double beta2,
                                       double eps, double weight_decay, long long step, unsigned int seed,
                                       const float* grad_scale, void* cuda_stream)
{
    const dion_status ok = list_ok(count, tensors, true);
    if (ok != DION_OK) return ok;
    if (!hyper_ok(lr, beta1, beta2, eps, weight_decay) || step < 1 || (uintptr_t)grad_scale % 4) return DION_ERR_INVALID_ARG;
    return step_all(count, tensors, constants(lr, beta1, beta2, eps, weight_decay, step, seed), nullptr, grad_scale,
                    (cudaStream_t)cuda_stream);
}

extern "C" dion_status dion_adamw_step_dev(int count, const dion_adamw_tensor* tensors, const double* hyper,
                                           long long* step, unsigned int seed, const float* grad_scale, void* workspace,
                                           size_t workspace_bytes, void* cuda_stream)
{
    const dion_status ok = list_ok(count, tensors, true);
    if (ok != DION_OK) return ok;
    if (!at_least(hyper, 8) || !at_least(step, 8) || (uintptr_t)grad_scale % 4) return DION_ERR_INVALID_ARG;
    if (!at_least(workspace, 16) || workspace_bytes < 256) return DION_ERR_WORKSPACE;
    Constants* c = (Constants*)workspace;
    DION_TRY(launch_overlapped("adamw_constants", adamw_constants_kernel, dim3(1), dim3(1), 0, (cudaStream_t)cuda_stream, hyper,
                               step, (uint32_t)seed, grad_scale, c));
    return step_all(count, tensors, Constants{}, c, grad_scale, (cudaStream_t)cuda_stream);
}

extern "C" dion_status dion_grad_norm_workspace_size(int count, size_t* bytes)
{
    if (count < 0 || !bytes) return DION_ERR_INVALID_ARG;
    *bytes = (size_t)norm_launches(count) * norm_ctas() * sizeof(double);
    return DION_OK;
}

extern "C" dion_status dion_grad_norm(int count, const dion_adamw_tensor* tensors, double max_norm, float* out,
                                      void* workspace, size_t workspace_bytes, void* cuda_stream)
{
    const dion_status ok = list_ok(count, tensors, false);
    if (ok != DION_OK) return ok;
    if (!(max_norm > 0) || !at_least(out, 4)) return DION_ERR_INVALID_ARG;
    if (few_values(count, tensors)) {
        const cudaStream_t s = (cudaStream_t)cuda_stream;
        DION_TRY(count <= kSmall ? norm_few<kSmall>(count, tensors, max_norm, out, s) : norm_few<kMedium>(count, tensors, max_norm, out, s));
        return DION_OK;
    }
    size_t need = 0;
    dion_grad_norm_workspace_size(count, &need);
    if (need && (!at_least(workspace, 8) || workspace_bytes < need)) return DION_ERR_WORKSPACE;
    const cudaStream_t st = (cudaStream_t)cuda_stream;
    double* part = (double*)workspace;
    int parts = 0;
    for (int i = 0; i < count;)
        DION_TRY(count - i <= kSmall ? norm_some<kSmall>(i, count, tensors, part, norm_ctas(), parts, st)
                                     : norm_some<kLarge>(i, count, tensors, part, norm_ctas(), parts, st));
    DION_TRY(launch_overlapped("grad_norm_join", grad_norm_join_kernel, dim3(1), dim3(kThreads), 0, st, (const double*)part, parts,
                               max_norm, out));
    return DION_OK;
}
