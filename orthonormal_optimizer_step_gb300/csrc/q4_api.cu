// q4_api.cu -- the C entry points of include/dion_q4.h: argument checks, then dispatch.
#include "q4.cuh"

using namespace dion;

namespace {

bool type_ok(dion_dtype dt) { return dt == DION_F32 || dt == DION_BF16; }
bool aligned(const void* p, size_t a) { return p && (uintptr_t)p % a == 0; }
bool matrix_ok(const void* p, dion_dtype dt, int cols, long long ld) { return aligned(p, dt == DION_F32 ? 4 : 2) && ld >= cols; }
bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }
bool weights_ok(const Q4Side& w)
{
    return aligned(w.q, 16) && w.ldq % 16 == 0 && w.ldq >= 64 * cdiv(w.cols, 128) && aligned(w.s, 2) &&
           w.lds >= cdiv(w.cols, w.group);
}
// Column indices round up to whole chunks, and chunks are numbered in 32 bits.
bool size_ok(int rows, int cols) { return cols <= 0x7fff0000 && cdiv(cols, 128) * rows <= 0x7fff0000ll; }

dion_status done(cudaError_t e) { return e == cudaSuccess ? DION_OK : DION_ERR_CUDA; }

}  // namespace

extern "C" dion_status dion_q4_quantize(int rows, int cols, int group, dion_dtype dt, const void* x, long long ldx,
                                        void* q, long long ldq, void* s, long long lds, void* cuda_stream)
{
    if (rows < 0 || cols < 0 || !group_ok(group) || !type_ok(dt)) return DION_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return DION_OK;
    const Q4Side w{rows, cols, group, (uint8_t*)q, ldq, (bf16*)s, lds};
    if (!matrix_ok(x, dt, cols, ldx) || !weights_ok(w)) return DION_ERR_INVALID_ARG;
    if (!size_ok(rows, cols)) return DION_ERR_UNSUPPORTED;
    return done(q4_quantize(w, dt, x, ldx, (cudaStream_t)cuda_stream));
}

extern "C" dion_status dion_q4_dequantize(int rows, int cols, int group, const void* q, long long ldq, const void* s,
                                          long long lds, dion_dtype dt, void* y, long long ldy, void* cuda_stream)
{
    if (rows < 0 || cols < 0 || !group_ok(group) || !type_ok(dt)) return DION_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return DION_OK;
    const Q4Side w{rows, cols, group, (uint8_t*)q, ldq, (bf16*)s, lds};
    if (!matrix_ok(y, dt, cols, ldy) || !weights_ok(w)) return DION_ERR_INVALID_ARG;
    if (!size_ok(rows, cols)) return DION_ERR_UNSUPPORTED;
    return done(q4_dequantize(w, dt, y, ldy, (cudaStream_t)cuda_stream));
}

extern "C" dion_status dion_q4_matmul(int m, int n, int k, dion_x_type xt, const void* x, long long ldx, const void* sx,
                                      long long ldsx, int group, const void* q, long long ldq, const void* s,
                                      long long lds, dion_dtype ydt, void* y, long long ldy, void* cuda_stream)
{
    if (m < 0 || n < 0 || k < 0 || !group_ok(group) || !type_ok(ydt) || xt < DION_X_F32 || xt > DION_X_E5M2)
        return DION_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return DION_OK;
    if (!matrix_ok(y, ydt, n, ldy)) return DION_ERR_INVALID_ARG;
    // a row's share of eight CTAs in shared memory; the grid's passes over the weights
    if (k > 1 << 17 || m > 65535) return DION_ERR_UNSUPPORTED;
    const Q4Side w{n, k, group, (uint8_t*)q, ldq, (bf16*)s, lds};
    if (k > 0) {
        const bool q8 = xt == DION_X_E4M3 || xt == DION_X_E5M2;
        if (!weights_ok(w) || ldx < k) return DION_ERR_INVALID_ARG;
        // (8-bit rows as dion_q8.h has them)
        if (q8 ? !aligned(x, 16) || ldx % 16 || !aligned(sx, 4) || ldsx % 4 || ldsx < cdiv(k, 128)
               : !aligned(x, xt == DION_X_F32 ? 4 : 2))
            return DION_ERR_INVALID_ARG;
        if (!size_ok(n, k)) return DION_ERR_UNSUPPORTED;
    }
    Q4MatArgs a{};
    a.m = m;
    a.xt = xt; a.x = x; a.ldx = ldx; a.sx = (const uint8_t*)sx; a.ldsx = ldsx;
    a.w = w;
    a.y = y; a.ldy = ldy; a.ydt = ydt;
    return done(q4_matmul(a, (cudaStream_t)cuda_stream));
}
