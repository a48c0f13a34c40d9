// q8_api.cu -- the C entry points of include/dion_q8.h: argument checks, then dispatch.
#include <cmath>

#include "q8.cuh"

using namespace dion;

namespace {

bool type_ok(dion_dtype dt) { return dt == DION_F32 || dt == DION_BF16; }
bool format_ok(dion_q8_format f) { return f == DION_E4M3 || f == DION_E5M2; }
size_t bytes_of(dion_dtype dt) { return dt == DION_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return p && (uintptr_t)p % a == 0; }

// A plain matrix of the given type: rows of `cols` elements that do not overlap.
bool matrix_ok(const void* p, dion_dtype dt, int cols, long long ld) { return aligned(p, bytes_of(dt)) && ld >= cols; }
// The bytes and the scales of a quantized matrix.
bool q8_data_ok(const void* p, int cols, long long ld) { return aligned(p, 16) && ld >= cols && ld % 16 == 0; }
bool q8_scale_ok(const void* p, int cols, long long ld)
{
    return aligned(p, 4) && ld >= cdiv(cols, 128) && ld % 4 == 0;
}

// Tiles of 128 x 128 in one launch.
bool tiles_fit(int rows, int cols) { return cdiv(rows, 128) * cdiv(cols, 128) <= 0x7fffffffll; }

// Whether two rows x cols matrices share an element's byte.  With one pitch
// (columns of a wider matrix, say) they may lie between each other's rows: the
// rows of one start at the same distance behind those of the other everywhere.
// Else their address ranges decide.
bool overlap(const void* p, long long ldp, const void* q, long long ldq, int rows, int cols, dion_dtype dt)
{
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q, row = (uintptr_t)cols * bytes_of(dt);
    const uintptr_t pitch_p = (uintptr_t)ldp * bytes_of(dt), pitch_q = (uintptr_t)ldq * bytes_of(dt);
    if (a >= b + (rows - 1) * pitch_q + row || b >= a + (rows - 1) * pitch_p + row) return false;
    if (ldp != ldq) return true;
    const uintptr_t behind = (a > b ? a - b : b - a) % pitch_p;
    return behind < row || pitch_p - behind < row;
}

dion_status done(cudaError_t e) { return e == cudaSuccess ? DION_OK : DION_ERR_CUDA; }

}  // namespace

extern "C" dion_status dion_q8_quantize(int batch, int rows, int cols, dion_dtype dt, const void* x, long long ldx,
                                        long long sx, const float* rstd, const void* weight, dion_dtype wdt,
                                        int square, dion_q8_format fmt, void* q, long long ldq, long long sq, void* s,
                                        long long lds, long long ss, void* qt, long long ldqt, long long sqt, void* st,
                                        long long ldst, long long sst, void* cuda_stream)
{
    if (batch < 0 || rows < 0 || cols < 0 || !type_ok(dt) || !type_ok(wdt) || !format_ok(fmt) || (square & ~1))
        return DION_ERR_INVALID_ARG;
    if (!q != !s || !qt != !st || (!q && !qt)) return DION_ERR_INVALID_ARG;
    if (!rstd != !weight || (rstd && batch > 1)) return DION_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || cols == 0) return DION_OK;
    if (!matrix_ok(x, dt, cols, ldx)) return DION_ERR_INVALID_ARG;
    if (rstd && (!aligned(rstd, 4) || !aligned(weight, bytes_of(wdt)))) return DION_ERR_INVALID_ARG;
    if (q && (!q8_data_ok(q, cols, ldq) || !q8_scale_ok(s, cols, lds))) return DION_ERR_INVALID_ARG;
    if (qt && (!q8_data_ok(qt, rows, ldqt) || !q8_scale_ok(st, rows, ldst))) return DION_ERR_INVALID_ARG;
    if (batch > 1) {
        const long long sr = square ? cdiv(rows, 128) : rows, sc = square ? cdiv(cols, 128) : cols;
        if (sx < (long long)(rows - 1) * ldx + cols) return DION_ERR_INVALID_ARG;
        if (q && (sq % 16 || sq < (long long)(rows - 1) * ldq + cols || ss % 4 || ss < (sr - 1) * lds + cdiv(cols, 128))) return DION_ERR_INVALID_ARG;
        if (qt && (sqt % 16 || sqt < (long long)(cols - 1) * ldqt + rows || sst % 4 || sst < (sc - 1) * ldst + cdiv(rows, 128)))
            return DION_ERR_INVALID_ARG;
    }
    // indices round up to whole tiles in 32 bits
    if (batch > 65535 || rows > 0x7fff0000 || cols > 0x7fff0000 || !tiles_fit(rows, cols)) return DION_ERR_UNSUPPORTED;
    Q8QuantArgs a{};
    a.batch = batch; a.rows = rows; a.cols = cols;
    a.x = x; a.ldx = ldx; a.sx = sx;
    a.rstd = rstd; a.weight = weight; a.wdt = wdt;
    a.square = square;
    a.q = (uint8_t*)q; a.ldq = ldq; a.sq = sq;
    a.s = (uint8_t*)s; a.lds = lds; a.ss = ss;
    a.qt = (uint8_t*)qt; a.ldqt = ldqt; a.sqt = sqt;
    a.st = (uint8_t*)st; a.ldst = ldst; a.sst = sst;
    return done(q8_quantize(a, dt, fmt, (cudaStream_t)cuda_stream));
}

extern "C" dion_status dion_q8_matmul(int m, int n, int k, const void* a, long long lda, dion_q8_format afmt,
                                      const void* sa, long long ldsa, int a_square, const void* b, long long ldb,
                                      dion_q8_format bfmt, const void* sb, long long ldsb, int b_square, void* c,
                                      long long ldc, dion_dtype cdt, int* status, void* cuda_stream)
{
    if (m < 0 || n < 0 || k < 0 || !type_ok(cdt) || !format_ok(afmt) || !format_ok(bfmt) || (a_square & ~1) ||
        (b_square & ~1) || (uintptr_t)status % 4)
        return DION_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return DION_OK;
    if (!matrix_ok(c, cdt, n, ldc)) return DION_ERR_INVALID_ARG;
    if (k > 0 && (!q8_data_ok(a, k, lda) || !q8_scale_ok(sa, k, ldsa) || !q8_data_ok(b, k, ldb) || !q8_scale_ok(sb, k, ldsb)))
        return DION_ERR_INVALID_ARG;
    // tile counts and the tensor maps' coordinates are 32-bit, their pitches 40-bit
    if (m > 0x7fffff00 || n > 0x7fffff00 || k > 0x7fffff00 || !tiles_fit(m, n) || lda >> 40 || ldb >> 40)
        return DION_ERR_UNSUPPORTED;
    Q8MatArgs g{};
    g.k = k;
    g.a = Q8Side{m, (const uint8_t*)a, lda, afmt, (const uint8_t*)sa, ldsa, a_square};
    g.b = Q8Side{n, (const uint8_t*)b, ldb, bfmt, (const uint8_t*)sb, ldsb, b_square};
    g.c = c; g.ldc = ldc; g.cdt = cdt;
    g.status = status;
    return done(q8_matmul(g, (cudaStream_t)cuda_stream));
}

extern "C" dion_status dion_rms_norm_q8(int rows, int cols, dion_dtype dt, const void* x, long long ldx,
                                        const void* residual, long long ldr, const void* weight, dion_dtype wdt,
                                        float eps, void* h, long long ldh, dion_q8_format fmt, void* q, long long ldq,
                                        void* s, long long lds, float* rstd, void* cuda_stream)
{
    if (rows < 0 || cols < 0 || !type_ok(dt) || !type_ok(wdt) || !format_ok(fmt) || !residual != !h ||
        !(eps >= 0.f) || !std::isfinite(eps))
        return DION_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return DION_OK;
    if (!matrix_ok(x, dt, cols, ldx) || !aligned(weight, bytes_of(wdt)) || (uintptr_t)rstd % 4) return DION_ERR_INVALID_ARG;
    if (residual && (!matrix_ok(residual, dt, cols, ldr) || !matrix_ok(h, dt, cols, ldh))) return DION_ERR_INVALID_ARG;
    if (!q8_data_ok(q, cols, ldq) || !q8_scale_ok(s, cols, lds)) return DION_ERR_INVALID_ARG;
    if (cols > 0x7fff0000) return DION_ERR_UNSUPPORTED;   // column indices round up to whole CTA strides
    Q8NormArgs a{};
    a.rows = rows; a.cols = cols;
    a.x = x; a.ldx = ldx; a.res = residual; a.ldr = ldr;
    a.w = weight; a.wdt = wdt; a.eps = eps;
    a.h = h; a.ldh = ldh;
    a.q = (uint8_t*)q; a.ldq = ldq; a.s = (uint8_t*)s; a.lds = lds;
    a.rstd = rstd;
    return done(rms_norm_q8(a, dt, fmt, (cudaStream_t)cuda_stream));
}

extern "C" dion_status dion_rms_norm_backward_workspace_size(int rows, int cols, size_t* bytes)
{
    if (rows < 0 || cols < 0 || !bytes) return DION_ERR_INVALID_ARG;
    *bytes = norm_backward_workspace(rows, cols);
    return DION_OK;
}

extern "C" dion_status dion_rms_norm_backward(int rows, int cols, dion_dtype dt, const void* dy, long long lddy,
                                              const void* h, long long ldh, const float* rstd, const void* weight,
                                              dion_dtype wdt, const void* dh, long long lddh, void* dx, long long lddx,
                                              float* dw, void* workspace, size_t workspace_bytes, void* cuda_stream)
{
    if (rows < 0 || cols < 0 || !type_ok(dt) || !type_ok(wdt)) return DION_ERR_INVALID_ARG;
    if (cols == 0) return DION_OK;
    if (!aligned(dw, 4)) return DION_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!matrix_ok(dy, dt, cols, lddy) || !matrix_ok(h, dt, cols, ldh) || !matrix_ok(dx, dt, cols, lddx) ||
            !aligned(rstd, 4) || !aligned(weight, bytes_of(wdt)))
            return DION_ERR_INVALID_ARG;
        if (dh && !matrix_ok(dh, dt, cols, lddh)) return DION_ERR_INVALID_ARG;
        if (cols > 0x7fff0000) return DION_ERR_UNSUPPORTED;
        const bool alone = norm_backward_small(rows, cols) && !overlap(dx, lddx, dy, lddy, rows, cols, dt) &&
                           !overlap(dx, lddx, h, ldh, rows, cols, dt);
        if (workspace ? (uintptr_t)workspace % 256 || workspace_bytes < norm_backward_workspace(rows, cols) : !alone)
            return DION_ERR_WORKSPACE;
        if (alone) workspace = nullptr;
    }
    NormBwdArgs a{};
    a.rows = rows; a.cols = cols;
    a.dy = dy; a.lddy = lddy; a.h = h; a.ldh = ldh; a.rstd = rstd;
    a.w = weight; a.wdt = wdt; a.dh = dh; a.lddh = lddh;
    a.dx = dx; a.lddx = lddx; a.dw = dw; a.part = (float*)workspace;
    return done(rms_norm_backward(a, dt, (cudaStream_t)cuda_stream));
}
