// q4.cuh -- 4-bit weights with group scales (include/dion_q4.h): what the
// kernels and the entry points share.
#pragma once

#include "q8.cuh"
#include "../../include/dion_q4.h"

namespace dion {

// A 4-bit matrix.
struct Q4Side {
    int rows, cols, group;
    uint8_t* q; long long ldq;
    bf16* s; long long lds;
};
cudaError_t q4_quantize(const Q4Side& w, dion_dtype dt, const void* x, long long ldx, cudaStream_t st);
cudaError_t q4_dequantize(const Q4Side& w, dion_dtype dt, void* y, long long ldy, cudaStream_t st);

struct Q4MatArgs {
    int m;
    dion_x_type xt;
    const void* x; long long ldx;
    const uint8_t* sx; long long ldsx;
    Q4Side w;
    void* y; long long ldy; dion_dtype ydt;
};
cudaError_t q4_matmul(const Q4MatArgs& a, cudaStream_t st);

}  // namespace dion
