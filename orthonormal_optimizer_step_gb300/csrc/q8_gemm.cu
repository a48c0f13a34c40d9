// q8_gemm.cu -- C = A B^T for 8-bit operands with a power-of-two scale for
// each 128 values along the contraction, on the 5th-generation tensor cores.
//
// The scales are applied by the tensor core itself: tcgen05.mma of
// kind::mxf8f6f4 multiplies each 32-value slice of the contraction by the
// operand rows' scales, read from tensor memory, so the accumulator needs no
// pass of its own per block.  The four slices of a 128-value block share one
// scale byte (the instruction descriptor selects it), and one 32-bit word per
// operand row carries the scales of four consecutive blocks.
//
// B's rows (the output's columns) are the instruction's M side and A's rows
// its N side, so an accumulator column is a run of consecutive elements of one
// row of C: a warp stores 32 neighbours at once whatever the shapes, and few
// rows of A (single tokens) make the narrow side of the instruction.
//
// Warps of a CTA: 0 loads operand tiles by TMA (128 bytes of the contraction
// a stage, 128-byte swizzle), 1 issues the MMAs and the copies of the scales
// from shared to tensor memory, 2 gathers the scale words into the layout
// that copy takes, 4 and up drain the accumulator.
#include <algorithm>

#include "q8.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace dion {

int num_sms();

namespace {

struct GemmParams {
    int m, n, k;
    int tiles_m, tiles_n;             // of BN rows of A, 128 rows of B
    const uint8_t* sa; long long ldsa; int sa_shift, sa_rows;   // scale row = row >> shift, rows in the table
    const uint8_t* sb; long long ldsb; int sb_shift, sb_rows;
    void* c; long long ldc;
    uint32_t idesc;
    int* status;
};

// Instruction descriptor of kind::mxf8f6f4: A and B formats, N, scale format
// UE8M0, M; the scale byte selectors are added per block.
__host__ uint32_t idesc_mx(int M, int N, uint32_t fmt_m, uint32_t fmt_n)
{
    return (fmt_m << 7) | (fmt_n << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}
__device__ __forceinline__ uint32_t idesc_sf(uint32_t sel) { return (sel << 4) | (sel << 29); }

__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 32 rows of 16 bytes from shared memory to 4 columns of tensor memory, in
// each of the four lane quarters: one scale word of 128 operand rows (row r
// in lane r % 32 of column r / 32).
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr)
{
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(128u >> 4) << 32;   // eight-row groups are 128 bytes apart
    d |= (uint64_t)1 << 46;             // descriptor version; no swizzle
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// A kernel that gave up waiting leaves its last copies and MMAs a millisecond
// to land before it returns its shared and tensor memory.
__device__ __noinline__ void drain_after_abort()
{
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    __syncthreads();
}

constexpr int kSfSlots = 4;

template <int BN>
struct Cfg {
    static constexpr int BM = 128;                     // rows of B a tile
    static constexpr uint32_t P_BYTES = BM * 128, Q_BYTES = BN * 128, STAGE = P_BYTES + Q_BYTES;
    static constexpr int STAGES = BN >= 128 ? 6 : 8;
    static constexpr int SFQ = (BN + 127) / 128;       // 128-row scale groups of A's side
    static constexpr uint32_t SF_BYTES = 512 * (1 + SFQ);
    static constexpr uint32_t ACC = BN < 32 ? 32 : BN; // accumulator columns
    static constexpr uint32_t SF_COL = 2 * ACC;        // scales: 4 (B) + 4 SFQ (A) columns a slot
    static constexpr uint32_t SF_COLS = 4 + 4 * SFQ;
    static constexpr uint32_t TMEM = BN <= 32 ? 128 : BN <= 64 ? 256 : 512;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + kSfSlots * SF_BYTES + 512;
    static_assert(SF_COL + kSfSlots * SF_COLS <= TMEM, "tensor memory columns");
    static_assert(SMEM <= 232448, "shared memory per CTA");
};

// The scale words of 128 rows from row0 on, blocks 4 g .. 4 g + 3: lane l
// takes rows l, l + 32, l + 64, l + 96 (one 16-byte row of the copy's source).
// Rows past the operand (their values are zero) get 2^0.
__device__ __forceinline__ uint4 scale_words(const uint8_t* s, long long ld, int shift, int rows, int row0, int nrows,
                                             int g, int lane)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 32 * i + lane, sr = (row0 + r) >> shift;
        w[i] = r < nrows && sr < rows ? *reinterpret_cast<const uint32_t*>(s + sr * ld + 4ll * g) : 0x7f7f7f7fu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int BN, bool F32>
__global__ void __launch_bounds__(256, 1)
    q8_gemm_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ, const GemmParams p)
{
    using C = Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* sf = smem + C::STAGES * C::STAGE;
    uint64_t* full = (uint64_t*)(sf + kSfSlots * C::SF_BYTES);
    uint64_t* empty = full + C::STAGES;
    uint64_t* sf_full = empty + C::STAGES;
    uint64_t* sf_empty = sf_full + kSfSlots;
    uint64_t* acc_full = sf_empty + kSfSlots;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = (uint32_t*)(acc_empty + 2);
    volatile int* abrt = (volatile int*)(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kSfSlots; ++s) {
            tc::mbar_init(&sf_full[s], 1);
            tc::mbar_init(&sf_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            tc::mbar_init(&acc_empty[b], 4);
        }
        *abrt = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, C::TMEM);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = p.tiles_m * p.tiles_n;
    const int kblocks = (p.k + 127) / 128;

    if (warp == 0) {
        if (lane == 0) {
            tc::tma_prefetch_desc(&tmP);
            tc::tma_prefetch_desc(&tmQ);
            int stage = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int tn = t % p.tiles_n, tm = t / p.tiles_n;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!(ok = tc::mbar_wait(&empty[stage], ph ^ 1, abrt, p.status))) break;
                    uint8_t* s = smem + stage * C::STAGE;
                    tc::mbar_arrive_expect_tx(&full[stage], C::STAGE);
                    tc::tma_load_3d(s, &tmP, &full[stage], kb * 128, tn * C::BM, 0);
                    tc::tma_load_3d(s + C::P_BYTES, &tmQ, &full[stage], kb * 128, tm * BN, 0);
                    if (++stage == C::STAGES) { stage = 0; ph ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0, slot = 0, it = 0;
            uint32_t ph = 0, sph = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++it) {
                const int buf = it & 1;
                if (!(ok = tc::mbar_wait(&acc_empty[buf], ((it >> 1) & 1) ^ 1, abrt, p.status))) break;
                tc::tc_fence_after();
                const uint32_t d = tmem + buf * C::ACC;
                for (int kb = 0; kb < kblocks; ++kb) {
                    const uint32_t sfp = tmem + C::SF_COL + slot * C::SF_COLS, sfq = sfp + 4;
                    if ((kb & 3) == 0) {
                        if (!(ok = tc::mbar_wait(&sf_full[slot], sph, abrt, p.status))) break;
                        tc::tc_fence_after();
                        const uint32_t src = tc::smem_u32(sf + slot * C::SF_BYTES);
                        tmem_cp_scales(sfp, src);
#pragma unroll
                        for (int i = 0; i < C::SFQ; ++i) tmem_cp_scales(sfq + 4 * i, src + 512 * (1 + i));
                    }
                    if (!(ok = tc::mbar_wait(&full[stage], ph, abrt, p.status))) break;
                    tc::tc_fence_after();
                    const uint32_t a0 = tc::smem_u32(smem + stage * C::STAGE), b0 = a0 + C::P_BYTES;
                    const uint32_t idesc = p.idesc | idesc_sf(kb & 3);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_mx(d, tc::make_sdesc(a0 + 32 * j, 16, 1024), tc::make_sdesc(b0 + 32 * j, 16, 1024), idesc,
                               sfp, sfq, (kb | j) != 0);
                    tc::mma_commit(&empty[stage]);
                    if (++stage == C::STAGES) { stage = 0; ph ^= 1; }
                    if ((kb & 3) == 3 || kb == kblocks - 1) {
                        tc::mma_commit(&sf_empty[slot]);
                        if (++slot == kSfSlots) { slot = 0; sph ^= 1; }
                    }
                }
                if (ok) tc::mma_commit(&acc_full[buf]);
            }
        }
    } else if (warp == 2) {
        int slot = 0;
        uint32_t sph = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const int tn = t % p.tiles_n, tm = t / p.tiles_n;
            for (int g = 0; 4 * g < kblocks; ++g) {
                uint4 w[1 + C::SFQ];
                w[0] = scale_words(p.sb, p.ldsb, p.sb_shift, p.sb_rows, tn * C::BM, C::BM, g, lane);
#pragma unroll
                for (int i = 0; i < C::SFQ; ++i)
                    w[1 + i] = scale_words(p.sa, p.ldsa, p.sa_shift, p.sa_rows, tm * BN + 128 * i, BN - 128 * i, g, lane);
                ok = tc::mbar_wait(&sf_empty[slot], sph ^ 1, abrt, p.status);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                uint4* dst = reinterpret_cast<uint4*>(sf + slot * C::SF_BYTES);
#pragma unroll
                for (int i = 0; i < 1 + C::SFQ; ++i) dst[32 * i + lane] = w[i];
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sf_full[slot]);
                if (++slot == kSfSlots) { slot = 0; sph ^= 1; }
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3;          // the lane quarter of tensor memory that this warp reads
        int it = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
            const int tn = t % p.tiles_n, tm = t / p.tiles_n;
            const int buf = it & 1;
            if (!tc::mbar_wait(&acc_full[buf], (it >> 1) & 1, abrt, p.status)) break;
            tc::tc_fence_after();
            const int col = tn * C::BM + q * 32 + lane;
#pragma unroll 1
            for (int j0 = 0; j0 < BN; j0 += 16) {
                uint32_t v[16];
                tc::tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + buf * C::ACC + j0, v);
                tc::tmem_ld_wait();
                const int row0 = tm * BN + j0;
                if (col < p.n) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (row0 + j >= p.m) break;
                        const long long o = (long long)(row0 + j) * p.ldc + col;
                        if (F32) reinterpret_cast<float*>(p.c)[o] = __uint_as_float(v[j]);
                        else reinterpret_cast<bf16*>(p.c)[o] = __float2bfloat16_rn(__uint_as_float(v[j]));
                    }
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
        }
    }
    __syncthreads();
    if (*abrt) drain_after_abort();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, C::TMEM);
    }
}

template <int BN, bool F32>
cudaError_t gemm_go(const Q8MatArgs& a, cudaStream_t st)
{
    using C = Cfg<BN>;
    static std::atomic<unsigned long long> attr{0};
    cudaError_t e = smem_attr_once((const void*)q8_gemm_kernel<BN, F32>, (int)C::SMEM, attr);
    if (e != cudaSuccess) return e;
    CUtensorMap tmP, tmQ;
    if (!make_tmap_3d(&tmP, a.b, TmapType::U8, a.k, a.n, 1, a.ldb, a.ldb, 128, C::BM) ||
        !make_tmap_3d(&tmQ, a.a, TmapType::U8, a.k, a.m, 1, a.lda, a.lda, 128, BN))
        return cudaErrorInvalidValue;
    GemmParams p{};
    p.m = a.m; p.n = a.n; p.k = a.k;
    p.tiles_m = (int)cdiv(a.m, BN);
    p.tiles_n = (int)cdiv(a.n, C::BM);
    p.sa = a.sa; p.ldsa = a.ldsa; p.sa_shift = a.a_square ? 7 : 0; p.sa_rows = a.a_square ? (int)cdiv(a.m, 128) : a.m;
    p.sb = a.sb; p.ldsb = a.ldsb; p.sb_shift = a.b_square ? 7 : 0; p.sb_rows = a.b_square ? (int)cdiv(a.n, 128) : a.n;
    p.c = a.c; p.ldc = a.ldc;
    p.idesc = idesc_mx(C::BM, BN, (uint32_t)a.bfmt, (uint32_t)a.afmt);
    p.status = a.status;
    const long long tiles = (long long)p.tiles_m * p.tiles_n;
    return launch("q8_matmul", q8_gemm_kernel<BN, F32>, dim3((unsigned)std::min<long long>(tiles, num_sms())), dim3(256),
                  C::SMEM, st, tmP, tmQ, p);
}

template <bool F32>
cudaError_t gemm_pick(const Q8MatArgs& a, cudaStream_t st)
{
    if (a.m <= 16) return gemm_go<16, F32>(a, st);
    if (a.m <= 32) return gemm_go<32, F32>(a, st);
    if (a.m <= 64) return gemm_go<64, F32>(a, st);
    return gemm_go<128, F32>(a, st);
}

}  // namespace

cudaError_t q8_matmul(const Q8MatArgs& a, cudaStream_t st)
{
    if (a.m == 0 || a.n == 0) return cudaSuccess;
    if (a.k == 0) {
        const size_t e = a.cdt == DION_F32 ? 4 : 2;
        return cudaMemset2DAsync(a.c, (size_t)a.ldc * e, 0, (size_t)a.n * e, (size_t)a.m, st);
    }
    return a.cdt == DION_F32 ? gemm_pick<true>(a, st) : gemm_pick<false>(a, st);
}

}  // namespace dion
