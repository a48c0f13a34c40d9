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
// Either operand can take the instruction's M side (its rows are then the
// accumulator's lanes), the other its N side (the accumulator's columns):
//   A on the M side (rows of C in the lanes): a thread holds consecutive
//     elements of one row of C and packs them into 16-byte words, if C's rows
//     start and end on 16-byte boundaries.
//   B on the M side (columns of C in the lanes): the lanes of a warp hold 32
//     consecutive elements of one row of C and store them together, whatever
//     C's alignment; and few rows of A (single tokens) make the narrow side
//     of the instruction.
// The first form's stores are fewer and wider: 4864 x 4096 x 512 (four
// blocks of contraction a tile, so the stores set the pace) takes 20.1 us
// against 24.9 us.
//
// Warps of a CTA: 0 loads operand tiles by TMA (128 bytes of the contraction
// a stage, 128-byte swizzle), 1 issues the MMAs and the copies of the scales
// from shared to tensor memory, 2 gathers the scale words into the layout
// that copy takes, 4 and up drain the accumulator.  Each of them waits for the
// stream's previous kernel before its first wait on a barrier, whose time limit
// would count that kernel's time otherwise; each in its own branch, as one wait
// of all warps before the branches costs 0.1 us (16x4096x4096 5.66 -> 5.79).
#include <algorithm>

#include "q8.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace dion {

int num_sms();

namespace {

// The operand on the instruction's M side is P, the other Q.
struct GemmParams {
    int np, nq, k;                    // rows of P and of Q, contraction
    int tiles_p, tiles_q;
    const uint8_t* sp; long long ldsp; int sp_shift, sp_rows;   // scale row = row >> shift, rows in the table
    const uint8_t* sq; long long ldsq; int sq_shift, sq_rows;
    void* c; long long ldc;
    int vec4;                         // rows of C start on boundaries of four elements
    int sf16;                         // scale rows start on 16-byte boundaries
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

// CG = 2: the two CTAs of a pair work on one tile, each with its 128 rows of P
// and half of the tile's rows of Q in its own shared memory; the pair's first
// CTA issues for both.
template <int CG>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate)
{
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// 32 rows of 16 bytes from shared memory to 4 columns of tensor memory, in
// each of the four lane quarters: one scale word of 128 operand rows (row r
// in lane r % 32 of column r / 32).  CG = 2: in both CTAs, each from its own
// shared memory.
template <int CG>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr)
{
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(128u >> 4) << 32;   // eight-row groups are 128 bytes apart
    d |= (uint64_t)1 << 46;             // descriptor version; no swizzle
    if (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// Arrives on `bar` (of both CTAs of a pair) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar)
{
    if (CG == 1)
        tc::mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(tc::smem_u32(bar)), "h"((uint16_t)3)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols)
{
    if (CG == 1) {
        tc::tmem_alloc(slot, cols);
        tc::tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(slot)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols)
{
    if (CG == 1)
        tc::tmem_dealloc(taddr, cols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

// One lane of a converged warp.  The branch on it tells the compiler that one
// thread runs: a branch on the lane number does not, and each tcgen05
// instruction behind it then costs about 200 cycles of issue (a pair of MMAs of
// 128 or of 256 columns alike took 205; measured at 4864 x 4096 x 32768).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

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
__device__ __forceinline__ float4 load_remote(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// The address, in the cluster's shared memory, of this CTA's variable in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
    return r;
}
// Arrives on the barrier of the pair's first CTA.
template <int CG>
__device__ __forceinline__ void arrive_first(uint64_t* bar)
{
    if (CG == 1)
        tc::mbar_arrive(bar);
    else
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_rank(bar, 0)) : "memory");
}
// Waits like tc::mbar_wait for arrivals that may come from the peer CTA.
template <int CG>
__device__ __forceinline__ bool wait_peer(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status)
{
    if (!tc::mbar_wait(bar, parity, abort_flag, status)) return false;
    if (CG == 2) {                       // complete: acquires at cluster scope without waiting again
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(tc::smem_u32(bar)), "r"(parity)
            : "memory");
    }
    return true;
}
// TMA load into this CTA's shared memory that completes on the first CTA's barrier.
template <int CG>
__device__ __forceinline__ void tma_load(void* dst, const void* tmap, uint64_t* bar, uint32_t bar_first, int c0, int c1)
{
    if (CG == 1)
        tc::tma_load_3d(dst, tmap, bar, c0, c1, 0);
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
            ::"r"(tc::smem_u32(dst)), "l"((uint64_t)tmap), "r"(bar_first), "r"(c0), "r"(c1), "r"(0)
            : "memory");
}

// A kernel that gave up waiting leaves its last copies and MMAs a millisecond
// to land before it returns its shared and tensor memory.
__device__ __noinline__ void drain_after_abort()
{
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    __syncthreads();
}

constexpr int kOutBytes = 2048;  // a block of C on its way out: 32 rows of 64 bytes
// Scales move in groups of four blocks of the contraction; a slot is what one
// barrier hands over, two groups: in a pair the hand-over is an arrival with
// release at cluster scope, about 1600 cycles beside the operands' traffic (a
// block of a 256 x 224 tile takes 490), and one for every group set the pace
// (8192 x 14336 x 4096 in short loops on one GPU: 293 us, with two groups 274).
constexpr int kSfSlots = 2;
constexpr int kSfGroups = 2;     // of a slot
constexpr int kSplitSlots = 4;   // of one group each, in the split kernel (one CTA)
constexpr int kSfBatch = 4;      // groups whose words are loaded together
static_assert(kSfBatch == 4, "scale_words4 loads four");

template <int CG, int BN>
struct Cfg {
    static constexpr int BM = 128;                     // rows of P that a CTA holds
    static constexpr int QROWS = BN / CG;              // rows of Q that a CTA holds
    static constexpr uint32_t P_BYTES = BM * 128, Q_BYTES = QROWS * 128, STAGE = P_BYTES + Q_BYTES;
    static constexpr int STAGES = QROWS >= 96 ? 6 : 8;
    static constexpr int SFQ = (BN + 127) / 128;       // 128-row scale groups of Q
    static constexpr uint32_t SFG_BYTES = 512 * (1 + SFQ), SF_BYTES = kSfGroups * SFG_BYTES;   // a group's, a slot's
    static constexpr uint32_t ACC = BN < 32 ? 32 : BN; // accumulator columns
    // 512 columns hold two accumulators and the scales up to 224 columns wide.
    // The 256-wide accumulator is single: its eight epilogue warps take it
    // into registers whole (128 columns each) and release it before they store.
    static constexpr int BUFS = BN > 224 ? 1 : 2;
    static constexpr int EW = CG == 2 ? 8 : 4;         // epilogue warps
    static constexpr int EGROUPS = EW / 4;             // warps on each lane quarter, and the columns of one
    static constexpr int ECOLS = EGROUPS == 1 ? BN : (BN / 2 + 31) / 32 * 32;
    static constexpr uint32_t SF_COL = BUFS * ACC;     // scales: 4 (P) + 4 SFQ (Q) columns a group
    static constexpr uint32_t SFG_COLS = 4 + 4 * SFQ, SF_COLS = kSfGroups * SFG_COLS;
    static constexpr uint32_t TMEM = BN <= 32 ? 128 : BN <= 64 ? 256 : 512;
    static constexpr int OUTS = BN < 32 ? 0 : BN > 224 ? 1 : 2;   // such blocks of an epilogue warp
    static constexpr uint32_t OUT = EW * OUTS * kOutBytes;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + OUT + kSfSlots * SF_BYTES + 512;
    static_assert(kSfSlots * SF_BYTES % 512 == 0, "the swizzle of C's blocks repeats every 512 bytes");
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

// The same for groups g0 .. g0 + 3 at once, of rows whose 16 bytes at 4 g0 are
// aligned: a quarter as many loads.
__device__ __forceinline__ void scale_words4(const uint8_t* s, long long ld, int shift, int rows, int row0, int nrows,
                                             int g0, int lane, uint4& w0, uint4& w1, uint4& w2, uint4& w3)
{
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 32 * i + lane, sr = (row0 + r) >> shift;
        u[i] = r < nrows && sr < rows ? *reinterpret_cast<const uint4*>(s + sr * ld + 4ll * g0)
                                      : make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
    }
    w0 = make_uint4(u[0].x, u[1].x, u[2].x, u[3].x);
    w1 = make_uint4(u[0].y, u[1].y, u[2].y, u[3].y);
    w2 = make_uint4(u[0].z, u[1].z, u[2].z, u[3].z);
    w3 = make_uint4(u[0].w, u[1].w, u[2].w, u[3].w);
}

// Tile t of the grid: bands of eight tiles of Q, walked along Q first, so that
// the tiles in flight share both operands' panels in L2.
__device__ __forceinline__ void tile_of(const GemmParams& p, int t, int& tq, int& tp)
{
    const int per_band = 8 * p.tiles_p, band = t / per_band, in = t - band * per_band;
    const int rows = min(8, p.tiles_q - 8 * band);
    tq = 8 * band + in % rows;
    tp = in / rows;
}

// N accumulator columns of a warp, B on the M side: lane l holds column col of
// rows row0 .. row0 + N - 1 of C.
template <bool F32, int N>
__device__ __forceinline__ void store_cols(const GemmParams& p, int row0, int col, const uint32_t (&v)[N])
{
    if (col >= p.np) return;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (row0 + j >= p.nq) break;
        const long long o = (long long)(row0 + j) * p.ldc + col;
        if (F32) reinterpret_cast<float*>(p.c)[o] = __uint_as_float(v[j]);
        else reinterpret_cast<bf16*>(p.c)[o] = __float2bfloat16_rn(__uint_as_float(v[j]));
    }
}

// A on the M side: this lane holds columns col0 .. col0 + 31 of row row0 + lane
// of C, whose rows start and end on 16-byte boundaries (TMA stores whole
// 16-byte words).  The warp's block leaves as stores of 32 rows x 64 bytes from
// shared memory (16-byte word c of row r at c ^ (r / 2 % 4), the 64-byte
// swizzle, so that the lanes' writes meet no bank twice); what lies outside C
// is not written.  Shared memory's bandwidth
// bounds the main loop (a block of a 256 x 224 tile moves 30 KB in by TMA and
// about 30 KB out to the MMAs, at 128 bytes a cycle 470 of its 490 cycles), so
// the epilogue's use of it counts: 8192 x 14336 x 4096 takes 254 us without
// stores, 293 with them, 298 through shared memory and back through registers
// (before the scales' hand-over was halved, see kSfGroups).
template <bool F32, int OUTS>
__device__ __forceinline__ void store_rows(const GemmParams& p, const CUtensorMap* tmC, int row0, int col0,
                                           const uint32_t (&v)[32], uint8_t* buf, int& turn, int lane)
{
    if (row0 >= p.np || col0 >= p.nq) return;
    constexpr int COLS = F32 ? 16 : 32;
#pragma unroll
    for (int h = 0; h < 32 / COLS; ++h) {
        if (col0 + h * COLS >= p.nq) break;
        uint8_t* b = buf + (OUTS == 2 ? turn * kOutBytes : 0);
        if (lane == 0) {                 // the block's last store has been read
            if (OUTS == 2) tc::tma_store_wait_read1();
            else tc::tma_store_wait_read();
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = F32 ? v[(h * COLS + 4 * c + i) % 32]
                           : tc::pack_bf16x2(__uint_as_float(v[(8 * c + 2 * i) % 32]), __uint_as_float(v[(8 * c + 2 * i + 1) % 32]));
            *reinterpret_cast<uint4*>(b + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tc::tma_store_3d(tmC, b, col0 + h * COLS, row0, 0);
            tc::tma_store_commit();
        }
        turn ^= 1;
    }
}

// ROWS: A is on the M side (P), else B is.
template <int CG, int BN, bool F32, bool ROWS>
__global__ void __launch_bounds__(128 + 32 * Cfg<CG, BN>::EW, 1)
    q8_gemm_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmC, const GemmParams p)
{
    using C = Cfg<CG, BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* sf = smem + C::STAGES * C::STAGE;
    uint8_t* out = sf + kSfSlots * C::SF_BYTES;
    uint64_t* full = (uint64_t*)(out + C::OUT);
    uint64_t* empty = full + C::STAGES;
    uint64_t* sf_full = empty + C::STAGES;
    uint64_t* sf_empty = sf_full + kSfSlots;
    uint64_t* acc_full = sf_empty + kSfSlots;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = (uint32_t*)(acc_empty + 2);
    volatile int* abrt = (volatile int*)(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = CG == 2 ? (int)cluster_rank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kSfSlots; ++s) {
            tc::mbar_init(&sf_full[s], CG);
            tc::mbar_init(&sf_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            tc::mbar_init(&acc_empty[b], CG * C::EW);
        }
        *abrt = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) tmem_alloc<CG>(tmem_slot, C::TMEM);
    tc::tc_fence_before();
    if (CG == 2) cluster_sync();
    else __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (threadIdx.x == 0) allow_next();
    const int tiles = p.tiles_p * p.tiles_q;
    const int kblocks = (p.k + 127) / 128;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;

    if (warp == 0) {
        if (elect_one()) {
            tc::tma_prefetch_desc(&tmP);
            tc::tma_prefetch_desc(&tmQ);
            wait_previous();             // (the epilogue's stores come after these loads)
            int stage = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                int tq, tp;
                tile_of(p, t, tq, tp);
                const int prow = (tp * CG + rank) * C::BM, qrow = tq * BN + rank * C::QROWS;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!(ok = tc::mbar_wait(&empty[stage], ph ^ 1, abrt, p.status))) break;
                    uint8_t* s = smem + stage * C::STAGE;
                    const uint32_t bar = CG == 2 ? map_rank(&full[stage], 0) : 0;
                    if (rank == 0) tc::mbar_arrive_expect_tx(&full[stage], CG * C::STAGE);
                    tma_load<CG>(s, &tmP, &full[stage], bar, kb * 128, prow);
                    tma_load<CG>(s + C::P_BYTES, &tmQ, &full[stage], bar, kb * 128, qrow);
                    if (++stage == C::STAGES) { stage = 0; ph ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            wait_previous();
            int stage = 0, slot = 0, buf = 0;
            uint32_t ph = 0, sph = 0, aph = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                if (!(ok = wait_peer<CG>(&acc_empty[buf], aph ^ 1, abrt, p.status))) break;
                tc::tc_fence_after();
                const uint32_t d = tmem + buf * C::ACC;
                for (int kb = 0; kb < kblocks; ++kb) {
                    const int grp = kb / 4 % kSfGroups;
                    const uint32_t sfp = tmem + C::SF_COL + slot * C::SF_COLS + grp * C::SFG_COLS, sfq = sfp + 4;
                    if ((kb & 3) == 0) {
                        if (grp == 0) {
                            if (!(ok = wait_peer<CG>(&sf_full[slot], sph, abrt, p.status))) break;
                            tc::tc_fence_after();
                        }
                        const uint32_t src = tc::smem_u32(sf + slot * C::SF_BYTES + grp * C::SFG_BYTES);
                        tmem_cp_scales<CG>(sfp, src);
#pragma unroll
                        for (int i = 0; i < C::SFQ; ++i) tmem_cp_scales<CG>(sfq + 4 * i, src + 512 * (1 + i));
                    }
                    if (!(ok = tc::mbar_wait(&full[stage], ph, abrt, p.status))) break;
                    tc::tc_fence_after();
                    const uint32_t a0 = tc::smem_u32(smem + stage * C::STAGE), b0 = a0 + C::P_BYTES;
                    const uint32_t idesc = p.idesc | idesc_sf(kb & 3);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_mx<CG>(d, tc::make_sdesc(a0 + 32 * j, 16, 1024), tc::make_sdesc(b0 + 32 * j, 16, 1024), idesc,
                                   sfp, sfq, (kb | j) != 0);
                    commit<CG>(&empty[stage]);
                    if (++stage == C::STAGES) { stage = 0; ph ^= 1; }
                    if (kb % (4 * kSfGroups) == 4 * kSfGroups - 1 || kb == kblocks - 1) {
                        commit<CG>(&sf_empty[slot]);
                        if (++slot == kSfSlots) { slot = 0; sph ^= 1; }
                    }
                }
                if (ok) commit<CG>(&acc_full[buf]);
                if (++buf == C::BUFS) { buf = 0; aph ^= 1; }
            }
        }
    } else if (warp == 2) {
        wait_previous();
        int slot = 0;
        uint32_t sph = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            int tq, tp;
            tile_of(p, t, tq, tp);
            // the words of kSfBatch groups are loaded together: one group at a
            // time, the loads' latency (more than the 2048 cycles of a
            // group's MMAs) set the pace
            const int groups = (kblocks + 3) / 4;
            for (int g0 = 0; g0 < groups && ok; g0 += kSfBatch) {
                uint4 w[kSfBatch][1 + C::SFQ] = {};
                if (p.sf16 && g0 + 4 <= groups) {
                    scale_words4(p.sp, p.ldsp, p.sp_shift, p.sp_rows, (tp * CG + rank) * C::BM, C::BM, g0, lane, w[0][0],
                                 w[1][0], w[2][0], w[3][0]);
#pragma unroll
                    for (int i = 0; i < C::SFQ; ++i)
                        scale_words4(p.sq, p.ldsq, p.sq_shift, p.sq_rows, tq * BN + 128 * i, BN - 128 * i, g0, lane,
                                     w[0][1 + i], w[1][1 + i], w[2][1 + i], w[3][1 + i]);
                } else {
#pragma unroll
                    for (int j = 0; j < kSfBatch; ++j) {
                        if (g0 + j >= groups) break;
                        w[j][0] = scale_words(p.sp, p.ldsp, p.sp_shift, p.sp_rows, (tp * CG + rank) * C::BM, C::BM, g0 + j, lane);
#pragma unroll
                        for (int i = 0; i < C::SFQ; ++i)
                            w[j][1 + i] = scale_words(p.sq, p.ldsq, p.sq_shift, p.sq_rows, tq * BN + 128 * i, BN - 128 * i,
                                                      g0 + j, lane);
                    }
                }
#pragma unroll
                for (int j = 0; j < kSfBatch; j += kSfGroups) {
                    if (g0 + j >= groups) break;
                    ok = tc::mbar_wait(&sf_empty[slot], sph ^ 1, abrt, p.status);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
#pragma unroll
                    for (int e = 0; e < kSfGroups; ++e) {        // (words past the last group are not read)
                        uint4* dst = reinterpret_cast<uint4*>(sf + slot * C::SF_BYTES + e * C::SFG_BYTES);
#pragma unroll
                        for (int i = 0; i < 1 + C::SFQ; ++i) dst[32 * i + lane] = w[j + e][i];
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_first<CG>(&sf_full[slot]);
                    if (++slot == kSfSlots) { slot = 0; sph ^= 1; }
                }
            }
        }
    } else if (warp >= 4) {
        wait_previous();
        const int q = warp & 3;          // the lane quarter of tensor memory that this warp reads
        const int c0 = (warp - 4) / 4 * C::ECOLS;
        uint8_t* outs = out + (warp - 4) * C::OUTS * kOutBytes;
        int turn = 0;
        int buf = 0;
        uint32_t aph = 0;
        for (int t = first; t < tiles; t += step) {
            int tq, tp;
            tile_of(p, t, tq, tp);
            if (!tc::mbar_wait(&acc_full[buf], aph, abrt, p.status)) break;
            tc::tc_fence_after();
            const int lrow = (tp * CG + rank) * C::BM + q * 32;
            const uint32_t src = tmem + ((uint32_t)(q * 32) << 16) + buf * C::ACC + c0;
            if constexpr (C::BUFS == 1) {
                uint32_t v[C::ECOLS / 32][32];
#pragma unroll
                for (int j = 0; j < C::ECOLS / 32; ++j) tc::tmem_ld32(src + 32 * j, v[j]);
                tc::tmem_ld_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_first<CG>(&acc_empty[buf]);
#pragma unroll
                for (int j = 0; j < C::ECOLS / 32; ++j) {
                    if constexpr (ROWS) store_rows<F32, C::OUTS>(p, &tmC, lrow, tq * BN + c0 + 32 * j, v[j], outs, turn, lane);
                    else store_cols<F32>(p, tq * BN + c0 + 32 * j, lrow + lane, v[j]);
                }
            } else {
                constexpr int N = BN < 32 ? 16 : 32;
                const int cols = min(C::ECOLS, BN - c0);
#pragma unroll 1
                for (int j = 0; j < cols; j += N) {
                    uint32_t v[N];
                    if constexpr (N == 16) tc::tmem_ld16(src + j, v);
                    else tc::tmem_ld32(src + j, v);
                    tc::tmem_ld_wait();
                    if constexpr (ROWS) store_rows<F32, C::OUTS>(p, &tmC, lrow, tq * BN + c0 + j, v, outs, turn, lane);
                    else store_cols<F32>(p, tq * BN + c0 + j, lrow + lane, v);
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_first<CG>(&acc_empty[buf]);
            }
            if (++buf == C::BUFS) { buf = 0; aph ^= 1; }
        }
        if (ROWS && lane == 0) tc::tma_store_wait_all();
    }
    __syncthreads();
    if (*abrt) drain_after_abort();
    if (CG == 2) cluster_sync();         // the pair's barriers and tensor memory are both CTAs' until here
    if (warp == 1) {
        tc::tc_fence_after();
        tmem_dealloc<CG>(tmem, C::TMEM);
    }
}

// -------------------------------------------- few tiles: the contraction split
// One tile a cluster of `splits` CTAs, B on the M side.  Each contracts its
// share of the blocks and leaves its sums in its shared memory; then every CTA
// finishes BN / splits of the tile's columns: it reads them from all CTAs (16
// bytes a lane through distributed shared memory; 4-byte remote stores of the
// sums took several times as long) and adds them in the order of the shares,
// so the bits are the same every time.
template <int BN>
struct SplitCfg {
    static constexpr int BM = 128;
    static constexpr uint32_t P_BYTES = BM * 128, Q_BYTES = BN * 128, STAGE = P_BYTES + Q_BYTES;
    static constexpr int STAGES = BN > 128 ? 4 : BN == 128 ? 6 : 8;
    static constexpr int SFQ = (BN + 127) / 128;
    static constexpr uint32_t SF_BYTES = 512 * (1 + SFQ);
    static constexpr uint32_t ACC = BN < 32 ? 32 : BN;
    static constexpr uint32_t SF_COL = ACC, SF_COLS = 4 + 4 * SFQ;
    static constexpr uint32_t TMEM = BN <= 32 ? 64 : BN == 64 ? 128 : BN == 128 ? 256 : 512;
    // Sums [column][128 rows] float, in the place of the stages, which the MMAs have all read by then.
    static constexpr uint32_t SUMS = BN * 512;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + kSplitSlots * SF_BYTES + 512;
    static_assert(SF_COL + kSplitSlots * SF_COLS <= TMEM, "tensor memory columns");
    static_assert(SUMS <= STAGES * STAGE, "sums in the stages' place");
    static_assert(SMEM <= 232448, "shared memory per CTA");
};

template <int BN, bool F32>
__global__ void __launch_bounds__(256, 1)
    q8_gemm_split_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                         const GemmParams p, const int splits)
{
    using C = SplitCfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* sf = smem + C::STAGES * C::STAGE;
    float* sums = (float*)smem;
    uint64_t* full = (uint64_t*)(sf + kSplitSlots * C::SF_BYTES);
    uint64_t* empty = full + C::STAGES;
    uint64_t* sf_full = empty + C::STAGES;
    uint64_t* sf_empty = sf_full + kSplitSlots;
    uint64_t* acc_full = sf_empty + kSplitSlots;
    uint32_t* tmem_slot = (uint32_t*)(acc_full + 1);
    volatile int* abrt = (volatile int*)(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int share = (int)cluster_rank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kSplitSlots; ++s) {
            tc::mbar_init(&sf_full[s], 1);
            tc::mbar_init(&sf_empty[s], 1);
        }
        tc::mbar_init(acc_full, 1);
        *abrt = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) tmem_alloc<1>(tmem_slot, C::TMEM);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (threadIdx.x == 0) allow_next();
    const int tile = blockIdx.x / splits, tq = tile % p.tiles_q, tp = tile / p.tiles_q;
    const int kblocks = (p.k + 127) / 128, per = (kblocks + splits - 1) / splits;
    const int kb0 = min(share * per, kblocks), kb1 = min(kb0 + per, kblocks);
    const int prow = tp * C::BM, qrow = tq * BN;

    if (warp == 0) {
        if (elect_one()) {
            wait_previous();             // (the stores to C come after these loads)
            int stage = 0;
            uint32_t ph = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!tc::mbar_wait(&empty[stage], ph ^ 1, abrt, p.status)) break;
                uint8_t* s = smem + stage * C::STAGE;
                tc::mbar_arrive_expect_tx(&full[stage], C::STAGE);
                tc::tma_load_3d(s, &tmP, &full[stage], kb * 128, prow, 0);
                tc::tma_load_3d(s + C::P_BYTES, &tmQ, &full[stage], kb * 128, qrow, 0);
                if (++stage == C::STAGES) { stage = 0; ph ^= 1; }
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            wait_previous();
            int stage = 0, slot = 0;
            uint32_t ph = 0, sph = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                const uint32_t sfp = tmem + C::SF_COL + slot * C::SF_COLS, sfq = sfp + 4;
                if ((kb & 3) == 0 || kb == kb0) {
                    if (!(ok = tc::mbar_wait(&sf_full[slot], sph, abrt, p.status))) break;
                    tc::tc_fence_after();
                    const uint32_t src = tc::smem_u32(sf + slot * C::SF_BYTES);
                    tmem_cp_scales<1>(sfp, src);
#pragma unroll
                    for (int i = 0; i < C::SFQ; ++i) tmem_cp_scales<1>(sfq + 4 * i, src + 512 * (1 + i));
                }
                if (!(ok = tc::mbar_wait(&full[stage], ph, abrt, p.status))) break;
                tc::tc_fence_after();
                const uint32_t a0 = tc::smem_u32(smem + stage * C::STAGE), b0 = a0 + C::P_BYTES;
                const uint32_t idesc = p.idesc | idesc_sf(kb & 3);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_mx<1>(tmem, tc::make_sdesc(a0 + 32 * j, 16, 1024), tc::make_sdesc(b0 + 32 * j, 16, 1024), idesc,
                               sfp, sfq, (kb != kb0) | (j != 0));
                commit<1>(&empty[stage]);
                if (++stage == C::STAGES) { stage = 0; ph ^= 1; }
                if ((kb & 3) == 3) {
                    commit<1>(&sf_empty[slot]);
                    if (++slot == kSplitSlots) { slot = 0; sph ^= 1; }
                }
            }
            if (ok && kb1 > kb0) commit<1>(acc_full);
        }
    } else if (warp == 2) {
        wait_previous();
        int slot = 0;
        uint32_t sph = 0;
        bool ok = true;
        const int g1 = kb1 > kb0 ? (kb1 + 3) / 4 : 0;
        for (int g0 = kb0 / 4; g0 < g1 && ok; g0 += kSfBatch) {
            uint4 w[kSfBatch][1 + C::SFQ];
#pragma unroll
            for (int j = 0; j < kSfBatch; ++j) {
                if (g0 + j >= g1) break;
                w[j][0] = scale_words(p.sp, p.ldsp, p.sp_shift, p.sp_rows, prow, C::BM, g0 + j, lane);
#pragma unroll
                for (int i = 0; i < C::SFQ; ++i)
                    w[j][1 + i] = scale_words(p.sq, p.ldsq, p.sq_shift, p.sq_rows, qrow + 128 * i, BN - 128 * i, g0 + j, lane);
            }
#pragma unroll
            for (int j = 0; j < kSfBatch; ++j) {
                if (g0 + j >= g1) break;
                ok = tc::mbar_wait(&sf_empty[slot], sph ^ 1, abrt, p.status);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                uint4* dst = reinterpret_cast<uint4*>(sf + slot * C::SF_BYTES);
#pragma unroll
                for (int i = 0; i < 1 + C::SFQ; ++i) dst[32 * i + lane] = w[j][i];
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sf_full[slot]);
                if (++slot == kSplitSlots) { slot = 0; sph ^= 1; }
            }
        }
    }
    if (warp >= 4) {
        wait_previous();
        const int q = warp & 3;          // the lane quarter of tensor memory that this warp reads
        float* dst = sums + q * 32 + lane;
        const bool some = kb1 > kb0;
        if (some) tc::mbar_wait(acc_full, 0, abrt, p.status);
        tc::tc_fence_after();
#pragma unroll 1
        for (int j0 = 0; j0 < BN; j0 += 16) {
            uint32_t v[16];
            if (some) {
                tc::tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + j0, v);
                tc::tmem_ld_wait();
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = 0;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) dst[(j0 + j) * 128] = __uint_as_float(v[j]);
        }
        tc::tc_fence_before();
    }
    __syncwarp();
    cluster_sync();
    // a warp takes one column at a time, a lane four rows of it
    const int mine = (BN + splits - 1) / splits, c1 = min(BN, (share + 1) * mine);
    const int n = prow + 4 * lane;
    for (int c = share * mine + warp; c < c1; c += 8) {
        const int m = qrow + c;
        if (m >= p.nq) break;
        const uint32_t at = tc::smem_u32(sums) + 512 * c + 16 * lane;
        float4 t[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            if (s >= splits) break;
            uint32_t addr;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(at), "r"(s));
            t[s] = load_remote(addr);
        }
#pragma unroll
        for (int s = 1; s < 8; ++s) {
            if (s >= splits) break;
            t[0].x += t[s].x;
            t[0].y += t[s].y;
            t[0].z += t[s].z;
            t[0].w += t[s].w;
        }
        const float v[4] = {t[0].x, t[0].y, t[0].z, t[0].w};
        const long long o = (long long)m * p.ldc + n;
        if (n + 4 <= p.np && p.vec4) {
            if (F32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.c) + o) = t[0];
            else *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(p.c) + o) =
                make_uint2(tc::pack_bf16x2(v[0], v[1]), tc::pack_bf16x2(v[2], v[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (n + i >= p.np) break;
                if (F32) reinterpret_cast<float*>(p.c)[o + i] = v[i];
                else reinterpret_cast<bf16*>(p.c)[o + i] = __float2bfloat16_rn(v[i]);
            }
        }
    }
    __syncwarp();
    cluster_sync();                      // the others have read this CTA's sums
    __syncthreads();
    if (*abrt) drain_after_abort();
    if (warp == 1) {
        tc::tc_fence_after();
        tmem_dealloc<1>(tmem, C::TMEM);
    }
}

// Tensor maps and parameters of a launch with tiles of prows rows of P (boxes
// of 128) and qrows rows of Q (boxes of qbox); false if a map cannot be made.
template <bool F32, bool ROWS>
bool make_params(const Q8MatArgs& a, int prows, int qrows, int qbox, GemmParams& p, CUtensorMap& tmP, CUtensorMap& tmQ)
{
    const Q8Side P = ROWS ? a.a : a.b, Q = ROWS ? a.b : a.a;
    if (!make_tmap_3d(&tmP, P.q, TmapType::U8, a.k, P.rows, 1, P.ld, P.ld, 128, 128) ||
        !make_tmap_3d(&tmQ, Q.q, TmapType::U8, a.k, Q.rows, 1, Q.ld, Q.ld, 128, qbox))
        return false;
    p.np = P.rows; p.nq = Q.rows; p.k = a.k;
    p.tiles_p = (int)cdiv(P.rows, prows);
    p.tiles_q = (int)cdiv(Q.rows, qrows);
    p.sp = P.s; p.ldsp = P.lds; p.sp_shift = P.square ? 7 : 0; p.sp_rows = P.square ? (int)cdiv(P.rows, 128) : P.rows;
    p.sq = Q.s; p.ldsq = Q.lds; p.sq_shift = Q.square ? 7 : 0; p.sq_rows = Q.square ? (int)cdiv(Q.rows, 128) : Q.rows;
    p.sf16 = (uintptr_t)P.s % 16 == 0 && (uintptr_t)Q.s % 16 == 0 && P.lds % 16 == 0 && Q.lds % 16 == 0;
    p.c = a.c; p.ldc = a.ldc;
    p.vec4 = (uintptr_t)a.c % (F32 ? 16 : 8) == 0 && a.ldc % 4 == 0;
    p.idesc = idesc_mx(prows, qrows, (uint32_t)P.fmt, (uint32_t)Q.fmt);
    p.status = a.status;
    return true;
}

template <int CG, int BN, bool F32, bool ROWS>
cudaError_t gemm_go(const Q8MatArgs& a, cudaStream_t st)
{
    using C = Cfg<CG, BN>;
    static std::atomic<unsigned long long> attr{0};
    cudaError_t e = smem_attr_once((const void*)q8_gemm_kernel<CG, BN, F32, ROWS>, (int)C::SMEM, attr);
    if (e != cudaSuccess) return e;
    GemmParams p{};
    CUtensorMap tmP, tmQ;
    if (!make_params<F32, ROWS>(a, C::BM * CG, BN, C::QROWS, p, tmP, tmQ)) return cudaErrorInvalidValue;
    CUtensorMap tmC = tmP;               // used with ROWS only
    if (ROWS && !make_tmap_3d_sw64(&tmC, a.c, F32 ? TmapType::F32 : TmapType::BF16, a.b.rows, a.a.rows, 1,
                                   (uint64_t)a.ldc * (F32 ? 4 : 2), (uint64_t)a.ldc * (F32 ? 4 : 2), F32 ? 16 : 32, 32))
        return cudaErrorInvalidValue;
    const long long tiles = (long long)p.tiles_p * p.tiles_q;
    const unsigned grid = (unsigned)(CG * std::min<long long>(tiles, num_sms() / CG));
    const dim3 block(128 + 32 * C::EW);
    if (CG == 1)
        return launch_overlapped("q8_matmul", q8_gemm_kernel<CG, BN, F32, ROWS>, dim3(grid), block, C::SMEM, st, tmP, tmQ, tmC,
                      p);
    return launch_cluster("q8_matmul_pair", q8_gemm_kernel<CG, BN, F32, ROWS>, dim3(grid), block, CG, C::SMEM, st, tmP, tmQ, tmC, p);
}

template <int BN, bool F32>
cudaError_t gemm_split(const Q8MatArgs& a, int splits, cudaStream_t st)
{
    using C = SplitCfg<BN>;
    static std::atomic<unsigned long long> attr{0};
    cudaError_t e = smem_attr_once((const void*)q8_gemm_split_kernel<BN, F32>, (int)C::SMEM, attr);
    if (e != cudaSuccess) return e;
    GemmParams p{};
    CUtensorMap tmP, tmQ;
    if (!make_params<F32, false>(a, C::BM, BN, BN, p, tmP, tmQ)) return cudaErrorInvalidValue;
    return launch_cluster("q8_matmul_split", q8_gemm_split_kernel<BN, F32>,
                          dim3((unsigned)(p.tiles_p * p.tiles_q * splits)), dim3(256), splits, C::SMEM, st, tmP, tmQ, p, splits);
}

// Shares of the contraction for `tiles` tiles of 128 rows of B: as many as the
// clusters that run at once allow (an SM group holds whole clusters only: 152
// SMs take 46 clusters of 3, 36 of 4, 28, 23, 15, 15 of 8), and none for short
// contractions.  Each takes ceil(kblocks / shares) blocks, the last what is left;
// a share that would have none is dropped (64x1920x2500, 20 blocks: five shares
// 6.3 us, six 6.6; 500x500x2048, four 7.4, five 7.9), but eight stay eight: they
// divide the join evenly, which the eighth does without a block of its own
// (64x1000x3200, 25 blocks: eight 5.6 us, seven 6.1).
// Measured, split / whole, operands from memory: 1x4096x14336 12.9 / 23.7 us,
// 64x4096x4096 8.3 / 10.4, 768x768x16384 16.4 / 29.0; 16x1024x1024 (8 blocks)
// 3.9 / 3.7, 1x4096x1024 4.1 / 4.0, though 12 to 15 blocks would gain
// (64x1500x1500 6.1 / 6.4).  Two shares lose where the tiles fill half the SMs
// with long contractions (1024x1024x8192 16.3 / 16.2), though others would gain
// (900x900x5000 15.4 / 19.5).
int shares(long long tiles, int kblocks)
{
    constexpr int at_once[9] = {0, 0, 0, 46, 36, 28, 23, 15, 15};
    if (kblocks < 16) return 1;
    for (int s = 8; s > 2; --s)
        if (3 * s <= kblocks && tiles <= at_once[s]) return s == 8 ? 8 : (int)cdiv(kblocks, cdiv(kblocks, s));
    return 1;
}

template <int BN, bool F32>
cudaError_t gemm_narrow(const Q8MatArgs& a, cudaStream_t st)
{
    const int s = shares(cdiv(a.b.rows, 128) * cdiv(a.a.rows, BN), (int)cdiv(a.k, 128));
    return s > 1 ? gemm_split<BN, F32>(a, s, st) : gemm_go<1, BN, F32, false>(a, st);
}

template <bool F32>
cudaError_t gemm_pick(const Q8MatArgs& a, cudaStream_t st)
{
    const int m = a.a.rows, n = a.b.rows, kb = (int)cdiv(a.k, 128);
    if (m <= 16) return gemm_narrow<16, F32>(a, st);
    if (m <= 32) return gemm_narrow<32, F32>(a, st);
    if (m <= 64) return gemm_narrow<64, F32>(a, st);
    // All rows of A in one 256-wide tile, where two 128-wide ones are too many
    // for shares (operands from memory): 200x4096x14336 23.1 us against 27.4,
    // 192x4096x9216 19.1 against 18.9, 192x2500x8192 13.8 against 18.8; short
    // contractions lose (200x4096x4096 13.9 against 10.2).  With 24 to 28 tiles in
    // five shares it wins from 112 blocks on only (192x3500x8192 22.0 against
    // 18.9, 192x3500x14336 26.3 against 28.9).
    if (m > 128 && m <= 256 && kb >= 64 && shares(2 * cdiv(n, 128), kb) == 1) {
        const int s = shares(cdiv(n, 128), kb);
        if (s > 1) return gemm_split<256, F32>(a, s, st);
    }
    // TMA stores move whole 16-byte words: C's rows start and end on such boundaries
    const bool aligned = (uintptr_t)a.c % 16 == 0 && (a.ldc * (F32 ? 4 : 2)) % 16 == 0 && n % (F32 ? 4 : 8) == 0;
    // 128 x 128 tiles of one CTA against tiles of a pair, 256 x 256 or 256 x 224
    // (which double the accumulator), by a model of what they were measured to
    // take: start + waves * (time a block * blocks + a tile's end), in us on 152
    // SMs.  A pair reads half as much a product but starts and ends later.
    // Measured, us:                  128     224     256
    //    512 x  4096 x  4096        10.4            17.1
    //   8192 x  2304 x   768        16.0    17.5    17.8
    //   4096 x  4096 x  4096        51.0    41.0    46.6
    //   8192 x  1024 x  4096        36.0    35.8    28.8    (the last wave of 224 is nearly empty)
    //   8192 x 14336 x  4096         372     274     321    (short loops; 293 to 306 in longer ones)
    // Without alignment for TMA stores a 224-wide tile's stores take longer
    // than its share of the main loop is worth (4096 x 4097 x 4096: 57.5, 256: 50.7).
    const long long t1 = cdiv(m, 128) * cdiv(n, 128);
    const int q = aligned ? n : m, other = aligned ? m : n;      // rows of the operand on the N side
    const float one = 3.5f + (float)cdiv(t1, 152) * (0.21f * kb + 0.35f);
    const float w256 = 5.f + (float)cdiv(cdiv(q, 256) * cdiv(other, 256), 76) * (0.30f * kb + 1.2f);
    const float w224 = 5.f + (float)cdiv(cdiv(q, 224) * cdiv(other, 256), 76) * (0.265f * kb + 0.8f);
    if (aligned && w224 < one && w224 < w256) return gemm_go<2, 224, F32, true>(a, st);
    if (w256 < one) return aligned ? gemm_go<2, 256, F32, true>(a, st) : gemm_go<2, 256, F32, false>(a, st);
    const int s = shares(t1, kb);
    if (s > 1) return gemm_split<128, F32>(a, s, st);
    return aligned ? gemm_go<1, 128, F32, true>(a, st) : gemm_go<1, 128, F32, false>(a, st);
}

}  // namespace

cudaError_t q8_matmul(const Q8MatArgs& a, cudaStream_t st)
{
    if (a.a.rows == 0 || a.b.rows == 0) return cudaSuccess;
    if (a.k == 0) {
        const size_t e = a.cdt == DION_F32 ? 4 : 2;
        return cudaMemset2DAsync(a.c, (size_t)a.ldc * e, 0, (size_t)a.b.rows * e, (size_t)a.a.rows, st);
    }
    return a.cdt == DION_F32 ? gemm_pick<true>(a, st) : gemm_pick<false>(a, st);
}

}  // namespace dion
