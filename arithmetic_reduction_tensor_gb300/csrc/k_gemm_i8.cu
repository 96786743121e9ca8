// k_gemm_i8.cu -- matrix product in 8-bit integers with a scale for each
// token and each channel.
//
//   C[t][n] = (float(S) * sa[t]) * sw[n],   S = sum over k of A[t][k] * W[n][k]
//
// with S exact in 32-bit integers, so C's bits depend on the inputs only,
// whatever path, tile, split or order computed S.
//
// A few tokens: gemv_i8_kernel, dot products of four codes at a time on the
// integer units, one warp to two channels; the weights are read once and
// bound it.
//
// More tokens: the fifth-generation tensor cores.  GB300's 8-bit integer
// MMA rate is a small fraction of its binary16 rate, and binary16 serves an
// exact integer product: codes are exact in binary16 (|q| <= 128), products
// (<= 2^14) and sums of up to 1024 of them (<= 2^24) are exact in the
// binary32 accumulator.  So K is cut into chunks of 1024, each one chain of
// tcgen05.mma.kind::f16 into a zeroed TMEM accumulator, and the epilogue adds
// the chunks as 32-bit integers in registers.
//
// The output channels are the MMA's rows (M = 256 over a pair of SMs) and
// the tokens its columns, so that the weights -- the operand that is large
// when tokens are few -- travel to the SM as the 8-bit codes they are and
// are converted there, once per tile: four warps read a 128 x 128 box of
// codes from shared memory, widen them in registers (bias to unsigned,
// a byte permute under the exponent of 1024, one packed subtraction for two
// values) and write them to tensor memory, where the MMA takes its A operand
// from.  Shared memory then carries one byte per weight instead of two,
// and the operand reads of A cost it nothing.  The tokens' codes are widened
// by a short kernel before (i8_prepare_kernel) into 16-bit scratch that TMA
// boxes feed to the MMA as the B operand, half of the tile's tokens per SM.
//
// With few tiles K is also split over CTA pairs: integer additions commute,
// so the splits add into a zeroed 32-bit scratch with atomics and the last
// to arrive scales the tile -- the same bits in any order.
//
// CTA roles (768 threads, one persistent CTA per SM, clusters of two):
//   warp 0        TMA producer: 128 weight rows x 128 codes, and 2 boxes of
//                 64 columns x tile/2 tokens, into a 7-stage ring
//   warp 1        TMEM allocation; the leader's issues the MMAs
//   warps 4..15   conversion, four TMEM stages of 128 k ahead of the MMA
//   warps 16..23  epilogue: two 128-column accumulators, so a chunk's
//                 readout runs beside the next chunk's MMAs
// Every wait gives up after about a second as in the split-K GEMM.
#include <cstring>

#include "kernels.cuh"
#include "rowvec.cuh"
#include "tc05.cuh"

namespace tcr {

__device__ unsigned int g_gemm_i8_fault;

__device__ __forceinline__ void store_out(void *C, int dtype, size_t i, int acc, float sa, float sw)
{
    if (dtype == kOutI32) {
        ((int *)C)[i] = acc;
        return;
    }
    const float v = __fmul_rn(__fmul_rn((float)acc, sa), sw);
    if (dtype == kF16)
        ((uint16_t *)C)[i] = float_to_elem<kF16>(v);
    else if (dtype == kBF16)
        ((uint16_t *)C)[i] = float_to_elem<kBF16>(v);
    else
        ((float *)C)[i] = v;
}

// ---------------------------------------------------------------- few tokens

// 16 codes at p, `left` of them inside the row (the rest read as 0).
__device__ __forceinline__ uint4 ld_codes(const int8_t *p, size_t left, bool aligned)
{
    if (aligned && left >= 16) return ld16(p);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 16; k++)
        if ((size_t)k < left) w[k / 4] |= (uint32_t)(uint8_t)p[k] << (8 * (k % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kGvR = 2;             // channels per warp

// Lane l of a channel's warp takes the codes 16 l + 512 i.
template <int MT>
__global__ void __launch_bounds__(128) gemv_i8_kernel(const I8Args a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    const size_t n0 = ((size_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * kGvR;
    const int lane = threadIdx.x & 31;
    if (n0 >= a.N) return;
    int acc[MT][kGvR];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int r = 0; r < kGvR; r++) acc[m][r] = 0;
#pragma unroll 4
    for (size_t k = (size_t)lane * 16; k < a.K; k += 512) {
        uint4 w[kGvR];
#pragma unroll
        for (int r = 0; r < kGvR; r++)
            w[r] = n0 + r < a.N ? ld_codes(a.W + (n0 + r) * a.ldw + k, a.K - k, a.al_w)
                                : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int m = 0; m < MT; m++) {
            if (m >= (int)a.M) break;
            const uint4 x = ld_codes(a.A + (size_t)m * a.lda + k, a.K - k, a.al_a);
#pragma unroll
            for (int r = 0; r < kGvR; r++) {
                acc[m][r] = __dp4a((int)x.x, (int)w[r].x, acc[m][r]);
                acc[m][r] = __dp4a((int)x.y, (int)w[r].y, acc[m][r]);
                acc[m][r] = __dp4a((int)x.z, (int)w[r].z, acc[m][r]);
                acc[m][r] = __dp4a((int)x.w, (int)w[r].w, acc[m][r]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int r = 0; r < kGvR; r++) {
            const int s = __reduce_add_sync(kFull, acc[m][r]);
            if (lane == m * kGvR + r && m < (int)a.M && n0 + r < a.N)
                store_out(a.C, a.c_dtype, (size_t)m * a.ldc + n0 + r, s, a.sa ? a.sa[m] : 1.0f,
                          a.sw ? a.sw[n0 + r] : 1.0f);
        }
}

// ---------------------------------------------------------------- the operands' preparation

// Four codes of a word as two words of two binary16 values each.  A code
// with its sign bit flipped is q + 128; as the low byte under 0x64 it reads
// 1024 + q + 128, and subtracting 1152 leaves q, exactly.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// Blocks [0, blocks_a): the tokens' codes as binary16, rows of ldf values,
// zero past K.  Blocks up to blocks_a + blocks_w: the weights' codes in rows
// of ldp bytes (only when their own pitch or base does not fit TMA).  The
// rest zero the integer scratch.  A team of 2^team_log2 threads to a row.
__global__ void __launch_bounds__(256) i8_prepare_kernel(const I8Prepare p)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    unsigned b = blockIdx.x;
    const int team = 1 << p.team_log2;
    const int in_team = threadIdx.x & (team - 1);
    const size_t rows_per_block = (size_t)256 >> p.team_log2;
    if (b < p.blocks_a) {
        const size_t r = b * rows_per_block + (threadIdx.x >> p.team_log2);
        if (r >= p.M) return;
        for (size_t c = (size_t)in_team * 16; c < p.ldf; c += (size_t)team * 16) {
            const uint4 q = ld_codes(p.A + r * p.lda + c, p.K > c ? p.K - c : 0, p.al_a);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; k++) widen4(w[k], o[2 * k], o[2 * k + 1]);
            uint4 *dst = reinterpret_cast<uint4 *>(p.Af + r * p.ldf + c);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        return;
    }
    b -= p.blocks_a;
    if (b < p.blocks_w) {
        const size_t r = b * rows_per_block + (threadIdx.x >> p.team_log2);
        if (r >= p.N) return;
        for (size_t c = (size_t)in_team * 16; c < p.ldp; c += (size_t)team * 16)
            *reinterpret_cast<uint4 *>(p.Wp + r * p.ldp + c) =
                ld_codes(p.W + r * p.ldw + c, p.K > c ? p.K - c : 0, false);
        return;
    }
    b -= p.blocks_w;
    const unsigned nz = gridDim.x - p.blocks_a - p.blocks_w;
    for (size_t i = (size_t)b * 256 + threadIdx.x; i < p.zero_words; i += (size_t)nz * 256) p.zero[i] = 0;
}

// ---------------------------------------------------------------- the tensor-core kernel

constexpr int kI8BM = 256;                     // channels of a tile (128 per CTA)
constexpr int kI8MaxTn = 160;                  // tokens of a tile, at most
constexpr int kI8BK = 128;                     // k per stage
constexpr int kI8ChunkSteps = 8;               // 1024 k per exact accumulation
constexpr int kI8WBytes = 128 * kI8BK;         // 16 KiB of codes
constexpr int kI8TBoxBytes = kI8MaxTn / 2 * 128;    // 64 binary16 columns of half the tokens
constexpr int kI8StageBytes = kI8WBytes + 2 * kI8TBoxBytes;
constexpr int kI8Stages = 6;
constexpr int kI8AStages = 3;                  // TMEM stages of the widened weights
constexpr int kI8DCols = kI8MaxTn;             // accumulators at columns 0 and 160
constexpr int kI8ACol = 2 * kI8DCols;          // 320: 64 columns per A stage
constexpr int kI8ConvGroups = 3;               // warpgroups that take the steps in turn
constexpr int kI8EpiWarps = 8;
constexpr int kI8EpiWarp0 = 4 + 4 * kI8ConvGroups;
constexpr int kI8Threads = 32 * (kI8EpiWarp0 + kI8EpiWarps);
// Registers a thread by role (setmaxnreg); their sum over the warpgroups is
// within what the launch holds: 768 threads of 80.
constexpr int kI8RegsLaunch = 80, kI8RegsIssue = 48, kI8RegsConv = 64, kI8RegsEpi = 120;
static_assert(kI8RegsIssue + kI8ConvGroups * kI8RegsConv + kI8EpiWarps / 4 * kI8RegsEpi <=
                  kI8Threads / 128 * kI8RegsLaunch,
              "registers of the launch");
constexpr int kI8OffBars = kI8Stages * kI8StageBytes;
// barriers: wfull[S] (this CTA's codes), full[S] (leader's: both CTAs' tokens
// and converted weights), empty[S], dfull[2], dempty[2] (leader's), drain
constexpr int kI8NumBars = 3 * kI8Stages + 4 + 1;
constexpr int kI8OffMisc = kI8OffBars + 8 * kI8NumBars;
constexpr int kI8SmemBytes = kI8OffMisc + 64 + 1024;
static_assert(kI8SmemBytes <= 232448, "one SM's 227 KiB");
static_assert(kI8ACol + kI8AStages * 64 <= 512, "tensor memory columns");

__device__ __forceinline__ uint32_t i8_cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t i8_map_leader(uint32_t addr)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// One lane of a converged warp.
__device__ __forceinline__ bool i8_elect()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void i8_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What is handed over is tensor memory, ordered by the tcgen05 fences on both
// sides; no generic memory needs the (slow) release.
__device__ __forceinline__ void i8_arrive_leader(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Two blocks of 64 k (block, block + 1) of the tile's tokens from `row` on,
// one after the other in shared memory.
__device__ __forceinline__ void i8_load_tokens(uint32_t dst, const CUtensorMap *map, int row, int block, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"((uint64_t)map), "r"(0), "r"(row), "r"(block), "r"(bar)
        : "memory");
}

// D (+)= A B with A in tensor memory, over the pair.
__device__ __forceinline__ void i8_mma(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void i8_commit(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void i8_commit_local(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void i8_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void i8_ld16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 16; j++) v[j] = __uint_as_float(r[j]);
}

struct I8Unit {
    int split, tc, tt;      // K split, channel tile, token tile
};

// Units in split-major order; within a split, groups of 8 channel tiles,
// the channel tile fastest, so that the tiles in flight share operands in L2.
__device__ __forceinline__ I8Unit i8_decode(const I8Gemm &g, int u)
{
    constexpr int kGroup = 8;
    const int tiles = g.tiles_c * g.tiles_t;
    I8Unit r;
    r.split = u / tiles;
    const int t = u - r.split * tiles;
    const int group = kGroup * g.tiles_t;
    const int first = t / group * kGroup;
    const int in_group = min(g.tiles_c - first, kGroup);
    const int q = t % group;
    r.tc = first + q % in_group;
    r.tt = q / in_group;
    return r;
}

__global__ void __launch_bounds__(kI8Threads, 1)
gemm_i8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_t,
               const I8Gemm g)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t ring = smem_addr(smem);
    const uint32_t bars = ring + kI8OffBars;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wfull = [&](int s) { return bar(s); };
    auto full = [&](int s) { return bar(kI8Stages + s); };
    auto empty = [&](int s) { return bar(2 * kI8Stages + s); };
    auto dfull = [&](int s) { return bar(3 * kI8Stages + s); };
    auto dempty = [&](int s) { return bar(3 * kI8Stages + 2 + s); };
    const uint32_t drain = bar(kI8NumBars - 1);
    uint32_t *misc = (uint32_t *)(smem + kI8OffMisc);
    volatile uint32_t *tmem_holder = misc;
    volatile uint32_t *abort = misc + 1;
    volatile uint32_t *last = misc + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = i8_cluster_rank();
    const bool leader = rank == 0;
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_f(b, parity, abort, &g_gemm_i8_fault); };

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kI8Stages; s++) {
            mbar_init(wfull(s), 1);
            // the tokens' expect and a conversion warpgroup in each CTA
            mbar_init(full(s), 1 + 2 * 4);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(dfull(b), 1);
            mbar_init(dempty(b), 2 * kI8EpiWarps);
        }
        mbar_init(drain, 1);
        *abort = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_w) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_t) : "memory");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr((const void *)tmem_holder)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    i8_cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait_primary();

    // the steps (128 k each) of a split
    auto split_steps = [&](int s) { return min(g.sps, g.steps - s * g.sps); };
    const int half = g.tn / 2;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kI8RegsIssue));
        if (warp == 0) {
            // ---------------- producer (a converged warp, one lane issuing)
            const uint32_t leader_full = i8_map_leader(full(0));
            const uint32_t token_bytes = (uint32_t)(4 * 128 * half);
            int st = 0;
            uint32_t phase = 0;
            uint32_t armed = 0, armed_phase = 0;
            bool ok = true;
            for (int u = pair; u < g.units && ok; u += pairs) {
                const I8Unit c = i8_decode(g, u);
                const int nb = split_steps(c.split);
                const int s0 = c.split * g.sps;
                const int row_w = c.tc * kI8BM + 128 * (int)rank, row_t = c.tt * g.tn + half * (int)rank;
                for (int j = 0; j < nb; j++) {
                    ok = __all_sync(kFull, wait(empty(st), phase ^ 1u));
                    if (!ok) break;
                    const uint32_t dst = ring + (uint32_t)st * kI8StageBytes;
                    if (i8_elect()) {
                        mbar_arrive_expect_tx(wfull(st), kI8WBytes);
                        tma_load_2d(dst, &map_w, (s0 + j) * kI8BK, row_w, wfull(st));
                        if (leader) mbar_arrive_expect_tx(full(st), token_bytes);
                        i8_load_tokens(dst + kI8WBytes, &map_t, row_t, 2 * (s0 + j), leader_full + 8u * (uint32_t)st);
                    }
                    __syncwarp();
                    armed |= 1u << st;
                    armed_phase = (armed_phase & ~(1u << st)) | (phase << st);
                    if (++st == kI8Stages) {
                        st = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort) {
                // let the copies in flight land; the tokens' share a barrier
                // with conversions that may never come, so those get the time
                // of a whole wait
                for (int i = 0; i < kI8Stages; i++)
                    if ((armed >> i) & 1u) (void)mbar_wait_limited(wfull(i), (armed_phase >> i) & 1u);
                const uint64_t t0 = global_ns();
                while (global_ns() - t0 < 10000000ull) {
                }
            }
        } else if (warp == 1 && leader) {
            // ---------------- MMA issuer: the whole warp walks the steps, so
            // that the operands stay in uniform registers; one lane issues
            // kind::f16, D binary32, A and B binary16, M = 256, N = tn
            const uint32_t idesc = (1u << 4) | ((uint32_t)(g.tn >> 3) << 17) | ((uint32_t)(kI8BM >> 4) << 24);
            const uint64_t t_desc0 = smem_desc_sw128(ring + kI8WBytes);
            int st = 0, ta = 0, b = 0;
            uint32_t phase = 0, dphase = 0;
            bool ok = true, withhold = g.inject_stall != 0u;
            for (int u = pair; u < g.units && ok; u += pairs) {
                const I8Unit c = i8_decode(g, u);
                const int nb = split_steps(c.split);
                int in_chunk = 0;
                for (int j = 0; j < nb && ok; j++) {
                    bool ready = true;
                    if (in_chunk == 0) ready = !*abort && wait(dempty(b), ((dphase >> b) & 1u) ^ 1u);
                    ready = ready && wait(full(st), phase);
                    ok = __all_sync(kFull, ready);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(b * kI8DCols);
                    const uint32_t a = tmem + (uint32_t)(kI8ACol + 64 * ta);
                    const uint64_t t_desc = t_desc0 + (uint64_t)st * (kI8StageBytes >> 4);
                    const bool end = in_chunk == kI8ChunkSteps - 1 || j == nb - 1;
                    if (i8_elect()) {
                        i8_mma(d, a, t_desc, idesc, in_chunk > 0 ? 1u : 0u);
#pragma unroll
                        for (int k = 1; k < 8; k++)
                            i8_mma(d, a + 8u * (uint32_t)k,
                                   t_desc + (uint64_t)((k >> 2) * (half << 3) + (k & 3) * 2), idesc, 1u);
                        i8_commit(empty(st));
                        if (end && !withhold) i8_commit(dfull(b));
                    }
                    __syncwarp();
                    if (++st == kI8Stages) {
                        st = 0;
                        phase ^= 1u;
                    }
                    ta = (ta + 1) % kI8AStages;
                    in_chunk++;
                    if (end) {
                        withhold = false;
                        in_chunk = 0;
                        dphase ^= 1u << b;
                        b ^= 1;
                    }
                }
            }
            if (i8_elect()) i8_commit_local(drain);
            __syncwarp();
            (void)mbar_wait_limited(drain, 0u);
        }
    } else if (warp < kI8EpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kI8RegsConv));
        // ---------------- conversion: thread m of a warpgroup widens weight row m
        // of the box; the warpgroups take the steps in turn, so that a step's
        // fixed costs (two waits, the handover) are spread over a whole box
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const int m = 32 * (warp & 3) + lane;
        const uint32_t sw = (uint32_t)(m & 7);         // 128-byte swizzle of the box
        int total = 0;                                 // steps of all units
        for (int u = pair; u < g.units; u += pairs) total += split_steps(i8_decode(g, u).split);
        bool ok = true;
        for (int i = (warp - 4) >> 2; i < total; i += kI8ConvGroups) {
            const int st = i % kI8Stages;
            ok = __all_sync(kFull, wait(wfull(st), (uint32_t)(i / kI8Stages) & 1u));
            if (!ok) break;
            const uint32_t row = ring + (uint32_t)(st * kI8StageBytes + m * kI8BK);
            const uint32_t dst = tmem + lane_base + (uint32_t)(kI8ACol + 64 * (i % kI8AStages));
#pragma unroll
            for (int h = 0; h < 2; h++) {
                uint32_t o[32];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const uint4 w = lds16(row + 16u * ((uint32_t)(4 * h + q) ^ sw));
                    widen4(w.x, o[8 * q], o[8 * q + 1]);
                    widen4(w.y, o[8 * q + 2], o[8 * q + 3]);
                    widen4(w.z, o[8 * q + 4], o[8 * q + 5]);
                    widen4(w.w, o[8 * q + 6], o[8 * q + 7]);
                }
                if (h == 0 && i >= kI8AStages) {
                    // the MMAs that read this TMEM stage last are done
                    const int e = i - kI8AStages;
                    ok = __all_sync(kFull, wait(empty(e % kI8Stages), (uint32_t)(e / kI8Stages) & 1u));
                    if (!ok) break;
                    tc_fence_after();
                }
                i8_st32(dst + 32u * (uint32_t)h, o);
            }
            if (!ok) break;
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) i8_arrive_leader(i8_map_leader(full(st)));
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kI8RegsEpi));
        // ---------------- epilogue: a thread holds one channel, half of the tile's tokens
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const int m = 32 * (warp & 3) + lane;
        const int col0 = warp < kI8EpiWarp0 + 4 ? 0 : half;
        const int nblk = half / 16;
        int b = 0;
        uint32_t dphase = 0;
        for (int u = pair; u < g.units; u += pairs) {
            const I8Unit c = i8_decode(g, u);
            const int nb = split_steps(c.split);
            int acc[kI8MaxTn / 2];
#pragma unroll
            for (int i = 0; i < kI8MaxTn / 2; i++) acc[i] = 0;
            bool live = true;
            for (int j = 0; j < nb; j += kI8ChunkSteps) {
                const bool ready = live && !*abort && wait(dfull(b), (dphase >> b) & 1u);
                live = __all_sync(kFull, ready);
                if (live) {
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < kI8MaxTn / 32; q++) {
                        if (q < nblk) {
                            float v[16];
                            i8_ld16(tmem + lane_base + (uint32_t)(b * kI8DCols + col0 + 16 * q), v);
#pragma unroll
                            for (int i = 0; i < 16; i++) acc[16 * q + i] += __float2int_rn(v[i]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) i8_arrive_leader(i8_map_leader(dempty(b)));
                }
                dphase ^= 1u << b;
                b ^= 1;
            }
            const size_t n = (size_t)c.tc * kI8BM + 128u * rank + (size_t)m;
            const size_t t0 = (size_t)c.tt * (size_t)g.tn + (size_t)col0;
            // the tokens of this thread that exist
            const int nt = n >= g.N || t0 >= g.M ? 0 : (int)min((size_t)half, g.M - t0);
            bool write = true;
            if (g.splits > 1 && live) {
                // this split's share of the tile, then the last split scales it
                int *ws = g.ws + t0 * g.N + n;
#pragma unroll
                for (int i = 0; i < kI8MaxTn / 2; i++) {
                    if (i < nt) atomicAdd(ws, acc[i]);
                    ws += g.N;
                }
                __threadfence();
                named_sync(1, 32 * kI8EpiWarps);
                if (threadIdx.x == 32 * kI8EpiWarp0) {
                    uint32_t *count = g.count + 2 * (c.tt * g.tiles_c + c.tc) + rank;
                    *last = !*abort && atomicAdd(count, 1u) == (uint32_t)(g.splits - 1);
                }
                named_sync(1, 32 * kI8EpiWarps);
                write = *last != 0u;
                if (*abort) {                 // a role of this CTA gave up: its tiles read NaN
                    live = false;
                    write = true;
                } else if (write) {
                    __threadfence();
                    ws = g.ws + t0 * g.N + n;
#pragma unroll
                    for (int i = 0; i < kI8MaxTn / 2; i++) {
                        if (i < nt) acc[i] = __ldcg(ws);
                        ws += g.N;
                    }
                }
            } else if (g.splits > 1) {
                named_sync(1, 32 * kI8EpiWarps);
                if (threadIdx.x == 32 * kI8EpiWarp0) *last = 0u;
                named_sync(1, 32 * kI8EpiWarps);
            }
            if (write && nt > 0) {
                // a wait that gave up leaves NaN (or the least integer)
                const float sw = !live ? __int_as_float(0x7fc00000) : g.sw ? g.sw[n] : 1.0f;
                size_t at = t0 * g.ldc + n;
#pragma unroll
                for (int i = 0; i < kI8MaxTn / 2; i++) {
                    if (i < nt)
                        store_out(g.C, g.c_dtype, at, live ? acc[i] : (int)0x80000000, g.sa ? g.sa[t0 + i] : 1.0f,
                                  sw);
                    at += g.ldc;
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    i8_cluster_sync();
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------- host

// The CTA pairs that can be resident at once on the current device; cached
// per device, 0 when none can.
int gemm_i8_pairs()
{
    static std::mutex mu;
    static std::vector<std::pair<int, int>> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lk(mu);
    for (auto &c : cache)
        if (c.first == dev) return c.second;
    int sms = 0, n = 0;
    if (set_smem_once((void *)gemm_i8_kernel, kI8SmemBytes) == cudaSuccess &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)sms & ~1u);
        cfg.blockDim = dim3(kI8Threads);
        cfg.dynamicSmemBytes = kI8SmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, gemm_i8_kernel, &cfg) != cudaSuccess) n = 0;
    }
    (void)cudaGetLastError();
    cache.emplace_back(dev, n);
    return n;
}

I8Plan gemm_i8_plan(size_t M, size_t N, size_t K, int pairs)
{
    I8Plan p;
    std::memset(&p, 0, sizeof p);
    if (M <= (size_t)kI8GemvTokens) {
        p.launches = 1;
        return p;
    }
    p.tensor = 1;
    p.launches = 2;
    p.steps = (int)((K + kI8BK - 1) / kI8BK);
    p.tiles_c = (int)((N + kI8BM - 1) / kI8BM);
    // the token tile: the one whose waves over the pairs come out shortest
    size_t best = SIZE_MAX;
    for (int tn = 32; tn <= kI8MaxTn; tn += 32) {
        const size_t tt = (M + (size_t)tn - 1) / (size_t)tn;
        const size_t tiles = tt * (size_t)p.tiles_c;
        const size_t waves = (tiles + (size_t)pairs - 1) / (size_t)pairs;
        const size_t cost = waves * (size_t)(tn + 16);
        if (cost <= best) {
            best = cost;
            p.tn = tn;
            p.tiles_t = (int)tt;
        }
    }
    const size_t tiles = (size_t)p.tiles_c * (size_t)p.tiles_t;
    size_t s = (size_t)pairs / tiles;
    if (s > (size_t)p.steps) s = (size_t)p.steps;
    if (s < 1) s = 1;
    p.sps = p.steps ? (p.steps + (int)s - 1) / (int)s : 1;
    p.splits = p.steps ? (p.steps + p.sps - 1) / p.sps : 1;
    p.units = (int)(tiles * (size_t)p.splits);
    p.ldf = (K + 63) / 64 * 64;
    return p;
}

// Scratch bytes of a call: the tokens as binary16, the repacked weights
// (repack_w), the integer scratch and its counters.
size_t gemm_i8_scratch(const I8Plan &p, size_t M, size_t N, bool repack_w)
{
    if (!p.tensor) return 0;
    size_t b = M * p.ldf * 2;
    if (repack_w) b += N * p.ldf;
    b = (b + 255) / 256 * 256;
    if (p.splits > 1) b += (M * N + 2 * (size_t)p.tiles_c * (size_t)p.tiles_t) * 4;
    return b;
}

cudaError_t launch_gemm_i8(const I8Args &a, const I8Plan &p, void *scratch, bool repack_w, bool inject_stall,
                           cudaStream_t stream)
{
    if (!p.tensor) {
        const size_t per_block = 4 * kGvR;
        const dim3 grid((unsigned)((a.N + per_block - 1) / per_block));
        const void *k = a.M <= 1   ? (const void *)gemv_i8_kernel<1>
                        : a.M <= 2 ? (const void *)gemv_i8_kernel<2>
                        : a.M <= 4 ? (const void *)gemv_i8_kernel<4>
                                   : (const void *)gemv_i8_kernel<8>;
        void *args[] = {(void *)&a};
        return launch_first(k, grid, dim3(128), args, 0, stream);
    }
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    I8Prepare q;
    std::memset(&q, 0, sizeof q);
    q.A = a.A;
    q.lda = a.lda;
    q.M = a.M;
    q.K = a.K;
    q.N = a.N;
    q.al_a = a.al_a;
    q.Af = (uint16_t *)scratch;
    q.ldf = p.ldf;
    while (q.team_log2 < 8 && ((size_t)16 << q.team_log2) < p.ldf) q.team_log2++;
    const size_t rpb = (size_t)256 >> q.team_log2;
    q.blocks_a = (unsigned)((a.M + rpb - 1) / rpb);
    const int8_t *w = a.W;
    size_t ldw = a.ldw;
    size_t off = a.M * p.ldf * 2;
    if (repack_w) {
        q.W = a.W;
        q.ldw = a.ldw;
        q.Wp = (int8_t *)scratch + off;
        q.ldp = p.ldf;
        q.blocks_w = (unsigned)((a.N + rpb - 1) / rpb);
        w = q.Wp;
        ldw = p.ldf;
        off += a.N * p.ldf;
    }
    off = (off + 255) / 256 * 256;
    I8Gemm g;
    std::memset(&g, 0, sizeof g);
    unsigned blocks_z = 0;
    if (p.splits > 1) {
        q.zero = (int *)((char *)scratch + off);
        q.zero_words = a.M * a.N + 2 * (size_t)p.tiles_c * (size_t)p.tiles_t;
        const size_t nb = (q.zero_words + 1023) / 1024;
        blocks_z = (unsigned)(nb < 304 ? nb : 304);
        g.ws = q.zero;
        g.count = (uint32_t *)(q.zero + a.M * a.N);
    }
    alignas(64) CUtensorMap mw, mt;
    const cuuint32_t estride[2] = {1, 1};
    const cuuint64_t dw[2] = {(cuuint64_t)(repack_w ? p.ldf : a.K), (cuuint64_t)a.N};
    const cuuint64_t sw[1] = {(cuuint64_t)ldw};
    const cuuint32_t bw[2] = {kI8BK, 128};
    // the tokens as (64 k, token, block of 64 k)
    const cuuint32_t estride3[3] = {1, 1, 1};
    const cuuint64_t dt[3] = {64, (cuuint64_t)a.M, (cuuint64_t)(p.ldf / 64)};
    const cuuint64_t stt[2] = {(cuuint64_t)p.ldf * 2, 128};
    const cuuint32_t bt[3] = {64, (cuuint32_t)(p.tn / 2), 2};
    if (encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)w, dw, sw, bw, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        encode(&mt, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, (void *)q.Af, dt, stt, bt, estride3,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    void *args1[] = {(void *)&q};
    cudaError_t e = launch_first((const void *)i8_prepare_kernel, dim3(q.blocks_a + q.blocks_w + blocks_z), dim3(256),
                                 args1, 0, stream);
    if (e != cudaSuccess) return e;
    g.sa = a.sa;
    g.sw = a.sw;
    g.C = a.C;
    g.ldc = a.ldc;
    g.M = a.M;
    g.N = a.N;
    g.c_dtype = a.c_dtype;
    g.tn = p.tn;
    g.tiles_c = p.tiles_c;
    g.tiles_t = p.tiles_t;
    g.steps = p.steps;
    g.sps = p.sps;
    g.splits = p.splits;
    g.units = p.units;
    g.inject_stall = inject_stall ? 1u : 0u;
    const int pairs = gemm_i8_pairs();
    void *args[] = {(void *)&mw, (void *)&mt, (void *)&g};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (p.units < pairs ? p.units : pairs)));
    cfg.blockDim = dim3(kI8Threads);
    cfg.dynamicSmemBytes = kI8SmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, (const void *)gemm_i8_kernel, args);
}

cudaError_t read_gemm_i8_faults(unsigned int *flags, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_gemm_i8_fault, sizeof(unsigned int));
    if (e != cudaSuccess || !clear) return e;
    const unsigned int zero = 0u;
    return cudaMemcpyToSymbol(g_gemm_i8_fault, &zero, sizeof(unsigned int));
}

}  // namespace tcr
