// k_gemm_i8.cu -- matrix product in 8-bit integers with a scale for each
// token and each channel.
//
//   C[t][n] = (float(S) * sa[t]) * sw[n],   S = sum over k of A[t][k] * W[n][k]
//
// with S exact in 32-bit integers, so C's bits depend on the inputs only,
// whatever path, tile, split or order computed S.
//
// Few tokens and small matrices go to k_gemm_i8_few.cu (gemm_i8_plan says
// when); the rest run here, on the fifth-generation tensor cores.  GB300's
// 8-bit integer MMA rate is a small fraction of its binary16 rate, and
// binary16 serves an exact integer product: codes are exact in binary16 (|q|
// <= 128), products (<= 2^14) and sums of up to 1024 of them (<= 2^24) are
// exact in the binary32 accumulator.  So K is cut into chunks of 1024, each
// one chain of tcgen05.mma.kind::f16 into a zeroed TMEM accumulator, and the
// epilogue adds the chunks as 32-bit integers in registers.
//
// The output channels are the MMA's rows (M = 256 over a pair of SMs) and
// the tokens its columns, so that the weights -- the operand that is large
// when tokens are few -- travel to the SM as the 8-bit codes they are and
// are converted there, once per tile: a warpgroup reads a 128 x 128 box of
// codes from shared memory, widen them in registers (bias to unsigned,
// a byte permute under the exponent of 1024, one packed subtraction for two
// values) and write them to tensor memory, where the MMA takes its A operand
// from.  Shared memory then carries one byte per weight instead of two,
// and the operand reads of A cost it nothing.  The tokens' codes are widened
// by a short kernel before (i8_prepare_kernel) into 16-bit scratch that TMA
// boxes feed to the MMA as the B operand, half of the tile's tokens per SM.
//
// Whole tiles go round the CTA pairs; the tiles left over after whole rounds
// (all of them, where tiles are few) are cut along K over several pairs if
// that ends sooner: integer additions commute, so the pieces go to slabs of
// 32-bit scratch and the CTA that completes the tile adds and scales them --
// the same bits in any order.
//
// What bounds it.  Many tokens: the tensor pipe under the power limit (8192
// x 8192 x 8192: 600 us in a burst, 650 sustained, 1.70 to 1.83 PFLOP/s), the
// preparation being 5% of it; a step's conversion (about 620 cycles of the
// SM, its ALU work half of that) is shorter than the MMAs of 160 tokens (640)
// and is hidden.  Few tokens: the weights' bytes (48 x 8192 x 8192: 11 of 24
// us, the rest being the preparation, the pipeline's start and the split's
// hand-over).  Measured on the way, 8192 x 8192 x 8192: release arrivals at
// cluster scope 1470 us, relaxed ones 1060; issuing from a converged warp
// 740; three conversion warpgroups that take whole steps in turn 660, with
// tiles of 128 tokens; 618 with 160.
//
// CTA roles (768 threads, one persistent CTA per SM, clusters of two):
//   warps 0, 2    TMA copies into a 6-stage ring: 128 weight rows x 128
//                 codes; 2 blocks of 64 columns x tile/2 tokens
//   warp 1        TMEM allocation; the leader's issues the MMAs
//   warps 4..15   conversion, three to six TMEM stages of 128 k ahead
//   warps 16..23  epilogue: two accumulators, so a chunk's
//                 readout runs beside the next chunk's MMAs
// Every wait gives up after about a second as in the split-K GEMM.
#include <cstring>
#include <type_traits>

#include "kernels.cuh"
#include "codes.cuh"
#include "tc05.cuh"

namespace tcr {

__device__ unsigned int g_gemm_i8_fault;

// ---------------------------------------------------------------- the operands' preparation

// Blocks [0, blocks_a): the tokens' codes as binary16, rows of ldf values,
// zero past K, 8 codes a thread.  Blocks up to blocks_a + blocks_w: the
// weights' codes in rows of ldf bytes (only when their own pitch or base does
// not fit TMA), 16 codes a thread by 16-byte granules (333 x 2051 x 4100: 22.2
// us the whole call, with 8 codes by 8-byte granules 24.3).  The last one
// zeroes the counters of the split tiles.
__global__ void __launch_bounds__(256) i8_prepare_kernel(const I8Prepare p)
{
    // in this order: the product's kernel may read the weights as soon as it
    // runs, so it must not start while a kernel that writes them still runs
    pdl_wait_primary();
    pdl_launch_dependents();
    unsigned b = blockIdx.x;
    if (b >= p.blocks_a + p.blocks_w) {
        for (size_t i = threadIdx.x; i < p.zero_words; i += 256) p.zero[i] = 0;
        return;
    }
    const bool tokens = b < p.blocks_a;
    if (!tokens) b -= p.blocks_a;
    const uint32_t codes = tokens ? 8u : 16u;
    const size_t item = (size_t)b * 256 + threadIdx.x;
    const uint32_t per_row = (uint32_t)p.ldf / codes;
    const size_t r = item <= 0xffffffffu ? (uint32_t)item / per_row : item / per_row;
    const uint32_t c = codes * (uint32_t)(item - r * per_row);
    if (r >= (tokens ? p.M : p.N)) return;
    const uint32_t left = p.K > c ? (uint32_t)(p.K - c) : 0u;
    if (tokens) {
        const int8_t *from = p.A + r * p.lda + c;
        const uint2 q = p.al_a && left >= 8 ? *reinterpret_cast<const uint2 *>(from) : ld_codes8(from, left);
        uint4 o;
        widen4(q.x, o.x, o.y);
        widen4(q.y, o.z, o.w);
        *reinterpret_cast<uint4 *>(p.Af + r * p.ldf + c) = o;
    } else {
        const int8_t *from = p.W + r * p.ldw + c;
        *reinterpret_cast<uint4 *>(p.Wp + r * p.ldf + c) =
            use_codes<true>(load_last_codes<true>(from, left), from, left, left >= 16);
    }
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
// Tensor memory: two accumulators of a tile's tokens at columns 0 and tn, the
// widened weights in stages of 64 columns behind them: 3 at 160 tokens, up to
// 6 at fewer -- no more than stages of the ring, whose `empty` barriers free
// both: a wait for step i - 6 must not meet the barrier a phase further on.
__host__ __device__ constexpr int i8_a_stages(int tn)
{
    return (512 - 2 * tn) / 64 < kI8Stages ? (512 - 2 * tn) / 64 : kI8Stages;
}
constexpr int kI8ConvGroups = 3;               // warpgroups that take the steps in turn
constexpr int kI8EpiWarps = 8;
constexpr int kI8EpiWarp0 = 4 + 4 * kI8ConvGroups;
constexpr int kI8Threads = 32 * (kI8EpiWarp0 + kI8EpiWarps);
// Registers a thread by role (setmaxnreg); their sum over the warpgroups is
// within what the launch holds: 768 threads of 80.
constexpr int kI8RegsLaunch = 80, kI8RegsIssue = 40, kI8RegsConv = 56, kI8RegsEpi = 136;
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
static_assert(i8_a_stages(kI8MaxTn) >= 3, "TMEM stages");

// mbar_wait_f with its limit (2^31 cycles: 1.0 to 1.5 s) on the SM's cycle
// counter, whose read is short beside the global timer's: the waits of a
// small product follow one another.
__device__ __forceinline__ bool i8_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t i = 1;; i++) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 0u) {
            if (*abort) return false;
            if (clock64() - t0 > (1ll << 31)) {
                *abort = 1u;
                atomicOr(&g_gemm_i8_fault, 1u);
                return false;
            }
        }
    }
}

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

// A CTA pair's work, in turn: whole tiles pair, pair + pairs, .. below
// g.full, then at most one piece of a tile from g.full on, each of which is
// cut into g.per pieces for as many pairs.
struct I8Walk {
    int tile, k0, nb, part; // the current piece: a tile's steps k0 .. k0 + nb - 1, which piece of it
    int u, piece;

    __device__ __forceinline__ I8Walk(const I8Gemm &g, int pair, int pairs)
    {
        u = pair;
        piece = pair < (g.tiles - g.full) * g.per ? pair : -1;
    }
    __device__ __forceinline__ bool next(const I8Gemm &g, int pairs)
    {
        if (u < g.full) {
            tile = u;
            k0 = 0;
            nb = g.steps;
            part = 0;
            u += pairs;
            return true;
        }
        if (piece < 0) return false;
        tile = piece / g.per;
        part = piece - tile * g.per;
        k0 = part * g.steps / g.per;
        nb = (part + 1) * g.steps / g.per - k0;
        tile += g.full;
        piece = -1;
        return true;
    }
};

// A tile's channel and token tile: groups of 8 channel tiles, the channel
// tile fastest, so that the tiles in flight share operands in L2.
__device__ __forceinline__ void i8_tile(const I8Gemm &g, int tile, int &tc, int &tt)
{
    constexpr int kGroup = 8;
    const int group = kGroup * g.tiles_t;
    const int first = tile / group * kGroup;
    const int in_group = min(g.tiles_c - first, kGroup);
    const int q = tile % group;
    tc = first + q % in_group;
    tt = q / in_group;
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
    auto wait = [&](uint32_t b, uint32_t parity) { return i8_wait(b, parity, abort); };

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
    const int half = g.tn / 2, a_stages = i8_a_stages(g.tn);
    I8Walk walk(g, pair, pairs);

    // The kernel before this one on the stream is i8_prepare_kernel, which
    // lets this one start only once the kernels before it are done.  So only
    // what reads its results waits for it: the tokens' copies, the integer
    // scratch, and the weights' copies where it repacked them.

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kI8RegsIssue));
        if (warp == 0) {
            // ---------------- the weights' copies (here and below a converged
            // warp walks, one lane issues)
            if (g.w_prepared) pdl_wait_primary();
            int st = 0;
            uint32_t phase = 0;
            uint32_t armed = 0, armed_phase = 0;
            bool ok = true;
            while (ok && walk.next(g, pairs)) {
                int tc, tt;
                i8_tile(g, walk.tile, tc, tt);
                for (int j = 0; j < walk.nb; j++) {
                    ok = __all_sync(kFull, wait(empty(st), phase ^ 1u));
                    if (!ok) break;
                    if (i8_elect()) {
                        mbar_arrive_expect_tx(wfull(st), kI8WBytes);
                        tma_load_2d(ring + (uint32_t)st * kI8StageBytes, &map_w, (walk.k0 + j) * kI8BK,
                                    tc * kI8BM + 128 * (int)rank, wfull(st));
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
            if (*abort)                   // let the copies in flight land
                for (int i = 0; i < kI8Stages; i++)
                    if ((armed >> i) & 1u) (void)mbar_wait_limited(wfull(i), (armed_phase >> i) & 1u);
        } else if (warp == 2) {
            // ---------------- the tokens' copies
            pdl_wait_primary();
            const uint32_t leader_full = i8_map_leader(full(0));
            const uint32_t token_bytes = (uint32_t)(4 * 128 * half);
            int st = 0;
            uint32_t phase = 0;
            bool ok = true;
            while (ok && walk.next(g, pairs)) {
                int tc, tt;
                i8_tile(g, walk.tile, tc, tt);
                for (int j = 0; j < walk.nb; j++) {
                    ok = __all_sync(kFull, wait(empty(st), phase ^ 1u));
                    if (!ok) break;
                    if (i8_elect()) {
                        if (leader) mbar_arrive_expect_tx(full(st), token_bytes);
                        i8_load_tokens(ring + (uint32_t)st * kI8StageBytes + kI8WBytes, &map_t,
                                       tt * g.tn + half * (int)rank, 2 * (walk.k0 + j),
                                       leader_full + 8u * (uint32_t)st);
                    }
                    __syncwarp();
                    if (++st == kI8Stages) {
                        st = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort) {
                // these copies share a barrier with conversions that may
                // never come, so they get time (10 ms) to land
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
            while (ok && walk.next(g, pairs)) {
                int in_chunk = 0;
                for (int j = 0; j < walk.nb && ok; j++) {
                    bool ready = true;
                    if (in_chunk == 0) ready = !*abort && wait(dempty(b), ((dphase >> b) & 1u) ^ 1u);
                    ready = ready && wait(full(st), phase);
                    ok = __all_sync(kFull, ready);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(b * g.tn);
                    const uint32_t a = tmem + (uint32_t)(2 * g.tn + 64 * ta);
                    const uint64_t t_desc = t_desc0 + (uint64_t)st * (kI8StageBytes >> 4);
                    const bool end = in_chunk == kI8ChunkSteps - 1 || j == walk.nb - 1;
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
                    if (++ta == a_stages) ta = 0;
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
        int total = 0;                                 // steps of all pieces
        while (walk.next(g, pairs)) total += walk.nb;
        bool ok = true;
        const int group = (warp - 4) >> 2;
        int ta = group % a_stages;                     // TMEM stage of step i
        for (int i = group; i < total; i += kI8ConvGroups) {
            const int st = i % kI8Stages;
            ok = __all_sync(kFull, wait(wfull(st), (uint32_t)(i / kI8Stages) & 1u));
            if (!ok) break;
            const uint32_t row = ring + (uint32_t)(st * kI8StageBytes + m * kI8BK);
            const uint32_t dst = tmem + lane_base + (uint32_t)(2 * g.tn + 64 * ta);
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
                if (h == 0 && i >= a_stages) {
                    // the MMAs that read this TMEM stage last are done
                    const int e = i - a_stages;
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
            ta += kI8ConvGroups;
            while (ta >= a_stages) ta -= a_stages;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kI8RegsEpi));
        // ---------------- epilogue: a thread holds one channel, half of the tile's
        // tokens, 16 at a time
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const int m = 32 * (warp & 3) + lane;
        const int col0 = warp < kI8EpiWarp0 + 4 ? 0 : half;
        const int nblk = half / 16;
        int b = 0;
        uint32_t dphase = 0;
        pdl_wait_primary();
        while (walk.next(g, pairs)) {
            int tc, tt;
            i8_tile(g, walk.tile, tc, tt);
            const bool split = walk.nb < g.steps;
            const uint32_t n = (uint32_t)(tc * kI8BM + 128 * (int)rank + m);
            const uint32_t t0 = (uint32_t)(tt * g.tn + col0);
            // the tokens of this thread that exist
            const int nt = n >= g.N || t0 >= g.M ? 0 : (int)min((uint32_t)half, (uint32_t)g.M - t0);
            // a split tile's slabs of sums, laid out (piece, token, channel)
            const int rt = walk.tile - g.full;
            auto slab = [&](int part, int q) {
                const size_t token = ((size_t)rt * g.per + part) * g.tn + col0 + 16 * q;
                return g.ws + token * kI8BM + 128u * rank + m;
            };
            bool live = true;
            // this thread's scales, loaded ahead of the sums: its channel's and,
            // 32 to a register over the lanes, the tokens'
            const float sw = g.sw && n < g.N ? g.sw[n] : 1.0f;
            constexpr int kSa = (kI8MaxTn / 2 + 31) / 32;
            float sa[kSa];
#pragma unroll
            for (int i = 0; i < kSa; i++) {
                const uint32_t t = t0 + 32 * i + lane;
                sa[i] = g.sa && t < g.M && 32 * i + lane < half ? g.sa[t] : 1.0f;
            }
            // C's tokens 16 q .. of this thread's channel from their sums; NaN (or
            // the least integer) where a wait gave up
            auto store_as = [&](auto type, int q, auto &v) {
                constexpr int kType = decltype(type)::value, kCount = sizeof v / sizeof v[0];
                using E = typename Elem<kType == kOutI32 ? kF32 : kType>::T;
                E *at = (E *)g.C + (size_t)(t0 + 16 * q) * g.ldc + n;
                const int left = nt - 16 * q;
                const float channel = live ? sw : __int_as_float(0x7fc00000);
                float mine = sa[0];
                if constexpr (kCount == 16) {
#pragma unroll
                    for (int i = 1; i < kSa; i++) mine = q / 2 == i ? sa[i] : mine;
                }
#pragma unroll
                for (int i = 0; i < kCount; i++) {
                    E e;
                    if constexpr (kType == kOutI32) {
                        e = (uint32_t)v[i];
                    } else {
                        const float token = kCount == 16 ? __shfl_sync(kFull, mine, 16 * (q & 1) + i)
                                                         : __shfl_sync(kFull, sa[i / 32], i % 32);
                        e = float_to_elem<kType>(__fmul_rn(__fmul_rn((float)v[i], token), channel));
                    }
                    if (i < left) *at = e;
                    at += g.ldc;
                }
            };
            auto store16 = [&](int q, const int (&v)[16]) {
                switch (g.c_dtype) {
                case kF16: store_as(std::integral_constant<int, kF16>(), q, v); break;
                case kBF16: store_as(std::integral_constant<int, kBF16>(), q, v); break;
                case kF32: store_as(std::integral_constant<int, kF32>(), q, v); break;
                default: store_as(std::integral_constant<int, kOutI32>(), q, v); break;
                }
            };
            // 16 sums to where they go: this piece's slab, or C
            auto put16 = [&](int q, const int (&v)[16]) {
                if (split) {
                    int *own = slab(walk.part, q);
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        if (i < nt - 16 * q) __stcg(own + i * kI8BM, v[i]);
                } else {
                    store16(q, v);
                }
            };
            auto chunk_ready = [&]() {
                const bool ready = !*abort && wait(dfull(b), (dphase >> b) & 1u);
                return __all_sync(kFull, ready) != 0;
            };
            auto chunk_done = [&](bool read) {
                if (read) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) i8_arrive_leader(i8_map_leader(dempty(b)));
                }
                dphase ^= 1u << b;
                b ^= 1;
            };
            // (Loops over the blocks of 16 are kept rolled where the sums need
            // not stay in registers: the code runs once a tile, and its length
            // is what a small product waits for.)
            if (walk.nb <= kI8ChunkSteps) {
                live = chunk_ready();
                if (live) tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < nblk; q++) {
                    float f[16];
                    int v[16];
                    if (live) i8_ld16(tmem + lane_base + (uint32_t)(b * g.tn + col0 + 16 * q), f);
#pragma unroll
                    for (int i = 0; i < 16; i++) v[i] = live ? __float2int_rn(f[i]) : (int)0x80000000;
                    if (live || !split) put16(q, v);
                }
                chunk_done(live);
            } else {
                int acc[kI8MaxTn / 2];
#pragma unroll
                for (int i = 0; i < kI8MaxTn / 2; i++) acc[i] = 0;
                for (int j = 0; j < walk.nb; j += kI8ChunkSteps) {
                    live = live && chunk_ready();
                    if (live) {
                        tc_fence_after();
#pragma unroll
                        for (int q = 0; q < kI8MaxTn / 32; q++) {
                            if (q < nblk) {
                                float v[16];
                                i8_ld16(tmem + lane_base + (uint32_t)(b * g.tn + col0 + 16 * q), v);
#pragma unroll
                                for (int i = 0; i < 16; i++) acc[16 * q + i] += __float2int_rn(v[i]);
                            }
                        }
                    }
                    chunk_done(live);
                }
                if (!live) {
#pragma unroll
                    for (int i = 0; i < kI8MaxTn / 2; i++) acc[i] = (int)0x80000000;
                }
                if (split) {
                    int *own = slab(walk.part, 0);
#pragma unroll
                    for (int i = 0; i < kI8MaxTn / 2; i++)
                        if (i < nt) __stcg(own + i * kI8BM, acc[i]);
                } else {
                    switch (g.c_dtype) {
                    case kF16: store_as(std::integral_constant<int, kF16>(), 0, acc); break;
                    case kBF16: store_as(std::integral_constant<int, kBF16>(), 0, acc); break;
                    case kF32: store_as(std::integral_constant<int, kF32>(), 0, acc); break;
                    default: store_as(std::integral_constant<int, kOutI32>(), 0, acc); break;
                    }
                }
            }
            if (!split) continue;
            // the CTA that brings the tile's last steps adds the slabs
            __threadfence();
            named_sync(1, 32 * kI8EpiWarps);
            if (threadIdx.x == 32 * kI8EpiWarp0)
                *last = live && !*abort &&
                        atomicAdd(g.count + 2 * rt + rank, (uint32_t)walk.nb) + walk.nb == (uint32_t)g.steps;
            named_sync(1, 32 * kI8EpiWarps);
            const bool gave_up = *abort != 0u;       // a role of this CTA did: its tiles read NaN
            if (__any_sync(kFull, gave_up))
                live = false;
            else if (*last == 0u)
                continue;
            __threadfence();
#pragma unroll 1
            for (int q = 0; q < nblk; q++) {
                int v[16];
#pragma unroll
                for (int i = 0; i < 16; i++) v[i] = live ? 0 : (int)0x80000000;
                if (live && nt > 16 * q) {
#pragma unroll 1
                    for (int part = 0; part < g.per; part++) {
                        // (tokens past the tile's end read the slab's own padding)
                        const int *from = slab(part, q);
#pragma unroll
                        for (int i = 0; i < 16; i++) v[i] += __ldcg(from + i * kI8BM);
                    }
                }
                store16(q, v);
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
    if (M <= 2 || pairs <= 0) return p;
    p.tensor = 1;
    p.steps = (int)((K + kI8BK - 1) / kI8BK);
    p.tiles_c = (int)((N + kI8BM - 1) / kI8BM);
    p.ldf = (K + 63) / 64 * 64;
    // The token tile and the split: the least time by what a step costs, in
    // cycles -- the conversion of its weights (about 620) or its MMAs (4 a
    // token, and the accumulators' readout beside them) -- and a split tile's
    // way through the scratch (a fence, a counter, the readback: 2 to 3 us).  Whole tiles go round the pairs; the steps of the tiles
    // left over after whole rounds are split over the pairs, as many pairs to
    // each tile, if that ends sooner.
    size_t best = SIZE_MAX;
    for (int tn = 32; tn <= kI8MaxTn; tn += 32) {
        const size_t tt = (M + (size_t)tn - 1) / (size_t)tn;
        const size_t tiles = tt * (size_t)p.tiles_c, steps = (size_t)p.steps;
        const size_t step = tn * 4 + 30 > 620 ? (size_t)tn * 4 + 30 : 620;
        size_t full = tiles / (size_t)pairs * (size_t)pairs;
        const size_t left = tiles - full;
        size_t per = left ? (size_t)pairs / left : 1;        // pairs a left-over tile
        if (per > steps) per = steps;
        size_t cost = full / (size_t)pairs * steps * step;
        const size_t split = (steps + per - 1) / per * step + 4000 + 10 * (size_t)tn, whole = steps * step;
        if (left > 0) cost += per > 1 && split < whole ? split : whole;
        if (left == 0 || per < 2 || split >= whole) {
            full = tiles;
            per = 1;
        }
        if (cost < best) {
            best = cost;
            p.tn = tn;
            p.tiles_t = (int)tt;
            p.full = (int)full;
            p.per = (int)per;
            p.pairs = full == 0 ? (int)(left * per) : (int)(tiles < (size_t)pairs ? tiles : (size_t)pairs);
        }
    }
    // Against the kernels of k_gemm_i8_few.cu, whose one launch costs 5 us less
    // than the two, the copies' and the conversion's latency and the hand-over
    // here, but which run 40 thousand multiply-adds a cycle and stream 1900
    // bytes of weights (64 x 2048 x 2048: 4.5 us, 10 here; 48 x 4096 x 4096:
    // 14.8 and 16.0; 1024 x 1024 x 1024: 18.8 and 9.4).
    const size_t macs = N * K * ((M + 7) / 8 * 8);
    const size_t few = 3800 + (macs / 39500 > N * K / 1900 ? macs / 39500 : N * K / 1900);
    if (M <= (size_t)kI8FewTokens && few < 14500 + best) std::memset(&p, 0, sizeof p);
    return p;
}

// 32-bit words of the split tiles' scratch: a slab a piece, and a counter a
// CTA and tile (which start at 0).
static size_t i8_split_words(const I8Plan &p)
{
    const size_t tiles = (size_t)p.tiles_c * (size_t)p.tiles_t - (size_t)p.full;
    return tiles * ((size_t)p.per * (size_t)p.tn * kI8BM + 2);
}

// Scratch bytes of a call: the tokens as binary16, the repacked weights
// (repack_w), the integer scratch and its counters.
size_t gemm_i8_scratch(const I8Plan &p, size_t M, size_t N, bool repack_w)
{
    if (!p.tensor) return 0;
    size_t b = M * p.ldf * 2;
    if (repack_w) b += N * p.ldf;
    b = (b + 255) / 256 * 256;
    return b + i8_split_words(p) * 4;
}

cudaError_t launch_gemm_i8(const I8Args &a, const I8Plan &p, void *scratch, bool repack_w, bool inject_stall,
                           cudaStream_t stream)
{
    if (!p.tensor) return launch_gemm_i8_few(a, stream);
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
    auto blocks_of = [&](size_t rows, size_t codes) { return (unsigned)((rows * (p.ldf / codes) + 255) / 256); };
    q.blocks_a = blocks_of(a.M, 8);
    const int8_t *w = a.W;
    size_t ldw = a.ldw;
    size_t off = a.M * p.ldf * 2;
    if (repack_w) {
        q.W = a.W;
        q.ldw = a.ldw;
        q.Wp = (int8_t *)scratch + off;
        q.blocks_w = blocks_of(a.N, 16);
        w = q.Wp;
        ldw = p.ldf;
        off += a.N * p.ldf;
    }
    off = (off + 255) / 256 * 256;
    I8Gemm g;
    std::memset(&g, 0, sizeof g);
    unsigned blocks_z = 0;
    if (p.per > 1) {
        const size_t tiles = (size_t)p.tiles_c * (size_t)p.tiles_t - (size_t)p.full;
        g.ws = (int *)((char *)scratch + off);
        q.zero = g.ws + tiles * (size_t)p.per * (size_t)p.tn * kI8BM;
        q.zero_words = 2 * tiles;
        blocks_z = 1;
        g.count = (uint32_t *)q.zero;
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
    // the split of the SM's memory that the product's kernel needs, so that
    // its CTAs can start beside the last of these
    cudaError_t e = set_smem_once((void *)i8_prepare_kernel, 0, 100);
    if (e != cudaSuccess) return e;
    void *args1[] = {(void *)&q};
    e = launch_first((const void *)i8_prepare_kernel, dim3(q.blocks_a + q.blocks_w + blocks_z), dim3(256),
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
    g.full = p.full;
    g.tiles = p.tiles_c * p.tiles_t;
    g.per = p.per;
    g.w_prepared = repack_w ? 1u : 0u;
    g.inject_stall = inject_stall ? 1u : 0u;
    void *args[] = {(void *)&mw, (void *)&mt, (void *)&g};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * p.pairs));
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
