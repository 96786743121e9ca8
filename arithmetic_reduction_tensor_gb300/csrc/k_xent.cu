// k_xent.cu -- the matrix products of the softmax cross entropy over a
// vocabulary, on pairs of SMs (tcgen05.mma.cta_group::2, 256 x 256 tiles).
//
// With l = X W^T the logits of n tokens over V entries (never in memory):
//   forward   a tile's epilogue leaves, of each of its rows, the largest logit
//             and the sum of exp(l - largest) over the others of 128 of its
//             columns, and the target's logit: 8 bytes for 128 logits.
//   gradient  over a piece of the vocabulary at a time: the logits' tiles again,
//             their epilogue writing P = (exp(l - lse) - [target]) g in 16 bits;
//             then one launch forms dX += P W (units of 256 tokens x 256 columns
//             of X, K along the piece, fp32 sums across the pieces) and the
//             piece's rows of dW = P^T X (K along the tokens).
// P is the only thing rounded on the way: to the inputs' type, half a step of
// each of its elements, as large an error as the rounding of the results;
// the products' sums are 32 bits.
//
// X is the compact, aligned copy of the tokens that count (k_xent_rows.cu; few
// aligned tokens in the forward pass: x itself), W is V x H, P is n x the piece.  Only the logits have both operands K-major as they
// lie in memory.  The gradient's products take W, P and X as they are, MN-major:
// a 64 x 64 box of a row-major matrix lands in shared memory as 64 rows of 128
// swizzled bytes, which is a K-major operand of 64 rows or an MN-major one of
// 64 k, as the descriptor and the instruction say; so no matrix is transposed.
//
// Roles, barriers, time limits as in gemm_splitk_pair_kernel (k_gemm.cu): a
// producer thread, an MMA thread, two accumulators; eight epilogue warps, each 32
// rows and 128 columns of the CTA's 128 x 256.
//
// The tensor cores' sums lose their last bits at every step, all in the same
// direction, so the logits take K in chains of 1024 and add the chains in
// registers (4096 columns: the loss' error against binary64 1.4e-6 in one chain,
// 3e-7 so, for 2% of the forward pass' time).  The gradient does the same, so that its
// logits are the forward pass' bit for bit: P of a token that is predicted well is a
// difference of l and lse, which other sums would shift by their own loss.  dX and dW
// are rounded to 16 bits, which chains of 16384 do not spoil (terms of one sign: 2e-5
// low after 16384 of them in one chain, 1.6e-4 after 65536, 1.4e-3 after 262144); a
// launch with longer ones adds them in registers (kXentBackLong), the others read
// the accumulators as they store.
//
// What the gradient's tiles write (P, dX's sums, dW) leaves by tensor-map
// stores from shared memory, dX's later pieces as additions in L2: threads that
// store a row each keep the memory pipe from the MMAs' operands (4096 x 2048 over
// 9728: P's launch 104 us that way, 98 so).
//
// Many tokens are bound by the tensor pipe: 4096 x 4096 over 65536 forward 1.18 ms in
// a burst (the product alone by cuBLAS, logits written in 16 bits, 1.09 to 1.15), 1.27 to
// 1.33 under the power limit (1.22 beside 1.27); with the gradient over 32768 2.37
// and 2.56 to 2.74 ms, 8 T V H operations at 1.86 and 1.61 to 1.72 PFLOP/s.  The producer
// is one thread, and a box more a stage costs it: operands that lie K-major come
// in one box of all their rows (two of 64 rows: 2.56 ms).  Few tokens are bound by
// reading W: 16 x 4096 over 131072 175 us, 6.1 TB/s.
#include "pair.cuh"
#include "piece.cuh"
#include "plan.h"
#include "rowvec.cuh"
#include "xent.h"

namespace tcr {

constexpr int kXBox = 64;                          // rows and columns of a box
constexpr int kXBoxBytes = kXBox * kXBox * 2;      // 8 KiB
constexpr int kXHalf = 128;                        // rows of an operand per CTA
constexpr int kXHalfBytes = 2 * kXBoxBytes;
constexpr int kXChain = 16, kXBackChain = kXentChain / kXBox;   // boxes of K added up in one chain: of the logits, of dX and dW
constexpr int kXDBuffers = 2;
constexpr uint32_t kXTmemCols = kXDBuffers * kXentTile;
constexpr int kXEpilogueWarps = 8;
constexpr int kXThreads = 64 + 32 * kXEpilogueWarps;
constexpr int kXGroup = 8;                         // tile rows per raster group (L2 reuse)
// Columns of a tile that an epilogue warp takes, and the warps that a tile's columns keep busy.
template <int TN>
struct XTile {
    static constexpr int kCols = TN < 128 ? TN : 128, kWarps = 4 * (TN / kCols);
    static constexpr int kBBytes = TN / 2 * kXBox * 2;       // B's share of a stage per CTA
    static constexpr int kStageBytes = kXHalfBytes + kBBytes;
};
constexpr int kXOutBytes = 32 * 128;               // its staging: 32 rows of 128 swizzled bytes
// The ring, the staging (not in the forward pass, whose ring is longer for it)
// and the barriers: full[S] (leader's: both CTAs' copies), empty[S], dfull[D],
// dempty[D] (leader's), drain.
template <int MODE, int TN>
struct XLayout {
    static constexpr int kStages = (MODE == kXentForward ? 224 : 192) * 1024 / XTile<TN>::kStageBytes;
    static constexpr int kOffOut = kStages * XTile<TN>::kStageBytes;
    static constexpr int kOffBars = kOffOut + (MODE == kXentForward ? 0 : kXEpilogueWarps * kXOutBytes);
    static constexpr int kNumBars = 2 * kStages + 2 * kXDBuffers + 1;
    static constexpr int kOffMisc = kOffBars + 8 * kNumBars;
    static constexpr int kSmemBytes = kOffMisc + 64 + 1024;
    static_assert(kSmemBytes <= 232448, "one SM's 227 KiB");
};

__device__ unsigned int g_xent_fault;

__device__ __forceinline__ bool x_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort)
{
    return mbar_wait_f(bar, parity, abort, &g_xent_fault);
}

// 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tc_ld_row16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 16; j++) v[j] = __uint_as_float(r[j]);
}

// COLS consecutive fp32 columns of this thread's TMEM lane, all on their way
// before the first is waited for.
template <int COLS>
__device__ __forceinline__ void tc_ld_row(uint32_t taddr, float (&v)[COLS])
{
    uint32_t r[COLS];
#pragma unroll
    for (int c = 0; c < COLS; c += 32)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
            "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
            : "=r"(r[c + 0]), "=r"(r[c + 1]), "=r"(r[c + 2]), "=r"(r[c + 3]), "=r"(r[c + 4]), "=r"(r[c + 5]),
              "=r"(r[c + 6]), "=r"(r[c + 7]), "=r"(r[c + 8]), "=r"(r[c + 9]), "=r"(r[c + 10]),
              "=r"(r[c + 11]), "=r"(r[c + 12]), "=r"(r[c + 13]), "=r"(r[c + 14]), "=r"(r[c + 15]),
              "=r"(r[c + 16]), "=r"(r[c + 17]), "=r"(r[c + 18]), "=r"(r[c + 19]), "=r"(r[c + 20]),
              "=r"(r[c + 21]), "=r"(r[c + 22]), "=r"(r[c + 23]), "=r"(r[c + 24]), "=r"(r[c + 25]),
              "=r"(r[c + 26]), "=r"(r[c + 27]), "=r"(r[c + 28]), "=r"(r[c + 29]), "=r"(r[c + 30]),
              "=r"(r[c + 31])
            : "r"(taddr + (uint32_t)c)
            : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int c = 0; c < COLS; c += 16)               // (not used before the wait)
        asm volatile(""
                     : "+r"(r[c + 0]), "+r"(r[c + 1]), "+r"(r[c + 2]), "+r"(r[c + 3]), "+r"(r[c + 4]),
                       "+r"(r[c + 5]), "+r"(r[c + 6]), "+r"(r[c + 7]), "+r"(r[c + 8]), "+r"(r[c + 9]),
                       "+r"(r[c + 10]), "+r"(r[c + 11]), "+r"(r[c + 12]), "+r"(r[c + 13]), "+r"(r[c + 14]),
                       "+r"(r[c + 15]));
#pragma unroll
    for (int j = 0; j < COLS; j++) v[j] = __uint_as_float(r[j]);
}

// The operand of 128 rows (or MN elements) at `addr`, two boxes: K-major (8-row
// groups 1024 bytes apart; a k-slice of 16 is 32 bytes further) or MN-major
// (64-element blocks a box apart, groups of 8 k 1024 bytes apart; a slice
// is 16 rows of 128 bytes further).  128-byte swizzle.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn)
{
    const uint64_t lbo = mn ? (uint64_t)(kXBoxBytes >> 4) : 1u;
    return (uint64_t)((addr >> 4) & 0x3fffu) | (lbo << 16) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// kind::f16, M = 256, N = TN, fp32 sums; bits 15 and 16: A and B MN-major.
template <int DT, int TN>
__device__ __forceinline__ uint32_t operand_instr(bool a_mn, bool b_mn)
{
    constexpr uint32_t ab = DT == kF16 ? 0u : 1u;
    return (1u << 4) | (ab << 7) | (ab << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(kXentTile >> 4) << 24);
}

// One tile's work: 64-boxes [k0, k0 + nk) of K; of A's four boxes of rows the
// first `rows` hold something that is wanted (tokens; the others are not read,
// and what the MMAs make of their places in shared memory is not looked at).
struct XUnit {
    bool x;                // dX (else dW, or the logits)
    int tm, tn, split, k0, nk, rows;
};

// The units of one launch, of which pair p of `pairs` runs the i-th of its own.
struct XUnits {
    int n, pairs, pair;
    bool back;
    int tm, tn, nk;                    // the logits, or dW: tiles, boxes of K
    int xm, xn, xnk, xkps, xsplits;    // dX: tiles, boxes of K, boxes a split
    int nx, nd, lead, rem;

    __device__ __forceinline__ XUnits(const XentGemm &g, int n_, bool back_, int tile_cols) : n(n_), back(back_)
    {
        pairs = (int)(gridDim.x >> 1);
        pair = (int)(blockIdx.x >> 1);
        const int rows = (n + kXentTile - 1) / kXentTile, cols = (g.vn + tile_cols - 1) / tile_cols;
        nx = 0;
        lead = rem = 0;
        xm = xn = xnk = xkps = xsplits = 0;
        if (!back) {
            tm = rows;
            tn = cols;
            nk = (g.H + kXBox - 1) / kXBox;
            nd = tm * tn;
            return;
        }
        const int hcols = (g.H + kXentTile - 1) / kXentTile;
        tm = cols;
        tn = hcols;
        nk = (n + kXBox - 1) / kXBox;
        nd = g.dw ? tm * tn : 0;
        if (g.ws) {
            xm = rows;
            xn = hcols;
            xnk = (g.vn + kXBox - 1) / kXBox;
            xkps = (xnk + g.splits - 1) / g.splits;
            xsplits = g.splits;
            nx = xm * xn * xsplits;
            // the long units first, one more on some pairs than on others: those
            // take fewer of the short ones (whose epilogue takes as long as 7 boxes)
            const int cost = max(nk, 7);
            rem = nx % pairs;
            lead = rem ? (xkps + cost / 2) / cost : 0;
            if (lead > nd / (pairs - rem)) lead = nd / (pairs - rem);
        }
    }
    __device__ __forceinline__ static void raster(int u, int tiles_m, int tiles_n, int &m, int &n)
    {
        const int group = kXGroup * tiles_n, first = u / group * kXGroup;
        const int in_group = min(tiles_m - first, kXGroup), r = u % group;
        m = first + r % in_group;
        n = r / in_group;
    }
    __device__ __forceinline__ bool get(int i, XUnit &u) const
    {
        const int mine = nx ? (nx - pair + pairs - 1) / pairs : 0;       // its dX units
        if (i < mine) {
            const int v = pair + i * pairs, tiles = xm * xn;
            u.x = true;
            u.split = v / tiles;
            raster(v % tiles, xm, xn, u.tm, u.tn);
            u.k0 = u.split * xkps;
            u.nk = max(0, min(xkps, xnk - u.k0));
            u.rows = boxes_of_tokens(u.tm);
            return true;
        }
        i -= mine;
        int d;
        const int free_pairs = pairs - rem;
        if (pair >= rem && i < lead) {
            d = pair - rem + i * free_pairs;
        } else {
            if (pair >= rem) i -= lead;
            d = lead * free_pairs + pair + i * pairs;
        }
        if (d >= nd) return false;
        u.x = false;
        u.split = 0;
        raster(d, tm, tn, u.tm, u.tn);
        u.k0 = 0;
        u.nk = nk;
        u.rows = back ? 4 : boxes_of_tokens(u.tm);
        return true;
    }
    __device__ __forceinline__ int boxes_of_tokens(int m) const
    {
        return min(4, (n - m * kXentTile + kXBox - 1) / kXBox);
    }
};

// ---------------------------------------------------------------- epilogues
//
// A lane has one row of the tile and its warp's 128 (64) columns of it: v, or `ld(c, v)`
// gives the columns 32 c .. 32 c + 31 of these.  Every lane of the warp calls
// ld and the stores.

// exp(l - about) of two logits (an instruction for both but for the exponentials).
__device__ __forceinline__ void exp_pair(float a, float b, uint64_t minus_about, float &x, float &y)
{
    uint64_t d = add_pair(pack_pair(a, b), minus_about);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(d), "l"(pack_pair(kLog2e, kLog2e)));
    unpack_pair(d, x, y);
    x = ex2(x);
    y = ex2(y);
}

// The smaller, or NaN where either is (fmaxf gives the other).
__device__ __forceinline__ float min_or_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest logit m of the row among 64 columns, and the sum of exp(l - m) over
// the others: without the largest's 1, in which small sums would drown, the loss
// of a token that is predicted well keeps its bits.  The differences are taken
// before they are scaled, so that the logits' size costs no bits and overflows
// nothing.  A tournament whose losers stay finds both (v is lost): comparing each with
// the largest and counting those alike took 4096 x 1024 over 16384 100 us, 95 so, 93 with
// the logits loaded at once (tc_ld_row).
template <int C0, int COLS>
__device__ __forceinline__ float2 part_of(float (&v)[COLS])
{
#pragma unroll
    for (int h = 32; h >= 1; h /= 2) {
#pragma unroll
        for (int j = C0; j < C0 + h; j++) {
            const float a = v[j], b = v[j + h];
            v[j] = fmaxf(a, b);
            v[j + h] = min_or_nan(a, b);
        }
    }
    const float mx = v[C0], minus = -xent_about(mx);
    const uint64_t minus_about = pack_pair(minus, minus);
    float e[4];
    exp_pair(v[C0 + 1], v[C0 + 1], minus_about, e[0], e[1]);
    e[1] = e[2] = e[3] = 0.0f;
    uint64_t s[2] = {pack_pair(e[0], e[1]), pack_pair(e[2], e[3])};
#pragma unroll
    for (int j = 2; j < 64; j += 2) {
        float x, y;
        exp_pair(v[C0 + j], v[C0 + j + 1], minus_about, x, y);
        s[(j >> 1) & 1] = add_pair(s[(j >> 1) & 1], pack_pair(x, y));
    }
    unpack_pair(add_pair(s[0], s[1]), e[0], e[1]);
    return make_float2(mx, __fadd_rn(e[0], e[1]));
}

template <int COLS>
__device__ __forceinline__ void epilogue_forward(const XentGemm &g, size_t row, int part, float (&v)[COLS])
{
    const int col0 = part * COLS, left = g.V - col0;
    const int lab = g.head ? g.lab[row] : row < (size_t)g.n ? xent_label(g.target[row], (size_t)g.V) : -1;
    const int at = lab - col0;
    if (left < COLS) {
#pragma unroll
        for (int j = 0; j < COLS; j++)
            if (j >= left) v[j] = -INFINITY;
    }
    if (at >= 0 && at < COLS) {
        float hit = 0.0f;
#pragma unroll
        for (int j = 0; j < COLS; j++)
            if (j == at) hit = v[j];
        g.hit[row] = hit;
    }
    float2 p = part_of<0>(v);
    if constexpr (COLS == 128) p = xent_join(p, part_of<64>(v));
    g.part[(size_t)part * g.tpad + row] = p;
}

// A warp's staging: 32 rows of 128 bytes, 16-byte granule k of row r at granule k ^
// (r % 8), as a tensor map with 128-byte swizzle reads them.
struct XOut {
    uint8_t *smem;
    uint32_t addr;
    __device__ __forceinline__ void ready() const        // the last store has read it
    {
        if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
    }
    __device__ __forceinline__ void put(int k, uint32_t a, uint32_t b, uint32_t c, uint32_t d) const
    {
        const uint32_t r = threadIdx.x & 31;
        *reinterpret_cast<uint4 *>(smem + 128 * r + 16 * ((uint32_t)k ^ (r & 7u))) = make_uint4(a, b, c, d);
    }
    // Store the box at column c0, row c1 of the map's matrix.
    template <bool ADD>
    __device__ __forceinline__ void send(const CUtensorMap *map, int c0, int c1) const
    {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if ((threadIdx.x & 31) != 0) return;
        if constexpr (ADD)
            asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];"
                         ::"l"((uint64_t)map), "r"(c0), "r"(c1), "r"(addr)
                         : "memory");
        else
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                         ::"l"((uint64_t)map), "r"(c0), "r"(c1), "r"(addr)
                         : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
};

// P of the row: (exp(l - lse) - [target]) * g, in units of the largest |g| so
// that the target's -1 times a common g is exact (binary16: times 2^15 on top,
// which keeps probabilities of 2^-29 normal).
template <int DT, int COLS>
__device__ __forceinline__ void epilogue_gradient(const XentGemm &g, const CUtensorMap *map, const XOut &out, int row0,
                                                  int n, int col0, const float (&v)[COLS])
{
    if (row0 >= (n + kXBox - 1) / kXBox * kXBox) return;     // not read: dW's K ends with the tokens' last box
    const int row = row0 + (threadIdx.x & 31);
    float about = 0.0f, gq = 0.0f;
    int at = -1;
    if (row < n) {
        const int tok = g.tok[row], lab = g.lab[row];
        const float gmax = __uint_as_float(g.head[1]);
        about = g.lse[tok];
        gq = g.dloss[(size_t)tok * g.inc_dloss];
        if (gmax > 0.0f) gq = __fdiv_rn(gq, gmax);       // (gmax is that of the finite ones)
        if (DT == kF16) gq = __fmul_rn(gq, kXentF16Scale);
        if (lab < 0) gq = __int_as_float(0x7fc00000);    // no such entry
        at = lab - g.v0 - col0;
    }
    const int left = gq == 0.0f ? 0 : g.vn - col0;
#pragma unroll
    for (int c = 0; c < COLS / 64; c++) {
        out.ready();
#pragma unroll
        for (int k = 0; k < 8; k++) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float q[2];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int col = 64 * c + 8 * k + j + i;
                    float p = xent_exp(v[col], about);               // (no product of a logit that overflows)
                    if (at == col) p = __fsub_rn(p, 1.0f);
                    q[i] = col < left ? __fmul_rn(p, gq) : 0.0f;
                }
                o[j / 2] = float2_to_word<DT>(q[0], q[1]);
            }
            out.put(k, o[0], o[1], o[2], o[3]);
        }
        out.send<false>(map, col0 + 64 * c, row0);
    }
}

// A split's sums of dX, added to those of the pieces before.
template <int UNROLL, class Ld>
__device__ __forceinline__ void epilogue_dx(const XentGemm &g, const CUtensorMap *map, const XOut &out, int row0,
                                            int n, int split, int col0, Ld ld)
{
#pragma unroll UNROLL
    for (int c = 0; c < XTile<kXentTile>::kCols / 32; c++) {
        float v[32];
        ld(c, v);
        if ((size_t)(col0 + 32 * c) >= g.ldws || row0 >= n) continue;
        out.ready();
#pragma unroll
        for (int k = 0; k < 8; k++)
            out.put(k, __float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                    __float_as_uint(v[4 * k + 3]));
        const int to = split * (int)g.tpad + row0;
        if (g.first)
            out.send<false>(map, col0 + 32 * c, to);
        else
            out.send<true>(map, col0 + 32 * c, to);
    }
}

// Rows of dW, rounded; row0 within the piece.  Rows that no tensor map takes (not
// 16-byte aligned) are written from the staging, 64 bytes of a row at a time.
template <int DT, int UNROLL, class Ld>
__device__ __forceinline__ void epilogue_dw(const XentGemm &g, const CUtensorMap *map, const XOut &out, int row0,
                                            int col0, Ld ld)
{
    const uint32_t lane = threadIdx.x & 31;
    float scale = __uint_as_float(g.head[1]);
    if (DT == kF16) scale = __fmul_rn(scale, 1.0f / kXentF16Scale);
#pragma unroll UNROLL
    for (int c = 0; c < XTile<kXentTile>::kCols / 64; c++) {
        uint32_t o[32];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float v[32];
            ld(2 * c + h, v);
#pragma unroll
            for (int j = 0; j < 16; j++)
                o[16 * h + j] = float2_to_word<DT>(__fmul_rn(v[2 * j], scale), __fmul_rn(v[2 * j + 1], scale));
        }
        const int col = col0 + 64 * c, left = g.H - col;
        if (left <= 0 || row0 >= g.vn) continue;
        out.ready();
#pragma unroll
        for (int k = 0; k < 8; k++) out.put(k, o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        if (g.al_dw) {
            out.send<false>(map, col, g.v0 + row0);
            continue;
        }
        __syncwarp();
        uint16_t *to = (uint16_t *)g.dw + (size_t)(g.v0 + row0) * g.lddw + col + lane;
        const int rows = min(32, g.vn - row0);
        const bool in0 = (int)lane < left, in1 = (int)lane + 32 < left;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 8) {               // eight rows' values read ahead of their stores
            uint16_t e[16];
#pragma unroll
            for (uint32_t i = 0; i < 16; i++) {              // (a row's number mod 8 is i / 2)
                const uint32_t at = 2 * (lane + 32 * (i & 1u));
                e[i] = *reinterpret_cast<const uint16_t *>(out.smem + 128 * (r0 + i / 2) + (at & 15u) +
                                                           16 * ((at >> 4) ^ (i / 2)));
            }
#pragma unroll
            for (int i = 0; i < 8; i++, to += g.lddw)
                if (r0 + i < rows) {
                    if (in0) to[0] = e[2 * i];
                    if (in1) to[32] = e[2 * i + 1];
                }
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- the kernel

// TN: columns of a tile, 256; of the logits also 64, where every such tile has a
// pair to itself.  A box of K takes the MMAs as long either way (their A, 128 rows
// an SM, comes from shared memory at 128 cycles a slice of 16), so a narrow tile
// saves its epilogue's time alone: 64 tokens x 2048 over 1000 15.2 us, 16.8 with
// 256 columns.
template <int DT, int MODE, int TN>
__global__ void __launch_bounds__(kXThreads, 1)
xent_kernel(const __grid_constant__ XentMaps maps, const XentGemm g)
{
    pdl_launch_dependents();
    using Y = XLayout<MODE, TN>;
    using N = XTile<TN>;
    constexpr int kStages = Y::kStages;
    constexpr bool kBack = MODE == kXentBack || MODE == kXentBackLong;
    constexpr int kChain = kBack ? kXBackChain : kXChain;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t ring = smem_addr(smem);
    const uint32_t bars = ring + Y::kOffBars;
    auto full_bar = [&](int s) { return bars + 8u * (uint32_t)s; };
    auto empty_bar = [&](int s) { return bars + 8u * (uint32_t)(kStages + s); };
    auto dfull_bar = [&](int b) { return bars + 8u * (uint32_t)(2 * kStages + b); };
    auto dempty_bar = [&](int b) { return bars + 8u * (uint32_t)(2 * kStages + kXDBuffers + b); };
    const uint32_t drain_bar = bars + 8u * (uint32_t)(2 * kStages + 2 * kXDBuffers);
    uint32_t *misc = (uint32_t *)(smem + Y::kOffMisc);
    volatile uint32_t *tmem_holder = misc;
    volatile uint32_t *abort = misc + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < kXDBuffers; b++) {
            mbar_init(dfull_bar(b), 1);
            mbar_init(dempty_bar(b), 2 * N::kWarps);              // both CTAs' epilogues
        }
        mbar_init(drain_bar, 1);
        *abort = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        auto fetch = [](const CUtensorMap *m) { asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)m) : "memory"); };
        fetch(&maps.x);
        fetch(kBack ? &maps.p : &maps.x128);
        fetch(kBack ? &maps.w : TN == 64 ? &maps.w32 : &maps.w128);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (warp == 1) {
        // together with the peer CTA's warp 1
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr((const void *)tmem_holder)), "r"(kXTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync_all();        // both CTAs' barriers and allocation are in place
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait_primary();
    const int n = g.head ? (int)g.head[0] : g.n;
    const XUnits units(g, n, kBack, TN);

    if (warp == 0) {
        // ---------------- producer: this CTA's halves; completion on the leader's full barrier
        if (lane == 0) {
            int st = 0;
            uint32_t phase = 0, armed = 0;                   // stages armed so far, in turn
            const uint32_t full0 = map_to_rank(full_bar(0), 0u);
            XUnit u;
            for (int i = 0; !*abort && units.get(i, u); i++) {
                const int m0 = u.tm * kXentTile + kXHalf * (int)rank, n0 = u.tn * TN + TN / 2 * (int)rank;
                const bool a_mn = kBack && !u.x, b_mn = kBack;
                // K-major operands come in boxes of all their rows, 128 (A: or 64) or 32; MN-major
                // ones in two of 64 x 64
                const int a_boxes = min(2, max(0, u.rows - 2 * (int)rank));
                const bool a_whole = !a_mn && a_boxes == 2;
                const CUtensorMap *ma = kBack ? (a_whole ? &maps.p128 : &maps.p) : (a_whole ? &maps.x128 : &maps.x);
                const CUtensorMap *mb = TN == 64 ? &maps.w32 : !kBack ? &maps.w128 : u.x ? &maps.w : &maps.x;
                const uint32_t bytes = (uint32_t)(u.rows * kXBoxBytes + 2 * N::kBBytes);
                // the vocabulary's coordinate counts from the piece's first entry in P only
                const int b_row = kBack ? (u.x ? g.v0 : 0) : n0 + g.v0;
                bool ok = true;
                for (int j = 0; j < u.nk; j++) {
                    if (!x_wait(empty_bar(st), phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = ring + (uint32_t)st * N::kStageBytes, fb = full0 + 8u * (uint32_t)st;
                    const int kc = (u.k0 + j) * kXBox;
                    if (leader) mbar_arrive_expect_tx(full_bar(st), bytes);
                    if (a_mn) {
                        tma_load_2d_pair(dst, ma, m0, kc, fb);
                        tma_load_2d_pair(dst + kXBoxBytes, ma, m0 + kXBox, kc, fb);
                    } else if (a_boxes > 0) {
                        tma_load_2d_pair(dst, ma, kc, m0, fb);
                    }
                    if (b_mn) {
                        tma_load_2d_pair(dst + kXHalfBytes, mb, n0, b_row + kc, fb);
                        tma_load_2d_pair(dst + kXHalfBytes + kXBoxBytes, mb, n0 + kXBox, b_row + kc, fb);
                    } else {
                        tma_load_2d_pair(dst + kXHalfBytes, mb, kc, b_row, fb);
                    }
                    armed++;
                    if (++st == kStages) {
                        st = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
            }
            if (*abort && leader) {
                // the full barriers count both CTAs' copies: let them land
                for (uint32_t i = armed < (uint32_t)kStages ? 0u : armed - kStages; i < armed; i++)
                    (void)mbar_wait_limited(full_bar((int)(i % kStages)), (i / kStages) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (the leader's lane 0)
        if (leader && lane == 0) {
            int st = 0, b = 0;
            uint32_t phase = 0, dphase = 0;       // bit b: uses of accumulator b so far, mod 2
            bool withhold = g.inject_stall != 0u;
            XUnit u;
            for (int i = 0; !*abort && units.get(i, u); i++) {
                const bool a_mn = kBack && !u.x, b_mn = kBack;
                const uint32_t idesc = operand_instr<DT, TN>(a_mn, b_mn);
                const uint64_t a_ring = operand_desc(ring, a_mn), b_ring = operand_desc(ring + kXHalfBytes, b_mn);
                const uint64_t a_step = a_mn ? 2048u >> 4 : 32u >> 4, b_step = b_mn ? 2048u >> 4 : 32u >> 4;
                bool ok = true;
                for (int j0 = 0; ok && (j0 < u.nk || j0 == 0); j0 += kChain) {
                    // both epilogues have read accumulator b
                    if (!x_wait(dempty_bar(b), ((dphase >> b) & 1u) ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(b * kXentTile);
                    const int end = min(u.nk, j0 + kChain);
                    for (int j = j0; j < end; j++) {
                        if (!x_wait(full_bar(st), phase, abort)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t at = (uint64_t)st * (uint64_t)(N::kStageBytes >> 4);
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            tc_mma_pair(d, a_ring + at + (uint64_t)k * a_step, b_ring + at + (uint64_t)k * b_step, idesc,
                                        (j > j0 || k > 0) ? 1u : 0u);
                        tc_commit_pair(empty_bar(st));           // both CTAs' stage is free
                        if (++st == kStages) {
                            st = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    if (withhold)
                        withhold = false;
                    else
                        tc_commit_pair(dfull_bar(b));            // the chain is in both CTAs' TMEM
                    dphase ^= 1u << b;
                    b ^= 1;
                }
                if (!ok) break;
            }
            tc_commit_pair_local(drain_bar);
            (void)mbar_wait_limited(drain_bar, 0u);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: a warp takes 32 rows and 128 columns of the tile
        const int q = warp & 3, half = (warp - 2) >> 2;          // (a warp reads the lanes of its number mod 4)
        const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * N::kCols);
        const XOut out = {smem + Y::kOffOut + (warp - 2) * kXOutBytes,
                          ring + (uint32_t)(Y::kOffOut + (warp - 2) * kXOutBytes)};
        int b = 0;
        uint32_t dphase = 0;
        bool live = false;
        auto begin = [&] {
            const bool ready = !*abort && x_wait(dfull_bar(b), (dphase >> b) & 1u, abort);
            live = __all_sync(kFull, ready);
            if (live) tc_fence_after();
        };
        auto done = [&] {
            if (live) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(dempty_bar(b), 0u));
            }
            dphase ^= 1u << b;
            b ^= 1;
        };
        XUnit u;
        for (int i = 0; warp - 2 < N::kWarps && units.get(i, u); i++) {
            const int row0 = u.tm * kXentTile + kXHalf * (int)rank + 32 * q, col0 = u.tn * TN + half * N::kCols;
            if constexpr (MODE != kXentBack) {                   // chains, added up in registers
                float v[N::kCols];
                begin();
                __syncwarp();
                // (without an MMA, K of nothing, the accumulator holds another tile's sums)
                if (live && !(kBack && u.nk == 0)) {
                    tc_ld_row(base + (uint32_t)(b * kXentTile), v);
                } else {
#pragma unroll
                    for (int j = 0; j < N::kCols; j++) v[j] = live ? 0.0f : __int_as_float(0x7fc00000);
                }
                done();
#pragma unroll 1
                for (int j0 = kChain; j0 < u.nk; j0 += kChain) {
                    begin();
#pragma unroll
                    for (int c = 0; c < N::kCols / 16; c++) {
                        float f[16];
                        __syncwarp();
                        if (live) {
                            tc_ld_row16(base + (uint32_t)(b * kXentTile + 16 * c), f);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; j++) f[j] = __int_as_float(0x7fc00000);
                        }
#pragma unroll
                        for (int j = 0; j < 16; j++) v[16 * c + j] = __fadd_rn(v[16 * c + j], f[j]);
                    }
                    done();
                }
                if constexpr (MODE == kXentForward) {
                    if (row0 < n) epilogue_forward<N::kCols>(g, (size_t)(row0 + lane), u.tn * (TN / N::kCols) + half, v);
                } else if constexpr (MODE == kXentGradient) {
                    epilogue_gradient<DT, N::kCols>(g, &maps.p_out, out, row0, n, col0, v);
                } else {
                    auto of = [&](int c, float (&w)[32]) {
#pragma unroll
                        for (int j = 0; j < 32; j++) w[j] = v[32 * c + j];
                    };
                    if (u.x)
                        epilogue_dx<4>(g, &maps.ws_out, out, row0, n, u.split, col0, of);
                    else
                        epilogue_dw<DT, 2>(g, &maps.dw_out, out, row0, col0, of);
                }
            } else {
                begin();
                // without an MMA (K of nothing) the accumulator holds another tile's sums
                const float fill = live ? 0.0f : __int_as_float(0x7fc00000);
                const bool read = live && u.nk > 0;
                auto ld = [&](int c, float (&v)[32]) {
                    __syncwarp();
                    if (read) {
                        tc_ld_row32(base + (uint32_t)(b * kXentTile + 32 * c), v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j++) v[j] = fill;
                    }
                };
                if (u.x)
                    epilogue_dx<1>(g, &maps.ws_out, out, row0, n, u.split, col0, ld);
                else
                    epilogue_dw<DT, 1>(g, &maps.dw_out, out, row0, col0, ld);
                done();
            }
        }
        if (MODE != kXentForward && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // the leader's MMAs read the peer's shared memory and write its tensor
    // memory: neither CTA leaves or frees before both are done
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kXTmemCols)
                     : "memory");
    }
}

// ---------------------------------------------------------------- host

namespace {

template <int DT>
const void *xent_pick(int mode, bool narrow)
{
    if (mode == kXentForward)
        return narrow ? (const void *)xent_kernel<DT, kXentForward, 64> : (const void *)xent_kernel<DT, kXentForward, 256>;
    if (mode == kXentGradient)
        return narrow ? (const void *)xent_kernel<DT, kXentGradient, 64>
                      : (const void *)xent_kernel<DT, kXentGradient, 256>;
    return mode == kXentBack ? (const void *)xent_kernel<DT, kXentBack, 256>
                             : (const void *)xent_kernel<DT, kXentBackLong, 256>;
}

const void *xent_pick(int dtype, int mode, bool narrow)
{
    return dtype == kF16 ? xent_pick<kF16>(mode, narrow) : xent_pick<kBF16>(mode, narrow);
}

int xent_smem(int mode, bool narrow)
{
    if (mode == kXentForward)
        return narrow ? XLayout<kXentForward, 64>::kSmemBytes : XLayout<kXentForward, 256>::kSmemBytes;
    if (mode == kXentGradient && narrow) return XLayout<kXentGradient, 64>::kSmemBytes;
    return XLayout<kXentBack, 256>::kSmemBytes;
}

cudaLaunchConfig_t pair_config(int mode, bool narrow, int pairs, cudaLaunchAttribute (&attr)[2], cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(kXThreads);
    cfg.dynamicSmemBytes = (size_t)xent_smem(mode, narrow);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

}  // namespace

// The pairs that can be resident at once on the current device, cached; -1, not
// cached, where the device could not be asked.
int xent_pairs()
{
    static std::mutex mu;
    static std::vector<std::pair<int, int>> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return -1;
    }
    {
        std::lock_guard<std::mutex> lk(mu);
        for (auto &c : cache)
            if (c.first == dev) return c.second;
    }
    int n = 0, sms = 0;
    bool ok = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
    for (int dt : {kF16, kBF16})
        for (int mode : {kXentForward, kXentGradient, kXentBack, kXentBackLong})
            for (bool narrow : {false, true})
                ok = ok && set_smem_once((void *)xent_pick(dt, mode, narrow), xent_smem(mode, narrow)) == cudaSuccess;
    if (ok) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = pair_config(kXentBack, false, sms / 2, attr, nullptr);
        cfg.numAttrs = 1;
        ok = cudaOccupancyMaxActiveClusters(&n, xent_pick(kBF16, kXentBack, false), &cfg) == cudaSuccess;
    }
    (void)cudaGetLastError();
    if (!ok || plan::fault_injected("query")) return -1;
    std::lock_guard<std::mutex> lk(mu);
    cache.emplace_back(dev, n);
    return n;
}

// A matrix of 16-bit values (or, `wide`, of binary32) in boxes of 128 bytes x
// box_rows rows.
cudaError_t xent_map(CUtensorMap *map, const void *base, size_t cols, size_t rows, size_t ld, int box_rows, bool wide)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint32_t box[2] = {wide ? 32u : (cuuint32_t)kXBox, (cuuint32_t)box_rows}, step[2] = {1, 1};
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, pitch[1] = {(cuuint64_t)ld * (wide ? 4 : 2)};
    return encode(map, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, (void *)base, dims,
                  pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

int xent_tile_cols(size_t tokens, size_t vn, int pairs)
{
    const size_t narrow = ((tokens + kXentTile - 1) / kXentTile) * ((vn + 63) / 64);
    return narrow <= (size_t)pairs ? 64 : kXentTile;
}

cudaError_t launch_xent(int dtype, int mode, const XentMaps &maps, const XentGemm &g, size_t units, int pairs,
                        int tile_cols, cudaStream_t stream)
{
    // a K of more than one chain: dX's, dW's
    if (mode == kXentBack && ((g.ws && ((g.vn + kXBox - 1) / kXBox + g.splits - 1) / g.splits > kXBackChain) ||
                              (g.dw && g.tpad > (size_t)(kXBackChain * kXBox))))
        mode = kXentBackLong;
    void *args[] = {(void *)&maps, (void *)&g};
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pair_config(mode, tile_cols == 64, (int)(units < (size_t)pairs ? units : (size_t)pairs), attr, stream);
    return cudaLaunchKernelExC(&cfg, xent_pick(dtype, mode, tile_cols == 64), args);
}

cudaError_t read_xent_faults(unsigned int *flags, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_xent_fault, sizeof(unsigned int));
    if (e != cudaSuccess || !clear) return e;
    const unsigned int zero = 0u;
    return cudaMemcpyToSymbol(g_xent_fault, &zero, sizeof(unsigned int));
}

}  // namespace tcr
