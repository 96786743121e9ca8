// k_layer_back.cu -- the gradient of the layer norm with dropout.
//
//   xh = (h - mean) * rstd,  g = dy * w,
//   a = (row sum of g) / cols,  c = (row sum of g * xh) / cols
//   dr = rstd * ((g - a) - xh * c) + dh     (of the residual, and of h)
//   dx = dropout(dr)                        (of x: the mask formed again)
//   dw_j = sum over rows of dy * xh,  db_j = sum over rows of dy
//
// Both row sums fold in one exchange, in the declared order of rowvec.cuh.
// dw and db: CTA b of G adds its rows b, b + G, .. in order, and a second kernel
// adds the G partials: 32 threads a column, thread k the partials k, k + 32, .. in
// order, then the halving fold over the 32.  G depends on rows, cols and the
// type only (layer_back_groups); there are no atomics.
#include "kernels.cuh"
#include "piece.cuh"
#include "plan.h"
#include "tc05.cuh"

namespace tcr {

// A thread's column sums, at any alignment of binary32.
template <int L>
__device__ __forceinline__ void store_sums(float *p, uint32_t n, const float (&acc)[kRv])
{
    if (L == kVectors && ((uintptr_t)p & 15u) == 0) {
        store_piece<kF32, kVectors>((uint32_t *)p, n, acc);
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < kRv; k++)
        if (k < n) p[value_at<L>(k)] = acc[k];
}

// xh from h.
__device__ __forceinline__ void normalise(float mean, float rstd, float (&xh)[kRv])
{
    add8(xh, xh, -mean);
    mul8(xh, xh, rstd);
}

// The trees over g and g * xh of n values: absent ones count as 0 whatever was
// read in their place and whatever mean and rstd are.
template <int L>
__device__ __forceinline__ void row_trees(uint32_t n, float (&xh)[kRv], float (&g)[kRv], float &sa, float &sc)
{
    zero_absent(n, xh);
    zero_absent(n, g);
    float e[kRv];
    mul8(e, g, xh);
    sa = piece_tree<L>(g);
    sc = piece_tree<L>(e);
}

// rstd * ((g - a) - xh * c), over g; xh is lost.
__device__ __forceinline__ void back_dr(float rstd, float a, float c, float (&xh)[kRv], float (&g)[kRv])
{
    add8(g, g, -a);
    mul8(xh, xh, -c);
    add8(g, g, xh);
    mul8(g, g, rstd);
}

// The thread's sums of eight columns in shared memory, `step` float4 apart.
__device__ __forceinline__ void add_sums(float4 *p, uint32_t step, const float (&e)[kRv])
{
    const float4 u = p[0], v = p[step];
    float f[kRv] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    add8(f, f, e);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[step] = make_float4(f[4], f[5], f[6], f[7]);
}

// The rows of one CTA, NV pieces a thread, of which the first LEAD are whole;
// ALL: there are a weight and a dh.
template <int DT, bool ELEM, int T, int NV, int LEAD, bool ALL>
__device__ __forceinline__ void layer_back_rows(const LayerBackArgs &a, const Drop &drop, float4 *sums, float *red)
{
    using E = typename Elem<DT>::T;
    constexpr int L = layout_of<DT, ELEM>();
    constexpr uint32_t kStep = kRv * T;
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    const bool has_w = ALL || a.w != nullptr, has_dh = ALL || a.dh != nullptr;
    const uint32_t at = piece_offset<L>(t);
    auto count = [&](int i) { return piece_count<L, T, LEAD>(cols, at, i); };
    int buf = 0;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x, buf ^= 1) {
        Piece<DT> dy[NV], h[NV], dh[NV];
        const E *pdy = (const E *)a.dy + r * a.lddy + at, *ph = (const E *)a.h + r * a.ldh + at;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t n = count(i);
            load_piece<DT, L>(pdy + i * kStep, n, dy[i], by_words(pdy));
            load_piece<DT, L>(ph + i * kStep, n, h[i], by_words(ph));
        }
        if (has_dh) {
            const E *pdh = (const E *)a.dh + r * a.lddh + at;
#pragma unroll
            for (int i = 0; i < NV; i++)
                load_piece<DT, L>(pdh + i * kStep, count(i), dh[i], by_words(pdh));
        }
        const float mean = a.mean[r], rstd = a.rstd[r];
        float sa[NV], sc[NV], g_of[NV][kRv];
        auto weigh = [&](int i, float (&g)[kRv]) {
            Piece<DT> w;
            float f[kRv];
            load_piece<DT, L>((const E *)a.w + at + i * kStep, count(i), w, by_words(a.w));
            piece_values<DT>(w, f);
            mul8(g, g, f);
        };
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float xh[kRv], (&g)[kRv] = g_of[i];
            piece_values<DT>(h[i], xh);
            piece_values<DT>(dy[i], g);
            normalise(mean, rstd, xh);
            float e[kRv];
            mul8(e, g, xh);
            add_sums(sums + 4 * i * T + t, T, e);
            add_sums(sums + (4 * i + 2) * T + t, T, g);
            if (has_w) weigh(i, g);
            row_trees<L>(count(i), xh, g, sa[i], sc[i]);
        }
        // two buffers: a thread reaches the next row's write of this one only
        // after every thread has passed the barrier of the row between
        float m[2] = {fold<NV>(sa), fold<NV>(sc)};
        team_sums<T, L>(m, red + buf * 2 * T);
        const float ma = __fdiv_rn(m[0], (float)cols), mc = __fdiv_rn(m[1], (float)cols);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t n = count(i);
            float xh[kRv], (&g)[kRv] = g_of[i];
            piece_values<DT>(h[i], xh);
            normalise(mean, rstd, xh);
            back_dr(rstd, ma, mc, xh, g);
            if (has_dh) {
                float d[kRv];
                piece_values<DT>(dh[i], d);
                add8(g, g, d);
            }
            if (a.dr) {
                E *p = (E *)a.dr + r * a.lddr + at + i * kStep;
                store_piece<DT, L>(p, n, g, by_words(p));
            }
            if (a.dx) {
                E *p = (E *)a.dx + r * a.lddx + at + i * kStep;
                drop_values<L>(drop, t + i * T, r, g);
                store_piece<DT, L>(p, n, g, by_words(p));
            }
        }
    }
}

// Rows of at most T NV vectors, NV pieces a thread.  A CTA walks the rows b, b +
// G, .. and keeps its sums of dw and db in shared memory, thread by thread, so
// that registers hold one row's g and its h and dh as they were read (xh is
// formed again after the barrier) and 1024 threads (binary32: 768) fit an SM:
// their rows are at different steps, and none is loaded ahead.  16384 x 4096
// bfloat16 with dropout, both gradients and sums 119 us (issuing on 63% of
// cycles; 83% of the copy rate, 87% without the sums' launch); with the sums in
// registers and the next row loaded ahead, two CTAs of 256 threads an SM, 163.
template <int DT, bool ELEM, int T, int NV, int LEAD, int MINB>
__global__ void __launch_bounds__(T, MINB)
layer_back_kernel(const __grid_constant__ LayerBackArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    extern __shared__ float4 sums[];                     // [4 NV][T]: a piece's dw, then its db
    __shared__ float red[4 * T];
    constexpr int L = layout_of<DT, ELEM>();
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    const Drop drop(a.drop);
#pragma unroll
    for (int i = 0; i < 4 * NV; i++) sums[i * T + t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (warp_whole<T, NV>(cols, t) && a.w && a.dh)
        layer_back_rows<DT, ELEM, T, NV, NV, true>(a, drop, sums, red);
    else
        layer_back_rows<DT, ELEM, T, NV, LEAD, false>(a, drop, sums, red);
    // partial[b * cols + j]: the sum of column j over the rows b, b + G, ..
#pragma unroll
    for (int i = 0; i < 2 * NV; i++) {
        float *to = i % 2 ? a.partial_b : a.partial_w;
        if (!to) continue;
        const uint32_t first = piece_offset<L>(t) + (uint32_t)(i / 2 * kRv * T);
        const float4 u = sums[2 * i * T + t], v = sums[(2 * i + 1) * T + t];
        const float f[kRv] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        store_sums<L>(to + (size_t)blockIdx.x * cols + first, piece_count<L>(cols, first), f);
    }
}

// Longer rows: the row sums first (sums[2 r], sums[2 r + 1]), then blocks of 8
// * 256 columns, which are the grid's x (2^27 columns are 65536 of them).
template <int DT>
__device__ __forceinline__ void load_back(const LayerBackArgs &a, size_t r, uint32_t v, float (&xh)[kRv],
                                          float (&g)[kRv], float (&w)[kRv])
{
    using E = typename Elem<DT>::T;
    const uint32_t cols = (uint32_t)a.cols;
    unpack<DT>(load_raw<DT>((const E *)a.h + r * a.ldh, cols, v, a.al_h), xh);
    unpack<DT>(load_raw<DT>((const E *)a.dy + r * a.lddy, cols, v, a.al_dy), g);
    if (a.w) unpack<DT>(load_raw<DT>((const E *)a.w, cols, v, a.al_w), w);
}

template <int DT>
__global__ void __launch_bounds__(kRowLongT)
layer_back_sums_kernel(const __grid_constant__ LayerBackArgs a, float *sums)
{
    constexpr uint32_t T = kRowLongT;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2 * T];
    const size_t r = blockIdx.x;
    const uint32_t cols = (uint32_t)a.cols, nvec = (cols + kRv - 1) / kRv, steps = (nvec + T - 1) / T;
    const int bits = ceil_log2_sz(steps);
    const float mean = a.mean[r], rstd = a.rstd[r];
    TreeCounter<16> ta, tc;
    for (uint32_t j = 0; j < (1u << bits); j++) {
        const uint32_t v = threadIdx.x + bit_reverse(j, bits) * T;
        float sa = 0.0f, sc = 0.0f;
        if (v < nvec) {
            float xh[kRv], g[kRv], w[kRv];
            load_back<DT>(a, r, v, xh, g, w);
            normalise(mean, rstd, xh);
            if (a.w) mul8(g, g, w);
            row_trees<kVectors>(vec_left(cols, v), xh, g, sa, sc);
        }
        ta.push(sa);
        tc.push(sc);
    }
    float m[2] = {ta.finish(), tc.finish()};
    team_sums<(int)T, kVectors>(m, red);
    if (threadIdx.x == 0) {
        sums[2 * r] = __fdiv_rn(m[0], (float)cols);
        sums[2 * r + 1] = __fdiv_rn(m[1], (float)cols);
    }
}

constexpr int kBackLongT = 256;
template <int DT>
__global__ void __launch_bounds__(kBackLongT)
layer_back_long_kernel(const __grid_constant__ LayerBackArgs a, const float *sums)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    using E = typename Elem<DT>::T;
    const uint32_t v = blockIdx.x * kBackLongT + threadIdx.x, cols = (uint32_t)a.cols;
    const Drop drop(a.drop);
    const uint32_t left = vec_left(cols, v);
    float accw[kRv], accb[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) accw[k] = accb[k] = 0.0f;
    for (size_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float rstd = a.rstd[r];
        float xh[kRv], g[kRv], w[kRv], e[kRv];
        load_back<DT>(a, r, v, xh, g, w);
        normalise(a.mean[r], rstd, xh);
        mul8(e, g, xh);
        add8(accw, accw, e);
        add8(accb, accb, g);
        if (a.w) mul8(g, g, w);
        back_dr(rstd, sums[2 * r], sums[2 * r + 1], xh, g);
        if (a.dh) {
            float d[kRv];
            unpack<DT>(load_raw<DT>((const E *)a.dh + r * a.lddh, cols, v, a.al_dh), d);
#pragma unroll
            for (int k = 0; k < kRv; k++) g[k] = __fadd_rn(g[k], d[k]);
        }
        if (a.dr) store_vec<DT>((E *)a.dr + r * a.lddr, cols, v, a.al_dr, g);
        if (a.dx) {
            drop_values<kVectors>(drop, v, r, g);
            store_vec<DT>((E *)a.dx + r * a.lddx, cols, v, a.al_dx, g);
        }
    }
    const size_t to = (size_t)blockIdx.y * cols + kRv * v;
    if (a.partial_w) store_sums<kVectors>(a.partial_w + to, left, accw);
    if (a.partial_b) store_sums<kVectors>(a.partial_b + to, left, accb);
}

// dw[j] (block y = 0) and db[j] (1) from the G partials of column j.
__global__ void __launch_bounds__(1024)
layer_sums_kernel(const float *partial_w, const float *partial_b, size_t cols, int G, float *dw, float *db)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    const float *partial = blockIdx.y ? partial_b : partial_w;
    float *out = blockIdx.y ? db : dw;
    if (!out) return;
    __shared__ float s[32][33];
    const size_t j = (size_t)blockIdx.x * 32 + threadIdx.x;
    float acc = 0.0f;
    if (j < cols) {
#pragma unroll 8
        for (int g = threadIdx.y; g < G; g += 32) acc = __fadd_rn(acc, partial[(size_t)g * cols + j]);
    }
    s[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    // warp y folds column y of the 32
    const float v = halving_lanes(s[threadIdx.x][threadIdx.y]);
    const size_t jo = (size_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && jo < cols) out[jo] = v;
}

// ---------------------------------------------------------------- host

namespace {

// The kernel of a row length, and the CTAs of it that an SM holds (what registers
// and shared memory let it): they make the number of partial sums.
template <int DT, bool ELEM>
const void *pick(size_t nvec, unsigned &threads, size_t &smem, int &ctas)
{
#define TCR_BACK(T_, NV_, MINB_)                                      \
    return (threads = T_, smem = (size_t)T_ * NV_ * 64, ctas = MINB_, \
            (const void *)layer_back_kernel<DT, ELEM, T_, NV_, NV_ - 1, MINB_>)
    // The fastest of those measured (with dropout and the sums; threads whose last
    // pieces are past the row's end issue for nothing): bfloat16 16384 x 4096 256 x 2
    // in 119 us, 128 x 4 in 124; 32768 x 1536 64 x 3 97, 128 x 2 129; 20000 x 2560
    // 64 x 5 101, 128 x 3 123; 10000 x 5120 128 x 5 101, 256 x 3 139; 10000 x 6144
    // 256 x 3 127, 128 x 6 130; 8000 x 7168 128 x 7 125, 512 x 2 142.  binary32, 2^26
    // elements: 512 columns 64 x 1 224, 128 x 1 278; 3000 128 x 3 217, 256 x 2 241; 4096 256 x
    // 2 236, 128 x 4 229; 6144 256 x 3 222, 128 x 6 216.  Not the fastest: 1024 64 x 2 240,
    // 128 x 1 205; 2048 128 x 2 238, 256 x 1 219; 5120 128 x 5 227, 256 x 3 219; 8192 512 x 2 249,
    // 128 x 8 213.  A shape's CTAs are the order of dw's and db's sums, which stays.
    if constexpr (DT == kF32) {
        if (nvec <= 64) TCR_BACK(64, 1, 12);
        if (nvec <= 128) TCR_BACK(64, 2, 12);
        if (nvec <= 256) TCR_BACK(128, 2, 6);
        if (nvec <= 384) TCR_BACK(128, 3, 4);
        if (nvec <= 512) TCR_BACK(256, 2, 3);
        if (nvec <= 640) TCR_BACK(128, 5, 3);
        if (nvec <= 768) TCR_BACK(256, 3, 2);
        TCR_BACK(512, 2, 1);
    } else {
        if (nvec <= 64) TCR_BACK(64, 1, 16);
        if (nvec <= 128) TCR_BACK(64, 2, 16);
        if (nvec <= 192) TCR_BACK(64, 3, 12);
        if (nvec <= 256) TCR_BACK(128, 2, 8);
        if (nvec <= 320) TCR_BACK(64, 5, 8);
        if (nvec <= 384) TCR_BACK(128, 3, 5);
        if (nvec <= 512) TCR_BACK(256, 2, 4);
        if (nvec <= 640) TCR_BACK(128, 5, 4);
        if (nvec <= 768) TCR_BACK(256, 3, 2);
        if (nvec <= 896) TCR_BACK(128, 7, 3);
        TCR_BACK(512, 2, 2);
    }
#undef TCR_BACK
}

int back_ctas(size_t nvec, int dtype)
{
    unsigned threads;
    size_t smem;
    int ctas = 0;
    if (dtype == kF32)
        pick<kF32, false>(nvec, threads, smem, ctas);
    else
        pick<kBF16, false>(nvec, threads, smem, ctas);           // (binary16's are the same)
    return ctas;
}

}  // namespace

// As many CTAs as fit the SMs, but (above one an SM) no more than half the rows: a
// partial costs as much traffic as a row (1001 x 1537 binary32 12.4 us, with a
// quarter of the rows 16.3, with all of them 12.3).
// Longer rows: as many as make, with their blocks of columns, two rounds of the
// three CTAs that an SM holds, or one of the four in binary32.  As many as the rule
// above counts were 64 CTAs a group here, and their partials as large as the
// inputs: bfloat16 304 x 131072 277 us and 159 MB of partials, so 192 and 15; 152 x 2^20
// 1491 and 921; 4096 x 16384 309 and 312, 20000 x 12288 1168 and 1164 (with four an SM 209,
// 921, 339, 1308, with eight 199, 873, 315, 1206); binary32 152 x 2^19 with four 409,
// three 489, six 463, 4096 x 16384 305, 318, 328, 8192 x 8200 411, 461, 447.
int layer_back_groups(size_t rows, size_t cols, int dtype)
{
    const size_t nvec = (cols + kRv - 1) / kRv;
    size_t g;
    if (nvec > kBackMaxVecs) {
        g = (size_t)plan::kRuleSMs * (dtype == kF32 ? 4 : 6) / ((nvec + kBackLongT - 1) / kBackLongT);
        if (g < 1) g = 1;
    } else {
        const size_t full = (size_t)plan::kRuleSMs * back_ctas(nvec, dtype);
        const size_t one = plan::kRuleSMs, half = (rows + 1) / 2 > one ? (rows + 1) / 2 : one;
        g = full < half ? full : half;
    }
    return (int)(rows < g ? rows : g);
}

size_t layer_back_scratch(size_t rows, size_t cols, int dtype, bool dweight, bool dbias)
{
    const size_t part = (size_t)layer_back_groups(rows, cols, dtype) * cols;
    const size_t sums = (cols + kRv - 1) / kRv > kBackMaxVecs ? 2 * rows : 0;
    return ((dweight ? part : 0) + (dbias ? part : 0) + sums) * sizeof(float);
}

namespace {

template <int DT>
cudaError_t launch_back(LayerBackArgs a, int G, float *sums, cudaStream_t stream)
{
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    if (nvec <= kBackMaxVecs) {
        void *args[] = {(void *)&a};
        unsigned threads = 0;
        size_t smem = 0;
        int ctas = 0;
        const bool elem = !a.al_dy || !a.al_h || (a.w && !a.al_w) || (a.dh && !a.al_dh) || (a.dx && !a.al_dx) || (a.dr && !a.al_dr);
        const void *k = elem ? pick<DT, true>(nvec, threads, smem, ctas) : pick<DT, false>(nvec, threads, smem, ctas);
        if (smem + 16 * threads > 48 * 1024) {               // beside red
            cudaError_t e = set_smem_once((void *)k, (int)smem);
            if (e != cudaSuccess) return e;
        }
        // A grid that fills every SM is not launched while the kernel before it
        // finishes: where that one holds little shared memory, an SM would take
        // its first CTAs with a small share of it and the rest in a second wave
        // (100 calls back to back, 65536 x 1024 bfloat16: 148 us, 119 this way).
        if (G == plan::kRuleSMs * ctas)
            return cudaLaunchKernel(k, dim3((unsigned)G), dim3(threads), args, smem, stream);
        return launch_first(k, dim3((unsigned)G), dim3(threads), args, smem, stream);
    }
    void *args[] = {(void *)&a, (void *)&sums};
    cudaError_t e = launch_first((const void *)layer_back_sums_kernel<DT>, dim3((unsigned)a.rows), dim3(kRowLongT),
                                 args, 0, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((nvec + kBackLongT - 1) / kBackLongT), (unsigned)G);
    return launch_first((const void *)layer_back_long_kernel<DT>, grid, dim3(kBackLongT), args, 0, stream);
}

}  // namespace

cudaError_t launch_layer_back(int dtype, LayerBackArgs a, float *scratch, float *dw, float *db, cudaStream_t stream)
{
    int G = layer_back_groups(a.rows, a.cols, dtype);
    const size_t part = (size_t)G * a.cols;
    a.partial_w = dw ? scratch : nullptr;
    a.partial_b = db ? scratch + (dw ? part : 0) : nullptr;
    float *sums = scratch + (dw ? part : 0) + (db ? part : 0);
    cudaError_t e = dtype == kF16    ? launch_back<kF16>(a, G, sums, stream)
                    : dtype == kBF16 ? launch_back<kBF16>(a, G, sums, stream)
                                     : launch_back<kF32>(a, G, sums, stream);
    if (e != cudaSuccess || (!dw && !db)) return e;
    const float *pw = a.partial_w, *pb = a.partial_b;
    size_t cols = a.cols;
    void *args[] = {(void *)&pw, (void *)&pb, (void *)&cols, (void *)&G, (void *)&dw, (void *)&db};
    return launch_first((const void *)layer_sums_kernel, dim3((unsigned)((cols + 31) / 32), 2), dim3(32, 32), args, 0,
                        stream);
}

}  // namespace tcr
