// k_layer_back.cu -- the gradient of the layer norm with dropout.
//
//   xh = (h - mean) * rstd,  g = dy * w,
//   a = (row sum of g) / cols,  c = (row sum of g * xh) / cols
//   dr = rstd * ((g - a) - xh * c) + dh     (of the residual, and of h)
//   dx = dropout(dr)                        (of x: the mask formed again)
//   dw_j = sum over rows of dy * xh,  db_j = sum over rows of dy
//
// Both row sums fold in one exchange, in the declared order of rowvec.cuh.
// dw and db: CTA b of G adds its rows b, b + G, .. in order, each thread holding
// its columns' sums in registers, and a second kernel adds the G partials: 32
// threads a column, thread k the partials k, k + 32, .. in order, then the
// halving fold over the 32.  G depends on rows and cols only
// (norm_back_groups); there are no atomics.
#include "kernels.cuh"
#include "piece.cuh"

namespace tcr {

// team_sum of two values at once.
template <int T, bool ELEM>
__device__ __forceinline__ void team_sum2(float &a, float &b, float *red, uint32_t threads)
{
    const uint32_t lane = threadIdx.x & 31;
    float *ra = red, *rb = red + team_floats<T>();
    if constexpr (T >= 512) {
        float *ta = ra + T / 32 * 33, *tb = rb + T / 32 * 33;
        const uint32_t warp = threadIdx.x >> 5, warps = threads >> 5;
        ra[warp * 33 + lane] = a;
        rb[warp * 33 + lane] = b;
        __syncthreads();
        for (uint32_t c = warp; c < 64; c += warps) {
            const float *r = c < 32 ? ra : rb;
            const float s = halving_lanes(lane < warps ? r[lane * 33 + (c & 31u)] : 0.0f);
            if (lane == 0) (c < 32 ? ta : tb)[c & 31u] = s;
        }
        __syncthreads();
        a = ta[lane];
        b = tb[lane];
    } else if constexpr (T > 32) {
        ra[threadIdx.x] = a;
        rb[threadIdx.x] = b;
        __syncthreads();
        float fa[T / 32], fb[T / 32];
#pragma unroll
        for (int w = 0; w < T / 32; w++) {
            fa[w] = 32u * w < threads ? ra[32 * w + lane] : 0.0f;
            fb[w] = 32u * w < threads ? rb[32 * w + lane] : 0.0f;
        }
        a = halving<T / 32>(fa);
        b = halving<T / 32>(fb);
    }
    a = ELEM ? halving_lanes_elem(a) : halving_lanes(a);
    b = ELEM ? halving_lanes_elem(b) : halving_lanes(b);
}

// g and xh of a thread's values and the trees over g and g * xh; adds dy * xh
// and dy to the column sums.
template <int DT, bool ELEM>
__device__ __forceinline__ void back_values(const float *w, float mean, float rstd, uint32_t cols, uint32_t v,
                                            float (&xh)[kRv], float (&g)[kRv], float *accw, float *accb, float &sa,
                                            float &sc)
{
#pragma unroll
    for (int k = 0; k < kRv; k++) xh[k] = __fmul_rn(__fsub_rn(xh[k], mean), rstd);
    zero_absent<ELEM>(cols, v, xh);
    float e[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) {
        if (accw) {
            accw[k] = __fadd_rn(accw[k], __fmul_rn(g[k], xh[k]));
            accb[k] = __fadd_rn(accb[k], g[k]);
        }
        if (w) g[k] = __fmul_rn(g[k], w[k]);
        e[k] = __fmul_rn(g[k], xh[k]);
    }
    sa = piece_tree<ELEM>(g);
    sc = piece_tree<ELEM>(e);
}

__device__ __forceinline__ void back_dr(float rstd, float a, float c, const float (&xh)[kRv], float (&g)[kRv])
{
#pragma unroll
    for (int k = 0; k < kRv; k++) g[k] = __fmul_rn(rstd, __fsub_rn(__fsub_rn(g[k], a), __fmul_rn(xh[k], c)));
}

// partial[b * cols + j]: the sum of column j over the rows b, b + G, ..
template <bool ELEM>
__device__ __forceinline__ void store_sums(float *partial, size_t b, uint32_t cols, uint32_t v, const float (&acc)[kRv])
{
    if (!partial) return;
    store_piece_values_any<ELEM>(partial + b * cols, cols, v, acc);
}

// Rows of at most T NV vectors, NV pieces a thread; NV = 1: a CTA of 32
// ceil(vectors / 32) <= T threads.  The next row's inputs are loaded before
// the current row's sums are waited for.
template <int DT, bool ELEM, int T, int NV, int MINB>
__global__ void __launch_bounds__(T, MINB)
layer_back_kernel(const LayerBackArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][2 * team_floats<T>()];
    using E = typename Elem<DT>::T;
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    const bool has_w = a.w != nullptr, has_dh = a.dh != nullptr;
    const DropArgs drop = drop_resolve(a.drop);
    Piece<DT, ELEM> dy[NV], h[NV], dh[NV], w[NV];
    float accw[NV][kRv], accb[NV][kRv];
    auto load = [&](size_t r) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t v = t + i * T;
            load_piece<DT, ELEM>((const E *)a.dy + r * a.lddy, cols, v, dy[i]);
            load_piece<DT, ELEM>((const E *)a.h + r * a.ldh, cols, v, h[i]);
            if (has_dh) load_piece<DT, ELEM>((const E *)a.dh + r * a.lddh, cols, v, dh[i]);
        }
    };
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (has_w) load_weight_piece<DT, ELEM>((const E *)a.w, cols, t + i * T, a.al_w, w[i]);
#pragma unroll
        for (int k = 0; k < kRv; k++) accw[i][k] = accb[i][k] = 0.0f;
    }
    load(blockIdx.x);
    float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
    int buf = 0;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x, buf ^= 1) {
        float sa[NV], sc[NV], xh[NV][kRv], g[NV][kRv];
        Piece<DT, ELEM> dh_now[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t v = t + i * T;
            float f[kRv];
            piece_values<DT, ELEM>(h[i], (const E *)a.h + r * a.ldh, cols, v, xh[i]);
            piece_values<DT, ELEM>(dy[i], (const E *)a.dy + r * a.lddy, cols, v, g[i]);
            if (has_w) piece_values<DT, ELEM>(w[i], (const E *)a.w, cols, v, f);
            back_values<DT, ELEM>(has_w ? f : nullptr, mean, rstd, cols, v, xh[i], g[i], accw[i], accb[i], sa[i],
                                  sc[i]);
            dh_now[i] = dh[i];
        }
        const size_t next = r + gridDim.x;
        const float rstd_now = rstd;
        if (next < a.rows) {
            load(next);
            mean = a.mean[next];
            rstd = a.rstd[next];
        }
        // two buffers: a thread reaches the next row's write of this one only
        // after every thread has passed the barrier of the row between
        float ma = halving<NV>(sa), mc = halving<NV>(sc);
        team_sum2<T, ELEM>(ma, mc, red[buf], blockDim.x);
        ma = __fdiv_rn(ma, (float)cols);
        mc = __fdiv_rn(mc, (float)cols);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t v = t + i * T;
            if (kRv * (v & ~31u) >= cols) continue;          // whole warps: stores are warp-wide
            back_dr(rstd_now, ma, mc, xh[i], g[i]);
            if (has_dh) {
                float d[kRv];
                piece_values<DT, ELEM>(dh_now[i], (const E *)a.dh + r * a.lddh, cols, v, d);
#pragma unroll
                for (int k = 0; k < kRv; k++) g[i][k] = __fadd_rn(g[i][k], d[k]);
            }
            if (a.dr) store_piece_values<DT, ELEM>((E *)a.dr + r * a.lddr, cols, v, g[i]);
            if (a.dx) {
                drop_values<ELEM>(drop, v, r, g[i]);
                store_piece_values<DT, ELEM>((E *)a.dx + r * a.lddx, cols, v, g[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const uint32_t v = t + i * T;
        store_sums<ELEM>(a.partial_w, blockIdx.x, cols, v, accw[i]);
        store_sums<ELEM>(a.partial_b, blockIdx.x, cols, v, accb[i]);
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
layer_back_sums_kernel(const LayerBackArgs a, float *sums)
{
    constexpr uint32_t T = kRowLongT;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2 * team_floats<T>()];
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
            back_values<DT, false>(a.w ? w : nullptr, mean, rstd, cols, v, xh, g, nullptr, nullptr, sa, sc);
        }
        ta.push(sa);
        tc.push(sc);
    }
    float ma = ta.finish(), mc = tc.finish();
    team_sum2<(int)T, false>(ma, mc, red, T);
    if (threadIdx.x == 0) {
        sums[2 * r] = __fdiv_rn(ma, (float)cols);
        sums[2 * r + 1] = __fdiv_rn(mc, (float)cols);
    }
}

template <int DT>
__global__ void __launch_bounds__(256)
layer_back_long_kernel(const LayerBackArgs a, const float *sums)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    using E = typename Elem<DT>::T;
    const uint32_t v = blockIdx.x * 256 + threadIdx.x, cols = (uint32_t)a.cols;
    const DropArgs drop = drop_resolve(a.drop);
    float accw[kRv], accb[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) accw[k] = accb[k] = 0.0f;
    for (size_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float rstd = a.rstd[r];
        float xh[kRv], g[kRv], w[kRv], sa, sc;
        load_back<DT>(a, r, v, xh, g, w);
        back_values<DT, false>(a.w ? w : nullptr, a.mean[r], rstd, cols, v, xh, g, accw, accb, sa, sc);
        back_dr(rstd, sums[2 * r], sums[2 * r + 1], xh, g);
        if (a.dh) {
            float d[kRv];
            unpack<DT>(load_raw<DT>((const E *)a.dh + r * a.lddh, cols, v, a.al_dh), d);
#pragma unroll
            for (int k = 0; k < kRv; k++) g[k] = __fadd_rn(g[k], d[k]);
        }
        if (a.dr) store_vec<DT>((E *)a.dr + r * a.lddr, cols, v, a.al_dr, g);
        if (a.dx) {
            drop_values<false>(drop, v, r, g);
            store_vec<DT>((E *)a.dx + r * a.lddx, cols, v, a.al_dx, g);
        }
    }
    store_sums<false>(a.partial_w, blockIdx.y, cols, v, accw);
    store_sums<false>(a.partial_b, blockIdx.y, cols, v, accb);
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

static size_t sums_floats(size_t rows, size_t cols)
{
    return (cols + kRv - 1) / kRv > kBackMaxVecs ? 2 * rows : 0;
}

size_t layer_back_scratch(size_t rows, size_t cols, bool dweight, bool dbias)
{
    const size_t part = (size_t)norm_back_groups(rows, cols) * cols;
    return ((dweight ? part : 0) + (dbias ? part : 0) + sums_floats(rows, cols)) * sizeof(float);
}

namespace {

template <int DT>
const void *pick(size_t nvec, bool elem, unsigned &threads)
{
#define TCR_BACK(ELEM_, T_, NV_, MINB_) \
    return (threads = NV_ == 1 ? (unsigned)((nvec + 31) / 32 * 32) : T_, \
            (const void *)layer_back_kernel<DT, ELEM_, T_, NV_, MINB_>)
    if (elem) {
        if (nvec <= 64) TCR_BACK(true, 64, 1, 8);
        if (nvec <= 128) TCR_BACK(true, 128, 1, 4);
        if (nvec <= 256) TCR_BACK(true, 256, 1, 2);
        if (nvec <= 512) TCR_BACK(true, 512, 1, 1);
        TCR_BACK(true, 1024, 1, 1);
    }
    if constexpr (DT == kF32) {
        if (nvec <= 64) TCR_BACK(false, 64, 1, 8);
        if (nvec <= 128) TCR_BACK(false, 128, 1, 4);
        if (nvec <= 256) TCR_BACK(false, 256, 1, 2);
        if (nvec <= 512) TCR_BACK(false, 512, 1, 1);
        TCR_BACK(false, 1024, 1, 1);
    } else {
        if (nvec <= 64) TCR_BACK(false, 64, 1, 12);
        if (nvec <= 128) TCR_BACK(false, 128, 1, 6);
        if (nvec <= 256) TCR_BACK(false, 256, 1, 3);
        if (nvec <= 512) TCR_BACK(false, 512, 1, 1);
        TCR_BACK(false, 512, 2, 1);
    }
#undef TCR_BACK
}

template <int DT>
cudaError_t launch_back(LayerBackArgs a, int G, float *sums, cudaStream_t stream)
{
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    if (nvec <= kBackMaxVecs) {
        void *args[] = {(void *)&a};
        unsigned threads = 0;
        const bool elem = !a.al_dy || !a.al_h || (a.dh && !a.al_dh) || (a.dx && !a.al_dx) || (a.dr && !a.al_dr);
        const void *k = pick<DT>(nvec, elem, threads);
        return launch_first(k, dim3((unsigned)G), dim3(threads), args, 0, stream);
    }
    void *args[] = {(void *)&a, (void *)&sums};
    cudaError_t e = launch_first((const void *)layer_back_sums_kernel<DT>, dim3((unsigned)a.rows), dim3(kRowLongT),
                                 args, 0, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((nvec + 255) / 256), (unsigned)G);
    return launch_first((const void *)layer_back_long_kernel<DT>, grid, dim3(256), args, 0, stream);
}

}  // namespace

cudaError_t launch_layer_back(int dtype, LayerBackArgs a, float *scratch, float *dw, float *db, cudaStream_t stream)
{
    int G = norm_back_groups(a.rows, a.cols);
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
