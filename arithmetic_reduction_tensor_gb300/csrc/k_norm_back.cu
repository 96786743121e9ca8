// k_norm_back.cu -- the gradient of the RMS norm.
//
//   xh = h * rstd,  g = dy * w,  c = (row sum of g * xh) / cols
//   dx = rstd * (g - xh * c) + dh
//   dw_j = sum over rows of dy * xh
//
// Per row the sum has the declared order of rowvec.cuh.  dw: CTA b of G adds
// its rows b, b + G, .. in order, each thread holding its columns' sums in
// registers, and a second kernel adds the G partials: 32 threads a column,
// thread k the partials k, k + 32, .. in order, then the halving fold over
// the 32.  G depends on rows and cols only, so the bits of dw do too; there
// are no atomics.  One pass over dy, h and dh; bound by memory traffic.
#include "kernels.cuh"
#include "rowvec.cuh"

namespace tcr {

template <int DT>
struct BackRow {
    RawVec<DT> dy, h, dh;
};

template <int DT>
__device__ __forceinline__ void load_row(const BackArgs &a, size_t r, uint32_t v, BackRow<DT> &b)
{
    using E = typename Elem<DT>::T;
    const uint32_t cols = (uint32_t)a.cols;
    b.dy = load_raw<DT>((const E *)a.dy + r * a.lddy, cols, v, a.al_dy);
    b.h = load_raw<DT>((const E *)a.h + r * a.ldh, cols, v, a.al_h);
    if (a.dh) b.dh = load_raw<DT>((const E *)a.dh + r * a.lddh, cols, v, a.al_dh);
}

template <int DT>
__device__ __forceinline__ RawVec<DT> load_weight(const BackArgs &a, uint32_t v)
{
    return load_raw<DT>((const typename Elem<DT>::T *)a.w, (uint32_t)a.cols, v, a.al_w);
}

// xh and g of a vector; returns the tree over g * xh and, where `acc` is
// given, adds dy * xh to it.
template <int DT>
__device__ __forceinline__ float back_products(const BackArgs &a, const BackRow<DT> &b, const RawVec<DT> &wr,
                                               float rstd, float (&xh)[kRv], float (&g)[kRv], float *acc)
{
    float w[kRv], e[kRv];
    unpack<DT>(b.h, xh);
    unpack<DT>(b.dy, g);
    if (a.w) unpack<DT>(wr, w);
#pragma unroll
    for (int k = 0; k < kRv; k++) {
        xh[k] = __fmul_rn(xh[k], rstd);
        if (acc) acc[k] = __fadd_rn(acc[k], __fmul_rn(g[k], xh[k]));
        if (a.w) g[k] = __fmul_rn(g[k], w[k]);
        e[k] = __fmul_rn(g[k], xh[k]);
    }
    return tree8(e);
}

template <int DT>
__device__ __forceinline__ void store_dx(const BackArgs &a, size_t r, uint32_t v, const BackRow<DT> &b, float rstd,
                                         float c, const float (&xh)[kRv], const float (&g)[kRv])
{
    float dx[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) dx[k] = __fmul_rn(rstd, __fsub_rn(g[k], __fmul_rn(xh[k], c)));
    if (a.dh) {
        float d[kRv];
        unpack<DT>(b.dh, d);
#pragma unroll
        for (int k = 0; k < kRv; k++) dx[k] = __fadd_rn(dx[k], d[k]);
    }
    store_vec<DT>((typename Elem<DT>::T *)a.dx + r * a.lddx, (uint32_t)a.cols, v, a.al_dx, dx);
}

// partial[b * cols + j]: CTA b's sum of column j
__device__ __forceinline__ void store_partial(const BackArgs &a, uint32_t v, const float (&acc)[kRv])
{
    float *p = a.partial + (size_t)blockIdx.x * a.cols + kRv * v;
    const uint32_t left = vec_left((uint32_t)a.cols, v);
    if (left == kRv && (a.cols & 3) == 0) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < kRv; k++)
        if (k < left) p[k] = acc[k];
}

// Rows of at most 8 T vectors, one a thread; a CTA of 32 ceil(vectors / 32)
// <= T threads.  The next row's inputs are loaded before the current row's
// sum is waited for, so that loads stay in flight across the barrier (16384
// rows of 4096 bfloat16: 165 us without, one vector a thread either way).
template <int DT, int T>
__global__ void __launch_bounds__(T, DT == kF32 ? 1 : 1024 / T)
back_kernel(const BackArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][team_floats<T>()];
    const uint32_t v = threadIdx.x;
    // lanes past the row take part in the row's sum with zeros
    const RawVec<DT> w = a.w ? load_weight<DT>(a, v) : RawVec<DT>();
    float acc[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) acc[k] = 0.0f;
    BackRow<DT> cur;
    load_row<DT>(a, blockIdx.x, v, cur);
    float rstd = a.rstd[blockIdx.x];
    int buf = 0;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x, buf ^= 1) {
        float xh[kRv], g[kRv];
        const float s = back_products<DT>(a, cur, w, rstd, xh, g, acc);
        const size_t next = r + gridDim.x;
        BackRow<DT> ahead = {};
        float rstd_ahead = 0.0f;
        if (next < a.rows) {
            load_row<DT>(a, next, v, ahead);
            rstd_ahead = a.rstd[next];
        }
        // two buffers: a thread reaches the next row's write of this one only
        // after every thread has passed the barrier of the row between
        const float c = __fdiv_rn(team_sum<T>(s, red[buf], blockDim.x), (float)a.cols);
        store_dx<DT>(a, r, v, cur, rstd, c, xh, g);
        cur = ahead;
        rstd = rstd_ahead;
    }
    store_partial(a, v, acc);
}

// Longer rows: the row sums first (c[r]), then blocks of 8 * 256 columns.
template <int DT>
__global__ void __launch_bounds__(kRowLongT)
back_long_sum_kernel(const BackArgs a, float *c_out)
{
    constexpr uint32_t T = kRowLongT;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[team_floats<T>()];
    const size_t r = blockIdx.x;
    const uint32_t nvec = (uint32_t)((a.cols + kRv - 1) / kRv);
    const uint32_t steps = (nvec + T - 1) / T;
    const int bits = ceil_log2_sz(steps);
    const float rstd = a.rstd[r];
    BackArgs b = a;
    b.dh = nullptr;
    TreeCounter<16> tc;
    for (uint32_t j = 0; j < (1u << bits); j++) {
        const uint32_t v = threadIdx.x + bit_reverse(j, bits) * T;
        float s = 0.0f;
        if (v < nvec) {
            BackRow<DT> row;
            float xh[kRv], g[kRv];
            load_row<DT>(b, r, v, row);
            const RawVec<DT> w = a.w ? load_weight<DT>(a, v) : RawVec<DT>();
            s = back_products<DT>(a, row, w, rstd, xh, g, nullptr);
        }
        tc.push(s);
    }
    const float c = __fdiv_rn(team_sum<T>(tc.finish(), red), (float)a.cols);
    if (threadIdx.x == 0) c_out[r] = c;
}

template <int DT>
__global__ void __launch_bounds__(256)
back_long_kernel(const BackArgs a, const float *c_in)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    const uint32_t v = blockIdx.y * 256 + threadIdx.x;
    const RawVec<DT> w = a.w ? load_weight<DT>(a, v) : RawVec<DT>();
    float acc[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) acc[k] = 0.0f;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float rstd = a.rstd[r];
        BackRow<DT> row;
        float xh[kRv], g[kRv];
        load_row<DT>(a, r, v, row);
        (void)back_products<DT>(a, row, w, rstd, xh, g, acc);
        store_dx<DT>(a, r, v, row, rstd, c_in[r], xh, g);
    }
    store_partial(a, v, acc);
}

// dw[j] from the G partials of column j.
__global__ void __launch_bounds__(1024) dweight_kernel(const float *partial, size_t cols, int G, float *dw)
{
    pdl_launch_dependents();
    pdl_wait_primary();
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
    if (threadIdx.x == 0 && jo < cols) dw[jo] = v;
}

// ---------------------------------------------------------------- host

namespace {

uint32_t team_of(size_t cols)
{
    const size_t nvec = (cols + kRv - 1) / kRv;
    return nvec > kBackMaxVecs ? 1024u : (uint32_t)((nvec + 31) / 32 * 32);
}

}  // namespace

// Enough CTAs for 1024 threads on each of 152 SMs, but (above one an SM) no
// more than a quarter of the rows: a partial costs as much traffic as a row.
int norm_back_groups(size_t rows, size_t cols)
{
    const size_t full = (size_t)152 * (1024 / team_of(cols));
    const size_t quarter = (rows + 3) / 4 > 152 ? (rows + 3) / 4 : 152;
    size_t g = full < quarter ? full : quarter;
    return (int)(rows < g ? rows : g);
}

size_t norm_back_scratch(size_t rows, size_t cols)
{
    const size_t nvec = (cols + kRv - 1) / kRv;
    return ((size_t)norm_back_groups(rows, cols) * cols + (nvec > kBackMaxVecs ? rows : 0)) * sizeof(float);
}

namespace {

template <int DT>
cudaError_t launch_back(BackArgs a, int G, cudaStream_t stream)
{
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    if (nvec <= kBackMaxVecs) {
        void *args[] = {(void *)&a};
        const void *k = nvec <= 64    ? (const void *)back_kernel<DT, 64>
                        : nvec <= 128 ? (const void *)back_kernel<DT, 128>
                        : nvec <= 256 ? (const void *)back_kernel<DT, 256>
                        : nvec <= 512 ? (const void *)back_kernel<DT, 512>
                                      : (const void *)back_kernel<DT, 1024>;
        return launch_first(k, dim3((unsigned)G), dim3(team_of(a.cols)), args, 0, stream);
    }
    float *c = a.partial + (size_t)G * a.cols;
    void *args[] = {(void *)&a, (void *)&c};
    cudaError_t e = launch_first((const void *)back_long_sum_kernel<DT>, dim3((unsigned)a.rows), dim3(kRowLongT),
                                 args, 0, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)G, (unsigned)((nvec + 255) / 256));
    return launch_first((const void *)back_long_kernel<DT>, grid, dim3(256), args, 0, stream);
}

}  // namespace

cudaError_t launch_norm_back(int dtype, const BackArgs &a, float *dw, cudaStream_t stream)
{
    int G = norm_back_groups(a.rows, a.cols);
    cudaError_t e = dtype == kF16    ? launch_back<kF16>(a, G, stream)
                    : dtype == kBF16 ? launch_back<kBF16>(a, G, stream)
                                     : launch_back<kF32>(a, G, stream);
    if (e != cudaSuccess || !dw) return e;
    const float *partial = a.partial;
    size_t cols = a.cols;
    void *args[] = {(void *)&partial, (void *)&cols, (void *)&G, (void *)&dw};
    return launch_first((const void *)dweight_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(32, 32), args, 0,
                        stream);
}

}  // namespace tcr
