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
__device__ __forceinline__ void back_products(const float (&dy)[kRv], const float (&h)[kRv],
                                              const float (&w)[kRv], float rstd, float (&xh)[kRv],
                                              float (&g)[kRv])
{
#pragma unroll
    for (int k = 0; k < kRv; k++) {
        xh[k] = __fmul_rn(h[k], rstd);
        g[k] = __fmul_rn(dy[k], w[k]);
    }
}

template <int DT>
__device__ __forceinline__ void load_weight(const BackArgs &a, size_t v, float (&w)[kRv])
{
    if (a.w) {
        unpack<DT>(load_raw<DT>((const typename Elem<DT>::T *)a.w, a.cols, v, a.al_w), w);
    } else {
#pragma unroll
        for (int k = 0; k < kRv; k++) w[k] = 1.0f;
    }
}

template <int DT>
__device__ __forceinline__ void store_dx(const BackArgs &a, size_t r, size_t v, float rstd, float c,
                                         const float (&xh)[kRv], const float (&g)[kRv])
{
    using E = typename Elem<DT>::T;
    float dx[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) dx[k] = __fmul_rn(rstd, __fsub_rn(g[k], __fmul_rn(xh[k], c)));
    if (a.dh) {
        float d[kRv];
        unpack<DT>(load_raw<DT>((const E *)a.dh + r * a.lddh, a.cols, v, a.al_dh), d);
#pragma unroll
        for (int k = 0; k < kRv; k++) dx[k] = __fadd_rn(dx[k], d[k]);
    }
    store_vec<DT>((E *)a.dx + r * a.lddx, a.cols, v, a.al_dx, dx);
}

// partial[b * cols + j]: CTA b's sum of column j
__device__ __forceinline__ void store_partial(const BackArgs &a, size_t v, const float (&acc)[kRv])
{
    float *p = a.partial + (size_t)blockIdx.x * a.cols + kRv * v;
#pragma unroll
    for (int k = 0; k < kRv; k++)
        if (kRv * v + k < a.cols) p[k] = acc[k];
}

// Rows of at most 8 T NV columns.
template <int DT, int T, int NV>
__global__ void __launch_bounds__(T)
back_kernel(const BackArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][T];
    using E = typename Elem<DT>::T;
    const int t = threadIdx.x;
    float acc[NV][kRv];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int k = 0; k < kRv; k++) acc[i][k] = 0.0f;
    int buf = 0;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x, buf ^= 1) {
        const float rstd = a.rstd[r];
        float xh[NV][kRv], g[NV][kRv], s[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const size_t v = (size_t)t + (size_t)i * T;
            s[i] = 0.0f;
            if (kRv * v >= a.cols) continue;
            float dy[kRv], h[kRv], w[kRv], e[kRv];
            unpack<DT>(load_raw<DT>((const E *)a.dy + r * a.lddy, a.cols, v, a.al_dy), dy);
            unpack<DT>(load_raw<DT>((const E *)a.h + r * a.ldh, a.cols, v, a.al_h), h);
            load_weight<DT>(a, v, w);
            back_products<DT>(dy, h, w, rstd, xh[i], g[i]);
#pragma unroll
            for (int k = 0; k < kRv; k++) {
                e[k] = __fmul_rn(g[i][k], xh[i][k]);
                acc[i][k] = __fadd_rn(acc[i][k], __fmul_rn(dy[k], xh[i][k]));
            }
            s[i] = tree8(e);
        }
        // two buffers: a thread reaches the next row's write of this one only
        // after every thread has passed the barrier of the row between
        const float c = __fdiv_rn(team_sum<T>(halving<NV>(s), red[buf]), (float)a.cols);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const size_t v = (size_t)t + (size_t)i * T;
            if (kRv * v < a.cols) store_dx<DT>(a, r, v, rstd, c, xh[i], g[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const size_t v = (size_t)t + (size_t)i * T;
        if (kRv * v < a.cols) store_partial(a, v, acc[i]);
    }
}

// Longer rows: the row sums first (c[r]), then blocks of 8 T columns.
template <int DT>
__global__ void __launch_bounds__(kRowLongT)
back_long_sum_kernel(const BackArgs a, float *c_out)
{
    constexpr int T = kRowLongT;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[T];
    using E = typename Elem<DT>::T;
    const size_t r = blockIdx.x;
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    const uint32_t steps = (uint32_t)((nvec + T - 1) / T);
    const int bits = ceil_log2_sz(steps);
    const float rstd = a.rstd[r];
    TreeCounter<32> tc;
    for (uint32_t j = 0; j < (1u << bits); j++) {
        const size_t v = (size_t)threadIdx.x + (size_t)bit_reverse(j, bits) * T;
        float s = 0.0f;
        if (v < nvec) {
            float dy[kRv], h[kRv], w[kRv], xh[kRv], g[kRv], e[kRv];
            unpack<DT>(load_raw<DT>((const E *)a.dy + r * a.lddy, a.cols, v, a.al_dy), dy);
            unpack<DT>(load_raw<DT>((const E *)a.h + r * a.ldh, a.cols, v, a.al_h), h);
            load_weight<DT>(a, v, w);
            back_products<DT>(dy, h, w, rstd, xh, g);
#pragma unroll
            for (int k = 0; k < kRv; k++) e[k] = __fmul_rn(g[k], xh[k]);
            s = tree8(e);
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
    using E = typename Elem<DT>::T;
    const size_t v = (size_t)blockIdx.y * 256 + threadIdx.x;
    if (kRv * v >= a.cols) return;
    float acc[kRv], w[kRv];
    load_weight<DT>(a, v, w);
#pragma unroll
    for (int k = 0; k < kRv; k++) acc[k] = 0.0f;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float rstd = a.rstd[r];
        float dy[kRv], h[kRv], xh[kRv], g[kRv];
        unpack<DT>(load_raw<DT>((const E *)a.dy + r * a.lddy, a.cols, v, a.al_dy), dy);
        unpack<DT>(load_raw<DT>((const E *)a.h + r * a.ldh, a.cols, v, a.al_h), h);
        back_products<DT>(dy, h, w, rstd, xh, g);
#pragma unroll
        for (int k = 0; k < kRv; k++) acc[k] = __fadd_rn(acc[k], __fmul_rn(dy[k], xh[k]));
        store_dx<DT>(a, r, v, rstd, c_in[r], xh, g);
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
    if (j < cols)
        for (int g = threadIdx.y; g < G; g += 32) acc = __fadd_rn(acc, partial[(size_t)g * cols + j]);
    s[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    // warp y folds column y of the 32
    const float v = halving_lanes(s[threadIdx.x][threadIdx.y]);
    const size_t jo = (size_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && jo < cols) dw[jo] = v;
}

// ---------------------------------------------------------------- host

int norm_back_groups(size_t rows, size_t cols)
{
    // about two CTAs on each of 152 SMs; fewer, larger CTAs for long rows
    const size_t g = cols > 4096 ? 152 : 304;
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
    void *args[] = {(void *)&a};
    const dim3 grid((unsigned)G);
#define TCR_BACK(T_, NV_) launch_first((const void *)back_kernel<DT, T_, NV_>, grid, dim3(T_), args, 0, stream)
    if (nvec <= 64) return TCR_BACK(64, 1);
    if (nvec <= 128) return TCR_BACK(128, 1);
    if (nvec <= 256) return TCR_BACK(256, 1);
    if (nvec <= 512) return TCR_BACK(256, 2);
    if (nvec <= 1024) return TCR_BACK(512, 2);
    if (nvec <= kBackMaxVecs) return TCR_BACK(1024, 2);
#undef TCR_BACK
    float *c = a.partial + (size_t)G * a.cols;
    void *args1[] = {(void *)&a, (void *)&c};
    cudaError_t e = launch_first((const void *)back_long_sum_kernel<DT>, dim3((unsigned)a.rows), dim3(kRowLongT),
                                 args1, 0, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid2((unsigned)G, (unsigned)((nvec + 255) / 256));
    return launch_first((const void *)back_long_kernel<DT>, grid2, dim3(256), args1, 0, stream);
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
