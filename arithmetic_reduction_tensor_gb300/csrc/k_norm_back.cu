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
// are no atomics.  Rows of up to 8192 columns: one pass over dy, h and dh, bound
// by memory traffic (65536 x 4096 binary16 351 us, 6.1 TB/s), the barrier of
// each row and, for few rows, by the latency of two launches.  Longer rows: a
// pass over dy and h for the row sums, then one over all three (4096 x 12288
// bfloat16 174 us, 59 at the copy rate).
#include "kernels.cuh"
#include "rowvec.cuh"

namespace tcr {

template <int DT, bool GRAN>
struct BackRow {
    LoadedVec<DT, GRAN> dy, h, dh;
};

template <int DT, bool GRAN>
__device__ __forceinline__ void load_row(const BackArgs &a, size_t r, uint32_t v, BackRow<DT, GRAN> &b)
{
    using E = typename Elem<DT>::T;
    const uint32_t cols = (uint32_t)a.cols;
    b.dy = load_vec<DT, GRAN>((const E *)a.dy + r * a.lddy, cols, v);
    b.h = load_vec<DT, GRAN>((const E *)a.h + r * a.ldh, cols, v);
    if (a.dh) b.dh = load_vec<DT, GRAN>((const E *)a.dh + r * a.lddh, cols, v);
}

template <int DT>
__device__ __forceinline__ RawVec<DT> load_weight(const BackArgs &a, uint32_t v)
{
    return load_raw<DT>((const typename Elem<DT>::T *)a.w, (uint32_t)a.cols, v, a.al_w);
}

// The tree over g * xh of a vector's `left` elements: for an infinite rstd,
// which makes the absent ones, 0 * rstd, NaN.
__device__ __forceinline__ float sum_present(const float (&xh)[kRv], const float (&g)[kRv], uint32_t left)
{
    float e[kRv];
#pragma unroll
    for (uint32_t k = 0; k < kRv; k++) e[k] = k < left ? __fmul_rn(g[k], xh[k]) : 0.0f;
    return tree8(e);
}

// xh and g of a vector; returns the tree over g * xh (MASK = false: the
// caller sees to an infinite rstd) and, where `acc` is given, adds dy * xh to
// it.
template <int DT, bool GRAN, bool MASK>
__device__ __forceinline__ float back_products(const BackArgs &a, size_t r, uint32_t v, const BackRow<DT, GRAN> &b,
                                               const RawVec<DT> &wr, float rstd, float (&xh)[kRv], float (&g)[kRv],
                                               float *acc)
{
    using E = typename Elem<DT>::T;
    const uint32_t cols = (uint32_t)a.cols;
    float w[kRv], e[kRv];
    unpack<DT>(use_vec<DT, GRAN>(b.h, (const E *)a.h + r * a.ldh, cols, v), xh);
    unpack<DT>(use_vec<DT, GRAN>(b.dy, (const E *)a.dy + r * a.lddy, cols, v), g);
    if (a.w) unpack<DT>(wr, w);
#pragma unroll
    for (int k = 0; k < kRv; k++) {
        xh[k] = __fmul_rn(xh[k], rstd);
        if (acc) acc[k] = __fadd_rn(acc[k], __fmul_rn(g[k], xh[k]));
        if (a.w) g[k] = __fmul_rn(g[k], w[k]);
        e[k] = __fmul_rn(g[k], xh[k]);
    }
    if (MASK && isinf(rstd)) return sum_present(xh, g, vec_left(cols, v));
    return tree8(e);
}

template <int DT, bool GRAN>
__device__ __forceinline__ void store_dx(const BackArgs &a, size_t r, uint32_t v, const LoadedVec<DT, GRAN> &dh,
                                         float rstd, float c, const float (&xh)[kRv], const float (&g)[kRv])
{
    using E = typename Elem<DT>::T;
    const uint32_t cols = (uint32_t)a.cols;
    float dx[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) dx[k] = __fmul_rn(rstd, __fsub_rn(g[k], __fmul_rn(xh[k], c)));
    if (a.dh) {
        float d[kRv];
        unpack<DT>(use_vec<DT, GRAN>(dh, (const E *)a.dh + r * a.lddh, cols, v), d);
#pragma unroll
        for (int k = 0; k < kRv; k++) dx[k] = __fadd_rn(dx[k], d[k]);
    }
    store_vec<DT>((E *)a.dx + r * a.lddx, cols, v, a.al_dx, dx);
}

// partial[b * cols + j]: the sum of column j over the rows b, b + G, ..; not
// stored where the weight's gradient is not wanted.
__device__ __forceinline__ void store_partial(const BackArgs &a, unsigned b, uint32_t v, const float (&acc)[kRv])
{
    if (!a.partial) return;
    float *p = a.partial + (size_t)b * a.cols + kRv * v;
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

// Rows of at most T NV vectors, NV a thread; NV = 1: a CTA of 32 ceil(vectors
// / 32) <= T threads.  The next row's inputs are loaded before the current
// row's sum is waited for, so that loads stay in flight across the barrier.
// Rows are 16-byte aligned.
template <int DT, int T, int NV, int MINB>
__global__ void __launch_bounds__(T, MINB)
back_kernel(const BackArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][team_floats<T>()];
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    // where an infinite rstd is seen to: of two vectors at once behind the next
    // row's loads (16384 x 4096 bfloat16 91.1 us, in the products 92.2, not at
    // all 90.8), else in the products (x 2560 87.6 us, behind the loads 90.1)
    constexpr bool kLate = NV == 2 && DT != kF32;
    // lanes past the row take part in the row's sum with zeros
    RawVec<DT> w[NV];
    float acc[NV][kRv];
    BackRow<DT, false> cur[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        w[i] = a.w ? load_weight<DT>(a, t + i * T) : RawVec<DT>();
        load_row<DT, false>(a, blockIdx.x, t + i * T, cur[i]);
#pragma unroll
        for (int k = 0; k < kRv; k++) acc[i][k] = 0.0f;
    }
    float rstd = a.rstd[blockIdx.x];
    int buf = 0;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x, buf ^= 1) {
        float s[NV];
        LoadedVec<DT, false> dh[NV];
        float xh[NV][kRv], g[NV][kRv];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            s[i] = back_products<DT, false, !kLate>(a, r, t + i * T, cur[i], w[i], rstd, xh[i], g[i], acc[i]);
            dh[i] = cur[i].dh;
        }
        const size_t next = r + gridDim.x;
        const float rstd_now = rstd;
        if (next < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; i++) load_row<DT, false>(a, next, t + i * T, cur[i]);
            rstd = a.rstd[next];
        }
        if (kLate && isinf(rstd_now)) {
#pragma unroll
            for (int i = 0; i < NV; i++) s[i] = sum_present(xh[i], g[i], vec_left(cols, t + i * T));
        }
        // two buffers: a thread reaches the next row's write of this one only
        // after every thread has passed the barrier of the row between
        const float c = __fdiv_rn(team_sum<T>(halving<NV>(s), red[buf], blockDim.x), (float)a.cols);
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (kRv * ((t & ~31u) + i * T) < cols)           // whole warps: stores are warp-wide
                store_dx<DT, false>(a, r, t + i * T, dh[i], rstd_now, c, xh[i], g[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; i++) store_partial(a, blockIdx.x, t + i * T, acc[i]);
}

// The same for rows at any alignment, one vector's worth a thread, in the
// layout of tree8_lanes: lane l of warp w holds elements 256 w + 32 j + l.
// 16384 x 4090 binary16 145 us, 20000 x 2001 binary32 105, 6000 x 8003
// binary32 138; with granules shifted in registers 189, 122 and 295.
template <int DT, int T, int MINB>
__global__ void __launch_bounds__(T, MINB)
back_elem_kernel(const BackArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][team_floats<T>()];
    using E = typename Elem<DT>::T;
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    const uint32_t e0 = 8 * (t & ~31u) + (t & 31);
    const bool whole = 8 * (t & ~31u) + 256 <= cols;         // the warp's 256 elements all exist
    auto load8 = [&](const void *base, size_t at, E (&v)[kRv]) {
        const E *row = (const E *)base + at;
        if (whole) {
#pragma unroll
            for (int j = 0; j < kRv; j++) v[j] = row[e0 + 32 * j];
        } else {
#pragma unroll
            for (int j = 0; j < kRv; j++) v[j] = e0 + 32 * j < cols ? row[e0 + 32 * j] : (E)0;
        }
    };
    E dy[kRv], h[kRv], dh[kRv], w[kRv];
    float acc[kRv];
    auto load = [&](size_t r) {
        load8(a.dy, r * a.lddy, dy);
        load8(a.h, r * a.ldh, h);
        if (a.dh) load8(a.dh, r * a.lddh, dh);
    };
#pragma unroll
    for (int j = 0; j < kRv; j++) {
        w[j] = dh[j] = (E)0;
        acc[j] = 0.0f;
    }
    if (a.w) load8(a.w, 0, w);
    load(blockIdx.x);
    float rstd = a.rstd[blockIdx.x];
    int buf = 0;
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x, buf ^= 1) {
        float xh[kRv], g[kRv], d[kRv], e[kRv];
#pragma unroll
        for (int j = 0; j < kRv; j++) {
            xh[j] = __fmul_rn(elem_to_float<DT>(h[j]), rstd);
            g[j] = elem_to_float<DT>(dy[j]);
            d[j] = elem_to_float<DT>(dh[j]);
            acc[j] = __fadd_rn(acc[j], __fmul_rn(g[j], xh[j]));
            if (a.w) g[j] = __fmul_rn(g[j], elem_to_float<DT>(w[j]));
            e[j] = __fmul_rn(g[j], xh[j]);
        }
        if (isinf(rstd)) {                                   // (absent elements, as in sum_present)
#pragma unroll
            for (int j = 0; j < kRv; j++)
                if (e0 + 32 * j >= cols) e[j] = 0.0f;
        }
        const float s = tree8_lanes(e);
        const size_t next = r + gridDim.x;
        const float rstd_now = rstd;
        if (next < a.rows) {
            load(next);
            rstd = a.rstd[next];
        }
        // (two buffers, as in back_kernel)
        const float c = __fdiv_rn(team_sum<T, true>(s, red[buf], blockDim.x), (float)a.cols);
        E *dx = (E *)a.dx + r * a.lddx;
#pragma unroll
        for (int j = 0; j < kRv; j++) {
            float v = __fmul_rn(rstd_now, __fsub_rn(g[j], __fmul_rn(xh[j], c)));
            if (a.dh) v = __fadd_rn(v, d[j]);
            if (whole || e0 + 32 * j < cols) dx[e0 + 32 * j] = float_to_elem<DT>(v);
        }
    }
    if (!a.partial) return;
    float *p = a.partial + (size_t)blockIdx.x * a.cols;
#pragma unroll
    for (int j = 0; j < kRv; j++)
        if (e0 + 32 * j < cols) p[e0 + 32 * j] = acc[j];
}

// Longer rows: the row sums first (c[r]), then blocks of 8 * 256 columns, which
// are the grid's x: 2^27 columns are 65536 of them, one more than its y holds.
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
            BackRow<DT, true> row;
            float xh[kRv], g[kRv];
            load_row<DT, true>(b, r, v, row);
            const RawVec<DT> w = a.w ? load_weight<DT>(a, v) : RawVec<DT>();
            s = back_products<DT, true, true>(a, r, v, row, w, rstd, xh, g, nullptr);
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
    const uint32_t v = blockIdx.x * 256 + threadIdx.x;
    const RawVec<DT> w = a.w ? load_weight<DT>(a, v) : RawVec<DT>();
    float acc[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) acc[k] = 0.0f;
    for (size_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float rstd = a.rstd[r];
        BackRow<DT, true> row;
        float xh[kRv], g[kRv];
        load_row<DT, true>(a, r, v, row);
        (void)back_products<DT, true, true>(a, r, v, row, w, rstd, xh, g, acc);
        store_dx<DT, true>(a, r, v, row.dh, rstd, c_in[r], xh, g);
    }
    store_partial(a, blockIdx.y, v, acc);
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

// Floats of the partials; 0 where no weight gradient is wanted.
static size_t partial_floats(size_t rows, size_t cols, bool dweight)
{
    return dweight ? (size_t)norm_back_groups(rows, cols) * cols : 0;
}

size_t norm_back_scratch(size_t rows, size_t cols, bool dweight)
{
    const size_t nvec = (cols + kRv - 1) / kRv;
    return (partial_floats(rows, cols, dweight) + (nvec > kBackMaxVecs ? rows : 0)) * sizeof(float);
}

namespace {

// The fastest shapes measured: the registers of two rows decide how many
// threads fit, so binary32 takes half as many of an SM's threads as the 16-bit
// types, and 16-bit rows of more than 2048 columns go two vectors to a thread
// (16384 x 4096 bfloat16 91 us, 108 with one).  At 257 to 320 vectors
// norm_back_groups gives an SM three CTAs, which 64 registers hold at once and
// 128 do not: 16384 x 2560 bfloat16 88 us and 94, by elements 16384 x 2051
// bfloat16 108 and 132, binary32 117 and 136; aligned binary32 loses more by
// spills (16384 x 2560 150 and 128).  Few rows leave two CTAs an SM: 1000 x
// 2560 bfloat16 14.5 us with 64 registers, 10.5 with 128.
template <int DT>
const void *pick(size_t nvec, int G, bool elem, unsigned &threads)
{
    const bool three = nvec > 256 && nvec <= 320 && G > 2 * 152;
#define TCR_BACK(T_, NV_, MINB_) \
    return (threads = NV_ == 1 ? (unsigned)((nvec + 31) / 32 * 32) : T_, \
            (const void *)back_kernel<DT, T_, NV_, MINB_>)
#define TCR_ELEM(T_, MINB_) \
    return (threads = (unsigned)((nvec + 31) / 32 * 32), (const void *)back_elem_kernel<DT, T_, MINB_>)
    if (elem) {
        if (nvec <= 64) TCR_ELEM(64, 8);
        if (nvec <= 128) TCR_ELEM(128, 4);
        if (nvec <= 256) TCR_ELEM(256, 2);
        if (three) TCR_ELEM(512, 2);
        if (nvec <= 512) TCR_ELEM(512, 1);
        if (nvec <= 768) TCR_ELEM(768, 1);
        TCR_ELEM(1024, 1);
    }
    if constexpr (DT == kF32) {
        if (nvec <= 64) TCR_BACK(64, 1, 8);
        if (nvec <= 128) TCR_BACK(128, 1, 4);
        if (nvec <= 256) TCR_BACK(256, 1, 2);
        if (nvec <= 512) TCR_BACK(512, 1, 1);
    } else {
        if (nvec <= 64) TCR_BACK(64, 1, 16);
        if (nvec <= 128) TCR_BACK(128, 1, 8);
        if (nvec <= 256) TCR_BACK(256, 1, 4);
        if (three) TCR_BACK(512, 1, 2);
        if (nvec <= 512) TCR_BACK(256, 2, 2);
    }
    TCR_BACK(512, 2, 1);
#undef TCR_ELEM
#undef TCR_BACK
}

template <int DT>
cudaError_t launch_back(BackArgs a, int G, float *c, cudaStream_t stream)
{
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    if (nvec <= kBackMaxVecs) {
        void *args[] = {(void *)&a};
        unsigned threads = 0;
        const bool elem = !a.al_dy || !a.al_h || (a.dh && !a.al_dh) || !a.al_dx;
        const void *k = pick<DT>(nvec, G, elem, threads);
        return launch_first(k, dim3((unsigned)G), dim3(threads), args, 0, stream);
    }
    void *args[] = {(void *)&a, (void *)&c};
    cudaError_t e = launch_first((const void *)back_long_sum_kernel<DT>, dim3((unsigned)a.rows), dim3(kRowLongT),
                                 args, 0, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((nvec + 255) / 256), (unsigned)G);
    return launch_first((const void *)back_long_kernel<DT>, grid, dim3(256), args, 0, stream);
}

}  // namespace

cudaError_t launch_norm_back(int dtype, BackArgs a, float *scratch, float *dw, cudaStream_t stream)
{
    int G = norm_back_groups(a.rows, a.cols);
    a.partial = dw ? scratch : nullptr;
    float *c = scratch + partial_floats(a.rows, a.cols, dw != nullptr);
    cudaError_t e = dtype == kF16    ? launch_back<kF16>(a, G, c, stream)
                    : dtype == kBF16 ? launch_back<kBF16>(a, G, c, stream)
                                     : launch_back<kF32>(a, G, c, stream);
    if (e != cudaSuccess || !dw) return e;
    const float *partial = a.partial;
    size_t cols = a.cols;
    void *args[] = {(void *)&partial, (void *)&cols, (void *)&G, (void *)&dw};
    return launch_first((const void *)dweight_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(32, 32), args, 0,
                        stream);
}

}  // namespace tcr
