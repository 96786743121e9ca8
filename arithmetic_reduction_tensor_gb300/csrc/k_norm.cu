// k_norm.cu -- RMS norm with the residual's addition, and rows into 8-bit
// integers with one scale a row: one pass over the data per row.
//
//   norm      h = x + r (binary32),  y = (h * rstd) * w,
//             rstd = 1 / sqrt(S / cols + eps), S the row sum of fl32(h * h)
//   quantise  y = x, or (g / (1 + exp(-g))) * x with a gate g
//   codes     scale = max|y| / 127, q = rint(y * (127 / max|y|))
//
// A team of T threads (a warp for short rows, else a CTA) keeps the row in
// registers, NV vectors a thread, so every byte is read once; S is summed
// in the declared order of rowvec.cuh.  Every step outside expf is one
// binary32 operation rounded to nearest, so the norm's results are pinned
// bit for bit by the inputs.  The work is bound by memory traffic.
#include "kernels.cuh"
#include "rowvec.cuh"

namespace tcr {

constexpr int kOutSame = 0, kOutI8 = 1;

template <int DT, int OP>
__device__ __forceinline__ void row_value(const RowArgs &a, size_t r, size_t v, bool al, float (&y)[kRv])
{
    using E = typename Elem<DT>::T;
    unpack<DT>(load_raw<DT>((const E *)a.x + r * a.ldx, a.cols, v, al), y);
    if constexpr (OP == kRowNorm) {
        if (a.r) {
            float b[kRv];
            unpack<DT>(load_raw<DT>((const E *)a.r + r * a.ldr, a.cols, v, al), b);
#pragma unroll
            for (int k = 0; k < kRv; k++) y[k] = __fadd_rn(y[k], b[k]);
        }
    } else if (a.r) {
        float g[kRv];
        unpack<DT>(load_raw<DT>((const E *)a.r + r * a.ldr, a.cols, v, al), g);
#pragma unroll
        for (int k = 0; k < kRv; k++)
            y[k] = __fmul_rn(__fdiv_rn(g[k], __fadd_rn(1.0f, expf(-g[k]))), y[k]);
    }
}

__device__ __forceinline__ float squares8(const float (&h)[kRv])
{
    float e[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) e[k] = __fmul_rn(h[k], h[k]);
    return tree8(e);
}

__device__ __forceinline__ float rstd_of(float s, size_t cols, float eps)
{
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(s, (float)cols), eps));
}

template <int DT>
__device__ __forceinline__ void apply_norm(const RowArgs &a, size_t v, float rstd, float (&h)[kRv])
{
    float w[kRv];
    if (a.w) unpack<DT>(load_raw<DT>((const typename Elem<DT>::T *)a.w, a.cols, v, a.al_w), w);
#pragma unroll
    for (int k = 0; k < kRv; k++) {
        h[k] = __fmul_rn(h[k], rstd);
        if (a.w) h[k] = __fmul_rn(h[k], w[k]);
    }
}

__device__ __forceinline__ uint32_t amax8(const float (&y)[kRv], uint32_t m)
{
#pragma unroll
    for (int k = 0; k < kRv; k++) m = max(m, __float_as_uint(y[k]) & 0x7fffffffu);
    return m;
}

// Rows of at most 8 T NV columns, one team of T threads each (T = 32: four
// to a CTA).
template <int DT, int OP, int OUT, int T, int NV>
__global__ void __launch_bounds__(T == 32 ? 128 : T)
row_kernel(const RowArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[T == 32 ? 1 : T];
    __shared__ uint32_t redm[32];
    using E = typename Elem<DT>::T;
    const size_t r = T == 32 ? (size_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (r >= a.rows) return;               // T = 32 only: whole warps leave
    const int t = T == 32 ? threadIdx.x & 31 : threadIdx.x;
    float y[NV][kRv];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const size_t v = (size_t)t + (size_t)i * T;
        if (kRv * v < a.cols) {
            row_value<DT, OP>(a, r, v, a.al_in, y[i]);
        } else {
#pragma unroll
            for (int k = 0; k < kRv; k++) y[i][k] = 0.0f;
        }
    }
    float rstd = 0.0f;
    if constexpr (OP == kRowNorm) {
        float s[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) s[i] = squares8(y[i]);
        rstd = rstd_of(team_sum<T>(halving<NV>(s), red), a.cols, a.eps);
        if (a.rstd && t == 0) a.rstd[r] = rstd;
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const size_t v = (size_t)t + (size_t)i * T;
        if (kRv * v >= a.cols) continue;
        if constexpr (OP == kRowNorm) {
            if (a.h) store_vec<DT>((E *)a.h + r * a.ldh, a.cols, v, a.al_h, y[i]);
            apply_norm<DT>(a, v, rstd, y[i]);
        }
        if constexpr (OUT == kOutSame)
            store_vec<DT>((E *)a.y + r * a.ldy, a.cols, v, a.al_y, y[i]);
        else
            m = amax8(y[i], m);
    }
    if constexpr (OUT == kOutI8) {
        float scale, per;
        i8_scale(team_max<T>(m, redm), scale, per);
        if (t == 0) a.scale[r] = scale;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const size_t v = (size_t)t + (size_t)i * T;
            if (kRv * v < a.cols) store_codes((int8_t *)a.y + r * a.ldy, a.cols, v, a.al_y, y[i], per);
        }
    }
}

// Longer rows: a CTA of T threads reads the row once per step (the sum, the
// largest magnitude, the outputs).  h may be written over x or r: it is
// stored in the last step only.
template <int DT, int OP, int OUT>
__global__ void __launch_bounds__(kRowLongT)
row_long_kernel(const RowArgs a)
{
    constexpr int T = kRowLongT;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[T];
    __shared__ uint32_t redm[32];
    using E = typename Elem<DT>::T;
    const size_t r = blockIdx.x;
    const int t = threadIdx.x;
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    const uint32_t steps = (uint32_t)((nvec + T - 1) / T);
    const int bits = ceil_log2_sz(steps);
    float rstd = 0.0f;
    float y[kRv];
    if constexpr (OP == kRowNorm) {
        TreeCounter<32> tc;
        for (uint32_t j = 0; j < (1u << bits); j++) {
            const size_t v = (size_t)t + (size_t)bit_reverse(j, bits) * T;
            float s = 0.0f;
            if (v < nvec) {
                row_value<DT, OP>(a, r, v, a.al_in, y);
                s = squares8(y);
            }
            tc.push(s);
        }
        rstd = rstd_of(team_sum<T>(tc.finish(), red), a.cols, a.eps);
        if (a.rstd && t == 0) a.rstd[r] = rstd;
    }
    float per = 0.0f;
    if constexpr (OUT == kOutI8) {
        uint32_t m = 0u;
        for (size_t v = t; v < nvec; v += T) {
            row_value<DT, OP>(a, r, v, a.al_in, y);
            if constexpr (OP == kRowNorm) apply_norm<DT>(a, v, rstd, y);
            m = amax8(y, m);
        }
        float scale;
        i8_scale(team_max<T>(m, redm), scale, per);
        if (t == 0) a.scale[r] = scale;
    }
    for (size_t v = t; v < nvec; v += T) {
        row_value<DT, OP>(a, r, v, a.al_in, y);
        if constexpr (OP == kRowNorm) {
            if (a.h) store_vec<DT>((E *)a.h + r * a.ldh, a.cols, v, a.al_h, y);
            apply_norm<DT>(a, v, rstd, y);
        }
        if constexpr (OUT == kOutSame)
            store_vec<DT>((E *)a.y + r * a.ldy, a.cols, v, a.al_y, y);
        else
            store_codes((int8_t *)a.y + r * a.ldy, a.cols, v, a.al_y, y, per);
    }
}

// ---------------------------------------------------------------- codes read back

// y = q * scale[row], 16 codes a thread; a team of `team` threads (a power
// of two, at most 256) walks each row.
template <int DT>
__global__ void __launch_bounds__(256)
dequant_kernel(const int8_t *q, size_t ldq, const float *scale, typename Elem<DT>::T *y, size_t ldy,
               size_t rows, size_t cols, int team_log2, bool al_q, bool al_y)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    const size_t r = ((size_t)blockIdx.x << (8 - team_log2)) + (threadIdx.x >> team_log2);
    if (r >= rows) return;
    const float s = scale[r];
    const int8_t *row = q + r * ldq;
    const size_t step = (size_t)16 << team_log2;
    for (size_t c = (size_t)(threadIdx.x & ((1 << team_log2) - 1)) * 16; c < cols; c += step) {
        float f[2][kRv];
        if (al_q && c + 16 <= cols) {
            const uint4 u = ld16(row + c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 16; k++)
                f[k / 8][k % 8] = __fmul_rn((float)(int8_t)(w[k / 4] >> (8 * (k % 4))), s);
        } else {
#pragma unroll
            for (int k = 0; k < 16; k++)
                f[k / 8][k % 8] = c + k < cols ? __fmul_rn((float)row[c + k], s) : 0.0f;
        }
        store_vec<DT>(y + r * ldy, cols, c / kRv, al_y, f[0]);
        if (c + kRv < cols) store_vec<DT>(y + r * ldy, cols, c / kRv + 1, al_y, f[1]);
    }
}

// ---------------------------------------------------------------- host

namespace {

template <int DT, int OP, int OUT>
const void *pick(size_t nvec, size_t rows, int &threads, size_t &grid)
{
    grid = rows;
    // few rows: more threads to a row, fewer values to a thread (the same bits)
    const bool few = rows <= 304;
#define TCR_ROW(T_, NV_) (threads = T_, (const void *)row_kernel<DT, OP, OUT, T_, NV_>)
    if (nvec <= 128 && !(few && nvec > 32)) {
        threads = 128;
        grid = (rows + 3) / 4;
        if (nvec <= 32) return (const void *)row_kernel<DT, OP, OUT, 32, 1>;
        if (nvec <= 64) return (const void *)row_kernel<DT, OP, OUT, 32, 2>;
        return (const void *)row_kernel<DT, OP, OUT, 32, 4>;
    }
    if (few) {
        if (nvec <= 128) return TCR_ROW(128, 1);
        if (nvec <= 256) return TCR_ROW(256, 1);
        if (nvec <= 512) return TCR_ROW(512, 1);
    }
    if (nvec <= 256) return TCR_ROW(128, 2);
    if (nvec <= 512) return TCR_ROW(128, 4);
    if (nvec <= 1024) return few ? TCR_ROW(512, 2) : TCR_ROW(256, 4);
    if (nvec <= 2048) return TCR_ROW(512, 4);
    if (nvec <= 4096) return TCR_ROW(1024, 4);
#undef TCR_ROW
    threads = kRowLongT;
    return (const void *)row_long_kernel<DT, OP, OUT>;
}

template <int DT>
const void *pick_op(int op, int out_i8, size_t nvec, size_t rows, int &threads, size_t &grid)
{
    if (op == kRowNorm)
        return out_i8 ? pick<DT, kRowNorm, kOutI8>(nvec, rows, threads, grid)
                      : pick<DT, kRowNorm, kOutSame>(nvec, rows, threads, grid);
    return pick<DT, kRowQuant, kOutI8>(nvec, rows, threads, grid);
}

}  // namespace

cudaError_t launch_rows_op(int op, int dtype, bool out_i8, const RowArgs &a, cudaStream_t stream)
{
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    int threads = 0;
    size_t grid = 0;
    const void *k = dtype == kF16    ? pick_op<kF16>(op, out_i8, nvec, a.rows, threads, grid)
                    : dtype == kBF16 ? pick_op<kBF16>(op, out_i8, nvec, a.rows, threads, grid)
                                     : pick_op<kF32>(op, out_i8, nvec, a.rows, threads, grid);
    void *args[] = {(void *)&a};
    return launch_first(k, dim3((unsigned)grid), dim3((unsigned)threads), args, 0, stream);
}

cudaError_t launch_dequant(int dtype, const int8_t *q, size_t ldq, const float *scale, void *y, size_t ldy,
                           size_t rows, size_t cols, cudaStream_t stream)
{
    int team_log2 = 0;
    while (team_log2 < 8 && ((size_t)16 << team_log2) < cols) team_log2++;
    const size_t grid = (rows + ((size_t)256 >> team_log2) - 1) / ((size_t)256 >> team_log2);
    const size_t es = dtype == kF32 ? 4 : 2;
    bool al_q = ((uintptr_t)q & 15u) == 0 && (rows == 1 || ldq % 16 == 0);
    bool al_y = ((uintptr_t)y & 15u) == 0 && (rows == 1 || (ldy * es) % 16 == 0);
    const void *k = dtype == kF16    ? (const void *)dequant_kernel<kF16>
                    : dtype == kBF16 ? (const void *)dequant_kernel<kBF16>
                                     : (const void *)dequant_kernel<kF32>;
    void *args[] = {(void *)&q,    (void *)&ldq,  (void *)&scale,     (void *)&y,    (void *)&ldy,
                    (void *)&rows, (void *)&cols, (void *)&team_log2, (void *)&al_q, (void *)&al_y};
    return launch_first(k, dim3((unsigned)grid), dim3(256), args, 0, stream);
}

}  // namespace tcr
