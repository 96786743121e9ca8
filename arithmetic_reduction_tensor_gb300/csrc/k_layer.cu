// k_layer.cu -- dropout, and the layer norm with dropout and the residual's
// addition: one pass over the data per row.
//
//   h = r + dropout(x) (binary32),  mean = S1 / cols, S1 the row sum of h,
//   rstd = 1 / sqrt(S2 / cols + eps), S2 the row sum of (h - mean)^2,
//   y = ((h - mean) * rstd) * w + b, rounded, or as 8-bit codes
//
// The row stays in registers, so the squares are taken about the mean itself
// (the difference of two large sums would lose small variances) at the price
// of a second barrier and no second read.  Both sums have the declared order
// of rowvec.cuh, every step is one binary32 operation rounded to nearest, and
// the mask is that of drop.cuh: the results are pinned bit for bit.
#include "kernels.cuh"
#include "piece.cuh"

namespace tcr {

constexpr int kOutSame = 0, kOutI8 = 1;

__device__ __forceinline__ float rstd_of(float s, uint32_t cols, float eps)
{
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(s, (float)cols), eps));
}

// Rows of at most 8 T NV columns, NV pieces a thread: teams of T threads (T =
// 32: eight to a CTA; else the CTA) walk the rows, each loading its next row
// before it finishes the current one.  The sums' two buffers and the largest
// magnitude's are each written again only after a barrier that every reader
// of the last values has passed.
template <int DT, int OUT, bool ELEM, int T, int NV, int MINB>
__global__ void __launch_bounds__(T == 32 ? 256 : T, MINB)
layer_kernel(const LayerArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][team_floats<T>()];
    __shared__ uint32_t redm[32];
    using E = typename Elem<DT>::T;
    const uint32_t t = T == 32 ? threadIdx.x & 31 : threadIdx.x, cols = (uint32_t)a.cols;
    const uint32_t threads = T == 32 ? 32 : blockDim.x;
    const size_t team = T == 32 ? (size_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    const size_t teams = T == 32 ? (size_t)gridDim.x * 8 : gridDim.x;
    const bool has_r = a.r != nullptr, has_w = a.w != nullptr, has_b = a.b != nullptr;
    const DropArgs drop = drop_resolve(a.drop);
    Piece<DT, ELEM> x[NV], res[NV], w[NV], b[NV];
    auto load = [&](size_t r) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            load_piece<DT, ELEM>((const E *)a.x + r * a.ldx, cols, t + i * T, x[i]);
            if (has_r) load_piece<DT, ELEM>((const E *)a.r + r * a.ldr, cols, t + i * T, res[i]);
        }
    };
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (has_w) load_weight_piece<DT, ELEM>((const E *)a.w, cols, t + i * T, a.al_w, w[i]);
        if (has_b) load_weight_piece<DT, ELEM>((const E *)a.b, cols, t + i * T, a.al_b, b[i]);
    }
    if (team < a.rows) load(team);
    for (size_t r = team; r < a.rows; r += teams) {
        float y[NV][kRv], s[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t v = t + i * T;
            piece_values<DT, ELEM>(x[i], (const E *)a.x + r * a.ldx, cols, v, y[i]);
            drop_values<ELEM>(drop, v, r, y[i]);
            if (has_r) {
                float g[kRv];
                piece_values<DT, ELEM>(res[i], (const E *)a.r + r * a.ldr, cols, v, g);
#pragma unroll
                for (int k = 0; k < kRv; k++) y[i][k] = __fadd_rn(g[k], y[i][k]);
            }
            s[i] = piece_tree<ELEM>(y[i]);
        }
        if (r + teams < a.rows) load(r + teams);
        const float mean = __fdiv_rn(team_sum<T, ELEM>(halving<NV>(s), red[0], threads), (float)cols);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t v = t + i * T;
            if (a.h && kRv * (v & ~31u) < cols)              // whole warps: stores are warp-wide
                store_piece_values<DT, ELEM>((E *)a.h + r * a.ldh, cols, v, y[i]);
            centre(y[i], mean);
            zero_absent<ELEM>(cols, v, y[i]);
            float e[kRv];
#pragma unroll
            for (int k = 0; k < kRv; k++) e[k] = __fmul_rn(y[i][k], y[i][k]);
            s[i] = piece_tree<ELEM>(e);
        }
        const float rstd = rstd_of(team_sum<T, ELEM>(halving<NV>(s), red[1], threads), cols, a.eps);
        if (t == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t v = t + i * T;
            if (kRv * (v & ~31u) >= cols) continue;
#pragma unroll
            for (int k = 0; k < kRv; k++) y[i][k] = __fmul_rn(y[i][k], rstd);
            float f[kRv];
            if (has_w) {
                piece_values<DT, ELEM>(w[i], (const E *)a.w, cols, v, f);
#pragma unroll
                for (int k = 0; k < kRv; k++) y[i][k] = __fmul_rn(y[i][k], f[k]);
            }
            if (has_b) {
                piece_values<DT, ELEM>(b[i], (const E *)a.b, cols, v, f);
#pragma unroll
                for (int k = 0; k < kRv; k++) y[i][k] = __fadd_rn(y[i][k], f[k]);
            }
            if constexpr (OUT == kOutSame) {
                store_piece_values<DT, ELEM>((E *)a.y + r * a.ldy, cols, v, y[i]);
            } else {
                zero_absent<ELEM>(cols, v, y[i]);            // 0 times a possibly infinite rstd
                m = amax8(y[i], m);
            }
        }
        if constexpr (OUT == kOutI8) {
            float scale, per;
            i8_scale(team_max<T>(__float_as_uint(m), redm, threads), scale, per);
            if (t == 0) a.scale[r] = scale;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const uint32_t v = t + i * T;
                if (kRv * (v & ~31u) < cols) store_piece_codes<ELEM>((int8_t *)a.y + r * a.ldy, cols, v, y[i], per);
            }
        }
    }
}

// Rows at any alignment and length, read once a step (mean, variance, the
// largest magnitude, the outputs): a CTA a row.
template <int DT>
struct LayerRow {
    using E = typename Elem<DT>::T;
    const LayerArgs &a;
    const DropArgs &drop;
    size_t r;
    uint32_t cols;
    __device__ __forceinline__ void h(uint32_t v, float (&y)[kRv]) const
    {
        unpack<DT>(load_raw<DT>((const E *)a.x + r * a.ldx, cols, v, a.al_x), y);
        drop_values<false>(drop, v, r, y);
        if (!a.r) return;
        float g[kRv];
        unpack<DT>(load_raw<DT>((const E *)a.r + r * a.ldr, cols, v, a.al_r), g);
#pragma unroll
        for (int k = 0; k < kRv; k++) y[k] = __fadd_rn(g[k], y[k]);
    }
    __device__ __forceinline__ void norm(uint32_t v, float mean, float rstd, float (&y)[kRv]) const
    {
        float f[kRv];
        centre(y, mean);
#pragma unroll
        for (int k = 0; k < kRv; k++) y[k] = __fmul_rn(y[k], rstd);
        if (a.w) {
            unpack<DT>(load_raw<DT>((const E *)a.w, cols, v, a.al_w), f);
#pragma unroll
            for (int k = 0; k < kRv; k++) y[k] = __fmul_rn(y[k], f[k]);
        }
        if (a.b) {
            unpack<DT>(load_raw<DT>((const E *)a.b, cols, v, a.al_b), f);
#pragma unroll
            for (int k = 0; k < kRv; k++) y[k] = __fadd_rn(y[k], f[k]);
        }
        zero_absent<false>(cols, v, y);
    }
};

template <int DT, int OUT>
__global__ void __launch_bounds__(kRowLongT)
layer_long_kernel(const LayerArgs a)
{
    constexpr uint32_t T = kRowLongT;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][team_floats<(int)T>()];
    __shared__ uint32_t redm[32];
    using E = typename Elem<DT>::T;
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    const DropArgs drop = drop_resolve(a.drop);
    const LayerRow<DT> row{a, drop, blockIdx.x, cols};
    const size_t r = blockIdx.x;
    const uint32_t nvec = (cols + kRv - 1) / kRv, steps = (nvec + T - 1) / T;
    const int bits = ceil_log2_sz(steps);
    float y[kRv], mean = 0.0f, rstd = 0.0f;
#pragma unroll 1
    for (int pass = 0; pass < 2; pass++) {
        TreeCounter<16> tc;
        for (uint32_t j = 0; j < (1u << bits); j++) {
            const uint32_t v = t + bit_reverse(j, bits) * T;
            float s = 0.0f;
            if (v < nvec) {
                row.h(v, y);
                if (pass == 1) {
                    centre(y, mean);
                    zero_absent<false>(cols, v, y);
#pragma unroll
                    for (int k = 0; k < kRv; k++) y[k] = __fmul_rn(y[k], y[k]);
                } else {
                    zero_absent<false>(cols, v, y);
                }
                s = tree8(y);
            }
            tc.push(s);
        }
        const float sum = team_sum<T>(tc.finish(), red[pass]);
        if (pass == 0)
            mean = __fdiv_rn(sum, (float)cols);
        else
            rstd = rstd_of(sum, cols, a.eps);
    }
    if (t == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
    float per = 0.0f;
    if constexpr (OUT == kOutI8) {
        float m = 0.0f;
        for (uint32_t v = t; v < nvec; v += T) {
            row.h(v, y);
            row.norm(v, mean, rstd, y);
            m = amax8(y, m);
        }
        float scale;
        i8_scale(team_max<T>(__float_as_uint(m), redm), scale, per);
        if (t == 0) a.scale[r] = scale;
    }
    for (uint32_t i = 0; i < steps; i++) {              // whole warps: stores are warp-wide
        const uint32_t v = t + i * T;
        row.h(v, y);
        if (a.h) store_vec<DT>((E *)a.h + r * a.ldh, cols, v, a.al_h, y);
        row.norm(v, mean, rstd, y);
        if constexpr (OUT == kOutSame)
            store_vec<DT>((E *)a.y + r * a.ldy, cols, v, a.al_y, y);
        else
            store_codes((int8_t *)a.y + r * a.ldy, cols, v, a.al_y, y, per);
    }
}

// ---------------------------------------------------------------- dropout alone

// y = r + dropout(x).  A CTA of 8 warps takes 256 * 2^wr columns of 8 / 2^wr
// rows at a time, kDropRows such steps with their loads issued together.
// Bound by memory traffic.
constexpr int kDropRows = 4;
template <int DT, bool ELEM>
__global__ void __launch_bounds__(256)
dropout_kernel(const LayerArgs a, int wr)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    using E = typename Elem<DT>::T;
    const uint32_t cols = (uint32_t)a.cols, warp = threadIdx.x >> 5;
    const uint32_t v = 32u * ((blockIdx.x << wr) + (warp & ((1u << wr) - 1))) + (threadIdx.x & 31);
    if (kRv * (v & ~31u) >= cols) return;
    const DropArgs drop = drop_resolve(a.drop);
    const size_t step = (size_t)gridDim.y << (3 - wr);       // rows of one step of the grid
    const bool has_r = a.r != nullptr;
    for (size_t r0 = ((size_t)blockIdx.y << (3 - wr)) + (warp >> wr); r0 < a.rows; r0 += kDropRows * step) {
        Piece<DT, ELEM> x[kDropRows], res[kDropRows];
#pragma unroll
        for (int i = 0; i < kDropRows; i++) {
            const size_t r = r0 + i * step;
            if (r >= a.rows) break;
            load_piece<DT, ELEM>((const E *)a.x + r * a.ldx, cols, v, x[i]);
            if (has_r) load_piece<DT, ELEM>((const E *)a.r + r * a.ldr, cols, v, res[i]);
        }
#pragma unroll
        for (int i = 0; i < kDropRows; i++) {
            const size_t r = r0 + i * step;
            if (r >= a.rows) break;
            float y[kRv];
            piece_values<DT, ELEM>(x[i], (const E *)a.x + r * a.ldx, cols, v, y);
            drop_values<ELEM>(drop, v, r, y);
            if (has_r) {
                float g[kRv];
                piece_values<DT, ELEM>(res[i], (const E *)a.r + r * a.ldr, cols, v, g);
#pragma unroll
                for (int k = 0; k < kRv; k++) y[k] = __fadd_rn(g[k], y[k]);
            }
            store_piece_values<DT, ELEM>((E *)a.y + r * a.ldy, cols, v, y);
        }
    }
}

// ---------------------------------------------------------------- host

namespace {

template <int DT, int OUT, bool ELEM, int T, int NV, int MINB>
const void *shape_of(size_t nvec, size_t rows, int &threads, size_t &grid)
{
    threads = T == 32 ? 256 : NV == 1 ? (int)((nvec + 31) / 32 * 32) : T;
    const size_t need = T == 32 ? (rows + 7) / 8 : rows;
    const size_t full = (size_t)152 * (size_t)(T == 32 ? MINB : MINB * T / threads);
    grid = need < full ? need : full;
    return (const void *)layer_kernel<DT, OUT, ELEM, T, NV, MINB>;
}

template <int DT, int OUT>
const void *pick(size_t nvec, size_t rows, bool elem, int &threads, size_t &grid)
{
#define TCR_SHAPE(ELEM_, T_, NV_, MINB_) return shape_of<DT, OUT, ELEM_, T_, NV_, MINB_>(nvec, rows, threads, grid)
    if (elem) {
        if (nvec <= 32) TCR_SHAPE(true, 32, 1, 4);
        if (nvec <= 64) TCR_SHAPE(true, 32, 2, 2);
        if (nvec <= 128) TCR_SHAPE(true, 128, 1, 8);
        if (nvec <= 256) TCR_SHAPE(true, 256, 1, 4);
        if (nvec <= 512) TCR_SHAPE(true, 256, 2, 2);
        if (nvec <= 1024) TCR_SHAPE(true, 512, 2, 1);
    } else if constexpr (DT == kF32) {
        if (nvec <= 32) TCR_SHAPE(false, 32, 1, 3);
        if (nvec <= 64) TCR_SHAPE(false, 32, 2, 2);
        if (nvec <= 128) TCR_SHAPE(false, 128, 1, 8);
        if (nvec <= 256) TCR_SHAPE(false, 256, 1, 4);
        if (nvec <= 512) TCR_SHAPE(false, 512, 1, 2);
        if (nvec <= 1024) TCR_SHAPE(false, 512, 2, 1);
    } else {
        if (nvec <= 32) TCR_SHAPE(false, 32, 1, 4);
        if (nvec <= 64) TCR_SHAPE(false, 32, 2, 3);
        if (nvec <= 128) TCR_SHAPE(false, 64, 2, 12);
        if (nvec <= 256) TCR_SHAPE(false, 128, 2, 6);
        if (nvec <= 512) TCR_SHAPE(false, 256, 2, 3);
        if (nvec <= 1024) TCR_SHAPE(false, 256, 4, 2);
        if (nvec <= 2048) TCR_SHAPE(false, 512, 4, 1);
    }
#undef TCR_SHAPE
    grid = rows;
    threads = kRowLongT;
    return (const void *)layer_long_kernel<DT, OUT>;
}

template <int DT>
const void *pick_out(bool out_i8, size_t nvec, size_t rows, bool elem, int &threads, size_t &grid)
{
    return out_i8 ? pick<DT, kOutI8>(nvec, rows, elem, threads, grid)
                  : pick<DT, kOutSame>(nvec, rows, elem, threads, grid);
}

}  // namespace

cudaError_t launch_layer(int dtype, bool out_i8, const LayerArgs &a, cudaStream_t stream)
{
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    int threads = 0;
    size_t grid = 0;
    const bool elem = !a.al_x || (a.r && !a.al_r) || (a.h && !a.al_h) || !a.al_y;
    const void *k = dtype == kF16    ? pick_out<kF16>(out_i8, nvec, a.rows, elem, threads, grid)
                    : dtype == kBF16 ? pick_out<kBF16>(out_i8, nvec, a.rows, elem, threads, grid)
                                     : pick_out<kF32>(out_i8, nvec, a.rows, elem, threads, grid);
    void *args[] = {(void *)&a};
    return launch_first(k, dim3((unsigned)grid), dim3((unsigned)threads), args, 0, stream);
}

cudaError_t launch_dropout(int dtype, const LayerArgs &a, cudaStream_t stream)
{
    int wr = 0;
    while (wr < 3 && ((size_t)256 << wr) < a.cols) wr++;
    const size_t gx = (a.cols + ((size_t)256 << wr) - 1) / ((size_t)256 << wr);
    const size_t steps = (a.rows + ((size_t)8 >> wr) - 1) / ((size_t)8 >> wr);
    // kDropRows steps a CTA; few rows: one, spread over the SMs
    size_t gy = (steps + kDropRows - 1) / kDropRows;
    if (gx * gy < 4 * 152) gy = steps;
    if (gy > 65535) gy = 65535;
    const bool elem = !a.al_x || (a.r && !a.al_r) || !a.al_y;
    const void *k;
    if (elem)
        k = dtype == kF16    ? (const void *)dropout_kernel<kF16, true>
            : dtype == kBF16 ? (const void *)dropout_kernel<kBF16, true>
                             : (const void *)dropout_kernel<kF32, true>;
    else
        k = dtype == kF16    ? (const void *)dropout_kernel<kF16, false>
            : dtype == kBF16 ? (const void *)dropout_kernel<kBF16, false>
                             : (const void *)dropout_kernel<kF32, false>;
    void *args[] = {(void *)&a, (void *)&wr};
    return launch_first(k, dim3((unsigned)gx, (unsigned)gy), dim3(256), args, 0, stream);
}

}  // namespace tcr
