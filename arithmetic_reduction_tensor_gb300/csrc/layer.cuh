// layer.cuh -- the layer norm with dropout and the residual's addition: one pass
// over the data per row.  Its shapes take long to compile, so each type has a
// file of its own (k_layer_*.cu).
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
#pragma once

#include "kernels.cuh"
#include "piece.cuh"

namespace tcr {

__device__ __forceinline__ float rstd_of(float s, uint32_t cols, float eps)
{
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(s, (float)cols), eps));
}

// One row, NV pieces a thread, of which the first LEAD are whole.
template <int DT, bool ELEM, int T, int NV, int LEAD>
__device__ __forceinline__ void layer_row(const LayerArgs &a, const Drop &drop, size_t r, uint32_t t, float *red,
                                          uint32_t *redm)
{
    using E = typename Elem<DT>::T;
    constexpr int L = layout_of<DT, ELEM>();
    constexpr uint32_t kStep = kRv * T;                  // elements between a thread's pieces
    const uint32_t cols = (uint32_t)a.cols;
    const bool has_r = a.r != nullptr;
    const uint32_t at = piece_offset<L>(t);
    auto count = [&](int i) { return piece_count<L, T, LEAD>(cols, at, i); };
    float y[NV][kRv], s[NV];
    {
        const E *px = (const E *)a.x + r * a.ldx + at, *pr = (const E *)a.r + r * a.ldr + at;
        Piece<DT> x[NV], res[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) load_piece<DT, L>(px + i * kStep, count(i), x[i], by_words(px));
        if (has_r) {
#pragma unroll
            for (int i = 0; i < NV; i++)
                load_piece<DT, L>(pr + i * kStep, count(i), res[i], by_words(pr));
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            piece_values<DT>(x[i], y[i]);
            drop_values<L>(drop, t + i * T, r, y[i]);
        }
        if (has_r) {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float g[kRv];
                piece_values<DT>(res[i], g);
                add8(y[i], g, y[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        zero_absent(count(i), y[i]);
        s[i] = piece_tree<L>(y[i]);
    }
    float sum[1] = {fold<NV>(s)};
    team_sums<T, L>(sum, red);
    const float mean = __fdiv_rn(sum[0], (float)cols);
    if (a.h) {
        E *ph = (E *)a.h + r * a.ldh + at;
#pragma unroll
        for (int i = 0; i < NV; i++)
            store_piece<DT, L>(ph + i * kStep, count(i), y[i], by_words(ph));
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        float e[kRv];
        add8(y[i], y[i], -mean);
        zero_absent(count(i), y[i]);
        mul8(e, y[i], y[i]);
        s[i] = piece_tree<L>(e);
    }
    sum[0] = fold<NV>(s);
    team_sums<T, L>(sum, red + team_sums_floats<T, 1>());
    const float rstd = rstd_of(sum[0], cols, a.eps);
    if (t == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; i++) mul8(y[i], y[i], rstd);
    if (a.w) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float f[kRv];
            Piece<DT> w;
            load_piece<DT, L>((const E *)a.w + at + i * kStep, count(i), w, by_words(a.w));
            piece_values<DT>(w, f);
            mul8(y[i], y[i], f);
        }
    }
    if (a.b) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float f[kRv];
            Piece<DT> b;
            load_piece<DT, L>((const E *)a.b + at + i * kStep, count(i), b, by_words(a.b));
            piece_values<DT>(b, f);
            add8(y[i], y[i], f);
        }
    }
    if (!a.scale) {
        E *py = (E *)a.y + r * a.ldy + at;
#pragma unroll
        for (int i = 0; i < NV; i++)
            store_piece<DT, L>(py + i * kStep, count(i), y[i], by_words(py));
        return;
    }
    float m = 0.0f, scale, per;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        zero_absent(count(i), y[i]);                         // 0 times a possibly infinite rstd
        m = amax8(y[i], m);
    }
    i8_scale(team_most<T>(__float_as_uint(m), redm), scale, per);
    if (t == 0) a.scale[r] = scale;
    int8_t *py = (int8_t *)a.y + r * a.ldy + at;
#pragma unroll
    for (int i = 0; i < NV; i++) store_piece_codes<L>(py + i * kStep, count(i), y[i], per);
}

// Rows of at most 8 T NV columns, NV pieces a thread, a team of T threads a row
// (T = 32: four to a CTA; else the CTA); the first LEAD pieces are whole in
// every warp, and warps whose last is whole, too, run code without masks (most
// of a row's warps; masks everywhere cost 16384 x 4096 bfloat16 rows a third).  No
// team walks rows and none loads ahead: weight and bias come from L1 or L2 row
// by row, so that registers hold one row alone and up to 1024 threads' rows
// are in flight on an SM, at different steps.  That takes 16384 x 4096 bfloat16
// 79 us (the copy rate), where teams that walk rows, with the weight in
// registers and the next row's loads in flight, took 93.
template <int DT, bool ELEM, int T, int NV, int LEAD, int MINB>
__global__ void __launch_bounds__(T == 32 ? 128 : T, MINB)
layer_kernel(const __grid_constant__ LayerArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2 * team_sums_floats<T, 1>()];
    __shared__ uint32_t redm[32];
    const uint32_t t = T == 32 ? threadIdx.x & 31 : threadIdx.x;
    const size_t r = T == 32 ? (size_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (T == 32 && r >= a.rows) return;
    const Drop drop(a.drop);
    if (warp_whole<T, NV>((uint32_t)a.cols, t))
        layer_row<DT, ELEM, T, NV, NV>(a, drop, r, t, red, redm);
    else
        layer_row<DT, ELEM, T, NV, LEAD>(a, drop, r, t, red, redm);
}

// Rows at any alignment and length, read once a step (mean, variance, the
// largest magnitude, the outputs): a CTA a row.
template <int DT>
struct LayerRow {
    using E = typename Elem<DT>::T;
    const LayerArgs &a;
    const Drop &drop;
    size_t r;
    uint32_t cols;
    __device__ __forceinline__ void h(uint32_t v, float (&y)[kRv]) const
    {
        unpack<DT>(load_raw<DT>((const E *)a.x + r * a.ldx, cols, v, a.al_x), y);
        drop_values<kVectors>(drop, v, r, y);
        if (!a.r) return;
        float g[kRv];
        unpack<DT>(load_raw<DT>((const E *)a.r + r * a.ldr, cols, v, a.al_r), g);
#pragma unroll
        for (int k = 0; k < kRv; k++) y[k] = __fadd_rn(g[k], y[k]);
    }
    __device__ __forceinline__ void norm(uint32_t v, float mean, float rstd, float (&y)[kRv]) const
    {
        float f[kRv];
        add8(y, y, -mean);
        mul8(y, y, rstd);
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
        zero_absent(vec_left(cols, v), y);
    }
};

template <int DT>
__global__ void __launch_bounds__(kRowLongT)
layer_long_kernel(const __grid_constant__ LayerArgs a)
{
    constexpr uint32_t T = kRowLongT;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][team_floats<(int)T>()];
    __shared__ uint32_t redm[32];
    using E = typename Elem<DT>::T;
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    const Drop drop(a.drop);
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
                    add8(y, y, -mean);
                    zero_absent(vec_left(cols, v), y);
#pragma unroll
                    for (int k = 0; k < kRv; k++) y[k] = __fmul_rn(y[k], y[k]);
                } else {
                    zero_absent(vec_left(cols, v), y);
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
    if (a.scale) {
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
        if (!a.scale)
            store_vec<DT>((E *)a.y + r * a.ldy, cols, v, a.al_y, y);
        else
            store_codes((int8_t *)a.y + r * a.ldy, cols, v, a.al_y, y, per);
    }
}

// Which shape serves a row length: as many pieces of T threads as the row needs,
// T by what was measured (bfloat16, with dropout).  Threads whose last pieces
// are past the row's end issue for nothing: 6151 x 5120 128 x 5 40 us, 256 x 3 49;
// 4500 x 7168 128 x 7 42, 256 x 4 46; unaligned 32768 x 1500 64 x 3 114, 64 x 4 194.
// 8192 x 8192 256 x 4 with 4 CTAs an SM 83, 4096 x 16384 512 x 4 with 2 CTAs 100,
// with 1 146.  binary32, 2^26 elements: 512 columns 32 x 2 155, 64 x 1 154; 1024 64 x 2
// 155, 128 x 1 153, 32 x 4 156; 2048 128 x 2 155, 256 x 1 160; 4096 256 x 2 161, 128 x 4 157, 512
// x 1 191; 8192 512 x 2 195, 256 x 4 203, 1024 x 1 259; 16384 1024 x 2 216, 512 x 4 216.  MINB_:
// CTAs an SM at 64 registers a thread (80 from five pieces on and in binary32).
template <int DT, bool ELEM>
const void *layer_shape(size_t nvec, int &team)
{
#define TCR_SHAPE(T_, NV_, LEAD_, MINB_) return (team = T_, (const void *)layer_kernel<DT, ELEM, T_, NV_, LEAD_, MINB_>)
    if constexpr (DT == kF32) {
        if (nvec <= 64) TCR_SHAPE(32, 2, 0, 6);
        if (nvec <= 128) TCR_SHAPE(64, 2, 1, 12);
        if (nvec <= 256) TCR_SHAPE(128, 2, 1, 6);
        if (nvec <= 512) TCR_SHAPE(256, 2, 1, 3);
        if (nvec <= 1024) TCR_SHAPE(512, 2, 1, 1);
        if (nvec <= 2048) TCR_SHAPE(1024, 2, 1, 1);
    } else {
        if (nvec <= 64) TCR_SHAPE(32, 2, 0, 8);
        if (nvec <= 128) TCR_SHAPE(32, 4, 2, 8);
        if (nvec <= 192) TCR_SHAPE(64, 3, 2, 16);
        if (nvec <= 256) TCR_SHAPE(64, 4, 3, 16);
        if (nvec <= 384) TCR_SHAPE(128, 3, 2, 8);
        if (nvec <= 512) TCR_SHAPE(128, 4, 3, 8);
        if (nvec <= 640) TCR_SHAPE(128, 5, 4, 6);
        if (nvec <= 768) TCR_SHAPE(128, 6, 5, 5);
        if (nvec <= 896) TCR_SHAPE(128, 7, 6, 5);
        if (nvec <= 1024) TCR_SHAPE(256, 4, 3, 4);
        if (nvec <= 1536) TCR_SHAPE(512, 3, 2, 2);
        if (nvec <= 2048) TCR_SHAPE(512, 4, 3, 2);
        if (nvec <= 4096) TCR_SHAPE(1024, 4, 2, 1);
    }
#undef TCR_SHAPE
    team = 0;
    return (const void *)layer_long_kernel<DT>;
}

// The kernel for a row of nvec vectors, its team's threads in *team (0: a CTA of
// kRowLongT a row); elem: some of the call's rows are not 16-byte aligned.
template <int DT>
const void *layer_kernel_of(size_t nvec, bool elem, int &team)
{
    return elem ? layer_shape<DT, true>(nvec, team) : layer_shape<DT, false>(nvec, team);
}

}  // namespace tcr
