// k_layer.cu -- dropout, and the launch of the layer norm (layer.cuh).
#include "kernels.cuh"
#include "piece.cuh"
#include "plan.h"

namespace tcr {

// y = r + dropout(x).  A CTA of 8 warps takes 256 * 2^wr columns of 8 / 2^wr
// rows at a time, kDropRows such steps with their loads issued together.
// Bound by memory traffic.
constexpr int kDropRows = 4;
template <int DT, bool ELEM>
__global__ void __launch_bounds__(256)
dropout_kernel(const __grid_constant__ LayerArgs a, int wr)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    using E = typename Elem<DT>::T;
    const uint32_t cols = (uint32_t)a.cols, warp = threadIdx.x >> 5;
    const uint32_t v = 32u * ((blockIdx.x << wr) + (warp & ((1u << wr) - 1))) + (threadIdx.x & 31);
    if (kRv * (v & ~31u) >= cols) return;
    const Drop drop(a.drop);
    constexpr int L = layout_of<DT, ELEM>();
    const uint32_t at = piece_offset<L>(v), n = piece_count<L>(cols, at);
    const size_t step = (size_t)gridDim.y << (3 - wr);       // rows of one step of the grid
    const bool has_r = a.r != nullptr;
    for (size_t r0 = ((size_t)blockIdx.y << (3 - wr)) + (warp >> wr); r0 < a.rows; r0 += kDropRows * step) {
        Piece<DT> x[kDropRows], res[kDropRows];
#pragma unroll
        for (int i = 0; i < kDropRows; i++) {
            const size_t r = r0 + i * step;
            if (r >= a.rows) break;
            const E *px = (const E *)a.x + r * a.ldx + at, *pr = (const E *)a.r + r * a.ldr + at;
            load_piece<DT, L>(px, n, x[i], by_words(px));
            if (has_r) load_piece<DT, L>(pr, n, res[i], by_words(pr));
        }
#pragma unroll
        for (int i = 0; i < kDropRows; i++) {
            const size_t r = r0 + i * step;
            if (r >= a.rows) break;
            float y[kRv];
            piece_values<DT>(x[i], y);
            drop_values<L>(drop, v, r, y);
            if (has_r) {
                float g[kRv];
                piece_values<DT>(res[i], g);
                add8(y, g, y);
            }
            E *py = (E *)a.y + r * a.ldy + at;
            store_piece<DT, L>(py, n, y, by_words(py));
        }
    }
}

// ---------------------------------------------------------------- host

cudaError_t launch_layer(int dtype, const LayerArgs &a, cudaStream_t stream)
{
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    int team = 0;
    const bool elem = !a.al_x || (a.r && !a.al_r) || (a.w && !a.al_w) || (a.b && !a.al_b) || (a.h && !a.al_h) || !a.al_y;
    const void *k = dtype == kF16    ? layer_kernel_f16(nvec, elem, team)
                    : dtype == kBF16 ? layer_kernel_bf16(nvec, elem, team)
                                     : layer_kernel_f32(nvec, elem, team);
    void *args[] = {(void *)&a};
    if (team == 32) return launch_first(k, dim3((unsigned)((a.rows + 3) / 4)), dim3(128), args, 0, stream);
    return launch_first(k, dim3((unsigned)a.rows), dim3((unsigned)(team ? team : kRowLongT)), args, 0, stream);
}

cudaError_t launch_dropout(int dtype, const LayerArgs &a, cudaStream_t stream)
{
    int wr = 0;
    while (wr < 3 && ((size_t)256 << wr) < a.cols) wr++;
    const size_t gx = (a.cols + ((size_t)256 << wr) - 1) / ((size_t)256 << wr);
    const size_t steps = (a.rows + ((size_t)8 >> wr) - 1) / ((size_t)8 >> wr);
    // kDropRows steps a CTA; few rows: one, spread over the SMs
    size_t gy = (steps + kDropRows - 1) / kDropRows;
    if (gx * gy < 4 * (size_t)plan::kRuleSMs) gy = steps;
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
