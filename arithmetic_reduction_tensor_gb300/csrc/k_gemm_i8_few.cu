// k_gemm_i8_few.cu -- the 8-bit product for a few tokens (a decoding step).
//
// At these sizes the weights, read once, and the fixed cost of a launch bound
// it: one launch, no scratch, no preparation, K split only inside a CTA.
// Dot products of four codes at a time run on the integer units.  A CTA owns
// 4 R channels; a warp reads 128 consecutive codes of each of four channels at
// once (8 lanes of 16 codes to a channel), so that a token's 128 codes, the
// same for all four, are one shared-bandwidth access instead of four, and its
// eight warps take the blocks of 128 k in turn.  The lanes' integer sums meet
// by shuffles and shared-memory atomics, in any order: they are exact.
//
// (Warp-level binary16 MMAs on the same layout were measured beside it:
// m16n8k16 runs at about 80 TFLOP/s here, so from 8 tokens on they took
// longer -- 8 x 8192 x 8192 28 us, 48 x 8192 x 8192 81 us.)
#include "kernels.cuh"
#include "codes.cuh"

namespace tcr {

constexpr int kFwWarps = 8;

// Tokens blockIdx.y * MT ..; the weights of a token tile after the first come
// from L2.
template <int MT, int R>
__global__ void __launch_bounds__(32 * kFwWarps, MT * R <= 16 ? 3 : 2)
gemm_i8_few_kernel(const I8Args a)
{
    constexpr int kCh = 4 * R;
    __shared__ int sum[MT][kCh];
    pdl_launch_dependents();
    if (threadIdx.x < MT * kCh) (&sum[0][0])[threadIdx.x] = 0;
    __syncthreads();
    pdl_wait_primary();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 3;
    const uint32_t K = (uint32_t)a.K;
    const size_t n0 = (size_t)blockIdx.x * kCh, m0 = (size_t)blockIdx.y * MT;
    const int tokens = (int)min((size_t)MT, a.M - m0);
    int acc[MT][R];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int r = 0; r < R; r++) acc[m][r] = 0;
    // channels and tokens past the end read the first one's codes; their sums
    // are not stored
    const int8_t *w[R];
#pragma unroll
    for (int r = 0; r < R; r++) w[r] = a.W + (n0 + 4 * r + row < a.N ? n0 + 4 * r + row : n0) * a.ldw;
    const int8_t *x0 = a.A + m0 * a.lda;
    auto add = [&](const uint4 &q, const uint4 &c, int &s) {
        s = __dp4a((int)q.x, (int)c.x, s);
        s = __dp4a((int)q.y, (int)c.y, s);
        s = __dp4a((int)q.z, (int)c.z, s);
        s = __dp4a((int)q.w, (int)c.w, s);
    };
    const uint32_t step = 128 * kFwWarps;
    uint32_t k = 128 * warp + 16 * (lane & 7);
    if (a.al_a && a.al_w && K >= 16) {
        // whole 16-byte words, the next step's weights loaded ahead
        uint4 q[R];
        const bool any = k + 16 <= K;
        if (any) {
#pragma unroll
            for (int r = 0; r < R; r++) q[r] = ld_stream(w[r] + k);
        }
        while (k + 16 <= K) {
            uint4 next[R];
            const bool more = k + step + 16 <= K;
#pragma unroll
            for (int r = 0; r < R; r++) next[r] = more ? ld_stream(w[r] + k + step) : q[r];
#pragma unroll
            for (int m = 0; m < MT; m++) {
                const uint4 c = ld16(x0 + (m < tokens ? m : 0) * a.lda + k);
#pragma unroll
                for (int r = 0; r < R; r++) add(q[r], c, acc[m][r]);
            }
#pragma unroll
            for (int r = 0; r < R; r++) q[r] = next[r];
            k += step;
        }
    }
    for (; k < K; k += step) {
        uint4 q[R];
#pragma unroll
        for (int r = 0; r < R; r++) q[r] = ld_codes(w[r] + k, K - k, a.al_w);
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const uint4 c = ld_codes(x0 + (m < tokens ? m : 0) * a.lda + k, K - k, a.al_a);
#pragma unroll
            for (int r = 0; r < R; r++) add(q[r], c, acc[m][r]);
        }
    }
    // the eight lanes of a channel, then the warps
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int r = 0; r < R; r++) {
            int s = acc[m][r];
#pragma unroll
            for (int h = 4; h >= 1; h /= 2) s += __shfl_xor_sync(kFull, s, h);
            if ((lane & 7) == 0) atomicAdd(&sum[m][4 * r + row], s);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < MT * kCh; i += 32 * kFwWarps) {
        const int m = i / kCh, c = i % kCh;
        const size_t n = n0 + c;
        if (m < tokens && n < a.N)
            store_out(a.C, a.c_dtype, (m0 + m) * a.ldc + n, sum[m][c], a.sa ? a.sa[m0 + m] : 1.0f,
                      a.sw ? a.sw[n] : 1.0f);
    }
}

// ---------------------------------------------------------------- host

namespace {

template <int MT, int R>
cudaError_t launch_few(const I8Args &a, cudaStream_t stream)
{
    void *args[] = {(void *)&a};
    const dim3 grid((unsigned)((a.N + 4 * R - 1) / (4 * R)), (unsigned)((a.M + MT - 1) / MT));
    return launch_first((const void *)gemm_i8_few_kernel<MT, R>, grid, dim3(32 * kFwWarps), args, 0, stream);
}

}  // namespace

cudaError_t launch_gemm_i8_few(const I8Args &a, cudaStream_t stream)
{
#ifdef FEWCFG
    switch (atoi(getenv("FEWCFG"))) {
    case 12: return launch_few<1, 2>(a, stream);
    case 14: return launch_few<1, 4>(a, stream);
    case 22: return launch_few<2, 2>(a, stream);
    case 24: return launch_few<2, 4>(a, stream);
    case 42: return launch_few<4, 2>(a, stream);
    case 44: return launch_few<4, 4>(a, stream);
    case 82: return launch_few<8, 2>(a, stream);
    case 84: return launch_few<8, 4>(a, stream);
    case 161: return launch_few<16, 1>(a, stream);
    case 162: return launch_few<16, 2>(a, stream);
    case 164: return launch_few<16, 4>(a, stream);
    }
#endif
    if (a.M <= 1) return launch_few<1, 4>(a, stream);
    if (a.M <= 2) return launch_few<2, 4>(a, stream);
    if (a.M <= 4) return launch_few<4, 4>(a, stream);
    if (a.M <= 8) return launch_few<8, 4>(a, stream);
    return launch_few<16, 4>(a, stream);
}

}  // namespace tcr
