// k_gemm_i8_few.cu -- the 8-bit product for a few tokens (a decoding step) and
// for small matrices.
//
// At these sizes the weights, read from memory once (a token tile after the
// first finds them in L2), and the fixed cost of a launch bound it: one launch,
// no scratch, no preparation, K split only inside a CTA.
//
// One or two tokens: dot products of four codes at a time on the integer
// units (240 multiply-adds a cycle and SM).  A CTA owns 4 R channels; a warp
// reads 128 consecutive codes of each of four channels at once (8 lanes of 16
// codes to a channel), so that a token's 128 codes, the same for all four,
// are one access, and its eight warps take the blocks of 128 k in turn.
//
// More tokens: warp-level MMAs (m16n8k16 on binary16 operands, 1000 a cycle
// and SM; the 8-bit integer MMA, 250, gains nothing), exact as in
// k_gemm_i8.cu, the channels as rows and the tokens as columns.  Both operands
// come straight from global memory as codes: the order of k inside a sum is
// free as long as both operands agree, so lane (g, t) of a warp reads 16
// codes, k = 16 t .. 16 t + 15 of a block of 64, of channels g and g + 8 and
// of token g, and the four words of each are the fragments of four MMAs.  A
// CTA owns 16 MB channels and 8 NB tokens; its eight warps take the blocks of
// 64 k in turn (512 consecutive bytes of each row at a time), the next
// block's codes loaded ahead, and add their sums as integers in shared
// memory, in any order: they are exact.
#include "kernels.cuh"
#include "codes.cuh"

namespace tcr {

constexpr int kFwWarps = 8;

// Tokens blockIdx.y * MT ..; the weights of a token tile after the first come
// from L2.
template <int MT, int R, bool GRAN>
__global__ void __launch_bounds__(32 * kFwWarps, 3)
gemm_i8_dot_kernel(const I8Args a)
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
    // the next step's weights are loaded ahead; a warp's steps are whole
    // blocks of 128 k but for the row's last
    const uint32_t step = 128 * kFwWarps;
    uint32_t k = 128 * warp + 16 * (lane & 7);
    auto left = [&](uint32_t at) { return at < K ? K - at : 0u; };
    auto whole = [&](uint32_t at) { return (at & ~127u) + 128 <= K; };
    LoadedCodes<GRAN> q[R];
    auto load = [&](uint32_t at) {
        if (whole(at)) {
#pragma unroll
            for (int r = 0; r < R; r++) q[r] = load_codes<GRAN, true>(w[r] + at);
        } else {
#pragma unroll
            for (int r = 0; r < R; r++) q[r] = load_last_codes<GRAN>(w[r] + at, left(at));
        }
    };
    load(k);
    for (; k < K; k += step) {
        const bool all = whole(k);
        uint4 now[R];
#pragma unroll
        for (int r = 0; r < R; r++) now[r] = use_codes<GRAN>(q[r], w[r] + k, left(k), all);
        load(k + step);
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const int8_t *x = x0 + (m < tokens ? m : 0) * a.lda + k;
            const LoadedCodes<GRAN> l = all ? load_codes<GRAN, false>(x) : load_last_codes<GRAN>(x, left(k));
            const uint4 c = use_codes<GRAN>(l, x, left(k), all);
#pragma unroll
            for (int r = 0; r < R; r++) add(now[r], c, acc[m][r]);
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

// ---------------------------------------------------------------- warp-level MMAs

constexpr int kFwChunk = 16;        // blocks of 64 k per exact binary32 sum

template <int NB, int MB, bool GRAN>
__global__ void __launch_bounds__(32 * kFwWarps, NB * MB == 1 ? 3 : 2)
gemm_i8_few_kernel(const I8Args a)
{
    constexpr int kTok = 8 * NB, kCh = 16 * MB;
    __shared__ int sum[kTok][kCh + 1];
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < kTok * (kCh + 1); i += 32 * kFwWarps) (&sum[0][0])[i] = 0;
    __syncthreads();
    pdl_wait_primary();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t K = (uint32_t)a.K, blocks = (K + 63) / 64;
    const size_t n0 = (size_t)blockIdx.x * kCh, m0 = (size_t)blockIdx.y * kTok;
    const int tokens = (int)min((size_t)kTok, a.M - m0);
    // rows past the end read the first one's codes; their sums are not stored
    const int8_t *w[2 * MB], *x[NB];
#pragma unroll
    for (int i = 0; i < 2 * MB; i++) w[i] = a.W + (n0 + 8 * i + g < a.N ? n0 + 8 * i + g : n0) * a.ldw + 16 * t;
#pragma unroll
    for (int i = 0; i < NB; i++) x[i] = a.A + (m0 + (8 * i + (int)g < tokens ? 8 * i + g : 0)) * a.lda + 16 * t;
    float d[MB][NB][4];
#pragma unroll
    for (int i = 0; i < MB; i++)
#pragma unroll
        for (int j = 0; j < NB; j++)
#pragma unroll
            for (int r = 0; r < 4; r++) d[i][j][r] = 0.0f;
    auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < MB; i++)
#pragma unroll
            for (int j = 0; j < NB; j++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    atomicAdd(&sum[8 * j + 2 * t + (r & 1)][16 * i + g + 8 * (r >> 1)], __float2int_rn(d[i][j][r]));
                    d[i][j][r] = 0.0f;
                }
    };
    LoadedCodes<GRAN> q[2 * MB], c[NB];
    auto left = [&](uint32_t b) { return 64 * b + 16 * t < K ? K - 64 * b - 16 * t : 0u; };
    auto whole = [&](uint32_t b) { return 64 * b + 64 <= K; };
    auto load = [&](uint32_t b) {
        if (whole(b)) {
#pragma unroll
            for (int i = 0; i < 2 * MB; i++) q[i] = load_codes<GRAN, true>(w[i] + 64 * b);
#pragma unroll
            for (int j = 0; j < NB; j++) c[j] = load_codes<GRAN, false>(x[j] + 64 * b);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * MB; i++) q[i] = load_last_codes<GRAN>(w[i] + 64 * b, left(b));
#pragma unroll
            for (int j = 0; j < NB; j++) c[j] = load_last_codes<GRAN>(x[j] + 64 * b, left(b));
        }
    };
    if (warp < blocks) load(warp);
    int in_sum = 0;
    for (uint32_t b = warp; b < blocks; b += kFwWarps) {
        const bool all = whole(b);
        uint32_t f[MB][4][4], e[NB][4][2];        // the fragments of four MMAs
#pragma unroll
        for (int i = 0; i < MB; i++) {
            const uint4 lo = use_codes<GRAN>(q[2 * i], w[2 * i] + 64 * b, left(b), all);
            const uint4 hi = use_codes<GRAN>(q[2 * i + 1], w[2 * i + 1] + 64 * b, left(b), all);
            const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int s = 0; s < 4; s++) {
                widen4(l[s], f[i][s][0], f[i][s][2]);
                widen4(u[s], f[i][s][1], f[i][s][3]);
            }
        }
#pragma unroll
        for (int j = 0; j < NB; j++) {
            const uint4 v = use_codes<GRAN>(c[j], x[j] + 64 * b, left(b), all);
            const uint32_t l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int s = 0; s < 4; s++) widen4(l[s], e[j][s][0], e[j][s][1]);
        }
        if (b + kFwWarps < blocks) load(b + kFwWarps);
#pragma unroll
        for (int s = 0; s < 4; s++)
#pragma unroll
            for (int j = 0; j < NB; j++)
#pragma unroll
                for (int i = 0; i < MB; i++)
                    mma_ab<kF16>(d[i][j][0], d[i][j][1], d[i][j][2], d[i][j][3], f[i][s][0], f[i][s][1], f[i][s][2],
                                 f[i][s][3], e[j][s][0], e[j][s][1]);
        if (++in_sum == kFwChunk) {
            flush();
            in_sum = 0;
        }
    }
    flush();
    __syncthreads();
    for (int i = threadIdx.x; i < kTok * kCh; i += 32 * kFwWarps) {
        const int tok = i / kCh, ch = i % kCh;
        const size_t n = n0 + ch;
        if (tok < tokens && n < a.N)
            store_out(a.C, a.c_dtype, (m0 + tok) * a.ldc + n, sum[tok][ch], a.sa ? a.sa[m0 + tok] : 1.0f,
                      a.sw ? a.sw[n] : 1.0f);
    }
}

// ---------------------------------------------------------------- host

namespace {

template <int MT, int R>
cudaError_t launch_dot(const I8Args &a, cudaStream_t stream)
{
    void *args[] = {(void *)&a};
    const dim3 grid((unsigned)((a.N + 4 * R - 1) / (4 * R)), (unsigned)((a.M + MT - 1) / MT));
    const void *k = a.al_a && a.al_w ? (const void *)gemm_i8_dot_kernel<MT, R, false>
                                     : (const void *)gemm_i8_dot_kernel<MT, R, true>;
    return launch_first(k, grid, dim3(32 * kFwWarps), args, 0, stream);
}

template <int NB, int MB>
cudaError_t launch_few(const I8Args &a, cudaStream_t stream)
{
    void *args[] = {(void *)&a};
    const dim3 grid((unsigned)((a.N + 16 * MB - 1) / (16 * MB)), (unsigned)((a.M + 8 * NB - 1) / (8 * NB)));
    const void *k = a.al_a && a.al_w ? (const void *)gemm_i8_few_kernel<NB, MB, false>
                                     : (const void *)gemm_i8_few_kernel<NB, MB, true>;
    return launch_first(k, grid, dim3(32 * kFwWarps), args, 0, stream);
}

}  // namespace

cudaError_t launch_gemm_i8_few(const I8Args &a, cudaStream_t stream)
{
    if (a.M <= 1) return launch_dot<1, 2>(a, stream);
    if (a.M <= 2) return launch_dot<2, 2>(a, stream);
    // 32 channels a CTA where that still gives every SM one (16 x 8192 x
    // 8192: 18.6 us, 28.5 with 16), else 16 (8 x 4096 x 4096: 7.8 us, 11.6
    // with 32)
    const bool wide = a.N > 152 * 32;
    if (a.M <= 8) return wide ? launch_few<1, 2>(a, stream) : launch_few<1, 1>(a, stream);
    if (wide) return launch_few<2, 2>(a, stream);
    return a.M <= 16 ? launch_few<2, 1>(a, stream) : launch_few<4, 1>(a, stream);
}

}  // namespace tcr
