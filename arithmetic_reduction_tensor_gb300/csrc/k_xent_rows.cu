// k_xent_rows.cu -- the passes over tokens around the products of the softmax
// cross entropy: the compact copy of the tokens that count, the loss from the
// tiles' parts, dX from its sums.
//
// Copying the tokens costs 4 bytes an element of X where the products cost 2 V
// operations or more; for it, ignored tokens cost nothing afterwards and what
// they hold (NaN included) reaches no sum, and X may have any pitch and
// alignment.  All are bound by memory traffic, or, for few tokens, by latency.
#include "kernels.cuh"
#include "plan.h"
#include "rowvec.cuh"
#include "xent.h"

namespace tcr {

constexpr int kTokThreads = 256, kTokWarps = kTokThreads / 32;
constexpr int kTokTail = 8;            // CTAs that count all tokens, and zero the rows behind the last (2 to 32: alike)

// The live tokens among [0, n).
__device__ __forceinline__ int count_live(const XentTokens &a, size_t n, int *red)
{
    int c = 0;
#pragma unroll 8
    for (size_t i = threadIdx.x; i < n; i += kTokThreads) c += a.target[i] != a.ignore;
    c = __reduce_add_sync(kFull, c);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = c;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kTokWarps; w++) s += red[w];
    __syncthreads();
    return s;
}

// One row by a warp, to a 16-byte aligned one of whole vectors; unaligned rows as
// the granules that hold their elements, shifted in registers (by elements a
// 5003 x 1001 matrix took 9.0 us instead of 5).
template <bool GRAN>
__device__ __forceinline__ void copy_row(const uint16_t *src, uint16_t *dst, uint32_t H)
{
    constexpr int kAtOnce = 8;       // (the loss of 16 x 4095 over 131072 549 us; 4 547, 2 and 16 581)
    const uint32_t lane = threadIdx.x & 31, nvec = (H + kRv - 1) / kRv;
    for (uint32_t v0 = lane; v0 < nvec + lane; v0 += 32 * kAtOnce) {     // (the same steps in every lane)
        LoadedVec<kBF16, GRAN> l[kAtOnce];
#pragma unroll
        for (uint32_t k = 0; k < kAtOnce; k++) l[k] = load_vec<kBF16, GRAN>(src, H, v0 + 32 * k);
#pragma unroll
        for (uint32_t k = 0; k < kAtOnce; k++)
            if (v0 + 32 * k < nvec)
                reinterpret_cast<uint4 *>(dst)[v0 + 32 * k] = use_vec<kBF16, GRAN>(l[k], src, H, v0 + 32 * k).q[0];
    }
}

// CTA b takes tokens [b chunk, (b + 1) chunk): their rows in the copy follow
// from the count of those before, which each CTA takes itself (a scan would
// be a launch more).  CTAs past those and the tail copy W where it has to be
// copied.
__global__ void __launch_bounds__(kTokThreads) xent_tokens_kernel(const XentTokens a, size_t chunk, unsigned blocks)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ int red[kTokWarps];
    __shared__ int ranks[kTokThreads];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x >= blocks + kTokTail) {
        const size_t step = (size_t)(gridDim.x - blocks - kTokTail) * kTokWarps;
        for (size_t r = (size_t)(blockIdx.x - blocks - kTokTail) * kTokWarps + warp; r < a.V; r += step)
            copy_row<true>((const uint16_t *)a.w + r * a.ldw, a.W + r * a.ldX, (uint32_t)a.H);
        return;
    }
    if (blockIdx.x >= blocks) {
        const unsigned part = blockIdx.x - blocks;
        const int n = count_live(a, a.tokens, red);
        const size_t end = ((size_t)n + 63) / 64 * 64;
        for (size_t r = (size_t)n + part * kTokWarps + warp; r < end; r += kTokTail * kTokWarps)
            for (size_t v = lane; v < a.ldX / 8; v += 32)
                reinterpret_cast<uint4 *>(a.X + r * a.ldX)[v] = make_uint4(0u, 0u, 0u, 0u);
        if (part != 0) return;
        unsigned int m = 0;
        if (a.dloss) {
#pragma unroll 8
            for (size_t i = threadIdx.x; i < a.tokens; i += kTokThreads)
                if (a.target[i] != a.ignore) {
                    const unsigned int b = __float_as_uint(a.dloss[i * a.inc_dloss]) & 0x7fffffffu;
                    if (b < 0x7f800000u) m = max(m, b);
                }
            m = __reduce_max_sync(kFull, m);
            if (lane == 0) red[warp] = (int)m;
            __syncthreads();
            for (int w = 0; w < kTokWarps; w++) m = max(m, (unsigned int)red[w]);
        }
        if (threadIdx.x == 0) {
            a.head[0] = (unsigned int)n;
            a.head[1] = m;
        }
        return;
    }
    const size_t first = (size_t)blockIdx.x * chunk, last = min(first + chunk, a.tokens);
    int base = count_live(a, first, red);
    for (size_t t0 = first; t0 < last; t0 += kTokThreads) {          // kTokThreads tokens at a time
        const size_t t = t0 + threadIdx.x;
        const long long y = t < last ? a.target[t] : a.ignore;
        const bool live = t < last && y != a.ignore;
        const unsigned mask = __ballot_sync(kFull, live);
        if (lane == 0) red[warp] = __popc(mask);
        __syncthreads();
        int r = base, all = 0;
#pragma unroll
        for (int w = 0; w < kTokWarps; w++) {
            if (w < (int)warp) r += red[w];
            all += red[w];
        }
        r += __popc(mask & ((1u << lane) - 1u));
        ranks[threadIdx.x] = live ? r : -1;
        if (t < last) a.rank[t] = live ? r : -1;
        if (live) {
            a.lab[r] = xent_label(y, a.V);
            a.tok[r] = (int)t;
        }
        __syncthreads();
        const int here = (int)min(last - t0, (size_t)kTokThreads);
        for (int i = (int)warp; i < here; i += kTokWarps) {
            const int to = ranks[i];
            if (to < 0) continue;
            const uint16_t *row = (const uint16_t *)a.x + (t0 + i) * a.ldx;
            if (a.al_x)
                copy_row<false>(row, a.X + (size_t)to * a.ldX, (uint32_t)a.H);
            else
                copy_row<true>(row, a.X + (size_t)to * a.ldX, (uint32_t)a.H);
        }
        base += all;
        __syncthreads();
    }
}

// Four tokens a CTA (32 bytes of each part's row), 64 threads a token over the
// parts.  With M the largest logit, h the target's and A the sum of exp(l - M) over
// the others,
//   lse = M + log1p(A),  loss = (M - h) + log1p(A).
// The loss is not lse - h: that difference of two numbers as large as the logits
// would leave a token that is predicted well (A << 1, h = M) no bit of its loss.
constexpr int kLossTokens = 4, kLossThreads = 256, kLossSlices = kLossThreads / kLossTokens;
template <bool NARROW>
__global__ void __launch_bounds__(kLossThreads) xent_loss_kernel(const XentLoss a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[3][kLossThreads / 32][kLossTokens];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = threadIdx.x % kLossTokens;
    const size_t t = (size_t)blockIdx.x * kLossTokens + k;
    const int first = (int)threadIdx.x / kLossTokens;
    int r = -1, lab = -1;
    if (t < a.tokens) {
        if (a.rank) {
            r = a.rank[t];
            if (r >= 0) lab = a.lab[r];
        } else {
            const long long y = a.target[t];
            if (y != a.ignore) r = (int)t;
            lab = xent_label(y, a.V);
        }
    }
    float m = -INFINITY, s = 0.0f, tops = 0.0f;
    // part j of 128 entries; narrow ones, each absent one -infinity, joined as the wide tiles' are
    const int parts = NARROW ? (a.parts + 1) / 2 : a.parts;
    auto part = [&](int j) {
        if constexpr (!NARROW) return a.part[(size_t)j * a.tpad + r];
        const float2 p = a.part[(size_t)(2 * j) * a.tpad + r];
        return xent_join(p, 2 * j + 1 < a.parts ? a.part[(size_t)(2 * j + 1) * a.tpad + r] : make_float2(-INFINITY, 0.0f));
    };
    if (r >= 0) {
        // two passes over the parts (8 bytes for 128 logits): the largest, then the sum about it
#pragma unroll 8
        for (int j = first; j < parts; j += kLossSlices) m = fmaxf(m, part(j).x);
    }
#pragma unroll
    for (int h = kLossTokens; h < 32; h *= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, h));
    if (lane < kLossTokens) red[0][warp][k] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLossThreads / 32; w++) m = fmaxf(m, red[0][w][k]);
    const float about = xent_about(m);
    if (r >= 0) {
#pragma unroll 8
        for (int j = first; j < parts; j += kLossSlices) {
            const float2 p = part(j);
            const float w = exp2f(__fmul_rn(__fsub_rn(p.x, about), kLog2e));
            // the part's largest counts beside its others, but for one that is M
            if (p.x == m)
                tops += 1.0f;
            else
                s = __fadd_rn(s, w);
            s = __fmaf_rn(p.y, w, s);
        }
    }
#pragma unroll
    for (int h = kLossTokens; h < 32; h *= 2) {
        s = __fadd_rn(s, __shfl_xor_sync(kFull, s, h));
        tops = __fadd_rn(tops, __shfl_xor_sync(kFull, tops, h));
    }
    if (lane < kLossTokens) {
        red[1][warp][k] = s;
        red[2][warp][k] = tops;
    }
    __syncthreads();
    if (threadIdx.x >= kLossTokens || t >= a.tokens) return;
    float loss = 0.0f, lse = 0.0f;
    if (r >= 0) {
        s = 0.0f;
        tops = -1.0f;
#pragma unroll
        for (int w = 0; w < kLossThreads / 32; w++) {
            s = __fadd_rn(s, red[1][w][k]);
            tops = __fadd_rn(tops, red[2][w][k]);
        }
        const float log_s = log1pf(__fadd_rn(s, tops));
        lse = __fadd_rn(m, log_s);
        loss = lab < 0 ? __int_as_float(0x7fc00000) : __fadd_rn(__fsub_rn(m, a.hit[r]), log_s);
    }
    a.loss[t] = loss;
    if (a.lse) a.lse[t] = lse;
}

// A CTA takes 1024 columns of a token, four a thread.
template <int DT>
__global__ void __launch_bounds__(256) xent_dx_kernel(const XentDx a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    const size_t j = (size_t)blockIdx.y * 1024 + 4 * threadIdx.x;
    if (j >= a.H) return;
    float scale = __uint_as_float(a.head[1]);
    if (DT == kF16) scale = __fmul_rn(scale, 1.0f / kXentF16Scale);
    for (size_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const int r = a.rank[t];
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r >= 0) {
            const float *p = a.ws + (size_t)r * a.ldws + j;
#pragma unroll 4
            for (int k = 0; k < a.splits; k++) {
                const float4 f = *reinterpret_cast<const float4 *>(p + (size_t)k * a.tpad * a.ldws);
                s = make_float4(__fadd_rn(s.x, f.x), __fadd_rn(s.y, f.y), __fadd_rn(s.z, f.z), __fadd_rn(s.w, f.w));
            }
            s = make_float4(__fmul_rn(s.x, scale), __fmul_rn(s.y, scale), __fmul_rn(s.z, scale), __fmul_rn(s.w, scale));
        }
        const uint32_t lo = float2_to_word<DT>(s.x, s.y), hi = float2_to_word<DT>(s.z, s.w);
        uint16_t *out = (uint16_t *)a.dx + t * a.lddx + j;
        if (a.al_dx && j + 4 <= a.H) {
            *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
        } else {
            out[0] = (uint16_t)lo;
            if (j + 1 < a.H) out[1] = (uint16_t)(lo >> 16);
            if (j + 2 < a.H) out[2] = (uint16_t)hi;
            if (j + 3 < a.H) out[3] = (uint16_t)(hi >> 16);
        }
    }
}

// ---------------------------------------------------------------- host

cudaError_t launch_xent_tokens(const XentTokens &a, cudaStream_t stream)
{
    // about a thousand CTAs at most: each reads the targets before its own
    size_t chunk = (a.tokens + 1023) / 1024;
    if (chunk < kTokWarps) chunk = kTokWarps;
    unsigned blocks = (unsigned)((a.tokens + chunk - 1) / chunk);
    const size_t need = (a.V + kTokWarps - 1) / kTokWarps, most = (size_t)plan::kRuleSMs * 8;
    const unsigned repack = a.w ? (unsigned)(need < most ? need : most) : 0u;
    void *args[] = {(void *)&a, (void *)&chunk, (void *)&blocks};
    return launch_first((const void *)xent_tokens_kernel, dim3(blocks + kTokTail + repack), dim3(kTokThreads), args, 0,
                        stream);
}

cudaError_t launch_xent_loss(const XentLoss &a, cudaStream_t stream)
{
    void *args[] = {(void *)&a};
    const void *k = a.narrow ? (const void *)xent_loss_kernel<true> : (const void *)xent_loss_kernel<false>;
    return launch_first(k, dim3((unsigned)((a.tokens + kLossTokens - 1) / kLossTokens)),
                        dim3(kLossThreads), args, 0, stream);
}

cudaError_t launch_xent_dx(int dtype, const XentDx &a, cudaStream_t stream)
{
    void *args[] = {(void *)&a};
    const size_t gy = (a.H + 1023) / 1024, most = (size_t)plan::kRuleSMs * 32;
    const dim3 grid((unsigned)(a.tokens < most ? a.tokens : most), (unsigned)gy);
    return launch_first(dtype == kF16 ? (const void *)xent_dx_kernel<kF16> : (const void *)xent_dx_kernel<kBF16>, grid,
                        dim3(256), args, 0, stream);
}

}  // namespace tcr
