// xent.h -- the softmax cross entropy over a vocabulary: what its products
// (k_xent.cu), its passes over tokens (k_xent_rows.cu) and its entry points
// (tcr_train.cu) share.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace tcr {

constexpr int kXentChain = 16384;           // K of dX and dW that the tensor cores add up in one chain
constexpr int kXentTile = 256;             // tokens and vocabulary entries (or columns) of a tile
constexpr int kXentForward = 0, kXentGradient = 1, kXentBack = 2, kXentBackLong = 3;
constexpr float kXentF16Scale = 32768.0f;  // of P in binary16

// A target as an entry of the vocabulary, -1 where there is no such entry.
__host__ __device__ inline int xent_label(long long y, size_t V)
{
    return y >= 0 && y < (long long)V ? (int)y : -1;
}

#ifdef __CUDACC__
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What logits are taken about: their largest, m, but 0 where there is none.
__device__ __forceinline__ float xent_about(float m)
{
    return m == -INFINITY ? 0.0f : m;
}

// exp(l - about).
__device__ __forceinline__ float xent_exp(float l, float about)
{
    return ex2(__fmul_rn(__fsub_rn(l, about), kLog2e));
}

// Two parts of the vocabulary (largest logit, sum of the others about it) as one.
// A tile of 256 columns joins its parts of 64 in the epilogue, the parts of narrow
// tiles are joined where they are read: the same bits.
__device__ __forceinline__ float2 xent_join(float2 a, float2 b)
{
    const bool first = a.x >= b.x;
    const float2 hi = first ? a : b, lo = first ? b : a;
    return make_float2(hi.x, __fmaf_rn(__fadd_rn(lo.y, 1.0f), xent_exp(lo.x, xent_about(hi.x)), hi.y));
}
#endif

// The tokens that count, in their order: n of them, then at least zeros up to
// a multiple of 64 rows of X.
struct XentTokens {
    const void *x;
    size_t ldx;
    const long long *target;
    size_t tokens, H, V;
    long long ignore;
    bool al_x;
    const float *dloss;        // null in the forward pass
    size_t inc_dloss;
    // outputs
    uint16_t *X;               // the compact copy, ldX elements a row
    size_t ldX;
    const void *w;             // W to be copied to rows of ldX elements at W; null: not
    size_t ldw;
    uint16_t *W;
    int *lab, *tok, *rank;     // by compact row: label (-1: no entry of the vocabulary), token; by token: its row or -1
    unsigned int *head;        // n, and the bits of those tokens' largest finite |dloss|
};
cudaError_t launch_xent_tokens(const XentTokens &a, cudaStream_t stream);

struct XentGemm {
    const unsigned int *head;  // null: all of n tokens, their labels from target (the forward pass of few)
    int n;
    const long long *target;
    const int *lab, *tok;
    size_t tpad;               // rows of X, P, part and ws
    int V, H;
    int v0, vn;                // the piece of the vocabulary (the forward pass: all of it)
    // forward
    float2 *part;              // [part of the vocabulary][row]: largest logit, sum of the others about it
    float *hit;                // the target's logit
    // gradient
    const float *lse, *dloss;
    size_t inc_dloss;
    uint16_t *P;
    size_t ldp;
    // back
    float *ws;                 // [split][row][ldws]; null: dX not wanted
    size_t ldws;
    int splits, first;
    void *dw;                  // null: not wanted
    size_t lddw;
    bool al_dw;
    uint32_t inject_stall;     // withhold the first tile's publication (tests of the failure path)
};
// Read maps of X, W and P, in boxes of 64 rows or of the number named; write maps of P, of dX's sums (rows of all splits) and of dW.
struct XentMaps {
    CUtensorMap x, x128, w, w128, w32, p, p128, p_out, ws_out, dw_out;
};
int xent_pairs();
cudaError_t xent_map(CUtensorMap *map, const void *base, size_t cols, size_t rows, size_t ld, int box_rows,
                     bool wide = false);
// Columns of the logits' tiles over vn entries of the vocabulary, 256 or 64, and of a part.
int xent_tile_cols(size_t tokens, size_t vn, int pairs);
inline int xent_part_cols(int tile_cols) { return tile_cols < 128 ? tile_cols : 128; }
cudaError_t launch_xent(int dtype, int mode, const XentMaps &maps, const XentGemm &g, size_t units, int pairs,
                        int tile_cols, cudaStream_t stream);

// loss and lse of every token from its tiles' parts.
struct XentLoss {
    const float2 *part;
    const float *hit;
    const int *rank, *lab;     // null: as of target
    const long long *target;
    long long ignore;
    size_t tpad, tokens, V;
    int parts;
    bool narrow;               // parts of 64 entries, to be joined two by two
    float *loss, *lse;         // lse may be null
};
cudaError_t launch_xent_loss(const XentLoss &a, cudaStream_t stream);

// dX of every token from the splits' sums; tokens that do not count 0.
struct XentDx {
    const float *ws;
    size_t tpad, ldws;
    int splits;
    const int *rank;
    const unsigned int *head;
    size_t tokens, H;
    void *dx;
    size_t lddx;
    bool al_dx;
};
cudaError_t launch_xent_dx(int dtype, const XentDx &a, cudaStream_t stream);

cudaError_t read_xent_faults(unsigned int *flags, bool clear);

}  // namespace tcr
