// tcr_train.cu -- the C ABI of dropout, the layer norm and its gradient, and
// the softmax cross entropy over a vocabulary and its gradient.  Argument
// checks, then scratch from the library's pool and the launches.
#include <cmath>

#include "../../include/tcr.h"
#include "args.h"
#include "kernels.cuh"
#include "xent.h"

using namespace tcr;
using namespace tcr::plan;

namespace {

constexpr size_t kMaxTokens = (size_t)1 << 24;     // exclusive, as the next two
constexpr size_t kMaxVocab = (size_t)1 << 27;
constexpr size_t kMaxHidden = (size_t)1 << 20;
constexpr size_t kMaxP = (size_t)512 << 20;        // bytes of P in a piece of the vocabulary
constexpr size_t kSplitPairs = kRuleSMs / 2;                 // pairs that dX is split for: a constant, as its splits are its sums' order

// The kernel's form of a call's dropout; none where drop is null.
bool drop_of(const tcr_drop *drop, DropArgs &d)
{
    d = {};
    if (!drop) return true;
    if (!(drop->p >= 0.0 && drop->p <= 1.0) || !is_aligned(drop->state, 8)) return false;
    d.t = (uint32_t)std::nearbyint(65536.0 * drop->p);
    d.s = d.t < 65536u ? (float)(65536.0 / (65536.0 - d.t)) : 0.0f;
    for (uint32_t i = 0; i < 10; i++) {
        d.rk[2 * i] = (uint32_t)drop->seed + i * kPhiloxW0;
        d.rk[2 * i + 1] = (uint32_t)(drop->seed >> 32) + i * kPhiloxW1;
    }
    d.c2 = (uint32_t)drop->offset;
    d.c3 = (uint32_t)(drop->offset >> 32);
    d.state = drop->state;
    return true;
}

size_t round_up(size_t n, size_t to)
{
    return (n + to - 1) / to * to;
}

// What the two passes of the cross entropy have in common.
struct XentSizes {
    size_t T, V, H, tpad, ldX;
    int tiles_t;
    bool repack;
};

tcr_status xent_check(const void *x, size_t ldx, const void *w, size_t ldw, const long long *target, size_t T, size_t V,
                      size_t H, int dtype)
{
    if (dtype != TCR_F16 && dtype != TCR_BF16) return TCR_ERR_INVALID_ARG;
    if (T >= kMaxTokens || V >= kMaxVocab || H >= kMaxHidden) return TCR_ERR_UNSUPPORTED;
    if (T * V >= kMaxInputs || V * H >= kMaxInputs || V == 0 || H == 0) return TCR_ERR_INVALID_ARG;
    if (T > 0 && (!matrix_ok(x, ldx, T, H, dtype, true) || !target || !is_aligned(target, 8)))
        return TCR_ERR_INVALID_ARG;
    // W may be one row for all only if it is one row
    if (!matrix_ok(w, ldw, V, H, dtype, false)) return TCR_ERR_INVALID_ARG;
    return TCR_OK;
}

XentSizes xent_sizes(const void *w, size_t ldw, size_t T, size_t V, size_t H)
{
    XentSizes z;
    z.T = T;
    z.V = V;
    z.H = H;
    z.tpad = round_up(T, kXentTile);
    z.tiles_t = (int)(z.tpad / kXentTile);
    z.ldX = round_up(H, 8);
    z.repack = !rows_aligned(w, ldw, V, 2);
    return z;
}

// Parts of one allocation, each on a 256-byte boundary.
struct Parts {
    size_t bytes = 0;
    size_t add(size_t n)
    {
        const size_t at = bytes;
        bytes += round_up(n, 256);
        return at;
    }
};

struct XentCommon {
    size_t X, W, lab, tok, rank, head;
    void place(Parts &p, const XentSizes &z)
    {
        X = p.add(z.tpad * z.ldX * 2);
        W = p.add(z.repack ? z.V * z.ldX * 2 : 0);
        lab = p.add(z.tpad * 4);
        tok = p.add(z.tpad * 4);
        rank = p.add(z.T * 4);
        head = p.add(8);
    }
};

// The maps of X (rows of ldx elements) and W; those of the gradient are not used.
cudaError_t xent_read_maps(XentMaps &maps, const void *x, size_t ldx, size_t rows, const void *w, size_t ldw,
                           const XentSizes &z)
{
    cudaError_t e = xent_map(&maps.x, x, z.H, rows, ldx, 64);
    if (e == cudaSuccess) e = xent_map(&maps.x128, x, z.H, rows, ldx, 128);
    if (e == cudaSuccess) e = xent_map(&maps.w, w, z.H, z.V, ldw, 64);
    if (e == cudaSuccess) e = xent_map(&maps.w128, w, z.H, z.V, ldw, 128);
    if (e == cudaSuccess) e = xent_map(&maps.w32, w, z.H, z.V, ldw, 32);
    maps.p = maps.p128 = maps.p_out = maps.ws_out = maps.dw_out = maps.x;
    return e;
}

// The tokens' compact copy, W where it has to be copied, and the tensor maps.
cudaError_t xent_prepare(XentTokens &k, const XentSizes &z, const XentCommon &c, char *base, const void *w, size_t ldw,
                         XentMaps &maps, cudaStream_t s)
{
    k.X = (uint16_t *)(base + c.X);
    k.ldX = z.ldX;
    k.lab = (int *)(base + c.lab);
    k.tok = (int *)(base + c.tok);
    k.rank = (int *)(base + c.rank);
    k.head = (unsigned int *)(base + c.head);
    if (z.repack) {
        k.w = w;
        k.ldw = ldw;
        k.W = (uint16_t *)(base + c.W);
        w = base + c.W;
        ldw = z.ldX;
    } else if (z.V == 1) {
        ldw = z.ldX;            // not looked at by the caller; the map wants a pitch
    }
    cudaError_t e = launch_xent_tokens(k, s);
    return e == cudaSuccess ? xent_read_maps(maps, k.X, z.ldX, z.tpad, w, ldw, z) : e;
}

}  // namespace

extern "C" {

tcr_status tcr_dropout(const void *x, size_t ldx, const void *residual, size_t ldr, void *y, size_t ldy, size_t rows,
                       size_t cols, const tcr_drop *drop, int dtype, void *stream)
{
    LayerArgs a = {};
    if (!is_float(dtype) || !sizes_ok(rows, cols) || !drop || !drop_of(drop, a.drop)) return TCR_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return TCR_OK;
    if (!matrix_ok(x, ldx, rows, cols, dtype, true) || !matrix_ok(y, ldy, rows, cols, dtype, false) ||
        (residual && !matrix_ok(residual, ldr, rows, cols, dtype, true)))
        return TCR_ERR_INVALID_ARG;
    if (current_device() < 0 || fault_injected("launch")) return TCR_ERR_CUDA;
    const size_t eb = elem_bytes(dtype);
    a.x = x;
    a.ldx = ldx;
    a.r = residual;
    a.ldr = ldr;
    a.y = y;
    a.ldy = ldy;
    a.rows = rows;
    a.cols = cols;
    a.al_x = rows_aligned(x, ldx, rows, eb);
    a.al_r = rows_aligned(residual, ldr, rows, eb);
    a.al_y = rows_aligned(y, ldy, rows, eb);
    return of(launch_dropout(dtype, a, (cudaStream_t)stream));
}

tcr_status tcr_layernorm(const tcr_layernorm_args *args, void *stream)
{
    if (!args) return TCR_ERR_INVALID_ARG;
    const tcr_layernorm_args &a = *args;
    LayerArgs r = {};
    if (!is_float(a.dtype) || (a.y_dtype != a.dtype && a.y_dtype != TCR_I8)) return TCR_ERR_INVALID_ARG;
    if (!(a.eps >= 0.0f) || std::isinf(a.eps) || !sizes_ok(a.rows, a.cols) || !drop_of(a.drop, r.drop))
        return TCR_ERR_INVALID_ARG;
    if (a.rows == 0) return TCR_OK;
    const size_t eb = elem_bytes(a.dtype);
    if (a.cols > 0) {
        if (!matrix_ok(a.x, a.ldx, a.rows, a.cols, a.dtype, true) ||
            !matrix_ok(a.y, a.ldy, a.rows, a.cols, a.y_dtype, false))
            return TCR_ERR_INVALID_ARG;
        if (a.residual && !matrix_ok(a.residual, a.ldr, a.rows, a.cols, a.dtype, true)) return TCR_ERR_INVALID_ARG;
        if (a.h && !matrix_ok(a.h, a.ldh, a.rows, a.cols, a.dtype, false)) return TCR_ERR_INVALID_ARG;
        if (!is_aligned(a.weight, eb) || !is_aligned(a.bias, eb)) return TCR_ERR_INVALID_ARG;
    }
    if ((a.y_dtype == TCR_I8 && !floats_ok(a.scale)) || !is_aligned(a.mean, 4) || !is_aligned(a.rstd, 4))
        return TCR_ERR_INVALID_ARG;
    if (current_device() < 0 || fault_injected("launch")) return TCR_ERR_CUDA;
    r.x = a.x;
    r.ldx = a.ldx;
    r.r = a.residual;
    r.ldr = a.ldr;
    r.w = a.weight;
    r.b = a.bias;
    r.h = a.h;
    r.ldh = a.ldh;
    r.y = a.y;
    r.ldy = a.ldy;
    r.scale = a.y_dtype == TCR_I8 ? a.scale : nullptr;
    r.mean = a.mean;
    r.rstd = a.rstd;
    r.eps = a.eps;
    r.rows = a.rows;
    r.cols = a.cols;
    r.al_x = rows_aligned(a.x, a.ldx, a.rows, eb);
    r.al_r = rows_aligned(a.residual, a.ldr, a.rows, eb);
    r.al_w = is_aligned(a.weight, 16);
    r.al_b = is_aligned(a.bias, 16);
    r.al_h = rows_aligned(a.h, a.ldh, a.rows, eb);
    r.al_y = a.y_dtype == TCR_I8 ? rows_aligned(a.y, a.ldy, a.rows, 1, 8) : rows_aligned(a.y, a.ldy, a.rows, eb);
    return of(launch_layer(a.dtype, r, (cudaStream_t)stream));
}

tcr_status tcr_layernorm_backward(const tcr_layernorm_back_args *args, void *stream)
try {
    if (!args) return TCR_ERR_INVALID_ARG;
    const tcr_layernorm_back_args &a = *args;
    LayerBackArgs b = {};
    if (!is_float(a.dtype) || !sizes_ok(a.rows, a.cols) || !drop_of(a.drop, b.drop)) return TCR_ERR_INVALID_ARG;
    if (!is_aligned(a.dweight, 4) || !is_aligned(a.dbias, 4)) return TCR_ERR_INVALID_ARG;
    if (a.cols == 0) return TCR_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const int dev = current_device();
    if (a.rows == 0) {
        if (!a.dweight && !a.dbias) return TCR_OK;
        if (dev < 0 || fault_injected("launch")) return TCR_ERR_CUDA;
        cudaError_t e = a.dweight ? cudaMemsetAsync(a.dweight, 0, a.cols * sizeof(float), s) : cudaSuccess;
        if (e == cudaSuccess && a.dbias) e = cudaMemsetAsync(a.dbias, 0, a.cols * sizeof(float), s);
        return of(e);
    }
    const size_t eb = elem_bytes(a.dtype);
    if (!matrix_ok(a.dy, a.lddy, a.rows, a.cols, a.dtype, true) ||
        !matrix_ok(a.h, a.ldh, a.rows, a.cols, a.dtype, true) || !floats_ok(a.mean) || !floats_ok(a.rstd))
        return TCR_ERR_INVALID_ARG;
    if ((a.dh && !matrix_ok(a.dh, a.lddh, a.rows, a.cols, a.dtype, true)) ||
        (a.dx && !matrix_ok(a.dx, a.lddx, a.rows, a.cols, a.dtype, false)) ||
        (a.dresidual && !matrix_ok(a.dresidual, a.lddr, a.rows, a.cols, a.dtype, false)) || !is_aligned(a.weight, eb))
        return TCR_ERR_INVALID_ARG;
    if (!a.dx && !a.dresidual && !a.dweight && !a.dbias) return TCR_OK;
    if (dev < 0) return TCR_ERR_CUDA;
    Scratch scratch(s);
    tcr_status st = scratch.take(layer_back_scratch(a.rows, a.cols, a.dtype, a.dweight, a.dbias), dev);
    if (st != TCR_OK) return st;
    if (fault_injected("launch")) return TCR_ERR_CUDA;
    b.dy = a.dy;
    b.lddy = a.lddy;
    b.h = a.h;
    b.ldh = a.ldh;
    b.w = a.weight;
    b.mean = a.mean;
    b.rstd = a.rstd;
    b.dh = a.dh;
    b.lddh = a.lddh;
    b.dx = a.dx;
    b.lddx = a.lddx;
    b.dr = a.dresidual;
    b.lddr = a.lddr;
    b.rows = a.rows;
    b.cols = a.cols;
    b.al_dy = rows_aligned(a.dy, a.lddy, a.rows, eb);
    b.al_h = rows_aligned(a.h, a.ldh, a.rows, eb);
    b.al_w = is_aligned(a.weight, 16);
    b.al_dh = rows_aligned(a.dh, a.lddh, a.rows, eb);
    b.al_dx = rows_aligned(a.dx, a.lddx, a.rows, eb);
    b.al_dr = rows_aligned(a.dresidual, a.lddr, a.rows, eb);
    cudaError_t e = launch_layer_back(a.dtype, b, (float *)scratch.p, a.dweight, a.dbias, s);
    const cudaError_t f = scratch.release();
    return of(e == cudaSuccess ? f : e);
} catch (...) {         // the host's memory for a cache: nothing may cross the C boundary
    return TCR_ERR_CUDA;
}

tcr_status tcr_cross_entropy(const tcr_xent_args *args, void *stream)
try {
    if (!args) return TCR_ERR_INVALID_ARG;
    const tcr_xent_args &a = *args;
    tcr_status st = xent_check(a.x, a.ldx, a.weight, a.ldw, a.target, a.tokens, a.vocab, a.hidden, a.dtype);
    if (st != TCR_OK) return st;
    if (a.tokens == 0) return TCR_OK;
    if (!floats_ok(a.loss) || !is_aligned(a.lse, 4)) return TCR_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return TCR_ERR_CUDA;
    const int pairs = xent_pairs();
    if (pairs < 1) return pairs < 0 ? TCR_ERR_CUDA : TCR_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    const XentSizes z = xent_sizes(a.weight, a.ldw, a.tokens, a.vocab, a.hidden);
    const int tile = xent_tile_cols(z.T, z.V, pairs);
    const size_t tiles_v = (z.V + (size_t)tile - 1) / (size_t)tile;
    const size_t n_parts = tiles_v * (size_t)(tile / xent_part_cols(tile));
    // One tile of tokens, aligned: X is read where it lies, ignored tokens or not
    // (nothing of theirs reaches another token's row), and the launch that copies
    // is saved (64 tokens x 64 over 1000 10.7 -> 8.6 us, x 1024 14.0 -> 11.2).
    const bool al_x = rows_aligned(a.x, a.ldx, z.T, 2);
    const bool direct = z.T <= (size_t)kXentTile && !z.repack && al_x && (z.T == 1 || a.ldx >= z.H);
    Parts parts;
    XentCommon c;
    if (!direct) c.place(parts, z);
    const size_t at_part = parts.add(n_parts * z.tpad * sizeof(float2)), at_hit = parts.add(z.tpad * 4);
    Scratch scratch(s);
    if ((st = scratch.take(parts.bytes, dev)) != TCR_OK) return st;
    if (fault_injected("launch")) return TCR_ERR_CUDA;
    char *base = (char *)scratch.p;
    XentTokens k = {};
    XentMaps maps;
    cudaError_t e;
    if (direct) {
        e = xent_read_maps(maps, a.x, z.T == 1 ? z.ldX : a.ldx, z.T, a.weight, z.V == 1 ? z.ldX : a.ldw, z);
    } else {
        k.x = a.x;
        k.ldx = a.ldx;
        k.target = a.target;
        k.tokens = z.T;
        k.H = z.H;
        k.V = z.V;
        k.ignore = a.ignore_index;
        k.al_x = al_x;
        e = xent_prepare(k, z, c, base, a.weight, a.ldw, maps, s);
    }
    if (e == cudaSuccess) {
        XentGemm g = {};
        g.head = k.head;
        g.n = (int)z.T;
        g.target = a.target;
        g.lab = k.lab;
        g.tok = k.tok;
        g.tpad = z.tpad;
        g.V = g.vn = (int)z.V;
        g.H = (int)z.H;
        g.part = (float2 *)(base + at_part);
        g.hit = (float *)(base + at_hit);
        g.inject_stall = fault_injected("stall");
        e = launch_xent(a.dtype, kXentForward, maps, g, (size_t)z.tiles_t * tiles_v, pairs, tile, s);
        if (e == cudaSuccess) {
            XentLoss l = {g.part, g.hit,  k.rank, k.lab,        a.target, a.ignore_index,
                          z.tpad, z.T, z.V,    (int)n_parts, tile == 64, a.loss, a.lse};
            e = launch_xent_loss(l, s);
        }
    }
    const cudaError_t f = scratch.release();
    return of(e == cudaSuccess ? f : e);
} catch (...) {
    return TCR_ERR_CUDA;
}

tcr_status tcr_cross_entropy_backward(const tcr_xent_back_args *args, void *stream)
try {
    if (!args) return TCR_ERR_INVALID_ARG;
    const tcr_xent_back_args &a = *args;
    tcr_status st = xent_check(a.x, a.ldx, a.weight, a.ldw, a.target, a.tokens, a.vocab, a.hidden, a.dtype);
    if (st != TCR_OK) return st;
    if (a.inc_dloss > 1 || (a.dweight && !matrix_ok(a.dweight, a.lddw, a.vocab, a.hidden, a.dtype, false)))
        return TCR_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (a.tokens == 0) {
        if (!a.dweight) return TCR_OK;
        if (current_device() < 0 || fault_injected("launch")) return TCR_ERR_CUDA;
        return of(cudaMemset2DAsync(a.dweight, (a.vocab == 1 ? a.hidden : a.lddw) * 2, 0, a.hidden * 2, a.vocab, s));
    }
    if (!floats_ok(a.lse) || !floats_ok(a.dloss) || (a.dx && !matrix_ok(a.dx, a.lddx, a.tokens, a.hidden, a.dtype, false)))
        return TCR_ERR_INVALID_ARG;
    if (!a.dx && !a.dweight) return TCR_OK;
    const int dev = current_device();
    if (dev < 0) return TCR_ERR_CUDA;
    const int pairs = xent_pairs();
    if (pairs < 1) return pairs < 0 ? TCR_ERR_CUDA : TCR_ERR_UNSUPPORTED;
    const XentSizes z = xent_sizes(a.weight, a.ldw, a.tokens, a.vocab, a.hidden);
    // the piece of the vocabulary: equal ones, as few as kMaxP allows
    const size_t vpad = round_up(z.V, kXentTile);
    size_t most = kMaxP / 2 / z.tpad / kXentTile * kXentTile;
    if (most < 1024) most = 1024;
    const size_t pieces = (vpad + most - 1) / most, piece = round_up((vpad + pieces - 1) / pieces, kXentTile);
    // dX's K, the piece, in splits: enough for a unit a pair where tiles are few, of 4 boxes at
    // least (gradient of 64 x 512 over 1000 20.9 us; with 2, 8 or 16 boxes 23.1), 32 at most, for
    // the scratch's sake (8 to 64: alike)
    const size_t tiles_h = (z.H + kXentTile - 1) / kXentTile, tiles_x = (size_t)z.tiles_t * tiles_h;
    size_t splits = kSplitPairs / tiles_x, boxes = (z.V < piece ? z.V : piece) / 64 / 4;
    if (splits > boxes) splits = boxes;
    // Few tokens: a split a chain, too, so that the launch need not add chains up in
    // registers, which a short K of dW pays for (16 x 4096 over 131072 628 us, 685 with
    // 4 splits; 1024 tokens 2064 and 2118, 2048 4028 and 3989).
    const size_t chains = ((z.V < piece ? z.V : piece) + kXentChain - 1) / kXentChain;
    if (z.T <= 1024 && splits < chains) splits = chains;
    if (splits > 32) splits = 32;
    if (splits < 1) splits = 1;
    const size_t ldws = round_up(z.H, 32);
    Parts parts;
    XentCommon c;
    c.place(parts, z);
    const size_t at_P = parts.add(z.tpad * piece * 2), at_ws = parts.add(a.dx ? splits * z.tpad * ldws * 4 : 0);
    Scratch scratch(s);
    if ((st = scratch.take(parts.bytes, dev)) != TCR_OK) return st;
    if (fault_injected("launch")) return TCR_ERR_CUDA;
    char *base = (char *)scratch.p;
    XentTokens k = {};
    k.x = a.x;
    k.ldx = a.ldx;
    k.target = a.target;
    k.tokens = z.T;
    k.H = z.H;
    k.V = z.V;
    k.ignore = a.ignore_index;
    k.al_x = rows_aligned(a.x, a.ldx, z.T, 2);
    k.dloss = a.dloss;
    k.inc_dloss = a.inc_dloss;
    XentMaps maps;
    cudaError_t e = xent_prepare(k, z, c, base, a.weight, a.ldw, maps, s);
    if (e == cudaSuccess) e = xent_map(&maps.p, base + at_P, piece, z.tpad, piece, 64);
    if (e == cudaSuccess) e = xent_map(&maps.p128, base + at_P, piece, z.tpad, piece, 128);
    if (e == cudaSuccess) e = xent_map(&maps.p_out, base + at_P, piece, z.tpad, piece, 32);
    if (e == cudaSuccess && a.dx) e = xent_map(&maps.ws_out, base + at_ws, ldws, splits * z.tpad, ldws, 32, true);
    // a tensor-map store writes whole granules of 16 bytes, past a row's end as well
    const bool al_dw = rows_aligned(a.dweight, a.lddw, z.V, 2) && z.H % 8 == 0;
    if (e == cudaSuccess && a.dweight && al_dw)
        e = xent_map(&maps.dw_out, a.dweight, z.H, z.V, z.V == 1 ? z.ldX : a.lddw, 32);
    XentGemm g = {};
    g.head = k.head;
    g.lab = k.lab;
    g.tok = k.tok;
    g.tpad = z.tpad;
    g.V = (int)z.V;
    g.H = (int)z.H;
    g.lse = a.lse;
    g.dloss = a.dloss;
    g.inc_dloss = a.inc_dloss;
    g.P = (uint16_t *)(base + at_P);
    g.ldp = piece;
    g.ws = a.dx ? (float *)(base + at_ws) : nullptr;
    g.ldws = ldws;
    g.splits = (int)splits;
    g.dw = a.dweight;
    g.lddw = a.lddw;
    g.al_dw = al_dw;
    g.inject_stall = fault_injected("stall");
    for (size_t v0 = 0; v0 < z.V && e == cudaSuccess; v0 += piece) {
        g.v0 = (int)v0;
        g.vn = (int)(z.V - v0 < piece ? z.V - v0 : piece);
        g.first = v0 == 0;
        const size_t tiles_v = ((size_t)g.vn + kXentTile - 1) / kXentTile;
        const int tile = xent_tile_cols(z.T, (size_t)g.vn, pairs);
        const size_t logits = (size_t)z.tiles_t * (((size_t)g.vn + (size_t)tile - 1) / (size_t)tile);
        e = launch_xent(a.dtype, kXentGradient, maps, g, logits, pairs, tile, s);
        const size_t units = (g.ws ? tiles_x * splits : 0) + (g.dw ? tiles_v * tiles_h : 0);
        if (e == cudaSuccess) e = launch_xent(a.dtype, kXentBack, maps, g, units, pairs, kXentTile, s);
    }
    if (e == cudaSuccess && a.dx) {
        XentDx d = {g.ws, z.tpad, ldws, (int)splits, k.rank, k.head, z.T, z.H, a.dx, a.lddx,
                    rows_aligned(a.dx, a.lddx, z.T, 2, 8)};
        e = launch_xent_dx(a.dtype, d, s);
    }
    const cudaError_t f = scratch.release();
    return of(e == cudaSuccess ? f : e);
} catch (...) {
    return TCR_ERR_CUDA;
}

}  // extern "C"
