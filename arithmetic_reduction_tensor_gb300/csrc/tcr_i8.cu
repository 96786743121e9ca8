// tcr_i8.cu -- the C ABI of the 8-bit linear path: the norm and its
// gradient, the row quantiser and the 8-bit product.  Argument checks, then
// scratch from the library's pool and the launches.
#include <cmath>
#include <cstdint>

#include "../../include/tcr.h"
#include "kernels.cuh"
#include "plan.h"

namespace {

using namespace tcr;
using namespace tcr::plan;

constexpr size_t kMaxRows = (size_t)1 << 31;       // exclusive
constexpr size_t kMaxCols = (size_t)1 << 27;
constexpr size_t kMaxSpan = (size_t)1 << 48;       // rows * ld, exclusive
constexpr size_t kMaxK = 131071;                   // |S| <= 2^14 K < 2^31

bool is_float(int dtype)
{
    return dtype == TCR_F16 || dtype == TCR_BF16 || dtype == TCR_F32;
}

size_t dtype_bytes(int dtype)
{
    return dtype == TCR_I8 ? 1 : dtype == TCR_I32 ? 4 : elem_bytes(dtype);
}

bool is_aligned(const void *p, size_t bytes)
{
    return ((uintptr_t)p & (bytes - 1)) == 0;
}

bool sizes_ok(size_t rows, size_t cols)
{
    return rows < kMaxRows && cols <= kMaxCols && rows * cols < kMaxInputs;
}

// A matrix argument of a non-empty call: present, aligned to its element,
// with a leading dimension that holds a row (0 allowed for an input).
bool matrix_ok(const void *p, size_t ld, size_t rows, size_t cols, int dtype, bool input)
{
    if (!p || !is_aligned(p, dtype_bytes(dtype))) return false;
    if (rows <= 1) return true;
    if (ld < cols && !(input && ld == 0)) return false;
    return ld < kMaxSpan / rows;
}

bool floats_ok(const float *p)
{
    return p && is_aligned(p, 4);
}

// Whether every row starts on a 16-byte boundary (8 for codes written eight
// at a time).
bool rows_aligned(const void *p, size_t ld, size_t rows, size_t elem, size_t bytes = 16)
{
    return is_aligned(p, bytes) && (rows <= 1 || (ld * elem) % bytes == 0);
}

tcr_status of(cudaError_t e)
{
    return e == cudaSuccess ? TCR_OK : TCR_ERR_CUDA;
}

// Scratch of a call on its stream; freed (stream-ordered) with the object.
struct Scratch {
    void *p = nullptr;
    cudaStream_t s;
    explicit Scratch(cudaStream_t stream) : s(stream) {}
    tcr_status take(size_t bytes, int dev)
    {
        if (bytes == 0) return TCR_OK;
        if (fault_injected("alloc")) return TCR_ERR_CUDA;
        cudaMemPool_t pool = pool_for(dev);
        if (!pool) return TCR_ERR_CUDA;
        if (cudaMallocFromPoolAsync(&p, bytes, pool, s) != cudaSuccess) {
            p = nullptr;
            return TCR_ERR_CUDA;
        }
        return TCR_OK;
    }
    cudaError_t release()
    {
        void *q = p;
        p = nullptr;
        return q ? cudaFreeAsync(q, s) : cudaSuccess;
    }
    ~Scratch() { (void)release(); }
};

}  // namespace

extern "C" {

tcr_status tcr_rmsnorm(const tcr_norm_args *args, void *stream)
{
    if (!args) return TCR_ERR_INVALID_ARG;
    const tcr_norm_args &a = *args;
    if (!is_float(a.dtype) || (a.y_dtype != a.dtype && a.y_dtype != TCR_I8)) return TCR_ERR_INVALID_ARG;
    if (!(a.eps >= 0.0f) || std::isinf(a.eps) || !sizes_ok(a.rows, a.cols)) return TCR_ERR_INVALID_ARG;
    if (a.rows == 0) return TCR_OK;
    const size_t eb = elem_bytes(a.dtype);
    if (a.cols > 0) {
        if (!matrix_ok(a.x, a.ldx, a.rows, a.cols, a.dtype, true) ||
            !matrix_ok(a.y, a.ldy, a.rows, a.cols, a.y_dtype, false))
            return TCR_ERR_INVALID_ARG;
        if (a.residual && !matrix_ok(a.residual, a.ldr, a.rows, a.cols, a.dtype, true)) return TCR_ERR_INVALID_ARG;
        if (a.h && !matrix_ok(a.h, a.ldh, a.rows, a.cols, a.dtype, false)) return TCR_ERR_INVALID_ARG;
        if (a.weight && !is_aligned(a.weight, eb)) return TCR_ERR_INVALID_ARG;
    }
    if ((a.y_dtype == TCR_I8 && !floats_ok(a.scale)) || (a.rstd && !floats_ok(a.rstd))) return TCR_ERR_INVALID_ARG;
    if (current_device() < 0 || fault_injected("launch")) return TCR_ERR_CUDA;
    RowArgs r = {};
    r.x = a.x;
    r.ldx = a.ldx;
    r.r = a.residual;
    r.ldr = a.ldr;
    r.w = a.weight;
    r.h = a.h;
    r.ldh = a.ldh;
    r.y = a.y;
    r.ldy = a.ldy;
    r.scale = a.scale;
    r.rstd = a.rstd;
    r.eps = a.eps;
    r.rows = a.rows;
    r.cols = a.cols;
    r.al_x = rows_aligned(a.x, a.ldx, a.rows, eb);
    r.al_r = rows_aligned(a.residual, a.ldr, a.rows, eb);
    r.al_w = is_aligned(a.weight, 16);
    r.al_h = rows_aligned(a.h, a.ldh, a.rows, eb);
    r.al_y = a.y_dtype == TCR_I8 ? rows_aligned(a.y, a.ldy, a.rows, 1, 8) : rows_aligned(a.y, a.ldy, a.rows, eb);
    return of(launch_rows_op(kRowNorm, a.dtype, a.y_dtype == TCR_I8, r, (cudaStream_t)stream));
}

tcr_status tcr_rmsnorm_backward(const tcr_norm_back_args *args, void *stream)
try {
    if (!args) return TCR_ERR_INVALID_ARG;
    const tcr_norm_back_args &a = *args;
    if (!is_float(a.dtype) || !sizes_ok(a.rows, a.cols)) return TCR_ERR_INVALID_ARG;
    if (a.dweight && !floats_ok(a.dweight)) return TCR_ERR_INVALID_ARG;
    if (a.cols == 0) return TCR_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const int dev = current_device();
    if (a.rows == 0) {
        if (!a.dweight) return TCR_OK;
        if (dev < 0 || fault_injected("launch")) return TCR_ERR_CUDA;
        return of(cudaMemsetAsync(a.dweight, 0, a.cols * sizeof(float), s));
    }
    const size_t eb = elem_bytes(a.dtype);
    if (!matrix_ok(a.dy, a.lddy, a.rows, a.cols, a.dtype, true) ||
        !matrix_ok(a.h, a.ldh, a.rows, a.cols, a.dtype, true) ||
        !matrix_ok(a.dx, a.lddx, a.rows, a.cols, a.dtype, false) || !floats_ok(a.rstd))
        return TCR_ERR_INVALID_ARG;
    if (a.dh && !matrix_ok(a.dh, a.lddh, a.rows, a.cols, a.dtype, true)) return TCR_ERR_INVALID_ARG;
    if (a.weight && !is_aligned(a.weight, eb)) return TCR_ERR_INVALID_ARG;
    if (dev < 0) return TCR_ERR_CUDA;
    Scratch scratch(s);
    tcr_status st = scratch.take(norm_back_scratch(a.rows, a.cols, a.dweight != nullptr), dev);
    if (st != TCR_OK) return st;
    if (fault_injected("launch")) return TCR_ERR_CUDA;
    BackArgs b = {};
    b.dy = a.dy;
    b.lddy = a.lddy;
    b.h = a.h;
    b.ldh = a.ldh;
    b.w = a.weight;
    b.rstd = a.rstd;
    b.dh = a.dh;
    b.lddh = a.lddh;
    b.dx = a.dx;
    b.lddx = a.lddx;
    b.rows = a.rows;
    b.cols = a.cols;
    b.al_dy = rows_aligned(a.dy, a.lddy, a.rows, eb);
    b.al_h = rows_aligned(a.h, a.ldh, a.rows, eb);
    b.al_w = is_aligned(a.weight, 16);
    b.al_dh = rows_aligned(a.dh, a.lddh, a.rows, eb);
    b.al_dx = rows_aligned(a.dx, a.lddx, a.rows, eb);
    cudaError_t e = launch_norm_back(a.dtype, b, (float *)scratch.p, a.dweight, s);
    const cudaError_t f = scratch.release();
    return of(e == cudaSuccess ? f : e);
} catch (...) {         // the host's memory for a cache: nothing may cross the C boundary
    return TCR_ERR_CUDA;
}

tcr_status tcr_quantize_rows_i8(const void *x, size_t ldx, const void *gate, size_t ldg, void *q, size_t ldq,
                                float *scale, size_t rows, size_t cols, int dtype, void *stream)
{
    if (!is_float(dtype) || !sizes_ok(rows, cols)) return TCR_ERR_INVALID_ARG;
    if (rows == 0) return TCR_OK;
    if (!floats_ok(scale)) return TCR_ERR_INVALID_ARG;
    if (cols > 0) {
        if (!matrix_ok(x, ldx, rows, cols, dtype, true) || !matrix_ok(q, ldq, rows, cols, TCR_I8, false))
            return TCR_ERR_INVALID_ARG;
        if (gate && !matrix_ok(gate, ldg, rows, cols, dtype, true)) return TCR_ERR_INVALID_ARG;
    }
    if (current_device() < 0 || fault_injected("launch")) return TCR_ERR_CUDA;
    const size_t eb = elem_bytes(dtype);
    RowArgs r = {};
    r.x = x;
    r.ldx = ldx;
    r.r = gate;
    r.ldr = ldg;
    r.y = q;
    r.ldy = ldq;
    r.scale = scale;
    r.rows = rows;
    r.cols = cols;
    r.al_x = rows_aligned(x, ldx, rows, eb);
    r.al_r = rows_aligned(gate, ldg, rows, eb);
    r.al_y = rows_aligned(q, ldq, rows, 1, 8);
    return of(launch_rows_op(kRowQuant, dtype, true, r, (cudaStream_t)stream));
}

tcr_status tcr_dequantize_rows_i8(const void *q, size_t ldq, const float *scale, void *y, size_t ldy,
                                  size_t rows, size_t cols, int dtype, void *stream)
{
    if (!is_float(dtype) || !sizes_ok(rows, cols)) return TCR_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return TCR_OK;
    if (!matrix_ok(q, ldq, rows, cols, TCR_I8, true) || !matrix_ok(y, ldy, rows, cols, dtype, false) ||
        !floats_ok(scale))
        return TCR_ERR_INVALID_ARG;
    if (current_device() < 0 || fault_injected("launch")) return TCR_ERR_CUDA;
    return of(launch_dequant(dtype, (const int8_t *)q, ldq, scale, y, ldy, rows, cols, (cudaStream_t)stream));
}

tcr_status tcr_gemm_i8(const void *A, size_t lda, const void *W, size_t ldw, const float *scale_a,
                       const float *scale_w, void *C, size_t ldc, size_t M, size_t N, size_t K, int c_dtype,
                       void *stream)
try {
    if (!is_float(c_dtype) && c_dtype != TCR_I32) return TCR_ERR_INVALID_ARG;
    if (M >= kMaxRows || N >= kMaxRows) return TCR_ERR_INVALID_ARG;
    if (K > kMaxK) return TCR_ERR_UNSUPPORTED;
    if (M * N >= kMaxInputs || M * K >= kMaxInputs || N * K >= kMaxInputs) return TCR_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TCR_OK;
    if (!matrix_ok(C, ldc, M, N, c_dtype, false)) return TCR_ERR_INVALID_ARG;
    if ((scale_a && !floats_ok(scale_a)) || (scale_w && !floats_ok(scale_w))) return TCR_ERR_INVALID_ARG;
    if (K > 0) {
        // one row for all is no use here: its pitch would not fit a tensor map
        if (!matrix_ok(A, lda, M, K, TCR_I8, false) || !matrix_ok(W, ldw, N, K, TCR_I8, false))
            return TCR_ERR_INVALID_ARG;
    }
    const int dev = current_device();
    if (dev < 0) return TCR_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    const size_t cb = dtype_bytes(c_dtype);
    if (K == 0) {
        if (fault_injected("launch")) return TCR_ERR_CUDA;
        return of(cudaMemset2DAsync(C, (M == 1 ? N : ldc) * cb, 0, N * cb, M, s));
    }
    I8Args a = {};
    a.A = (const int8_t *)A;
    a.lda = M == 1 ? K : lda;
    a.W = (const int8_t *)W;
    a.ldw = N == 1 ? (K + 15) / 16 * 16 : ldw;
    a.M = M;
    a.N = N;
    a.K = K;
    a.sa = scale_a;
    a.sw = scale_w;
    a.C = C;
    a.ldc = ldc;
    a.c_dtype = c_dtype == TCR_I32 ? kOutI32 : c_dtype;
    a.al_a = rows_aligned(A, lda, M, 1);
    a.al_w = rows_aligned(W, ldw, N, 1);
    const I8Plan p = gemm_i8_plan(M, N, K, M <= 2 ? 0 : gemm_i8_pairs());
    // without CTA pairs the one-launch kernels serve what their grid covers
    if (!p.tensor && M >= ((size_t)1 << 19)) return TCR_ERR_UNSUPPORTED;
    const bool repack = p.tensor && !a.al_w;
    Scratch scratch(s);
    tcr_status st = scratch.take(gemm_i8_scratch(p, M, N, repack), dev);
    if (st != TCR_OK) return st;
    if (fault_injected("launch")) return TCR_ERR_CUDA;
    cudaError_t e = launch_gemm_i8(a, p, scratch.p, repack, fault_injected("stall"), s);
    const cudaError_t f = scratch.release();
    return of(e == cudaSuccess ? f : e);
} catch (...) {
    return TCR_ERR_CUDA;
}

}  // extern "C"
