// args.h -- what the entry points over matrices of rows (tcr_i8.cu,
// tcr_train.cu) share: checks of their arguments, and scratch of a call.
#pragma once

#include <cstdint>

#include "plan.h"

namespace tcr {
namespace plan {

constexpr size_t kMaxRows = (size_t)1 << 31;       // exclusive
constexpr size_t kMaxCols = (size_t)1 << 27;
constexpr size_t kMaxSpan = (size_t)1 << 48;       // rows * ld, exclusive

inline bool is_float(int dtype)
{
    return dtype == TCR_F16 || dtype == TCR_BF16 || dtype == TCR_F32;
}

inline size_t dtype_bytes(int dtype)
{
    return dtype == TCR_I8 ? 1 : dtype == TCR_I32 ? 4 : elem_bytes(dtype);
}

inline bool is_aligned(const void *p, size_t bytes)
{
    return ((uintptr_t)p & (bytes - 1)) == 0;
}

inline bool sizes_ok(size_t rows, size_t cols)
{
    return rows < kMaxRows && cols <= kMaxCols && rows * cols < kMaxInputs;
}

// A matrix argument of a non-empty call: present, aligned to its element,
// with a leading dimension that holds a row (0 allowed for an input).
inline bool matrix_ok(const void *p, size_t ld, size_t rows, size_t cols, int dtype, bool input)
{
    if (!p || !is_aligned(p, dtype_bytes(dtype))) return false;
    if (rows <= 1) return true;
    if (ld < cols && !(input && ld == 0)) return false;
    return ld < kMaxSpan / rows;
}

inline bool floats_ok(const float *p)
{
    return p && is_aligned(p, 4);
}

// Whether every row starts on a 16-byte boundary (8 for codes written eight
// at a time).
inline bool rows_aligned(const void *p, size_t ld, size_t rows, size_t elem, size_t bytes = 16)
{
    return is_aligned(p, bytes) && (rows <= 1 || (ld * elem) % bytes == 0);
}

inline tcr_status of(cudaError_t e)
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

}  // namespace plan
}  // namespace tcr
