// piece.cuh -- a thread's share of a row in the layer norm's kernels and its
// gradient's: eight values, held as a vector of rowvec.cuh or, for rows at any
// alignment, as one element in each of eight consecutive warp-wide accesses.
#pragma once

#include "drop.cuh"

namespace tcr {

// A thread's eight values of piece i of a row, T threads to a piece: vector
// t + i T (ELEM = false: rows are 16-byte aligned), or, for rows at any
// alignment, the elements 32 j + lane of its warp's 256.
template <int DT, bool ELEM>
struct Piece {
    using E = typename Elem<DT>::T;
    E e[ELEM ? kRv : 1];
    LoadedVec<DT, false> v;
};

template <int DT, bool ELEM>
__device__ __forceinline__ void load_piece(const typename Elem<DT>::T *row, uint32_t cols, uint32_t v,
                                           Piece<DT, ELEM> &p)
{
    using E = typename Elem<DT>::T;
    if constexpr (ELEM) {
        const uint32_t base = kRv * (v & ~31u), e = base + (v & 31u);
        if (base + 256 <= cols) {
#pragma unroll
            for (int j = 0; j < kRv; j++) p.e[j] = row[e + 32 * j];
        } else {
#pragma unroll
            for (int j = 0; j < kRv; j++) p.e[j] = e + 32 * j < cols ? row[e + 32 * j] : (E)0;
        }
    } else {
        p.v = load_vec<DT, false>(row, cols, v);
    }
}

template <int DT, bool ELEM>
__device__ __forceinline__ void piece_values(const Piece<DT, ELEM> &p, const typename Elem<DT>::T *row, uint32_t cols,
                                             uint32_t v, float (&f)[kRv])
{
    if constexpr (ELEM) {
#pragma unroll
        for (int j = 0; j < kRv; j++) f[j] = elem_to_float<DT>(p.e[j]);
    } else {
        unpack<DT>(use_vec<DT, false>(p.v, row, cols, v), f);
    }
}

// Zero the values that the row does not have.
template <bool ELEM>
__device__ __forceinline__ void zero_absent(uint32_t cols, uint32_t v, float (&f)[kRv])
{
    if constexpr (ELEM) {
        const uint32_t base = kRv * (v & ~31u), e = base + (v & 31u);
        if (base + 256 <= cols) return;
#pragma unroll
        for (int j = 0; j < kRv; j++)
            if (e + 32 * j >= cols) f[j] = 0.0f;
    } else {
        const uint32_t left = vec_left(cols, v);
        if (left == kRv) return;
#pragma unroll
        for (uint32_t k = 0; k < kRv; k++)
            if (k >= left) f[k] = 0.0f;
    }
}

// Every lane of the warp calls it (rows are as in load_piece).
template <int DT, bool ELEM>
__device__ __forceinline__ void store_piece_values(typename Elem<DT>::T *row, uint32_t cols, uint32_t v,
                                                   const float (&f)[kRv])
{
    if constexpr (ELEM) {
        const uint32_t base = kRv * (v & ~31u), e = base + (v & 31u);
        if (base + 256 <= cols) {
#pragma unroll
            for (int j = 0; j < kRv; j++) row[e + 32 * j] = float_to_elem<DT>(f[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kRv; j++)
                if (e + 32 * j < cols) row[e + 32 * j] = float_to_elem<DT>(f[j]);
        }
    } else {
        store_vec<DT>(row, cols, v, true, f);
    }
}

template <bool ELEM>
__device__ __forceinline__ void store_piece_codes(int8_t *row, uint32_t cols, uint32_t v, const float (&f)[kRv],
                                                  float per)
{
    if constexpr (ELEM) {
        const uint32_t base = kRv * (v & ~31u), e = base + (v & 31u);
        const bool whole = base + 256 <= cols;
#pragma unroll
        for (int j = 0; j < kRv; j++)
            if (whole || e + 32 * j < cols) row[e + 32 * j] = (int8_t)i8_code(f[j], per);
    } else {
        store_codes(row, cols, v, true, f, per);
    }
}

// The same of binary32 sums at any alignment.
template <bool ELEM>
__device__ __forceinline__ void store_piece_values_any(float *row, uint32_t cols, uint32_t v, const float (&f)[kRv])
{
    if constexpr (ELEM) {
        store_piece_values<kF32, true>((uint32_t *)row, cols, v, f);
    } else {
        const uint32_t left = vec_left(cols, v);
        float *p = row + kRv * v;
        if (left == kRv && ((uintptr_t)p & 15u) == 0) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
            return;
        }
#pragma unroll
        for (uint32_t k = 0; k < kRv; k++)
            if (k < left) p[k] = f[k];
    }
}

// A piece of the weight, whose own alignment may differ from the rows'.
template <int DT, bool ELEM>
__device__ __forceinline__ void load_weight_piece(const typename Elem<DT>::T *w, uint32_t cols, uint32_t v, bool aligned,
                                                  Piece<DT, ELEM> &p)
{
    if constexpr (ELEM) {
        load_piece<DT, true>(w, cols, v, p);
    } else {
        const RawVec<DT> raw = load_raw<DT>(w, cols, v, aligned);
#pragma unroll
        for (int k = 0; k < (DT == kF32 ? 2 : 1); k++) p.v.q[k] = raw.q[k];
    }
}

template <bool ELEM>
__device__ __forceinline__ float piece_tree(const float (&e)[kRv])
{
    if constexpr (ELEM)
        return tree8_lanes(e);
    else
        return tree8(e);
}

__device__ __forceinline__ void centre(float (&y)[kRv], float mean)
{
#pragma unroll
    for (int k = 0; k < kRv; k++) y[k] = __fsub_rn(y[k], mean);
}

}  // namespace tcr
