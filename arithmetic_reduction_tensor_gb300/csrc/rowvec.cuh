// rowvec.cuh -- rows cut into vectors of 8 values, for the row operators
// whose sums have a declared order of their own (norm, its gradient, the
// 8-bit row quantiser).
//
// Vector v of a row holds its elements 8v .. 8v + 7 (absent ones 0).  A sum
// over a row is, for every launch shape, alignment and row count alike,
//   s_v   = ((e0 + e1) + (e2 + e3)) + ((e4 + e5) + (e6 + e7))   per vector,
//   a_v  += a_(v + h), h = P/2, P/4, .. 1                       (halving),
// with P the power of two that covers the vectors and absent vectors +0.0.
// Folding the upper half onto the lower one first means that the vectors a
// thread holds (v = t + i T) fold in its registers, the warps' partials fold
// lane by lane, and the lanes fold last by shuffles -- so any team of T
// threads gives the same bits, and a row's result depends on the row alone.
#pragma once

#include "common.cuh"

namespace tcr {

constexpr int kRv = 8;                 // values per vector

template <int DT>
__device__ __forceinline__ float elem_to_float(typename Elem<DT>::T e)
{
    if constexpr (DT == kF16)
        return __half2float(__ushort_as_half(e));
    else if constexpr (DT == kBF16)
        return __uint_as_float((uint32_t)e << 16);
    else
        return __uint_as_float(e);
}

// Round to the type, to nearest even (bfloat16: NaN stays NaN).
template <int DT>
__device__ __forceinline__ typename Elem<DT>::T float_to_elem(float f)
{
    if constexpr (DT == kF16) {
        return __half_as_ushort(__float2half_rn(f));
    } else if constexpr (DT == kBF16) {
        uint16_t r;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
        return r;
    } else {
        return __float_as_uint(f);
    }
}

// Two values rounded and packed, `lo` at the lower address.
template <int DT>
__device__ __forceinline__ uint32_t float2_to_word(float lo, float hi)
{
    uint32_t r;
    if constexpr (DT == kF16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 ld16(const void *p)
{
    return *reinterpret_cast<const uint4 *>(p);
}

// The 8 values of a vector in its storage: 16 bytes, or 32 of binary32.
template <int DT>
struct RawVec {
    uint4 q[DT == kF32 ? 2 : 1];
};

// Vector v (8 v < cols) of a row at any element alignment.  A whole vector
// of a 16-byte aligned row is one 16-byte load (two of binary32), anything
// else is read element by element.
template <int DT>
__device__ __forceinline__ RawVec<DT> load_raw(const typename Elem<DT>::T *row, size_t cols, size_t v,
                                               bool aligned)
{
    RawVec<DT> r;
    const typename Elem<DT>::T *p = row + kRv * v;
    if (aligned && kRv * v + kRv <= cols) {
#pragma unroll
        for (int k = 0; k < (DT == kF32 ? 2 : 1); k++) r.q[k] = ld16((const char *)p + 16 * k);
        return r;
    }
    const size_t left = kRv * v < cols ? cols - kRv * v : 0;
    if constexpr (DT == kF32) {
        uint32_t e[8];
#pragma unroll
        for (int k = 0; k < 8; k++) e[k] = (size_t)k < left ? p[k] : 0u;
        r.q[0] = make_uint4(e[0], e[1], e[2], e[3]);
        r.q[1] = make_uint4(e[4], e[5], e[6], e[7]);
    } else {
        uint16_t e[8];
#pragma unroll
        for (int k = 0; k < 8; k++) e[k] = (size_t)k < left ? p[k] : (uint16_t)0;
        r.q[0] = make_uint4(pack2(e[0], e[1]), pack2(e[2], e[3]), pack2(e[4], e[5]), pack2(e[6], e[7]));
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void unpack(const RawVec<DT> &r, float (&f)[kRv])
{
    if constexpr (DT == kF32) {
        const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
        for (int k = 0; k < 8; k++) f[k] = __uint_as_float(w[k]);
    } else {
        const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            f[2 * k] = leaf_lo<DT>(w[k]);
            f[2 * k + 1] = leaf_hi<DT>(w[k]);
        }
    }
}

template <int DT>
__device__ __forceinline__ void store_vec(typename Elem<DT>::T *row, size_t cols, size_t v, bool aligned,
                                          const float (&f)[kRv])
{
    typename Elem<DT>::T *p = row + kRv * v;
    if (aligned && kRv * v + kRv <= cols) {
        if constexpr (DT == kF32) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4 *>(p) =
                make_uint4(float2_to_word<DT>(f[0], f[1]), float2_to_word<DT>(f[2], f[3]),
                           float2_to_word<DT>(f[4], f[5]), float2_to_word<DT>(f[6], f[7]));
        }
        return;
    }
    const size_t left = kRv * v < cols ? cols - kRv * v : 0;
#pragma unroll
    for (int k = 0; k < kRv; k++)
        if ((size_t)k < left) p[k] = float_to_elem<DT>(f[k]);
}

// The tree over the 8 values of a vector.
__device__ __forceinline__ float tree8(const float (&e)[kRv])
{
    return __fadd_rn(__fadd_rn(__fadd_rn(e[0], e[1]), __fadd_rn(e[2], e[3])),
                     __fadd_rn(__fadd_rn(e[4], e[5]), __fadd_rn(e[6], e[7])));
}

// a[0] after the halving fold of n (a power of two) values.
template <int N>
__device__ __forceinline__ float halving(float (&a)[N])
{
#pragma unroll
    for (int h = N / 2; h >= 1; h /= 2)
#pragma unroll
        for (int i = 0; i < h; i++) a[i] = __fadd_rn(a[i], a[i + h]);
    return a[0];
}

// The halving fold over the lanes of a warp; every lane gets the result
// (the butterfly adds the same two values in both lanes of a pair).
__device__ __forceinline__ float halving_lanes(float v)
{
#pragma unroll
    for (int h = 16; h >= 1; h /= 2) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, h));
    return v;
}

// The fold over a team of T threads (a warp, or the whole CTA) of values
// already folded within each thread; every thread gets the result.  `red`:
// T floats of shared memory, not in use by an earlier call that some thread
// may still be reading.
template <int T>
__device__ __forceinline__ float team_sum(float v, float *red)
{
    if constexpr (T > 32) {
        red[threadIdx.x] = v;
        __syncthreads();
        float a[T / 32];
#pragma unroll
        for (int w = 0; w < T / 32; w++) a[w] = red[32 * w + (threadIdx.x & 31)];
        v = halving<T / 32>(a);
    }
    return halving_lanes(v);
}

// The largest of the team's values, each given as the bits of a
// non-negative binary32 (their order as integers is the values', with NaN
// above infinity, so a NaN is never lost).
template <int T>
__device__ __forceinline__ uint32_t team_max(uint32_t bits, uint32_t *red)
{
    bits = __reduce_max_sync(kFull, bits);
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = bits;
        __syncthreads();
        bits = __reduce_max_sync(kFull, (threadIdx.x & 31) < T / 32 ? red[threadIdx.x & 31] : 0u);
    }
    return bits;
}

// The scale of a row of 8-bit codes from the bits of its largest magnitude,
// and the factor that takes values to codes: scale = amax / 127, per =
// 127 / amax.  A row whose scale is below the smallest normal number counts
// as a row of zeros (scale 0, codes 0); a row with a NaN or an infinity has
// scale NaN and codes 0, so that every value read back is NaN.
__device__ __forceinline__ void i8_scale(uint32_t amax_bits, float &scale, float &per)
{
    const float amax = __uint_as_float(amax_bits);
    per = 0.0f;
    if (amax_bits >= 0x7f800000u) {
        scale = __uint_as_float(0x7fc00000u);
        return;
    }
    scale = __fdiv_rn(amax, 127.0f);
    if (scale < 1.17549435e-38f)
        scale = 0.0f;
    else
        per = __fdiv_rn(127.0f, amax);
}

// rint(y * per) as an 8-bit code, ties to even; 0 where per is 0 (y may
// then be NaN or infinite).
__device__ __forceinline__ uint32_t i8_code(float y, float per)
{
    return per == 0.0f ? 0u : (uint32_t)__float2int_rn(__fmul_rn(y, per)) & 0xffu;
}

__device__ __forceinline__ void store_codes(int8_t *row, size_t cols, size_t v, bool aligned8,
                                            const float (&y)[kRv], float per)
{
    uint32_t c[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) c[k] = i8_code(y[k], per);
    int8_t *p = row + kRv * v;
    if (aligned8 && kRv * v + kRv <= cols) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                                                   c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
        return;
    }
    const size_t left = kRv * v < cols ? cols - kRv * v : 0;
#pragma unroll
    for (int k = 0; k < kRv; k++)
        if ((size_t)k < left) p[k] = (int8_t)c[k];
}

// i with its `bits` low bits in reverse order: visiting a thread's vectors
// in this order makes the halving fold the tree over neighbours that
// TreeCounter forms.
__device__ __forceinline__ uint32_t bit_reverse(uint32_t i, int bits)
{
    return bits ? __brev(i) >> (32 - bits) : 0u;
}

}  // namespace tcr
