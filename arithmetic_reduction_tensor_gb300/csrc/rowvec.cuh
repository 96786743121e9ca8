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

// Bytes sh .. sh + 4 N - 1 of the words w[0 .. N + 3] (0 <= sh < 16), sh the
// same in every lane that runs together: one branch on its words, then a
// funnel shift a word by the rest.  (Selecting words by predicates instead
// took rows of 5001 bfloat16 a tenth longer.)
template <int N, int S>
__device__ __forceinline__ void shift_by(const uint32_t (&w)[N + 4], uint32_t bits, uint32_t (&o)[N])
{
#pragma unroll
    for (int k = 0; k < N; k++) o[k] = __funnelshift_r(w[k + S], w[k + S + (S < 4 ? 1 : 0)], bits);
}

template <int N>
__device__ __forceinline__ void shift_words(const uint32_t (&w)[N + 4], uint32_t sh, uint32_t (&o)[N])
{
    const uint32_t bits = 8u * (sh & 3u);
    switch (sh >> 2) {
    case 0: shift_by<N, 0>(w, bits, o); break;
    case 1: shift_by<N, 1>(w, bits, o); break;
    case 2: shift_by<N, 2>(w, bits, o); break;
    default: shift_by<N, 3>(w, bits, o); break;
    }
}

// The elements of vector v that the row has.
__device__ __forceinline__ uint32_t vec_left(uint32_t cols, uint32_t v)
{
    return kRv * v >= cols ? 0u : min(cols - kRv * v, (uint32_t)kRv);
}

// A vector as loaded: its storage, or (GRAN) the 16-byte granules that its
// elements touch, one more than it has, to be shifted when it is used -- a
// load issued ahead must not be waited for by its own shift.
template <int DT, bool GRAN>
struct LoadedVec {
    uint4 q[(DT == kF32 ? 2 : 1) + (GRAN ? 1 : 0)];
};

// Vector v of a row at any element alignment; elements past cols read as 0.
// GRAN = false (`aligned`: the rows are 16-byte aligned): one 16-byte load
// (two of binary32) for whole vectors.  Granules reach up to 15 bytes before
// the row's first or after its last element, but each holds one of the
// row's elements.
template <int DT, bool GRAN>
__device__ __forceinline__ LoadedVec<DT, GRAN> load_vec(const typename Elem<DT>::T *row, uint32_t cols, uint32_t v)
{
    constexpr int es = DT == kF32 ? 4 : 2, NQ = es / 2;
    LoadedVec<DT, GRAN> r;
    const uint32_t left = vec_left(cols, v);
    const char *p = (const char *)(row + kRv * v);
    const uint32_t m = GRAN ? (uint32_t)(uintptr_t)p & 15u : 0u;
    const uint32_t end = left ? m + left * es : 0u;          // bytes of the granules in use
#pragma unroll
    for (int k = 0; k < NQ + (GRAN ? 1 : 0); k++) {
        r.q[k] = make_uint4(0u, 0u, 0u, 0u);
        if (16u * k < end) r.q[k] = ld16(p - m + 16 * k);
    }
    return r;
}

template <int DT, bool GRAN>
__device__ __forceinline__ RawVec<DT> use_vec(const LoadedVec<DT, GRAN> &l, const typename Elem<DT>::T *row,
                                              uint32_t cols, uint32_t v)
{
    constexpr int es = DT == kF32 ? 4 : 2, NW = 2 * es;      // words of a vector
    RawVec<DT> r;
    uint32_t o[NW];
    if constexpr (GRAN) {
        uint32_t w[NW + 4];
#pragma unroll
        for (int k = 0; k < NW / 4 + 1; k++) {
            w[4 * k] = l.q[k].x;
            w[4 * k + 1] = l.q[k].y;
            w[4 * k + 2] = l.q[k].z;
            w[4 * k + 3] = l.q[k].w;
        }
        shift_words<NW>(w, (uint32_t)(uintptr_t)row & 15u, o);
    } else {
#pragma unroll
        for (int k = 0; k < NW / 4; k++) {
            o[4 * k] = l.q[k].x;
            o[4 * k + 1] = l.q[k].y;
            o[4 * k + 2] = l.q[k].z;
            o[4 * k + 3] = l.q[k].w;
        }
    }
    const uint32_t left = vec_left(cols, v);
    if (left < kRv) {
#pragma unroll
        for (int k = 0; k < NW; k++) {
            if constexpr (es == 4)
                o[k] = (uint32_t)k < left ? o[k] : 0u;
            else
                o[k] = 2u * k + 1u < left ? o[k] : 2u * k < left ? o[k] & 0xffffu : 0u;
        }
    }
#pragma unroll
    for (int k = 0; k < NW / 4; k++) r.q[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    return r;
}

// The same at once, for rows that may or may not be aligned.
template <int DT>
__device__ __forceinline__ RawVec<DT> load_raw(const typename Elem<DT>::T *row, uint32_t cols, uint32_t v,
                                               bool aligned)
{
    if (aligned) return use_vec<DT, false>(load_vec<DT, false>(row, cols, v), row, cols, v);
    return use_vec<DT, true>(load_vec<DT, true>(row, cols, v), row, cols, v);
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

template <int B>
__device__ __forceinline__ void store_piece(char *p, const uint32_t *w)
{
    if constexpr (B == 16)
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (B == 8)
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else if constexpr (B == 4)
        *reinterpret_cast<uint32_t *>(p) = w[0];
    else if constexpr (B == 2)
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
    else
        *reinterpret_cast<uint8_t *>(p) = (uint8_t)w[0];
}

// Store a vector of NW words (the elements es bytes each, `left` of them, 0
// for a lane without a vector) where rows are not aligned: the lanes of a
// warp hold consecutive vectors, and between them cover whole granules (16
// bytes, or 8 for codes), so a lane stores the granules that begin in the
// vector before its own (taken over by a shuffle) or in its own.  What has
// no partner (a warp's first and last vectors, a row's last) goes element by
// element.  Every lane of the warp calls this.
template <int NW, int es>
__device__ __forceinline__ void store_shifted(char *p, uint32_t left, const uint32_t (&o)[NW])
{
    constexpr uint32_t bytes = 4 * NW;                  // of a vector
    constexpr uint32_t G = bytes < 16 ? bytes : 16;     // granule
    constexpr int GW = G / 4;
    constexpr uint32_t n = bytes / es;
    const uint32_t m = (uint32_t)(uintptr_t)p & (G - 1);
    const uint32_t lane = threadIdx.x & 31;
    uint32_t w[NW + 4];
#pragma unroll
    for (int k = 0; k < GW; k++) w[k] = __shfl_up_sync(kFull, o[NW - GW + k], 1);
    const uint32_t after = __shfl_down_sync(kFull, left, 1);
    const bool whole = left == n;
    const bool joins = whole && lane > 0;               // (the vector before a vector is whole)
    const bool next_joins = after == n && lane < 31;
    if (m == 0u) {
#pragma unroll
        for (int k = 0; k < NW / GW; k++)
            if (whole) store_piece<G>(p + G * k, o + GW * k);
        if (whole || left == 0u) return;
    }
    uint32_t from = 0, to = left;                       // own elements that no granule covers
    if (m != 0u) {
#pragma unroll
        for (int k = 0; k < NW; k++) w[GW + k] = o[k];
#pragma unroll
        for (int k = GW + NW; k < NW + 4; k++) w[k] = 0u;
        uint32_t g[NW];
        shift_words<NW>(w, G - m, g);                   // from p - m on
        if (joins) {
#pragma unroll
            for (int k = 0; k < NW / GW; k++) store_piece<G>(p - m + G * k, g + GW * k);
            from = (bytes - m) / es;
        }
        if (next_joins) to = (bytes - m) / es;
    }
    if (from >= to) return;
#pragma unroll
    for (uint32_t k = 0; k < n; k++)
        if (k >= from && k < to) {
            const uint32_t x = o[es * k / 4] >> (8 * (es * k & 3u));
            store_piece<es>(p + es * k, &x);
        }
}

// Vector v of a row, rounded to the type.  `aligned` (uniform): the rows are
// 16-byte aligned.  Every lane of the warp calls it, with the vectors of
// consecutive lanes consecutive; lanes past the row store nothing.
template <int DT>
__device__ __forceinline__ void store_vec(typename Elem<DT>::T *row, uint32_t cols, uint32_t v, bool aligned,
                                          const float (&f)[kRv])
{
    constexpr int es = DT == kF32 ? 4 : 2, NW = 2 * es;
    uint32_t o[NW];
    if constexpr (DT == kF32) {
#pragma unroll
        for (int k = 0; k < 8; k++) o[k] = __float_as_uint(f[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) o[k] = float2_to_word<DT>(f[2 * k], f[2 * k + 1]);
    }
    char *p = (char *)(row + kRv * v);
    if (aligned && kRv * v + kRv <= cols) {
#pragma unroll
        for (int k = 0; k < NW / 4; k++)
            *reinterpret_cast<uint4 *>(p + 16 * k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    } else if (!aligned) {
        store_shifted<NW, es>(p, vec_left(cols, v), o);
    } else {
        const uint32_t left = vec_left(cols, v);
#pragma unroll
        for (uint32_t k = 0; k < kRv; k++)
            if (k < left) row[kRv * v + k] = (typename Elem<DT>::T)(es == 4 ? o[k] : o[k / 2] >> (16 * (k % 2)));
    }
}

// The tree over the 8 values of a vector.
__device__ __forceinline__ float tree8(const float (&e)[kRv])
{
    return __fadd_rn(__fadd_rn(__fadd_rn(e[0], e[1]), __fadd_rn(e[2], e[3])),
                     __fadd_rn(__fadd_rn(e[4], e[5]), __fadd_rn(e[6], e[7])));
}

// The halving fold of N values, absent ones up to a power of two +0.0 (a
// sum of non-negative values or of a row's products: x + 0.0 is x but for
// the sign of a zero).
template <int N>
__device__ __forceinline__ float halving(float (&a)[N])
{
    if constexpr (N == 3) {
        return __fadd_rn(__fadd_rn(a[0], a[2]), __fadd_rn(a[1], 0.0f));
    } else {
        static_assert((N & (N - 1)) == 0, "a power of two, or 3");
#pragma unroll
        for (int h = N / 2; h >= 1; h /= 2)
#pragma unroll
            for (int i = 0; i < h; i++) a[i] = __fadd_rn(a[i], a[i + h]);
        return a[0];
    }
}

// The halving fold over the lanes of a warp; every lane gets the result
// (the butterfly adds the same two values in both lanes of a pair).
__device__ __forceinline__ float halving_lanes(float v)
{
#pragma unroll
    for (int h = 16; h >= 1; h /= 2) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, h));
    return v;
}

// Rows read element by element: lane l of a warp holds elements 32 j + l, j =
// 0 .. 7, of a stretch of 256, so that accesses of rows at any alignment are
// consecutive over the lanes.  From its eight values the value of one of the
// stretch's 32 vectors (tree8 of elements 8v .. 8v + 7, which lie in eight
// lanes): three exchanges that each halve what a lane still carries.  Lane l
// ends with vector 4 j + l / 8, j = l % 8.
__device__ __forceinline__ float tree8_lanes(const float (&e)[kRv])
{
    const uint32_t lane = threadIdx.x & 31;
    float a[4], b[2];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const bool odd = lane & 1u;
        const float keep = odd ? e[2 * k + 1] : e[2 * k], give = odd ? e[2 * k] : e[2 * k + 1];
        a[k] = __fadd_rn(keep, __shfl_xor_sync(kFull, give, 1));
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const bool odd = lane & 2u;
        const float keep = odd ? a[2 * k + 1] : a[2 * k], give = odd ? a[2 * k] : a[2 * k + 1];
        b[k] = __fadd_rn(keep, __shfl_xor_sync(kFull, give, 2));
    }
    const bool odd = lane & 4u;
    return __fadd_rn(odd ? b[1] : b[0], __shfl_xor_sync(kFull, odd ? b[0] : b[1], 4));
}

// The halving fold over those lanes: vector bits 4, 3, 2, 1, 0 are lane bits
// 2, 1, 0, 4, 3.
__device__ __forceinline__ float halving_lanes_elem(float v)
{
#pragma unroll
    for (int k = 0; k < 5; k++) {
        constexpr int order[5] = {4, 2, 1, 16, 8};
        v = __fadd_rn(v, __shfl_xor_sync(kFull, v, order[k]));
    }
    return v;
}

// The fold over a team of T threads (a warp, or the whole CTA) of values
// already folded within each thread; every thread gets the result.  `red`:
// team_floats<T>() floats of shared memory, not in use by an earlier call
// that some thread may still be reading.  A CTA may have fewer than T
// `threads` (whole warps); the absent ones count as +0.0.  Small teams:
// every warp folds over the warps itself, one barrier.  From 16 warps on
// that is more shared-memory reads than a second barrier costs: each warp
// folds over the warps for some of the lanes and passes the results on.
template <int T>
__host__ __device__ constexpr int team_floats()
{
    return T <= 32 ? 1 : T < 512 ? T : T / 32 * 33 + 32;
}

// ELEM: lanes hold the vectors of tree8_lanes.
template <int T, bool ELEM = false>
__device__ __forceinline__ float team_sum(float v, float *red, uint32_t threads = T)
{
    const uint32_t lane = threadIdx.x & 31;
    if constexpr (T >= 512) {
        float *tot = red + T / 32 * 33;
        const uint32_t warp = threadIdx.x >> 5, warps = threads >> 5;
        red[warp * 33 + lane] = v;
        __syncthreads();
        for (uint32_t c = warp; c < 32; c += warps) {
            const float a = halving_lanes(lane < warps ? red[lane * 33 + c] : 0.0f);
            if (lane == 0) tot[c] = a;
        }
        __syncthreads();
        v = tot[lane];
    } else if constexpr (T > 32) {
        red[threadIdx.x] = v;
        __syncthreads();
        float a[T / 32];
#pragma unroll
        for (int w = 0; w < T / 32; w++) a[w] = 32u * w < threads ? red[32 * w + lane] : 0.0f;
        v = halving<T / 32>(a);
    }
    return ELEM ? halving_lanes_elem(v) : halving_lanes(v);
}

// The largest of the team's values, each given as the bits of a
// non-negative binary32 (their order as integers is the values', with NaN
// above infinity, so a NaN is never lost).
template <int T>
__device__ __forceinline__ uint32_t team_max(uint32_t bits, uint32_t *red, uint32_t threads = T)
{
    bits = __reduce_max_sync(kFull, bits);
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = bits;
        __syncthreads();
        bits = __reduce_max_sync(kFull, (threadIdx.x & 31) < threads / 32 ? red[threadIdx.x & 31] : 0u);
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

// A code, in the low byte: rint(y * per), ties to even, the product not
// rounded; 0 where per is 0 (y may then be NaN or infinite).  Adding
// 1.5 * 2^23 in the same operation leaves the integer in the low bits (a
// conversion instruction per value runs at an eighth of the rate).
__device__ __forceinline__ uint32_t i8_code(float y, float per)
{
    return per == 0.0f ? 0u : __float_as_uint(__fmaf_rn(y, per, 12582912.0f));
}

// The codes of a vector.  Called like store_vec; `aligned8`: the rows are
// 8-byte aligned.
__device__ __forceinline__ void store_codes(int8_t *row, uint32_t cols, uint32_t v, bool aligned8,
                                            const float (&y)[kRv], float per)
{
    uint32_t o[2] = {0u, 0u};
    if (per != 0.0f) {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; i++) c[i] = i8_code(y[4 * k + i], per);
            o[k] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        }
    }
    char *p = (char *)(row + kRv * v);
    if (aligned8 && kRv * v + kRv <= cols) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(o[0], o[1]);
    } else if (!aligned8) {
        store_shifted<2, 1>(p, vec_left(cols, v), o);
    } else {
        const uint32_t left = vec_left(cols, v);
#pragma unroll
        for (uint32_t k = 0; k < kRv; k++)
            if (k < left) row[kRv * v + k] = (int8_t)(o[k / 4] >> (8 * (k % 4)));
    }
}

// The largest magnitude of m and a vector's values; NaN if one is NaN.
__device__ __forceinline__ float amax8(const float (&y)[kRv], float m)
{
#pragma unroll
    for (int k = 0; k < kRv; k += 2)
        asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(y[k]), "f"(y[k + 1]));
    return m;
}

// i with its `bits` low bits in reverse order: visiting a thread's vectors
// in this order makes the halving fold the tree over neighbours that
// TreeCounter forms.
__device__ __forceinline__ uint32_t bit_reverse(uint32_t i, int bits)
{
    return bits ? __brev(i) >> (32 - bits) : 0u;
}

}  // namespace tcr
