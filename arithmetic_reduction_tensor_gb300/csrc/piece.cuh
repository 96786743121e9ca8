// piece.cuh -- a thread's share of a row in the layer norm's kernels and its
// gradient's, and in dropout's: eight values, in one of three layouts.
//   kVectors   the vector 8v .. 8v + 7 of rowvec.cuh (rows are 16-byte aligned);
// and for rows at any alignment, of a warp's 256 consecutive elements:
//   kSingles   (binary32) elements 32 k + l, l the lane;
//   kPairs     (16 bits) elements 64 (k / 2) + 2 l + k % 2, so that a row that
//              starts on a 4-byte boundary is read and written by words.
// In each the values that a row has are the thread's first n.
//
// These kernels issue more than they wait: what does not change from row to
// row is found once, masks are left out where they can be, and sums run on
// pairs of values (f32x2: two binary32 additions an instruction, each rounded as
// it would be alone).
#pragma once

#include "drop.cuh"

namespace tcr {

template <int DT, bool ELEM>
__host__ __device__ constexpr int layout_of()
{
    return !ELEM ? kVectors : DT == kF32 ? kSingles : kPairs;
}

// Elements of a row before a thread's first; T threads share the row, 8 T
// elements to a piece.
template <int L>
__device__ __forceinline__ uint32_t piece_offset(uint32_t t)
{
    return L == kVectors ? kRv * t : kRv * (t & ~31u) + (L == kSingles ? 1u : 2u) * (t & 31u);
}

// Elements from a thread's first value to its value k.
template <int L>
__device__ __forceinline__ constexpr uint32_t value_at(uint32_t k)
{
    return L == kVectors ? k : L == kSingles ? 32 * k : 64 * (k / 2) + k % 2;
}

// How many of its eight values the row has: values 0 .. n - 1.
template <int L>
__device__ __forceinline__ uint32_t piece_count(uint32_t cols, uint32_t first)
{
    if (first >= cols) return 0u;
    const uint32_t left = cols - first;
    if constexpr (L == kVectors)
        return min(left, (uint32_t)kRv);
    else if constexpr (L == kSingles)
        return min((left + 31) / 32, (uint32_t)kRv);
    else
        return min(left / 64 * 2 + min(left % 64, 2u), (uint32_t)kRv);
}

// The same of piece i, where the first LEAD pieces are known to be whole.
template <int L, int T, int LEAD>
__device__ __forceinline__ uint32_t piece_count(uint32_t cols, uint32_t first, int i)
{
    return i < LEAD ? (uint32_t)kRv : piece_count<L>(cols, first + (uint32_t)(i * kRv * T));
}

// The halving fold (rowvec.cuh) of a thread's N values, absent ones up to a power
// of two +0.0.
template <int N>
__device__ __forceinline__ float fold(const float (&s)[N])
{
    constexpr int P = N <= 1 ? 1 : N <= 2 ? 2 : N <= 4 ? 4 : 8;
    static_assert(N <= 8, "");
    float a[P];
#pragma unroll
    for (int i = 0; i < P; i++) a[i] = i < N ? s[i] : 0.0f;
    return halving<P>(a);
}

// Whether the first NV pieces, which T threads (t: the thread's number among
// them) share, are whole in this warp; the same for the warp.
template <int T, int NV>
__device__ __forceinline__ bool warp_whole(uint32_t cols, uint32_t t)
{
    return __all_sync(kFull, kRv * ((t & ~31u) + (uint32_t)((NV - 1) * T)) + 256 <= cols);
}

// A thread's values as stored: words of two 16-bit values, or of one.
template <int DT>
struct Piece {
    uint32_t w[DT == kF32 ? 8 : 4];
};

// Whether a row of kPairs is read by words (the same in every lane).
__device__ __forceinline__ bool by_words(const void *p)
{
    return ((uintptr_t)p & 3u) == 0u;
}

// At p, the thread's first element.  Vectors: a row's last granule may reach
// past its end; what it brings is not one of the n.  words: by_words(p).
template <int DT, int L>
__device__ __forceinline__ void load_piece(const typename Elem<DT>::T *p, uint32_t n, Piece<DT> &q, bool words = false)
{
    if constexpr (L == kVectors) {
#pragma unroll
        for (uint32_t k = 0; k < (DT == kF32 ? 2 : 1); k++) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (n > 4 * k) u = ld16((const char *)p + 16 * k);
            q.w[4 * k] = u.x;
            q.w[4 * k + 1] = u.y;
            q.w[4 * k + 2] = u.z;
            q.w[4 * k + 3] = u.w;
        }
    } else if constexpr (L == kSingles) {
        if (n == kRv) {
#pragma unroll
            for (int k = 0; k < kRv; k++) q.w[k] = p[32 * k];
        } else {
#pragma unroll
            for (uint32_t k = 0; k < kRv; k++) q.w[k] = k < n ? p[32 * k] : 0u;
        }
    } else if (words && n == kRv) {
#pragma unroll
        for (int k = 0; k < 4; k++) q.w[k] = *reinterpret_cast<const uint32_t *>(p + 64 * k);
    } else {
        uint16_t e[kRv];
#pragma unroll
        for (uint32_t k = 0; k < kRv; k++) e[k] = k < n ? p[value_at<L>(k)] : (uint16_t)0;
#pragma unroll
        for (int k = 0; k < 4; k++) q.w[k] = pack2(e[2 * k], e[2 * k + 1]);
    }
}

template <int DT>
__device__ __forceinline__ void piece_values(const Piece<DT> &q, float (&f)[kRv])
{
    if constexpr (DT == kF32) {
#pragma unroll
        for (int k = 0; k < kRv; k++) f[k] = __uint_as_float(q.w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            f[2 * k] = leaf_lo<DT>(q.w[k]);
            f[2 * k + 1] = leaf_hi<DT>(q.w[k]);
        }
    }
}

__device__ __forceinline__ void zero_absent(uint32_t n, float (&f)[kRv])
{
    if (n == kRv) return;
#pragma unroll
    for (uint32_t k = 0; k < kRv; k++)
        if (k >= n) f[k] = 0.0f;
}

template <int DT, int L>
__device__ __forceinline__ void store_piece(typename Elem<DT>::T *p, uint32_t n, const float (&f)[kRv],
                                            bool words = false)
{
    uint32_t o[DT == kF32 ? 8 : 4];
#pragma unroll
    for (int k = 0; k < (DT == kF32 ? 8 : 4); k++) {
        if constexpr (DT == kF32)
            o[k] = __float_as_uint(f[k]);
        else
            o[k] = float2_to_word<DT>(f[2 * k], f[2 * k + 1]);
    }
    if (L == kVectors && n == kRv) {
#pragma unroll
        for (int k = 0; k < (DT == kF32 ? 8 : 4); k += 4)
            *reinterpret_cast<uint4 *>((char *)p + 4 * k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
    } else if (L == kPairs && words && n == kRv) {
#pragma unroll
        for (int k = 0; k < 4; k++) *reinterpret_cast<uint32_t *>(p + 64 * k) = o[DT == kF32 ? 0 : k];
    } else {
#pragma unroll
        for (uint32_t k = 0; k < kRv; k++)
            if (k < n) {
                if constexpr (DT == kF32)
                    p[value_at<L>(k)] = o[k];
                else
                    p[value_at<L>(k)] = (uint16_t)(o[k / 2] >> (16 * (k % 2)));
            }
    }
}

// 8-bit codes (vectors: at 8-byte aligned rows).
template <int L>
__device__ __forceinline__ void store_piece_codes(int8_t *p, uint32_t n, const float (&f)[kRv], float per)
{
    uint32_t c[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) c[k] = i8_code(f[k], per);
    if (L == kVectors && n == kRv) {
        uint32_t o[2];
#pragma unroll
        for (int k = 0; k < 2; k++)
            o[k] = __byte_perm(__byte_perm(c[4 * k], c[4 * k + 1], 0x0040), __byte_perm(c[4 * k + 2], c[4 * k + 3], 0x0040),
                               0x5410);
        *reinterpret_cast<uint2 *>(p) = make_uint2(o[0], o[1]);
    } else {
#pragma unroll
        for (uint32_t k = 0; k < kRv; k++)
            if (k < n) p[value_at<L>(k)] = (int8_t)c[k];
    }
}

// ---------------------------------------------------------------- pairs of values

__device__ __forceinline__ uint64_t pack_pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

// Sums only: a product of pairs may be fused with the sum of pairs that it goes
// into, its .rn notwithstanding (seen: xh * c and what it is taken from), and
// then rounds once instead of twice.
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void unpack_pair(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ void add8(float (&r)[kRv], const float (&a)[kRv], const float (&b)[kRv])
{
#pragma unroll
    for (int k = 0; k < kRv; k += 2)
        unpack_pair(add_pair(pack_pair(a[k], a[k + 1]), pack_pair(b[k], b[k + 1])), r[k], r[k + 1]);
}

__device__ __forceinline__ void add8(float (&r)[kRv], const float (&a)[kRv], float b)
{
#pragma unroll
    for (int k = 0; k < kRv; k += 2)
        unpack_pair(add_pair(pack_pair(a[k], a[k + 1]), pack_pair(b, b)), r[k], r[k + 1]);
}

__device__ __forceinline__ void mul8(float (&r)[kRv], const float (&a)[kRv], const float (&b)[kRv])
{
#pragma unroll
    for (int k = 0; k < kRv; k++) r[k] = __fmul_rn(a[k], b[k]);
}

__device__ __forceinline__ void mul8(float (&r)[kRv], const float (&a)[kRv], float b)
{
#pragma unroll
    for (int k = 0; k < kRv; k++) r[k] = __fmul_rn(a[k], b);
}

// From a thread's eight values the value of one vector (tree8): its own, or one
// of its warp's 32, the exchanges as in tree8_lanes.  Lane l ends with vector 8
// (l % 4) + l / 4 of kPairs.
template <int L>
__device__ __forceinline__ float piece_tree(const float (&e)[kRv])
{
    if constexpr (L == kVectors) {
        return tree8(e);
    } else if constexpr (L == kSingles) {
        return tree8_lanes(e);
    } else {
        const uint32_t lane = threadIdx.x & 31;
        float a[4], b[2];
#pragma unroll
        for (int k = 0; k < 4; k++) a[k] = __fadd_rn(e[2 * k], e[2 * k + 1]);
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const bool odd = lane & 1u;
            const float keep = odd ? a[2 * k + 1] : a[2 * k], give = odd ? a[2 * k] : a[2 * k + 1];
            b[k] = __fadd_rn(keep, __shfl_xor_sync(kFull, give, 1));
        }
        const bool odd = lane & 2u;
        return __fadd_rn(odd ? b[1] : b[0], __shfl_xor_sync(kFull, odd ? b[0] : b[1], 2));
    }
}

// The halving fold over those lanes.
template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    if constexpr (L == kVectors) {
        return halving_lanes(v);
    } else if constexpr (L == kSingles) {
        return halving_lanes_elem(v);
    } else {
#pragma unroll
        for (int k = 0; k < 5; k++) {
            constexpr int order[5] = {2, 1, 16, 8, 4};       // vector bits 4, 3, 2, 1, 0
            v = __fadd_rn(v, __shfl_xor_sync(kFull, v, order[k]));
        }
        return v;
    }
}

// team_sum (rowvec.cuh) of N values at once, with a barrier that the warps of a
// CTA may meet at different places of the code; `red`: N T floats.
template <int T, int L, int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float *red)
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if constexpr (T > 512) {
        // each warp folds the warps' values for some of the lanes and passes them on
        constexpr int W = T / 32;
        float *tot = red + N * W * 33;
#pragma unroll
        for (int i = 0; i < N; i++) red[(i * W + warp) * 33 + lane] = v[i];
        asm volatile("bar.sync 0;" ::: "memory");
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float s = halving_lanes(lane < W ? red[(i * W + lane) * 33 + warp] : 0.0f);
            if (lane == 0) tot[32 * i + warp] = s;
        }
        asm volatile("bar.sync 0;" ::: "memory");
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = tot[32 * i + lane];
    } else if constexpr (T > 32) {
#pragma unroll
        for (int i = 0; i < N; i++) red[i * T + threadIdx.x] = v[i];
        asm volatile("bar.sync 0;" ::: "memory");
#pragma unroll
        for (int i = 0; i < N; i++) {
            float f[T / 32];
#pragma unroll
            for (int w = 0; w < T / 32; w++) f[w] = red[i * T + 32 * w + lane];
            v[i] = halving<T / 32>(f);
        }
    }
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = lanes_sum<L>(v[i]);
}

template <int T, int N>
__host__ __device__ constexpr int team_sums_floats()
{
    return T <= 32 ? 1 : T <= 512 ? N * T : N * (T / 32 * 33 + 32);
}

// The largest of the team's values as team_max (rowvec.cuh) takes them.
template <int T>
__device__ __forceinline__ uint32_t team_most(uint32_t bits, uint32_t *red)
{
    bits = __reduce_max_sync(kFull, bits);
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = bits;
        asm volatile("bar.sync 0;" ::: "memory");
        bits = __reduce_max_sync(kFull, (threadIdx.x & 31) < T / 32 ? red[threadIdx.x & 31] : 0u);
    }
    return bits;
}

}  // namespace tcr
