// drop.cuh -- dropout's mask from a counter-based generator.
//
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel Random Numbers: As
// Easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products on a
// counter of four words, keyed by two.  Element j of row r takes 16 bits of
// the block with counter (j / 8, r, offset's low word, its high word) and key
// (seed's low word, its high word): half j % 2 (0 the low one) of word
// (j % 8) / 2.  It is kept where those bits are at least t = rint(65536 p).  So
// the mask depends on seed, offset, row and column alone, and any pass over
// the rows forms it again instead of reading it.
//
// 16 bits an element, not 32: the generator's 64-bit products are what
// dropout computes, and one block then serves a whole vector of 8; p is met to
// 2^-17, and the factor 65536 / (65536 - t) is that of the t used.
#pragma once

#include "kernels.cuh"
#include "rowvec.cuh"

namespace tcr {

// Layouts of a thread's eight values (piece.cuh).
constexpr int kVectors = 0, kSingles = 1, kPairs = 2;

// A call's dropout as the kernel uses it.  The round keys of a seed that the
// host knows come with the launch, as constants that the rounds take as
// operands; those of a seed on the device are summed up in registers, round by
// round.
struct Drop {
    const DropArgs &a;
    uint32_t t, k0, k1, c2, c3;
    bool device;
    __device__ __forceinline__ explicit Drop(const DropArgs &args) : a(args), t(args.t)
    {
        k0 = k1 = 0u;
        c2 = a.c2;
        c3 = a.c3;
        device = t != 0u && a.state;
        if (device) {
            const unsigned long long seed = a.state[0], offset = a.state[1];
            k0 = (uint32_t)seed;
            k1 = (uint32_t)(seed >> 32);
            c2 = (uint32_t)offset;
            c3 = (uint32_t)(offset >> 32);
        }
    }
};

__device__ __forceinline__ void philox_round(uint32_t &c0, uint32_t &c1, uint32_t &c2, uint32_t &c3, uint32_t k0,
                                             uint32_t k1)
{
    const uint64_t a = (uint64_t)c0 * kPhiloxM0, b = (uint64_t)c2 * kPhiloxM1;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
}

__device__ __forceinline__ uint4 philox10(const Drop &d, uint32_t c0, uint32_t c1)
{
    uint32_t c2 = d.c2, c3 = d.c3;
    if (!d.device) {
#pragma unroll
        for (int i = 0; i < 10; i++) philox_round(c0, c1, c2, c3, d.a.rk[2 * i], d.a.rk[2 * i + 1]);
    } else {
        uint32_t k0 = d.k0, k1 = d.k1;
#pragma unroll 1
        for (int i = 0; i < 10; i++) {
            philox_round(c0, c1, c2, c3, k0, k1);
            k0 += kPhiloxW0;
            k1 += kPhiloxW1;
        }
    }
    return make_uint4(c0, c1, c2, c3);
}

// dropout of the values of vector v of row r.
__device__ __forceinline__ void drop8(const Drop &d, uint32_t v, uint32_t r, float (&x)[kRv])
{
    const uint4 q = philox10(d, v, r);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const uint32_t top = d.t << 16;                     // (t <= 65535 here)
#pragma unroll
    for (int k = 0; k < 4; k++) {
        x[2 * k] = (w[k] << 16) >= top ? __fmul_rn(x[2 * k], d.a.s) : 0.0f;
        x[2 * k + 1] = w[k] >= top ? __fmul_rn(x[2 * k + 1], d.a.s) : 0.0f;
    }
}

// The same where a warp shares 256 elements in another layout, `v` the vector of
// the lane's number among their 32: each lane forms the eight bits of its
// vector, and the lanes hand them round.  Every lane of the warp calls it.
template <int L>
__device__ __forceinline__ void drop8_lanes(const Drop &d, uint32_t v, uint32_t r, float (&x)[kRv])
{
    const uint4 q = philox10(d, v, r);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const uint32_t lane = threadIdx.x & 31;
    uint32_t keep = 0;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if ((w[k] & 0xffffu) >= d.t) keep |= 1u << (2 * k);
        if ((w[k] >> 16) >= d.t) keep |= 2u << (2 * k);
    }
    if constexpr (L == kSingles) {
#pragma unroll
        for (int j = 0; j < kRv; j++) {
            const uint32_t m = __shfl_sync(kFull, keep, 4 * j + (int)(lane >> 3)) >> (lane & 7u);
            x[j] = m & 1u ? __fmul_rn(x[j], d.a.s) : 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t m = __shfl_sync(kFull, keep, 8 * j + (int)(lane >> 2)) >> (2 * (lane & 3u));
            x[2 * j] = m & 1u ? __fmul_rn(x[2 * j], d.a.s) : 0.0f;
            x[2 * j + 1] = m & 2u ? __fmul_rn(x[2 * j + 1], d.a.s) : 0.0f;
        }
    }
}

// Dropout of a thread's eight values in a layout of piece.cuh; a uniform no-op
// where nothing is dropped.
template <int L>
__device__ __forceinline__ void drop_values(const Drop &d, uint32_t v, size_t r, float (&x)[kRv])
{
    if (d.t == 0u) return;
    if (d.t == 65536u) {
#pragma unroll
        for (int k = 0; k < kRv; k++) x[k] = 0.0f;
        return;
    }
    if constexpr (L == kVectors)
        drop8(d, v, (uint32_t)r, x);
    else
        drop8_lanes<L>(d, v, (uint32_t)r, x);
}

}  // namespace tcr
