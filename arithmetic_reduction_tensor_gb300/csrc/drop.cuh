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

// seed and offset as the kernel uses them.
__device__ __forceinline__ DropArgs drop_resolve(const DropArgs &a)
{
    DropArgs d = a;
    if (a.t != 0u && a.state) {
        const unsigned long long seed = a.state[0], offset = a.state[1];
        d.k0 = (uint32_t)seed;
        d.k1 = (uint32_t)(seed >> 32);
        d.c2 = (uint32_t)offset;
        d.c3 = (uint32_t)(offset >> 32);
    }
    return d;
}

__device__ __forceinline__ uint4 philox10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                          uint32_t k1)
{
#pragma unroll
    for (int i = 0; i < 10; i++) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// dropout of the values of vector v of row r.
__device__ __forceinline__ void drop8(const DropArgs &d, uint32_t v, uint32_t r, float (&x)[kRv])
{
    const uint4 q = philox10(v, r, d.c2, d.c3, d.k0, d.k1);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
        x[2 * k] = (w[k] & 0xffffu) >= d.t ? __fmul_rn(x[2 * k], d.s) : 0.0f;
        x[2 * k + 1] = (w[k] >> 16) >= d.t ? __fmul_rn(x[2 * k + 1], d.s) : 0.0f;
    }
}

// The same where lane l of a warp holds elements 32 j + l of the 256 of 32
// vectors, `v` the vector of the lane's number among them: each lane forms
// the eight bits of its vector, and the lanes hand them round.  Every lane
// of the warp calls it.
__device__ __forceinline__ void drop8_lanes(const DropArgs &d, uint32_t v, uint32_t r, float (&x)[kRv])
{
    const uint4 q = philox10(v, r, d.c2, d.c3, d.k0, d.k1);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const uint32_t lane = threadIdx.x & 31;
    uint32_t keep = 0;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if ((w[k] & 0xffffu) >= d.t) keep |= 1u << (2 * k);
        if ((w[k] >> 16) >= d.t) keep |= 2u << (2 * k);
    }
#pragma unroll
    for (int j = 0; j < kRv; j++) {
        const uint32_t m = __shfl_sync(kFull, keep, 4 * j + (int)(lane >> 3));
        x[j] = (m >> (lane & 7u)) & 1u ? __fmul_rn(x[j], d.s) : 0.0f;
    }
}

// Dropout of a thread's eight values, as vector v (ELEM = false) or in the
// layout of tree8_lanes; a warp-uniform no-op where nothing is dropped.
template <bool ELEM>
__device__ __forceinline__ void drop_values(const DropArgs &d, uint32_t v, size_t r, float (&x)[kRv])
{
    if (d.t == 0u) return;
    if constexpr (ELEM)
        drop8_lanes(d, v, (uint32_t)r, x);
    else
        drop8(d, v, (uint32_t)r, x);
}

}  // namespace tcr
