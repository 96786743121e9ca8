// codes.cuh -- 8-bit codes on their way into a product, and its results on
// their way out; shared by the kernels of the 8-bit product.
#pragma once

#include "rowvec.cuh"

namespace tcr {

// Four codes of a word as two words of two binary16 values each.  A code
// with its sign bit flipped is q + 128; as the low byte under 0x64 it reads
// 1024 + q + 128, and subtracting 1152 leaves q, exactly.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// 16 codes as loaded: the 16-byte word that they are, or (GRAN) the two
// granules that they touch, to be shifted when they are used.
template <bool GRAN>
struct LoadedCodes {
    uint4 q[GRAN ? 2 : 1];
};

// 16 codes at p, all inside the row; GRAN = false: p is 16-byte aligned.  A
// granule without one of them is not read.  STREAM: read once, not worth a
// place in L1.
template <bool GRAN, bool STREAM>
__device__ __forceinline__ LoadedCodes<GRAN> load_codes(const int8_t *p)
{
    LoadedCodes<GRAN> r;
    if constexpr (GRAN) {
        const uint32_t m = (uint32_t)(uintptr_t)p & 15u;
        r.q[0] = ld16(p - m);
        r.q[1] = m > 0 ? ld16(p - m + 16) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        r.q[0] = STREAM ? ld_stream(p) : ld16(p);
    }
    return r;
}

// The same with `left` of the 16 inside the row.
template <bool GRAN>
__device__ __forceinline__ LoadedCodes<GRAN> load_last_codes(const int8_t *p, uint32_t left)
{
    LoadedCodes<GRAN> r;
    const uint32_t m = GRAN ? (uint32_t)(uintptr_t)p & 15u : 0u;
#pragma unroll
    for (int k = 0; k < (GRAN ? 2 : 1); k++) {
        r.q[k] = make_uint4(0u, 0u, 0u, 0u);
        if (left > 0 && m + min(left, 16u) > 16u * k) r.q[k] = ld16(p - m + 16 * k);
    }
    return r;
}

// Their four words, codes past the row 0 (lanes may differ in their shift).
template <bool GRAN>
__device__ __forceinline__ uint4 use_codes(const LoadedCodes<GRAN> &l, const int8_t *p, uint32_t left, bool whole)
{
    uint32_t o[4] = {l.q[0].x, l.q[0].y, l.q[0].z, l.q[0].w};
    if constexpr (GRAN) {
        const uint32_t m = (uint32_t)(uintptr_t)p & 15u;
        const uint32_t w[8] = {o[0], o[1], o[2], o[3], l.q[1].x, l.q[1].y, l.q[1].z, l.q[1].w};
        uint32_t a[6], b[5];
#pragma unroll
        for (int k = 0; k < 6; k++) a[k] = (m & 8u) ? w[k + 2] : w[k];
#pragma unroll
        for (int k = 0; k < 5; k++) b[k] = (m & 4u) ? a[k + 1] : a[k];
#pragma unroll
        for (int k = 0; k < 4; k++) o[k] = __funnelshift_r(b[k], b[k + 1], 8u * (m & 3u));
    }
    if (!whole) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int in = (int)left - 4 * k;                // codes of this word inside the row
            if (in < 4) o[k] = in <= 0 ? 0u : o[k] & (0xffffffffu >> (32 - 8 * in));
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The same for 8 codes at any alignment, by 8-byte granules.
__device__ __forceinline__ uint2 ld_codes8(const int8_t *p, uint32_t left)
{
    left = min(left, 8u);
    const uint32_t m = (uint32_t)(uintptr_t)p & 7u;
    uint2 lo = make_uint2(0u, 0u), hi = lo;
    if (left > 0) lo = *reinterpret_cast<const uint2 *>(p - m);
    if (m + left > 8) hi = *reinterpret_cast<const uint2 *>(p - m + 8);
    const bool far = m & 4u;
    const uint32_t a = far ? lo.y : lo.x, b = far ? hi.x : lo.y, c = far ? hi.y : hi.x;
    uint2 r = make_uint2(__funnelshift_r(a, b, 8u * (m & 3u)), __funnelshift_r(b, c, 8u * (m & 3u)));
    if (left < 4)
        r = make_uint2(left ? r.x & (0xffffffffu >> (32 - 8 * left)) : 0u, 0u);
    else if (left < 8)
        r.y = left > 4 ? r.y & (0xffffffffu >> (32 - 8 * (left - 4))) : 0u;
    return r;
}

__device__ __forceinline__ void store_out(void *C, int dtype, size_t i, int acc, float sa, float sw)
{
    if (dtype == kOutI32) {
        ((int *)C)[i] = acc;
        return;
    }
    const float v = __fmul_rn(__fmul_rn((float)acc, sa), sw);
    if (dtype == kF16)
        ((uint16_t *)C)[i] = float_to_elem<kF16>(v);
    else if (dtype == kBF16)
        ((uint16_t *)C)[i] = float_to_elem<kBF16>(v);
    else
        ((float *)C)[i] = v;
}

}  // namespace tcr
