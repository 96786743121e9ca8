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

// 16 codes at p, `left` of them inside the row, the rest read as 0.
// `aligned`: p is 16-byte aligned.  Otherwise the aligned granules that the
// codes touch are read and shifted (lanes may differ in their shift).
__device__ __forceinline__ uint4 ld_codes(const int8_t *p, uint32_t left, bool aligned)
{
    if (aligned && left >= 16) return ld16(p);
    left = min(left, 16u);
    const uint32_t m = (uint32_t)(uintptr_t)p & 15u;
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (left > 0) lo = ld16(p - m);
    if (m + left > 16) hi = ld16(p - m + 16);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t a[6], b[5], o[4];
#pragma unroll
    for (int k = 0; k < 6; k++) a[k] = (m & 8u) ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; k++) b[k] = (m & 4u) ? a[k + 1] : a[k];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        o[k] = __funnelshift_r(b[k], b[k + 1], 8u * (m & 3u));
        const int in = (int)left - 4 * k;                // codes of this word inside the row
        if (in < 4) o[k] = in <= 0 ? 0u : o[k] & (0xffffffffu >> (32 - 8 * in));
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
