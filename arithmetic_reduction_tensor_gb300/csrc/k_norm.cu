// k_norm.cu -- RMS norm with the residual's addition, and rows into 8-bit
// integers with one scale a row: one pass over the data per row.
//
//   norm      h = x + r (binary32),  y = (h * rstd) * w,
//             rstd = 1 / sqrt(S / cols + eps), S the row sum of fl32(h * h)
//   quantise  y = x, or (g / (1 + exp(-g))) * x with a gate g
//   codes     scale = max|y| / 127, q = rint(y * (127 / max|y|))
//
// A team of T threads (a warp for short rows, else a CTA) keeps the row in
// registers, NV vectors a thread, so every byte is read once (rows of more than
// 32768 columns: once a step, row_long_kernel); S is summed in the declared
// order of rowvec.cuh.  Every step outside the gate is one
// binary32 operation rounded to nearest, so the norm's results are pinned
// bit for bit by the inputs.  The work is bound by memory traffic: 65536 x
// 4096 binary16 279 us to codes, 325 to binary16, 219 for gated codes, 135 for
// codes without a gate, 127 for reading codes back (6.0 to 6.7 TB/s).  Lengths
// that leave much of a team's vectors empty run slower (16384 x 2560 bfloat16 to
// codes 0.67 of the copy rate).  Rows that are not 16-byte aligned run at the
// full rate in binary32, at a third (6000 x 12001 to codes) to three quarters of
// it in 16 bits, bound by latency (row_elem_kernel).
#include "kernels.cuh"
#include "rowvec.cuh"

namespace tcr {

constexpr int kOutSame = 0, kOutI8 = 1;

// The rows of one call that a team works on.
template <int DT>
struct RowPtrs {
    using E = typename Elem<DT>::T;
    const E *x, *r;
    E *h;
    void *y;
    __device__ __forceinline__ RowPtrs(const RowArgs &a, size_t row, size_t y_bytes)
    {
        x = (const E *)a.x + row * a.ldx;
        r = a.r ? (const E *)a.r + row * a.ldr : nullptr;
        h = a.h ? (E *)a.h + row * a.ldh : nullptr;
        y = (char *)a.y + row * a.ldy * y_bytes;
    }
};

// The values of a vector from its inputs as loaded.  The gate's exponential and
// quotient are CUDA's fast ones: their error, (8 + 1.2 max(0, -g)) 2^-23, is
// far below a code's half step, 2^-8 of the row's largest value, and reaches
// the scale in its last bits.  The quotient is 0 once 1 + exp(-g) passes 2^126 (g
// below -87.34), where the factor is less than 1.1e-36.
template <int DT, int OP>
__device__ __forceinline__ void row_value(const RawVec<DT> &x, const RawVec<DT> &r, bool has_r, float (&y)[kRv])
{
    unpack<DT>(x, y);
    if (!has_r) return;
    float b[kRv];
    unpack<DT>(r, b);
#pragma unroll
    for (int k = 0; k < kRv; k++)
        y[k] = OP == kRowNorm ? __fadd_rn(y[k], b[k])
                              : __fmul_rn(__fdividef(b[k], __fadd_rn(1.0f, __expf(-b[k]))), y[k]);
}

template <int DT, int OP>
__device__ __forceinline__ void row_value(const RowArgs &a, const RowPtrs<DT> &p, uint32_t cols, uint32_t v,
                                          float (&y)[kRv])
{
    const RawVec<DT> x = load_raw<DT>(p.x, cols, v, a.al_x);
    const RawVec<DT> r = p.r ? load_raw<DT>(p.r, cols, v, a.al_r) : RawVec<DT>();
    row_value<DT, OP>(x, r, p.r != nullptr, y);
}

__device__ __forceinline__ float squares8(const float (&h)[kRv])
{
    float e[kRv];
#pragma unroll
    for (int k = 0; k < kRv; k++) e[k] = __fmul_rn(h[k], h[k]);
    return tree8(e);
}

__device__ __forceinline__ float rstd_of(float s, uint32_t cols, float eps)
{
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(s, (float)cols), eps));
}

template <int DT>
__device__ __forceinline__ RawVec<DT> load_weight(const RowArgs &a, uint32_t cols, uint32_t v)
{
    return a.w ? load_raw<DT>((const typename Elem<DT>::T *)a.w, cols, v, a.al_w) : RawVec<DT>();
}

template <int DT>
__device__ __forceinline__ void apply_norm(const RawVec<DT> &wr, bool has_w, float rstd, float (&h)[kRv])
{
    float w[kRv];
    if (has_w) unpack<DT>(wr, w);
#pragma unroll
    for (int k = 0; k < kRv; k++) {
        h[k] = __fmul_rn(h[k], rstd);
        if (has_w) h[k] = __fmul_rn(h[k], w[k]);
    }
}

// Rows of at most 8 T NV columns, NV vectors a thread: teams of T threads
// (T = 32: eight to a CTA; else the CTA) walk the rows, each loading its next
// row before it finishes the current one, so that loads stay in flight
// across the row's barriers.  Rows are 16-byte aligned (codes 8-byte).  MINB:
// the CTAs per SM that the registers allow.
template <int DT, int OP, int OUT, int T, int NV, int MINB>
__global__ void __launch_bounds__(T == 32 ? 256 : T, MINB)
row_stream_kernel(const RowArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][team_floats<T>()];
    __shared__ uint32_t redm[2][32];
    using E = typename Elem<DT>::T;
    constexpr size_t y_bytes = OUT == kOutI8 ? 1 : sizeof(E);
    const uint32_t t = T == 32 ? threadIdx.x & 31 : threadIdx.x, cols = (uint32_t)a.cols;
    const uint32_t threads = T == 32 ? 32 : blockDim.x;
    const size_t team = T == 32 ? (size_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    const size_t teams = T == 32 ? (size_t)gridDim.x * 8 : gridDim.x;
    const bool has_r = a.r != nullptr, has_w = a.w != nullptr;
    RawVec<DT> w[NV];
    LoadedVec<DT, false> x[NV], b[NV];
    auto load = [&](size_t r) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            x[i] = load_vec<DT, false>((const E *)a.x + r * a.ldx, cols, t + i * T);
            b[i] = has_r ? load_vec<DT, false>((const E *)a.r + r * a.ldr, cols, t + i * T) : LoadedVec<DT, false>();
        }
    };
#pragma unroll
    for (int i = 0; i < NV; i++) w[i] = OP == kRowNorm ? load_weight<DT>(a, cols, t + i * T) : RawVec<DT>();
    if (team < a.rows) load(team);
    int buf = 0;
    for (size_t r = team; r < a.rows; r += teams, buf ^= 1) {
        float y[NV][kRv];
#pragma unroll
        for (int i = 0; i < NV; i++)
            row_value<DT, OP>(use_vec<DT, false>(x[i], (const E *)a.x + r * a.ldx, cols, t + i * T),
                              use_vec<DT, false>(b[i], (const E *)a.r + r * a.ldr, cols, t + i * T), has_r, y[i]);
        if (r + teams < a.rows) load(r + teams);
        // two buffers each: a thread reaches the next row's write of one only
        // after every thread has passed a barrier of the row between
        float m = 0.0f;
        if constexpr (OP == kRowNorm) {
            float s[NV];
#pragma unroll
            for (int i = 0; i < NV; i++) s[i] = squares8(y[i]);
            const float rstd = rstd_of(team_sum<T>(halving<NV>(s), red[buf], threads), cols, a.eps);
            if (a.rstd && t == 0) a.rstd[r] = rstd;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                if (kRv * ((t & ~31u) + i * T) >= cols) continue;         // whole warps: stores are warp-wide
                if (a.h) store_vec<DT>((E *)a.h + r * a.ldh, cols, t + i * T, true, y[i]);
                apply_norm<DT>(w[i], has_w, rstd, y[i]);
            }
        }
        char *out = (char *)a.y + r * a.ldy * y_bytes;
        float scale, per = 0.0f;
        if constexpr (OUT == kOutI8) {
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (kRv * (t + i * T) < cols) m = amax8(y[i], m);
            i8_scale(team_max<T>(__float_as_uint(m), redm[buf], threads), scale, per);
            if (t == 0) a.scale[r] = scale;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (kRv * ((t & ~31u) + i * T) >= cols) continue;
            if constexpr (OUT == kOutSame)
                store_vec<DT>((E *)out, cols, t + i * T, true, y[i]);
            else
                store_codes((int8_t *)out, cols, t + i * T, true, y[i], per);
        }
    }
}

// The same for rows at any alignment, element by element: lane l of a team's
// warp w holds elements 8 T i + 256 w + 32 j + l, so every access is of
// consecutive elements, 32 a warp, whatever the alignment; the sums are those
// of the vectors all the same (tree8_lanes).  At 16 bits (two bytes a lane and
// access) bound by the latency of exchanges and barriers with 16 warps an SM,
// issuing on 54% of cycles; at 32 by memory.  Norm to codes 100000 x 1001
// binary16 165 us (0.62 of the copy rate), 20000 x 5001 bfloat16 206 (0.50),
// 20000 x 2001 binary32 81 (0.94).  Shifting 16-byte granules in registers and
// joining lanes' vectors for the stores took 272, 246 and 167.
template <int DT, int OP, int OUT, int T, int NV, int MINB>
__global__ void __launch_bounds__(T == 32 ? 256 : T, MINB)
row_elem_kernel(const RowArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[2][team_floats<T>()];
    __shared__ uint32_t redm[2][32];
    using E = typename Elem<DT>::T;
    const uint32_t t = T == 32 ? threadIdx.x & 31 : threadIdx.x, cols = (uint32_t)a.cols;
    const uint32_t threads = T == 32 ? 32 : blockDim.x;
    const uint32_t e0 = 8 * (t & ~31u) + (t & 31);           // the thread's first element
    const size_t team = T == 32 ? (size_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    const size_t teams = T == 32 ? (size_t)gridDim.x * 8 : gridDim.x;
    const bool has_r = a.r != nullptr, has_w = OP == kRowNorm && a.w != nullptr;
    // whether all 256 elements of a warp's stretch i exist
    auto whole = [&](int i) { return 8 * ((t & ~31u) + (uint32_t)(i * T)) + 256 <= cols; };
    auto load8 = [&](const E *row, int i, E (&v)[kRv]) {
        const uint32_t e = e0 + (uint32_t)(8 * T * i);
        if (whole(i)) {
#pragma unroll
            for (int j = 0; j < kRv; j++) v[j] = row[e + 32 * j];
        } else {
#pragma unroll
            for (int j = 0; j < kRv; j++) v[j] = e + 32 * j < cols ? row[e + 32 * j] : (E)0;
        }
    };
    E x[NV][kRv], b[NV][kRv], w[NV][kRv];
    auto load = [&](size_t r) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            load8((const E *)a.x + r * a.ldx, i, x[i]);
            if (has_r) load8((const E *)a.r + r * a.ldr, i, b[i]);
        }
    };
#pragma unroll
    for (int i = 0; i < NV; i++) {
#pragma unroll
        for (int j = 0; j < kRv; j++) w[i][j] = (E)0;
        if (has_w) load8((const E *)a.w, i, w[i]);
    }
    if (team < a.rows) load(team);
    int buf = 0;
    for (size_t r = team; r < a.rows; r += teams, buf ^= 1) {
        float y[NV][kRv];
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < kRv; j++) {
                y[i][j] = elem_to_float<DT>(x[i][j]);
                if (has_r) {
                    const float g = elem_to_float<DT>(b[i][j]);
                    y[i][j] = OP == kRowNorm ? __fadd_rn(y[i][j], g)
                                             : __fmul_rn(__fdividef(g, __fadd_rn(1.0f, __expf(-g))), y[i][j]);
                }
            }
        if (r + teams < a.rows) load(r + teams);
        // (two buffers, as in row_stream_kernel)
        if constexpr (OP == kRowNorm) {
            float s[NV];
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float e[kRv];
#pragma unroll
                for (int j = 0; j < kRv; j++) e[j] = __fmul_rn(y[i][j], y[i][j]);
                s[i] = tree8_lanes(e);
            }
            const float rstd = rstd_of(team_sum<T, true>(halving<NV>(s), red[buf], threads), cols, a.eps);
            if (a.rstd && t == 0) a.rstd[r] = rstd;
            E *h = a.h ? (E *)a.h + r * a.ldh : nullptr;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const uint32_t e = e0 + (uint32_t)(8 * T * i);
                const bool all = whole(i);
#pragma unroll
                for (int j = 0; j < kRv; j++) {
                    if (h && (all || e + 32 * j < cols)) h[e + 32 * j] = float_to_elem<DT>(y[i][j]);
                    y[i][j] = __fmul_rn(y[i][j], rstd);
                    if (has_w) y[i][j] = __fmul_rn(y[i][j], elem_to_float<DT>(w[i][j]));
                }
            }
        }
        if constexpr (OUT == kOutSame) {
            E *out = (E *)a.y + r * a.ldy;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const uint32_t e = e0 + (uint32_t)(8 * T * i);
                const bool all = whole(i);
#pragma unroll
                for (int j = 0; j < kRv; j++)
                    if (all || e + 32 * j < cols) out[e + 32 * j] = float_to_elem<DT>(y[i][j]);
            }
        } else {
            float m = 0.0f, scale, per;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const uint32_t e = e0 + (uint32_t)(8 * T * i);
                if (!whole(i)) {
                    // absent elements are 0 times a possibly infinite rstd
#pragma unroll
                    for (int j = 0; j < kRv; j++)
                        if (e + 32 * j >= cols) y[i][j] = 0.0f;
                }
                m = amax8(y[i], m);
            }
            i8_scale(team_max<T>(__float_as_uint(m), redm[buf], threads), scale, per);
            if (t == 0) a.scale[r] = scale;
            int8_t *out = (int8_t *)a.y + r * a.ldy;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const uint32_t e = e0 + (uint32_t)(8 * T * i);
                const bool all = whole(i);
#pragma unroll
                for (int j = 0; j < kRv; j++)
                    if (all || e + 32 * j < cols) out[e + 32 * j] = (int8_t)i8_code(y[i][j], per);
            }
        }
    }
}

// Rows of at most 8 T NV columns, one CTA a row, NV vectors a thread.
template <int DT, int OP, int OUT, int T, int NV>
__global__ void __launch_bounds__(T)
row_kernel(const RowArgs a)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[team_floats<T>()];
    __shared__ uint32_t redm[32];
    using E = typename Elem<DT>::T;
    const size_t r = blockIdx.x;
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    const RowPtrs<DT> p(a, r, OUT == kOutI8 ? 1 : sizeof(E));
    float y[NV][kRv];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const uint32_t v = t + (uint32_t)(i * T);
        if (kRv * v < cols) {
            row_value<DT, OP>(a, p, cols, v, y[i]);
        } else {
#pragma unroll
            for (int k = 0; k < kRv; k++) y[i][k] = 0.0f;
        }
    }
    float rstd = 0.0f;
    if constexpr (OP == kRowNorm) {
        float s[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) s[i] = squares8(y[i]);
        rstd = rstd_of(team_sum<T>(halving<NV>(s), red), cols, a.eps);
        if (a.rstd && t == 0) a.rstd[r] = rstd;
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const uint32_t v = t + (uint32_t)(i * T);
        if (kRv * (v & ~31u) >= cols) continue;         // whole warps: stores are warp-wide
        if constexpr (OP == kRowNorm) {
            if (p.h) store_vec<DT>(p.h, cols, v, a.al_h, y[i]);
            apply_norm<DT>(load_weight<DT>(a, cols, v), a.w != nullptr, rstd, y[i]);
        }
        if constexpr (OUT == kOutSame)
            store_vec<DT>((E *)p.y, cols, v, a.al_y, y[i]);
        else
            m = amax8(y[i], m);
    }
    if constexpr (OUT == kOutI8) {
        float scale, per;
        i8_scale(team_max<T>(__float_as_uint(m), redm), scale, per);
        if (t == 0) a.scale[r] = scale;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t v = t + (uint32_t)(i * T);
            if (kRv * (v & ~31u) < cols) store_codes((int8_t *)p.y, cols, v, a.al_y, y[i], per);
        }
    }
}

// Longer rows: a CTA of T threads reads the row once per step (the sum, the
// largest magnitude, the outputs).  h may be written over x or r: it is
// stored in the last step only.
template <int DT, int OP, int OUT>
__global__ void __launch_bounds__(kRowLongT)
row_long_kernel(const RowArgs a)
{
    constexpr uint32_t T = kRowLongT;
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float red[team_floats<(int)T>()];
    __shared__ uint32_t redm[32];
    using E = typename Elem<DT>::T;
    const size_t r = blockIdx.x;
    const uint32_t t = threadIdx.x, cols = (uint32_t)a.cols;
    const RowPtrs<DT> p(a, r, OUT == kOutI8 ? 1 : sizeof(E));
    const uint32_t nvec = (cols + kRv - 1) / kRv;
    const uint32_t steps = (nvec + T - 1) / T;
    const int bits = ceil_log2_sz(steps);
    float rstd = 0.0f;
    float y[kRv];
    if constexpr (OP == kRowNorm) {
        TreeCounter<16> tc;
        for (uint32_t j = 0; j < (1u << bits); j++) {
            const uint32_t v = t + bit_reverse(j, bits) * T;
            float s = 0.0f;
            if (v < nvec) {
                row_value<DT, OP>(a, p, cols, v, y);
                s = squares8(y);
            }
            tc.push(s);
        }
        rstd = rstd_of(team_sum<T>(tc.finish(), red), cols, a.eps);
        if (a.rstd && t == 0) a.rstd[r] = rstd;
    }
    float per = 0.0f;
    if constexpr (OUT == kOutI8) {
        float m = 0.0f;
        for (uint32_t v = t; v < nvec; v += T) {
            row_value<DT, OP>(a, p, cols, v, y);
            if constexpr (OP == kRowNorm) apply_norm<DT>(load_weight<DT>(a, cols, v), a.w != nullptr, rstd, y);
            m = amax8(y, m);
        }
        float scale;
        i8_scale(team_max<T>(__float_as_uint(m), redm), scale, per);
        if (t == 0) a.scale[r] = scale;
    }
    for (uint32_t i = 0; i < steps; i++) {              // whole warps: stores are warp-wide
        const uint32_t v = t + i * T;
        row_value<DT, OP>(a, p, cols, v, y);
        if constexpr (OP == kRowNorm) {
            if (p.h) store_vec<DT>(p.h, cols, v, a.al_h, y);
            apply_norm<DT>(load_weight<DT>(a, cols, v), a.w != nullptr, rstd, y);
        }
        if constexpr (OUT == kOutSame)
            store_vec<DT>((E *)p.y, cols, v, a.al_y, y);
        else
            store_codes((int8_t *)p.y, cols, v, a.al_y, y, per);
    }
}

// ---------------------------------------------------------------- codes read back

// Four codes as binary32: with its sign bit flipped a code is q + 128, as
// the low byte of 2^23's pattern 2^23 + q + 128, and one subtraction leaves q.
__device__ __forceinline__ void codes4(uint32_t w, float *f)
{
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int k = 0; k < 4; k++)
        f[k] = __fsub_rn(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650u | (uint32_t)k)), 8388736.0f);
}

// y = q * scale[row], 8 codes a thread and step; a team of 2^team_log2
// threads walks each row, a warp at least (short rows leave lanes idle
// rather than split a warp between rows).  ELEM: the codes or y are not
// aligned, and lane l of a warp takes elements 32 j + l of 256 (the accesses
// of row_elem_kernel): 6151 x 5001 bfloat16 17 us, 100000 x 1001 binary16 70,
// 6000 x 8003 binary32 44; with shifted granules 24, 82 and 42.
template <int DT, bool ELEM>
__global__ void __launch_bounds__(256)
dequant_kernel(const int8_t *q, size_t ldq, const float *scale, typename Elem<DT>::T *y, size_t ldy,
               size_t rows, uint32_t cols, int team_log2)
{
    pdl_launch_dependents();
    pdl_wait_primary();
    const size_t r = ((size_t)blockIdx.x << (8 - team_log2)) + (threadIdx.x >> team_log2);
    if (r >= rows) return;
    const float s = scale[r];
    const int8_t *row = q + r * ldq;
    typename Elem<DT>::T *out = y + r * ldy;
    const uint32_t team = 1u << team_log2;
    for (uint32_t v = threadIdx.x & (team - 1); kRv * (v & ~31u) < cols; v += team) {
        if constexpr (ELEM) {
            const uint32_t at = kRv * (v & ~31u) + (v & 31u);
            const bool whole = kRv * (v & ~31u) + 256 <= cols;
            uint32_t c[kRv];
#pragma unroll
            for (int j = 0; j < kRv; j++) c[j] = whole || at + 32 * j < cols ? (uint8_t)row[at + 32 * j] : 0u;
#pragma unroll
            for (int j = 0; j < kRv; j++) {
                const float f = __fsub_rn(__uint_as_float((c[j] ^ 0x80u) | 0x4b000000u), 8388736.0f);
                if (whole || at + 32 * j < cols) out[at + 32 * j] = float_to_elem<DT>(__fmul_rn(f, s));
            }
        } else {
            // the granule of a row's last codes reaches past its end, not
            // past its 8 bytes
            uint2 w = make_uint2(0u, 0u);
            if (vec_left(cols, v)) w = *reinterpret_cast<const uint2 *>(row + kRv * v);
            float f[kRv];
            codes4(w.x, f);
            codes4(w.y, f + 4);
#pragma unroll
            for (int k = 0; k < kRv; k++) f[k] = __fmul_rn(f[k], s);
            store_vec<DT>(out, cols, v, true, f);
        }
    }
}

// ---------------------------------------------------------------- host

namespace {

// A launch of row_stream_kernel: as many CTAs as 152 SMs hold (or one team
// a row).
template <int DT, int OP, int OUT, bool ELEM, int T, int NV, int MINB>
const void *stream_of(size_t nvec, size_t rows, int &threads, size_t &grid)
{
    threads = T == 32 ? 256 : NV == 1 ? (int)((nvec + 31) / 32 * 32) : T;
    const size_t need = T == 32 ? (rows + 7) / 8 : rows;
    const size_t full = (size_t)152 * (size_t)(T == 32 ? MINB : MINB * T / threads);
    grid = need < full ? need : full;
    if constexpr (ELEM)
        return (const void *)row_elem_kernel<DT, OP, OUT, T, NV, MINB>;
    else
        return (const void *)row_stream_kernel<DT, OP, OUT, T, NV, MINB>;
}

// Which shape serves a row length: the fastest of those measured at it, on
// aligned rows.  A CTA an SM holds too few rows across the barriers, and a
// thread's registers (its vectors, the next row's, the weight's) decide how
// many CTAs fit: 65536 x 4096 binary16 with codes takes 277 us with 256
// threads of 2 vectors and 3 CTAs an SM, 410 with 512 x 1 and 2, 314 with
// 256 x 2 and 4 (spills), 303 with 128 x 4 and 4; 16384 x 8192 bfloat16 150
// with 256 x 4 and 2, 189 with 1024 x 1.  The gate needs no weight and one
// barrier, so one CTA more fits.  By elements: norm 20000 x 5001 bfloat16 206
// us with 256 x 3, 232 with 1024 x 1; 6000 x 12001 232 with 1024 x 2 (some
// spills; binary32 234), 319 with row_kernel (binary32 227); the gate 133 with
// 1024 x 1 against 138, and 164 with 1024 x 2 against 139.  One CTA more an SM
// loses: norm to codes 100000 x 1001 binary16 218 against 166.  At 257 to 384 vectors two a thread leave
// much of the CTA idle: the gate 512 x 1 43 us, 256 x 2 60 (16384 x 2304
// bfloat16; x 3000 55 and 61), by elements 47 and 74 (x 2051; x 3001 61 and
// 74); norm to codes by elements 84 and 95 at 2051, 109 and 96 at 3001.
template <int DT, int OP, int OUT>
const void *pick(size_t nvec, size_t rows, bool elem, int &threads, size_t &grid)
{
#define TCR_STREAM(T_, NV_, MINB_) return stream_of<DT, OP, OUT, false, T_, NV_, MINB_>(nvec, rows, threads, grid)
#define TCR_ELEM(T_, NV_, MINB_) return stream_of<DT, OP, OUT, true, T_, NV_, MINB_>(nvec, rows, threads, grid)
    constexpr bool quant = OP == kRowQuant;
    if (elem) {
        if (nvec <= 32) TCR_ELEM(32, 1, 4);
        if (nvec <= 64) TCR_ELEM(32, 2, 2);
        if (nvec <= 128) TCR_ELEM(128, 1, 8);
        if (nvec <= 256) TCR_ELEM(256, 1, 4);
        if (nvec <= (quant ? 384 : 320)) TCR_ELEM(512, 1, 2);
        if (nvec <= 512) TCR_ELEM(256, 2, 2);
        if constexpr (quant) {
            if (nvec <= 1024) TCR_ELEM(1024, 1, 1);
        } else {
            if (nvec <= 768) TCR_ELEM(256, 3, 2);
            if (nvec <= 1024) TCR_ELEM(512, 2, 1);
            if (nvec <= 2048) TCR_ELEM(1024, 2, 1);
        }
    } else if constexpr (DT == kF32) {
        if (nvec <= 32) TCR_STREAM(32, 1, 3);
        if (nvec <= 64) TCR_STREAM(32, 2, 2);
        if (nvec <= 128) TCR_STREAM(128, 1, 8);
        if (nvec <= 256) TCR_STREAM(256, 1, 4);
        if (nvec <= 512) TCR_STREAM(512, 1, 2);
        if (nvec <= 1024) TCR_STREAM(512, 2, 1);
    } else {
        if (nvec <= 32) TCR_STREAM(32, 1, 4);
        if (nvec <= 64) TCR_STREAM(32, 2, 3);
        if (nvec <= 128) {
            if constexpr (OUT == kOutI8)
                TCR_STREAM(32, 4, 2);
            else
                TCR_STREAM(64, 2, 12);
        }
        if (nvec <= 256) TCR_STREAM(128, 2, 6);
        if constexpr (quant)
            if (nvec <= 384) TCR_STREAM(512, 1, 3);
        if (nvec <= 512) TCR_STREAM(256, 2, (quant ? 4 : 3));
        if (nvec <= 768) TCR_STREAM(256, 3, (quant ? 3 : 2));
        if (nvec <= 1024) {
            if constexpr (quant)
                TCR_STREAM(512, 2, 2);
            else
                TCR_STREAM(256, 4, 2);
        }
        if (nvec <= 2048) {
            if constexpr (quant)
                TCR_STREAM(1024, 2, 1);
            else
                TCR_STREAM(512, 4, 1);
        }
    }
#undef TCR_ELEM
#undef TCR_STREAM
    grid = rows;
    if (nvec <= 2048) {
        threads = 512;
        return (const void *)row_kernel<DT, OP, OUT, 512, 4>;
    }
    if (nvec <= 4096) {
        threads = 1024;
        return (const void *)row_kernel<DT, OP, OUT, 1024, 4>;
    }
    threads = kRowLongT;
    return (const void *)row_long_kernel<DT, OP, OUT>;
}

template <int DT>
const void *pick_op(int op, int out_i8, size_t nvec, size_t rows, bool elem, int &threads, size_t &grid)
{
    if (op == kRowNorm)
        return out_i8 ? pick<DT, kRowNorm, kOutI8>(nvec, rows, elem, threads, grid)
                      : pick<DT, kRowNorm, kOutSame>(nvec, rows, elem, threads, grid);
    return pick<DT, kRowQuant, kOutI8>(nvec, rows, elem, threads, grid);
}

}  // namespace

cudaError_t launch_rows_op(int op, int dtype, bool out_i8, const RowArgs &a, cudaStream_t stream)
{
    const size_t nvec = (a.cols + kRv - 1) / kRv;
    int threads = 0;
    size_t grid = 0;
    const bool elem = !a.al_x || (a.r && !a.al_r) || (a.h && !a.al_h) || !a.al_y;
    const void *k = dtype == kF16    ? pick_op<kF16>(op, out_i8, nvec, a.rows, elem, threads, grid)
                    : dtype == kBF16 ? pick_op<kBF16>(op, out_i8, nvec, a.rows, elem, threads, grid)
                                     : pick_op<kF32>(op, out_i8, nvec, a.rows, elem, threads, grid);
    void *args[] = {(void *)&a};
    return launch_first(k, dim3((unsigned)grid), dim3((unsigned)threads), args, 0, stream);
}

cudaError_t launch_dequant(int dtype, const int8_t *q, size_t ldq, const float *scale, void *y, size_t ldy,
                           size_t rows, size_t cols, cudaStream_t stream)
{
    int team_log2 = 5;
    while (team_log2 < 8 && ((size_t)kRv << team_log2) < cols) team_log2++;
    uint32_t ncols = (uint32_t)cols;
    const size_t grid = (rows + ((size_t)256 >> team_log2) - 1) / ((size_t)256 >> team_log2);
    const size_t es = dtype == kF32 ? 4 : 2;
    const bool al_q = ((uintptr_t)q & 7u) == 0 && (rows == 1 || ldq % 8 == 0);
    const bool al_y = ((uintptr_t)y & 15u) == 0 && (rows == 1 || (ldy * es) % 16 == 0);
    const void *k;
    if (al_q && al_y)
        k = dtype == kF16    ? (const void *)dequant_kernel<kF16, false>
            : dtype == kBF16 ? (const void *)dequant_kernel<kBF16, false>
                             : (const void *)dequant_kernel<kF32, false>;
    else
        k = dtype == kF16    ? (const void *)dequant_kernel<kF16, true>
            : dtype == kBF16 ? (const void *)dequant_kernel<kBF16, true>
                             : (const void *)dequant_kernel<kF32, true>;
    void *args[] = {(void *)&q,   (void *)&ldq,  (void *)&scale, (void *)&y,
                    (void *)&ldy, (void *)&rows, (void *)&ncols, (void *)&team_log2};
    return launch_first(k, dim3((unsigned)grid), dim3(256), args, 0, stream);
}

}  // namespace tcr
