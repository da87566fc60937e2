// What the kernels on rows share (gated.hip, rows.hip): eight bf16 of a lane,
// workgroups of a launch, and blocks of a row to FP8 and MXFP4.
#pragma once

#include "products.hpp"

namespace moe {

typedef __attribute__((ext_vector_type(2))) int i32x2;

__device__ __forceinline__ void unpack8(u32x4 q, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_bits_to_f32(q[i] & 0xFFFFu);
        v[2 * i + 1] = bf16_bits_to_f32(q[i] >> 16);
    }
}

__device__ __forceinline__ u32x4 pack8(const float v[8]) {
    return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7])};
}

// Rows that hold something: *n_rows of them (kept inside [0, R]), or all.
__device__ __forceinline__ int row_count(const int32_t *n_rows, int R) {
    if (!n_rows) return R;
    const int n = *as_scalar(n_rows);
    return n < 0 ? 0 : n < R ? n : R;
}

// Number of this workgroup: a launch's threads along x have to fit 32 bits (a
// product past them wraps without an error), so the rest go along y.
constexpr long kBlocksX = 1 << 23;
__device__ __forceinline__ long block_id() { return (long)blockIdx.y * gridDim.x + blockIdx.x; }

inline bool blocks_ok(long n) { return n <= 0x7FFFFFFFL; }
inline dim3 blocks_of(long n) {
    return n <= kBlocksX ? dim3((unsigned)n) : dim3((unsigned)kBlocksX, (unsigned)((n + kBlocksX - 1) / kBlocksX));
}

// Row of unit v of `per` to a row, 1 << log units to a workgroup. (A 64-bit
// division for every thread cost the FP8 conversion of 24576 x 2048 values 8 us of
// 58, which the arithmetic bounds as much as HBM.)
__device__ __forceinline__ long row_of_unit(long v, int log, int per, const Divisor &d) {
    return block_id() < (1L << (31 - log)) ? (long)((uint32_t)v / d) : v / per;
}

// The largest magnitude of 8 columns of each of LANES neighbouring lanes, as its
// bits: magnitudes compare as integers, NaN above infinity above every number.
template <int LANES>
__device__ __forceinline__ uint32_t block_amax(const float v[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = a > m ? a : m;
    }
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    return m;
}

// v / d by d's reciprocal r, corrected by the quotient's remainder; in this order
// of signs a zero keeps its own. The bits of a division (2.7e8 codes compared), and
// 46.5 us instead of 48.7 for the activation of 24576 x 2048 values with divisions.
__device__ __forceinline__ float quotient(float v, float d, float r) {
    const float q = v * r;
    return fmaf(-fmaf(q, d, -v), r, q);
}

// A block of 128 columns as E4M3, 8 columns a lane, 16 lanes: the scale, which
// every lane gets, and this lane's codes. An infinity or a NaN makes the whole
// block NaN (codes and scale).
__device__ __forceinline__ float block_to_fp8(const float v[8], i32x2 &code) {
    const uint32_t m = block_amax<16>(v);
    const float top = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(m), 0x1p-100f);
    const float sc = quotient(top, 448.0f, 1.0f / 448.0f);
    // (the reciprocal from the instruction's, by a step of Newton's; sc is 2^-109 to 2^120)
    const float r0 = __builtin_amdgcn_rcpf(sc), rc = fmaf(fmaf(-sc, r0, 1.0f), r0, r0);
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = quotient(v[i], sc, rc);
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(d[0], d[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(d[2], d[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(d[4], d[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(d[6], d[7], hi, true);
    code = i32x2{lo, hi};
    return sc;
}

// A block of 32 columns as MXFP4, 8 columns a lane, 4 lanes: the E8M0 scale byte
// and this lane's codes, the first column in the lowest bits. The scale is
// 2^(floor(log2 amax) - 2), at least 2^-127, which is amax's exponent field less 2;
// an infinity or a NaN makes it 255, NaN. v / scale lies below 8; the conversion
// divides exactly, rounds to the nearest E2M1 (ties to even) and saturates at 6
// (every bf16 and 1e6 floats around the borders compared, subnormal ones with
// the scale 2^-127 as well).
__device__ __forceinline__ uint32_t block_to_mxfp4(const float v[8], uint32_t &code) {
    const uint32_t m = block_amax<4>(v), e = m >> 23;
    const uint32_t s = m >= 0x7F800000u ? 255u : e > 2 ? e - 2 : 0u;
    const float sc = __uint_as_float(s << 23);      // (the conversion reads the exponent alone)
    uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], sc, 3);
    // a zero has no sign: bit 3 of a code stays where its other bits hold something
    const uint32_t mag = c & 0x77777777u, some = (mag + 0x77777777u) & 0x88888888u;
    code = s == 255u ? 0u : mag | (c & some);
    return s;
}

// Host: sizes of the calls on rows, and pointers that 16-byte accesses go through.
inline bool row_sizes_ok(int R, int I) {
    return R >= 0 && R <= kMaxRows && I >= 8 && I % 8 == 0 && I <= (1 << 24);
}
inline bool al16(const void *p) { return p && ((uintptr_t)p & 15) == 0; }

}  // namespace moe
