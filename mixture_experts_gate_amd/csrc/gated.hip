// What stands between the expert products: the gated activation with its
// gradient, and rows to FP8 with a scale per 128 columns.
//
//   a   = w silu(g) u,  silu(g) = g s,  s = 1 / (1 + e^-g),  h = [g | u]
//   dg  = w da u s (1 + g (1 - s)),  du = w da silu(g),
//   dw  = sum over the row of da silu(g) u
//   fp8: scale = max(amax, 2^-100) / 448 over 128 columns, code = E4M3(v / scale)
//
// All of it is fp32 in registers with one rounding at the end; each value is
// read once and written once, 16 bytes a lane, so HBM bounds the large sizes
// (5.7 TB/s for the gradient of 32768 x 768 and the conversion of 24576 x 2048
// activations, which the arithmetic bounds as much) and the launch the small ones.
#include "products.hpp"

namespace moe {

// s = 1 / (1 + e^-g) and c = 1 - s, each to a few units of 2^-24, from e^-|g| (so
// that nothing overflows and c does not cancel). e^-|g| = 2^t e^(-|g| - t ln 2),
// t the rounded -|g| log2(e): with 2^t alone scales and weights' gradients were up
// to 57 units off at |g| = 70 (now at most 8). From |g| = 128 on e^-|g| is 0.
struct Sigmoid {
    float s, c;
};
__device__ __forceinline__ Sigmoid sigmoid(float g) {
    constexpr float kLn2 = 0.6931471805599453f, kLn2Rest = (float)(0.6931471805599453 - (double)kLn2);
    const float a = __builtin_amdgcn_fmed3f(fabsf(g), 0.0f, 128.0f);     // (a NaN comes back in by the factor g)
    const float t = -1.4426950408889634f * a, rest = fmaf(-kLn2Rest, t, fmaf(-kLn2, t, -a));
    const float e0 = __builtin_amdgcn_exp2f(t), e = fmaf(e0, rest, e0);
    const float d = 1.0f + e, r0 = __builtin_amdgcn_rcpf(d), r = fmaf(fmaf(-d, r0, 1.0f), r0, r0);
    const float er = e * r;
    return g < 0.0f ? Sigmoid{er, r} : Sigmoid{r, er};
}

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

// Row of unit v of `per` to a row, 1 << log units to a workgroup. (A 64-bit
// division for every thread cost the FP8 conversion of 24576 x 2048 values 8 us of
// 58, which the arithmetic bounds as much as HBM.)
__device__ __forceinline__ long row_of_unit(long v, int log, int per, const Divisor &d) {
    return block_id() < (1L << (31 - log)) ? (long)((uint32_t)v / d) : v / per;
}

// Weight's place of row r: -1 where the index is outside the weights.
__device__ __forceinline__ int weight_at(const int32_t *w_rows, int w_n, int r) {
    const int i = w_rows ? w_rows[r] : r;
    return i >= 0 && i < w_n ? i : -1;
}

__global__ __launch_bounds__(256) void gated_kernel(const uint16_t *__restrict__ h,
                                                    const float *__restrict__ wt,
                                                    const int32_t *__restrict__ w_rows, int w_n,
                                                    const int32_t *__restrict__ n_rows, int R,
                                                    int I, Divisor by, uint16_t *__restrict__ a) {
    const int per = I / 8;
    const long id = block_id() * blockDim.x + threadIdx.x, row = row_of_unit(id, 8, per, by);
    if (row >= row_count(n_rows, R)) return;
    const int r = (int)row;
    const int c = (int)(id - (long)r * per) * 8;
    float w = 1.0f;
    if (wt) {
        const int at = weight_at(w_rows, w_n, r);
        if (at < 0) return;
        w = wt[at];
    }
    float g[8], u[8];
    unpack8(load_nt16(h + (size_t)r * 2 * I + c), g);
    unpack8(load_nt16(h + (size_t)r * 2 * I + I + c), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = w * (g[i] * sigmoid(g[i]).s * u[i]);
    *(MOE_GLOBAL u32x4 *)(a + (size_t)r * I + c) = pack8(g);
}

// One wavefront a row, for the row's sum.
__global__ __launch_bounds__(256) void gated_grad_kernel(
    const uint16_t *__restrict__ h, const uint16_t *__restrict__ da, const float *__restrict__ wt,
    const int32_t *__restrict__ w_rows, int w_n, const int32_t *__restrict__ n_rows, int R, int I,
    uint16_t *__restrict__ dh, float *__restrict__ dw, uint16_t *__restrict__ a) {
    const long row = block_id() * (blockDim.x / kWave) + threadIdx.x / kWave;
    if (row >= row_count(n_rows, R)) return;
    const int r = (int)row, l = lane_id();
    float w = 1.0f;
    int at = -1;
    if (wt) {
        at = weight_at(w_rows, w_n, r);
        if (at < 0) return;
        w = wt[at];
    }
    float sum = 0.0f;
    for (int c = 8 * l; c < I; c += 8 * kWave) {
        float g[8], u[8], d[8], act[8];
        unpack8(load_nt16(h + (size_t)r * 2 * I + c), g);
        unpack8(load_nt16(h + (size_t)r * 2 * I + I + c), u);
        unpack8(load_nt16(da + (size_t)r * I + c), d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Sigmoid s = sigmoid(g[i]);
            const float silu = g[i] * s.s, wd = w * d[i];
            act[i] = silu * u[i];
            sum += d[i] * act[i];
            act[i] *= w;
            g[i] = wd * u[i] * (s.s * (1.0f + g[i] * s.c));
            u[i] = wd * silu;
        }
        *(MOE_GLOBAL u32x4 *)(dh + (size_t)r * 2 * I + c) = pack8(g);
        *(MOE_GLOBAL u32x4 *)(dh + (size_t)r * 2 * I + I + c) = pack8(u);
        if (a) *(MOE_GLOBAL u32x4 *)(a + (size_t)r * I + c) = pack8(act);
    }
    if (dw) {
#pragma unroll
        for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
        if (l == 0) dw[at] = sum;
    }
}

// v / d by d's reciprocal r, corrected by the quotient's remainder; in this order
// of signs a zero keeps its own. The bits of a division (2.7e8 codes compared), and
// 46.5 us instead of 48.7 for the activation of 24576 x 2048 values with divisions.
__device__ __forceinline__ float quotient(float v, float d, float r) {
    const float q = v * r;
    return fmaf(-fmaf(q, d, -v), r, q);
}

// 16 lanes a block of 128 columns, 8 columns a lane.
template <bool GATED>
__global__ __launch_bounds__(256) void to_fp8_kernel(const uint16_t *__restrict__ x,
                                                     const int32_t *__restrict__ n_rows, int R,
                                                     int K, Divisor by, uint8_t *__restrict__ q,
                                                     float *__restrict__ s) {
    const int kb = (K + 127) / 128;
    const long id = (block_id() * blockDim.x + threadIdx.x) >> 4;
    const long row = row_of_unit(id, 4, kb, by);
    if (row >= row_count(n_rows, R)) return;
    const int r = (int)row;
    const int b = (int)(id - (long)r * kb), l = threadIdx.x & 15, c = 128 * b + 8 * l;
    const bool in = c < K;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in) {
        if (GATED) {
            float u[8];
            unpack8(load_nt16(x + (size_t)r * 2 * K + c), v);
            unpack8(load_nt16(x + (size_t)r * 2 * K + K + c), u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid(v[i]).s * u[i];
        } else {
            unpack8(load_nt16(x + (size_t)r * K + c), v);
        }
    }
    // magnitudes compare as integers, NaN above infinity above every number
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = a > m ? a : m;
    }
#pragma unroll
    for (int d = 8; d; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    // an infinity or a NaN makes the whole block NaN (codes and scale)
    const float top = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(m), 0x1p-100f);
    const float sc = quotient(top, 448.0f, 1.0f / 448.0f);
    if (l == 0) s[(size_t)r * kb + b] = sc;
    if (!in) return;
    // (the reciprocal from the instruction's, by a step of Newton's; sc is 2^-109 to 2^120)
    const float r0 = __builtin_amdgcn_rcpf(sc), rc = fmaf(fmaf(-sc, r0, 1.0f), r0, r0);
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = quotient(v[i], sc, rc);
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(d[0], d[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(d[2], d[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(d[4], d[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(d[6], d[7], hi, true);
    typedef __attribute__((ext_vector_type(2))) int i32x2;
    *(MOE_GLOBAL i32x2 *)(q + (size_t)r * K + c) = i32x2{lo, hi};
}

static bool sizes_ok(int R, int I) {
    return R >= 0 && R <= kMaxRows && I >= 8 && I % 8 == 0 && I <= (1 << 24);
}
static bool al(const void *p) { return p && ((uintptr_t)p & 15) == 0; }
static bool blocks_ok(long n) { return n <= 0x7FFFFFFFL; }
static dim3 blocks_of(long n) {
    return n <= kBlocksX ? dim3((unsigned)n) : dim3((unsigned)kBlocksX, (unsigned)((n + kBlocksX - 1) / kBlocksX));
}

}  // namespace moe

using namespace moe;

extern "C" int moe_swiglu(const uint16_t *h_bf16, const float *w, const int32_t *w_rows, int w_n,
                          const int32_t *n_rows, int R, int I, uint16_t *a_bf16, void *stream) {
    if (!sizes_ok(R, I)) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if (!al(h_bf16) || !al(a_bf16) || (w_rows && !w) || (w && w_n < (w_rows ? 1 : R)))
        return MOE_EINVAL;
    const long blocks = ((long)R * (I / 8) + 255) / 256;
    if (!blocks_ok(blocks)) return MOE_EINVAL;
    MOE_LAUNCH(K_GATED, gated_kernel, blocks_of(blocks), dim3(256), 0, (hipStream_t)stream,
               h_bf16, w, w_rows, w_n, n_rows, R, I, divisor(I / 8), a_bf16);
    return check_launch();
}

extern "C" int moe_swiglu_grad(const uint16_t *h_bf16, const uint16_t *da_bf16, const float *w,
                               const int32_t *w_rows, int w_n, const int32_t *n_rows, int R, int I,
                               uint16_t *dh_bf16, float *dw, uint16_t *a_bf16, void *stream) {
    if (!sizes_ok(R, I)) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if (!al(h_bf16) || !al(da_bf16) || !al(dh_bf16) || ((uintptr_t)a_bf16 & 15)) return MOE_EINVAL;
    if ((w_rows && !w) || (w && w_n < (w_rows ? 1 : R)) || (dw && !w)) return MOE_EINVAL;
    MOE_LAUNCH(K_GATED_GRAD, gated_grad_kernel, blocks_of(((long)R + 3) / 4), dim3(256), 0,
               (hipStream_t)stream, h_bf16, da_bf16, w, w_rows, w_n, n_rows, R, I, dh_bf16, dw,
               a_bf16);
    return check_launch();
}

template <bool GATED>
static int to_fp8(const uint16_t *x, const int32_t *n_rows, int R, int K, uint8_t *q, float *s,
                  void *stream) {
    if (!sizes_ok(R, K)) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if (!al(x) || !q || ((uintptr_t)q & 7) || !s) return MOE_EINVAL;
    const long blocks = ((long)R * ((K + 127) / 128) + 15) / 16;
    if (!blocks_ok(blocks)) return MOE_EINVAL;
    MOE_LAUNCH(K_TO_FP8, (to_fp8_kernel<GATED>), blocks_of(blocks), dim3(256), 0,
               (hipStream_t)stream, x, n_rows, R, K, divisor((K + 127) / 128), q, s);
    return check_launch();
}

extern "C" int moe_quant_fp8(const uint16_t *x_bf16, const int32_t *n_rows, int R, int K,
                             uint8_t *q_e4m3, float *scale, void *stream) {
    return to_fp8<false>(x_bf16, n_rows, R, K, q_e4m3, scale, stream);
}

extern "C" int moe_swiglu_quant_fp8(const uint16_t *h_bf16, const int32_t *n_rows, int R, int I,
                                    uint8_t *q_e4m3, float *scale, void *stream) {
    return to_fp8<true>(h_bf16, n_rows, R, I, q_e4m3, scale, stream);
}
