// What stands between the expert products: the gated activation with its
// gradient, and rows to FP8 (a scale per 128 columns) and MXFP4 (one per 32).
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
#include "rows.hpp"

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
    i32x2 code;
    const float sc = block_to_fp8(v, code);
    if (l == 0) s[(size_t)r * kb + b] = sc;
    if (in) *(MOE_GLOBAL i32x2 *)(q + (size_t)r * K + c) = code;
}

// 4 lanes a block of 32 columns, 8 columns a lane. (One lane a block would load 64
// bytes in pieces of 16, four lines a request.) HBM bounds the large sizes: 2 (GATED 4)
// bytes in and 17/32 out for a value. 8192 x 2048 values 10.6 us (4.0 TB/s), the
// activation of 24576 x 2048 40 us (228 MB, 5.7 TB/s), one token's 2 us.
template <bool GATED>
__global__ __launch_bounds__(256) void to_mxfp4_kernel(const uint16_t *__restrict__ x,
                                                       const int32_t *__restrict__ n_rows, int R,
                                                       int K, Divisor by, uint32_t *__restrict__ q,
                                                       uint8_t *__restrict__ s) {
    const int kb = K / 32;
    const long id = (block_id() * blockDim.x + threadIdx.x) >> 2;
    const long row = row_of_unit(id, 6, kb, by);
    if (row >= row_count(n_rows, R)) return;
    const int r = (int)row;
    const int b = (int)(id - (long)r * kb), l = threadIdx.x & 3, c = 32 * b + 8 * l;
    float v[8];
    if (GATED) {
        float u[8];
        unpack8(load_nt16(x + (size_t)r * 2 * K + c), v);
        unpack8(load_nt16(x + (size_t)r * 2 * K + K + c), u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid(v[i]).s * u[i];
    } else {
        unpack8(load_nt16(x + (size_t)r * K + c), v);
    }
    uint32_t code;
    const uint32_t sc = block_to_mxfp4(v, code);
    q[((size_t)r * K + c) / 8] = code;
    if (l == 0) s[(size_t)r * kb + b] = (uint8_t)sc;
}

// Matrices to MXFP4 in the kernel layout: a wavefront takes 32 columns of 16 rows,
// whose codes are 256 and whose scales are 16 consecutive bytes there. HBM bounds it:
// 128 x 1536 x 2048 210 us (4.8 TB/s).
__global__ __launch_bounds__(256) void matrix_to_mxfp4_kernel(const uint16_t *__restrict__ w, long groups,
                                                              int K, uint32_t *__restrict__ q,
                                                              uint8_t *__restrict__ s) {
    const long id = (block_id() * blockDim.x + threadIdx.x) / kWave;      // (16 rows, 32 columns)
    if (id >= groups) return;
    const int l = lane_id(), per = K / 32;
    const long rb = id / per;
    const int b = (int)(id - rb * per), r = l >> 2, c = 8 * (l & 3);
    float v[8];
    unpack8(load_nt16(w + ((size_t)rb * 16 + r) * K + 32 * b + c), v);
    uint32_t code;
    const uint32_t sc = block_to_mxfp4(v, code);
    q[(size_t)id * 64 + l] = code;
    if ((l & 3) == 0) s[(size_t)id * 16 + r] = (uint8_t)sc;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_swiglu(const uint16_t *h_bf16, const float *w, const int32_t *w_rows, int w_n,
                          const int32_t *n_rows, int R, int I, uint16_t *a_bf16, void *stream) {
    if (!row_sizes_ok(R, I)) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if (!al16(h_bf16) || !al16(a_bf16) || (w_rows && !w) || (w && w_n < (w_rows ? 1 : R)))
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
    if (!row_sizes_ok(R, I)) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if (!al16(h_bf16) || !al16(da_bf16) || !al16(dh_bf16) || ((uintptr_t)a_bf16 & 15)) return MOE_EINVAL;
    if ((w_rows && !w) || (w && w_n < (w_rows ? 1 : R)) || (dw && !w)) return MOE_EINVAL;
    MOE_LAUNCH(K_GATED_GRAD, gated_grad_kernel, blocks_of(((long)R + 3) / 4), dim3(256), 0,
               (hipStream_t)stream, h_bf16, da_bf16, w, w_rows, w_n, n_rows, R, I, dh_bf16, dw,
               a_bf16);
    return check_launch();
}

template <bool GATED>
static int to_fp8(const uint16_t *x, const int32_t *n_rows, int R, int K, uint8_t *q, float *s,
                  void *stream) {
    if (!row_sizes_ok(R, K)) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if (!al16(x) || !q || ((uintptr_t)q & 7) || !s) return MOE_EINVAL;
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

template <bool GATED>
static int to_mxfp4(const uint16_t *x, const int32_t *n_rows, int R, int K, uint8_t *q, uint8_t *s,
                    void *stream) {
    if (!row_sizes_ok(R, K) || K % 32) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if (!al16(x) || !al16(q) || !s) return MOE_EINVAL;
    const long blocks = ((long)R * (K / 32) + 63) / 64;
    if (!blocks_ok(blocks)) return MOE_EINVAL;
    MOE_LAUNCH(K_TO_MXFP4, (to_mxfp4_kernel<GATED>), blocks_of(blocks), dim3(256), 0,
               (hipStream_t)stream, x, n_rows, R, K, divisor(K / 32), (uint32_t *)q, s);
    return check_launch();
}

extern "C" int moe_quant_mxfp4(const uint16_t *x_bf16, const int32_t *n_rows, int R, int K,
                               uint8_t *q_e2m1, uint8_t *scale_e8m0, void *stream) {
    return to_mxfp4<false>(x_bf16, n_rows, R, K, q_e2m1, scale_e8m0, stream);
}

extern "C" int moe_swiglu_quant_mxfp4(const uint16_t *h_bf16, const int32_t *n_rows, int R, int I,
                                      uint8_t *q_e2m1, uint8_t *scale_e8m0, void *stream) {
    return to_mxfp4<true>(h_bf16, n_rows, R, I, q_e2m1, scale_e8m0, stream);
}

extern "C" int moe_quant_mxfp4_matrices(const uint16_t *w_bf16, int E, int N, int K, uint8_t *q_e2m1,
                                        uint8_t *scale_e8m0, void *stream) {
    if (E < 0 || N < 16 || N % 16 || N > (1 << 20) || K < 128 || K % 128 || K > (1 << 20)) return MOE_EINVAL;
    if (E == 0) return MOE_OK;
    if (!al16(w_bf16) || !al16(q_e2m1) || !scale_e8m0) return MOE_EINVAL;
    const long groups = (long)E * (N / 16) * (K / 32);
    if (!blocks_ok((groups + 3) / 4)) return MOE_EINVAL;
    MOE_LAUNCH(K_TO_MXFP4, matrix_to_mxfp4_kernel, blocks_of((groups + 3) / 4), dim3(256), 0,
               (hipStream_t)stream, w_bf16, groups, K, (uint32_t *)q_e2m1, scale_e8m0);
    return check_launch();
}
