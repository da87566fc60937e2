// What stands around the experts: the norm before the layer, with the residual's
// addition and its output in 8 or 4 bits, its gradient, and the moves of rows
// between tokens and sorted order with the router's weights and their gradients.
//
//   norm      t = bf16(x + residual), inv = 1 / sqrt(mean(t^2) + eps), y = t inv w
//   gradient  g = dy w, n = t inv:  dx = inv (g - n mean(g n)) + dtotal,
//             dw = sum over the rows of dy n
//   dispatch  out[at] = x[t],  at = pair_row[t][j]
//   combine   out[t] = sum_j w[t][j] y[at] + add[t];
//   gradient  dy[at] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[at]>
//
// fp32 in registers with one rounding at each output; every value is read once
// and written once, 16 bytes a lane: HBM bounds the large sizes, the launch and
// one trip to memory the small ones. A row of the norm whose sums leave fp32's range
// is summed again in 64 bits, where every product of three bf16 has its place.
#include "rows.hpp"

namespace moe {

// 16 bytes that the kernel does not read again: past the caches' other contents (norm
// of 8192 x 2048 with a residual 27.2 -> 21.8 us, of 8192 x 4096 to FP8 59.5 -> 55.8).
__device__ __forceinline__ void store_nt(void *to, u32x4 v) {
    __builtin_nontemporal_store(v, (MOE_GLOBAL u32x4 *)to);
}

// ------------------------------------------------------------------- norm --

constexpr int kNormThreads = 256;
enum NormQuant { kNone = 0, kFp8 = 1, kMxfp4 = 2 };

// Sum over the TPR threads of a row, in a fixed order, in every thread.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *part) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if (TPR == kWave) return v;
    __syncthreads();                        // (the last sum's readers are done)
    if (lane_id() == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < TPR / kWave; ++i) v += part[i];
    return v;
}

// The same in 64 bits.
template <int TPR>
__device__ __forceinline__ double row_sum64(double v, double *part) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if (TPR == kWave) return v;
    __syncthreads();
    if (lane_id() == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < TPR / kWave; ++i) v += part[i];
    return v;
}

// Whether a row's fp32 sum of squares, or the mean of them with eps, is not to be used:
// past 2^120, or so small that squares below 2^-126 lost bits that count (a NaN too,
// which stays one). The same in all threads of a row, whose sums have the same bits.
__device__ __forceinline__ bool far_row(float squares, float mean) {
    return !(squares < 0x1p120f && mean > 0x1p-90f);
}

struct NormArgs {
    const uint16_t *x, *res, *w;
    float eps;
    int R, H;
    uint16_t *total, *y;
    uint8_t *q;
    void *qs;
};

// 8 columns of a row of t: x, or the rounded sum, which is stored. (total may be x
// or res: a thread reads its columns before it writes them.)
template <bool AGAIN>
__device__ __forceinline__ void norm_row(const NormArgs &a, size_t at, float v[8]) {
    unpack8(load16(a.x + at), v);
    if (!a.res) return;
    float b[8];
    unpack8(load16(a.res + at), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
    const u32x4 t = pack8(v);
    unpack8(t, v);
    if (!a.total) return;
    if (AGAIN) *(MOE_GLOBAL u32x4 *)(a.total + at) = t;       // (read again soon)
    else store_nt(a.total + at, t);
}

template <int QUANT>
__device__ __forceinline__ void norm_out(const NormArgs &a, int r, int c, const float v[8]) {
    const bool in = c < a.H;
    if (in && a.y) store_nt(a.y + (size_t)r * a.H + c, pack8(v));
    if (QUANT == kFp8) {
        i32x2 code;
        const float s = block_to_fp8(v, code);
        if (!in) return;
        __builtin_nontemporal_store(code, (MOE_GLOBAL i32x2 *)(a.q + (size_t)r * a.H + c));
        if ((c & 127) == 0) ((MOE_GLOBAL float *)a.qs)[(size_t)r * ((a.H + 127) / 128) + c / 128] = s;
    }
    if (QUANT == kMxfp4) {
        uint32_t code;
        const uint32_t s = block_to_mxfp4(v, code);
        if (!in) return;
        ((MOE_GLOBAL uint32_t *)a.q)[((size_t)r * a.H + c) / 8] = code;
        if ((c & 31) == 0) ((MOE_GLOBAL uint8_t *)a.qs)[(size_t)r * (a.H / 32) + c / 32] = (uint8_t)s;
    }
}

// TPR threads a row (a wavefront up to 1024 columns, or the workgroup), NV vectors of 8
// columns a thread: the row stays in registers between the sum and the outputs. NV = 0:
// rows of any length, read again (t from total, where it was rounded; from the caches).
// HBM bounds it: 8192 x 4096 with the residual's sum 49 us in bf16 (268 MB, 5.5 TB/s),
// with bf16 and FP8 (303 MB) 49 to 54, in MXFP4 alone 40; 8192 x 2048 21 us; 2048 x
// 16384, read again, 53 us (5.1 TB/s). One token: 2.3 us, one trip to memory and two
// barriers.
template <int TPR, int NV, int QUANT>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormArgs a) {
    __shared__ float part[kNormThreads / kWave];
    __shared__ double part64[kNormThreads / kWave];
    const long row = block_id() * (kNormThreads / TPR) + threadIdx.x / TPR;
    if (row >= a.R) return;                 // (whole wavefronts; whole workgroups where they meet)
    const int r = (int)row, t = threadIdx.x % TPR;
    const size_t at = (size_t)r * a.H;
    float v[NV ? NV : 1][8], sum = 0.0f;
    u32x4 w[NV ? NV : 1];
    const int per = (a.H + 8 * TPR - 1) / (8 * TPR);
    for (int i = 0; i < (NV ? NV : per); ++i) {
        const int c = 8 * (t + TPR * i), k = NV ? i : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
        if (c < a.H) {
            if (NV) w[k] = load16(a.w + c);
            norm_row<NV == 0>(a, at + c, v[k]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(v[k][j], v[k][j], sum);
    }
    const float squares = row_sum<TPR>(sum, part), mean = squares / (float)a.H + a.eps;
    const float inv = 1.0f / sqrtf(mean);
    const bool far = far_row(squares, mean);
    // columns c .. c + 7 of t again: from total, where they were rounded, or the inputs
    auto read_again = [&](int c, float u[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = 0.0f;
        if (c >= a.H) return;
        if (a.res && !a.total) norm_row<true>(a, at + c, u);
        else unpack8(load16((a.res ? a.total : a.x) + at + c), u);
    };
    if (far) {
        // (read again, a vector at a time: from registers this code would take up to 40 more
        // of them than an ordinary row does, and 4096 x 8192 to MXFP4 42.8 us instead of 38.7)
        double sum64 = 0.0;
#pragma unroll 1
        for (int c = 8 * t; c < a.H; c += 8 * TPR) {
            float u[8];
            read_again(c, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum64 = fma((double)u[j], (double)u[j], sum64);
        }
        const double inv64 = 1.0 / sqrt(row_sum64<TPR>(sum64, part64) / a.H + (double)a.eps);
#pragma unroll 1
        for (int i = 0; i < per; ++i) {          // (all lanes of a block of codes together)
            const int c = 8 * (t + TPR * i);
            float u[8], y[8];
            read_again(c, u);
            unpack8(c < a.H ? load16(a.w + c) : u32x4{0, 0, 0, 0}, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = c < a.H ? (float)((double)u[j] * inv64 * (double)y[j]) : 0.0f;
            norm_out<QUANT>(a, r, c, y);
        }
        return;
    }
    for (int i = 0; i < (NV ? NV : per); ++i) {
        const int c = 8 * (t + TPR * i), k = NV ? i : 0;
        if (!NV) {
            if (c < a.H) w[k] = load16(a.w + c);
            read_again(c, v[k]);
        }
        float y[8];
        unpack8(w[k], y);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = c < a.H ? v[k][j] * inv * y[j] : 0.0f;
        norm_out<QUANT>(a, r, c, y);
    }
}

struct NormGradArgs {
    const uint16_t *x, *w, *dy, *dt;
    float eps;
    int R, H;
    uint16_t *dx;
    float *part;              // [slots][H], or NULL
    int slots;
};

// Row r of the gradient in 64 bits: dx, and its part of dw. (A thread reads its columns
// before it writes them: dx may be dy's or dtotal's rows.)
template <int TPR, int NV>
__device__ __forceinline__ void far_grad(const NormGradArgs &a, long r, int t, float (&dw)[NV][8], double *part) {
    const uint16_t *const x = a.x + (size_t)r * a.H, *const g = a.dy + (size_t)r * a.H;
    double ss = 0.0, dot = 0.0;
#pragma unroll 1
    for (int c = 8 * t; c < a.H; c += 8 * TPR) {
        float u[8], v[8], f[8];
        unpack8(load16(x + c), u), unpack8(load16(g + c), v), unpack8(load16(a.w + c), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ss = fma((double)u[j], (double)u[j], ss);
            dot = fma((double)v[j] * f[j], (double)u[j], dot);
        }
    }
    const double inv = 1.0 / sqrt(row_sum64<TPR>(ss, part) / a.H + (double)a.eps);
    const double mean = row_sum64<TPR>(dot, part) * inv / a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        asm volatile("" ::: "memory");          // (one vector after the other: few registers)
        const int c = 8 * (t + TPR * i);
        if (c >= a.H) continue;
        float u[8], v[8], f[8], d[8];
        unpack8(load16(x + c), u), unpack8(load16(g + c), v), unpack8(load16(a.w + c), f);
        unpack8(a.dt ? load16(a.dt + (size_t)r * a.H + c) : u32x4{0, 0, 0, 0}, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double n = u[j] * inv;
            dw[i][j] = fmaf(v[j], (float)n, dw[i][j]);
            d[j] = (float)(d[j] + inv * ((double)v[j] * f[j] - n * mean));
        }
        store_nt(a.dx + (size_t)r * a.H + c, pack8(d));
    }
}

// Slot s takes the rows s, s + slots, ...: TPR threads, whose part of dw stays in
// registers over the rows and goes to row s of `part`, which norm_join adds up (no
// atomics: the order is fixed). The next row is on its way while this one's two sums
// meet. HBM bounds it: 8192 x 4096 with dtotal 46 us (268 MB, 5.8 TB/s), and 5 for the
// join; 4096 x 8192 53 and 5, 2048 x 16384 59 and 7, where the parts of dw are 17 and 34
// MB more; 301 x 2048 5 us, a row a workgroup, and 4.
template <int TPR, int NV>
__global__ __launch_bounds__(kNormThreads) void norm_grad_kernel(NormGradArgs a) {
    constexpr int W = TPR / kWave;
    __shared__ float part[2][2][kNormThreads / kWave];
    __shared__ double part64[kNormThreads / kWave];
    const int slot = blockIdx.x * (kNormThreads / TPR) + threadIdx.x / TPR, t = threadIdx.x % TPR;
    if (slot >= a.slots) return;
    struct Row {
        u32x4 x[NV], g[NV], t[NV];
    };
    auto load = [&](long r, Row &v) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (t + TPR * i);
            v.x[i] = v.g[i] = v.t[i] = u32x4{0, 0, 0, 0};
            if (c < a.H && r < a.R) {
                const size_t at = (size_t)r * a.H + c;
                v.x[i] = load_nt16(a.x + at);
                v.g[i] = load_nt16(a.dy + at);
                if (a.dt) v.t[i] = load_nt16(a.dt + at);
            }
        }
    };
    u32x4 w[NV];
    float dw[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (t + TPR * i);
        w[i] = u32x4{0, 0, 0, 0};
        if (c < a.H) w[i] = load16(a.w + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    }
    int turn = 0;
    // Rows in turns of 2048. Row n of a turn that is far (its dx is not stored, nor its
    // part of dw added) has bit n / 64 of lane n % 64's mask, which every wavefront of the
    // row holds, and follows at the turn's end: 64-bit code inside the loop would take
    // registers and time from every row (8192 x 2048 25.3 -> 32 us).
    for (long first = slot; first < a.R; first += 2048L * a.slots) {
        Row cur, next;
        load(first, cur);
        // (here, lest the compiler wait for it inside the loop, and so for `next` too)
        __builtin_amdgcn_s_waitcnt(0x0F70);         // vmcnt(0)
        uint32_t far = 0;
        int row = 0;
        for (long r = first; r < a.R && row < 2048; r += a.slots, turn ^= 1, ++row) {
            load(r + a.slots, next);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[8], g[8], f[8];
                unpack8(cur.x[i], x), unpack8(cur.g[i], g), unpack8(w[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ss = fmaf(x[j], x[j], ss);
                    dot = fmaf(g[j] * f[j], x[j], dot);
                }
            }
#pragma unroll
            for (int d = 32; d; d >>= 1) ss += __shfl_xor(ss, d), dot += __shfl_xor(dot, d);
            if (W > 1) {
                // (two places in turn: a barrier a row)
                if (lane_id() == 0)
                    part[turn][0][threadIdx.x / kWave] = ss, part[turn][1][threadIdx.x / kWave] = dot;
                wait_lds();
                bare_barrier();             // (one that leaves the loads in flight)
                ss = part[turn][0][0], dot = part[turn][1][0];
#pragma unroll
                for (int i = 1; i < W; ++i) ss += part[turn][0][i], dot += part[turn][1][i];
            }
            const float squares = ss / (float)a.H + a.eps, inv = 1.0f / sqrtf(squares);
            const float mean = dot * inv / (float)a.H;              // mean(g n)
            const bool is_far = far_row(ss, squares) || !(fabsf(mean) < 0x1p120f);
            far |= is_far && lane_id() == (row & 63) ? 1u << (row >> 6) : 0u;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = 8 * (t + TPR * i);
                // (unpacked once more: there are not registers for all values of 16384 columns)
                if (NV > 4) asm volatile("" : "+v"(w[i]));
                float x[8], g[8], f[8], d[8];
                unpack8(cur.x[i], x), unpack8(cur.g[i], g), unpack8(w[i], f), unpack8(cur.t[i], d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = x[j] * inv;
                    dw[i][j] = is_far ? dw[i][j] : fmaf(g[j], n, dw[i][j]);
                    d[j] += inv * (g[j] * f[j] - n * mean);
                }
                if (c < a.H && !is_far) store_nt(a.dx + (size_t)r * a.H + c, pack8(d));
            }
            cur = next;
        }
        if (!__ballot(far != 0)) continue;
        for (int b = 0; b < 32; ++b)
            for (unsigned long long m = __ballot(far >> b & 1); m; m &= m - 1)
                far_grad<TPR, NV>(a, first + (64L * b + __ffsll(m) - 1) * a.slots, t, dw, part64);
    }
    if (!a.part) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (t + TPR * i);
        if (c >= a.H) continue;
        float *const o = a.part + (size_t)slot * a.H + c;
        *(MOE_GLOBAL f32x4 *)o = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        *(MOE_GLOBAL f32x4 *)(o + 4) = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
}

// dw: the slots' parts, 32 columns a workgroup: 32 groups of slots, each in order,
// then the groups in order.
__global__ __launch_bounds__(256) void norm_join_kernel(const float *__restrict__ part, int slots, int H,
                                                        int accumulate, float *__restrict__ dw) {
    __shared__ f32x4 sums[32][8];
    const int l = threadIdx.x & 7, g = threadIdx.x >> 3, c = 32 * blockIdx.x + 4 * l;
    const int s0 = (int)((long)slots * g / 32), s1 = (int)((long)slots * (g + 1) / 32);
    f32x4 v = {0, 0, 0, 0};
    if (c < H) {
#pragma unroll 8
        for (int s = s0; s < s1; ++s) v += *(const MOE_GLOBAL f32x4 *)(part + (size_t)s * H + c);
    }
    sums[g][l] = v;
    __syncthreads();
    if (g || c >= H) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) v += sums[i][l];
    MOE_GLOBAL f32x4 *const o = (MOE_GLOBAL f32x4 *)(dw + c);
    *o = accumulate ? *o + v : v;
}

// ------------------------------------------------------------------ moves --

// Row that pair p stands at, or -1 where it is none of the n there are.
__device__ __forceinline__ int pair_at(const int32_t *pair_row, size_t p, int n) {
    const int r = pair_row[p];
    return r >= 0 && r < n ? r : -1;
}

// 8 columns of one token a thread: read once, written to its k rows. HBM's stores bound
// it. (8192 tokens of 2048 to 8 rows each: 52 us, 5.8 TB/s; writing scattered rows
// alone takes 51; with stores that stay in the caches, or a non-temporal load of rows
// that the caches may hold, 60.)
__global__ __launch_bounds__(256) void dispatch_kernel(const uint16_t *__restrict__ x,
                                                       const int32_t *__restrict__ pair_row, int T, int k,
                                                       int H, Divisor by, uint16_t *__restrict__ out,
                                                       int out_n) {
    const int per = H / 8;
    const long id = block_id() * blockDim.x + threadIdx.x, t = row_of_unit(id, 8, per, by);
    if (t >= T) return;
    const int c = (int)(id - t * per) * 8;
    const u32x4 v = load16(x + (size_t)t * H + c);
    for (int j0 = 0; j0 < k; j0 += 8) {
        int r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = j0 + j < k ? pair_at(pair_row, (size_t)t * k + j0 + j, out_n) : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r[j] >= 0) store_nt(out + (size_t)r[j] * H + c, v);
    }
}

// 8 columns of one token a thread; the rows of KB pairs are loaded together, one that
// exists (and whose values are cleared) in the place of one that does not: no branch
// stands between the loads. HBM bounds it: 4096 tokens of 8 rows of 2048 26 us in bf16
// (151 MB, 5.9 TB/s), 55 in fp32; 64 tokens of 6 rows of 4096 4 us, two
// trips to memory (indices, rows) on 512 workgroups of one wavefront.
template <bool F32, int KB>
__global__ __launch_bounds__(64) void combine_rows_kernel(const void *__restrict__ y, int y_n,
                                                          const int32_t *__restrict__ pair_row,
                                                          const float *__restrict__ w,
                                                          const uint16_t *__restrict__ add, int T, int k,
                                                          int H, Divisor by, uint16_t *__restrict__ out) {
    const int per = H / 8;
    const long id = block_id() * blockDim.x + threadIdx.x, t = row_of_unit(id, 6, per, by);
    if (t >= T) return;
    const int c = (int)(id - t * per) * 8;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < k; j0 += KB) {
        u32x4 v[KB][F32 ? 2 : 1];
        float f[KB];
        int r[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const size_t p = (size_t)t * k + (j0 + j < k ? j0 + j : k - 1);
            r[j] = pair_at(pair_row, p, y_n);
            f[j] = w ? w[p] : 1.0f;
            if (j0 + j >= k) r[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const size_t at = (size_t)(r[j] < 0 ? 0 : r[j]) * H + c;
            if (F32) {
                v[j][0] = load_nt16((const float *)y + at);
                v[j][F32 ? 1 : 0] = load_nt16((const float *)y + at + 4);
            } else {
                v[j][0] = load_nt16((const uint16_t *)y + at);
            }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const uint32_t keep = r[j] < 0 ? 0u : ~0u;
            const float fj = r[j] < 0 ? 0.0f : f[j];
            float u[8];
            if (F32) {
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = __uint_as_float(v[j][F32 ? i >> 2 : 0][i & 3] & keep);
            } else {
                unpack8(v[j][0] & u32x4{keep, keep, keep, keep}, u);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(fj, u[i], sum[i]);
        }
    }
    if (add) {
        float v[8];
        unpack8(load_nt16(add + (size_t)t * H + c), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
    store_nt(out + (size_t)t * H + c, pack8(sum));
}

// One wavefront a pair; the pairs of a token are neighbours, so that dout's row
// comes from the caches for all but one of them. HBM bounds it: 4096 tokens of 8 rows of
// 2048 53 us (286 MB, half of it written to scattered rows, 5.4 TB/s).
__global__ __launch_bounds__(256) void combine_rows_grad_kernel(
    const uint16_t *__restrict__ dout, const uint16_t *__restrict__ y, int y_n,
    const int32_t *__restrict__ pair_row, const float *__restrict__ w, long pairs, int k, Divisor by, int H,
    uint16_t *__restrict__ dy, float *__restrict__ dw) {
    constexpr int U = 4;
    const long p = block_id() * (blockDim.x / kWave) + threadIdx.x / kWave;
    if (p >= pairs) return;
    const int l = lane_id(), r = pair_at(pair_row, (size_t)p, y_n);
    const size_t from = (size_t)((uint32_t)p / by) * H, at = (size_t)(r < 0 ? 0 : r) * H;
    const float f = w ? w[p] : 1.0f;
    float sum = 0.0f;
    if (r >= 0) {
        for (int c0 = 8 * l; c0 < H; c0 += 8 * kWave * U) {
            u32x4 dq[U], yq[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + 8 * kWave * i;
                dq[i] = yq[i] = u32x4{0, 0, 0, 0};
                if (c < H) {
                    dq[i] = load16(dout + from + c);
                    if (dw) yq[i] = load_nt16(y + at + c);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + 8 * kWave * i;
                float d[8], v[8];
                unpack8(dq[i], d), unpack8(yq[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum = fmaf(d[j], v[j], sum);
                    d[j] *= f;
                }
                if (dy && c < H) store_nt(dy + at + c, pack8(d));
            }
        }
    }
    if (!dw) return;
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if (l == 0) dw[p] = sum;
}

// ------------------------------------------------------------------- host --

template <int QUANT>
static void launch_norm(const NormArgs &a, hipStream_t s) {
    const dim3 block(kNormThreads);
    if (a.H <= 1024) {
        const dim3 grid = blocks_of(((long)a.R + 3) / 4);
        if (a.H <= 512) MOE_LAUNCH(K_NORM, (norm_kernel<64, 1, QUANT>), grid, block, 0, s, a);
        else MOE_LAUNCH(K_NORM, (norm_kernel<64, 2, QUANT>), grid, block, 0, s, a);
        return;
    }
    const dim3 grid = blocks_of(a.R);
    if (a.H <= 2048) MOE_LAUNCH(K_NORM, (norm_kernel<256, 1, QUANT>), grid, block, 0, s, a);
    else if (a.H <= 4096) MOE_LAUNCH(K_NORM, (norm_kernel<256, 2, QUANT>), grid, block, 0, s, a);
    else if (a.H <= 8192) MOE_LAUNCH(K_NORM, (norm_kernel<256, 4, QUANT>), grid, block, 0, s, a);
    else MOE_LAUNCH(K_NORM, (norm_kernel<256, 0, QUANT>), grid, block, 0, s, a);
}

constexpr int kMaxGradH = 16384;     // columns whose dw stays in the registers of 256 threads

// Two workgroups a compute unit, eight wavefronts. (The parts of dw are written and
// read again: with 1, 2, 4 workgroups the gradient of 8192 x 4096 takes 52, 50, 54 us
// with the join, of 32768 x 512 36, 30, 35.) Past 4096 columns a wavefront holds more
// than half of a SIMD's registers, so that the second workgroup of a compute unit
// follows the first: with 1, 2, 4 of them 4096 x 8192 takes 51, 55, 64 us, 16384 x 8192
// 173, 177, 184, 2048 x 16384 57, 65, 83, 600 x 16384 28, 34, 41.
static int grad_slots(int R, int H) {
    const int most = (H <= 1024 ? 8 : 2) * compute_units();
    return R < most ? R : most;
}

}  // namespace moe

using namespace moe;

static bool eps_ok(float eps) { return eps >= 0.0f && eps <= 3.0e38f; }

extern "C" int moe_rms_norm(const uint16_t *x_bf16, const uint16_t *residual_bf16,
                            const uint16_t *weight_bf16, float eps, int R, int H, uint16_t *total_bf16,
                            uint16_t *y_bf16, int quant, uint8_t *q, void *q_scale, void *stream) {
    if (!row_sizes_ok(R, H) || !eps_ok(eps) || quant < kNone || quant > kMxfp4) return MOE_EINVAL;
    if (quant == kMxfp4 && H % 32) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if (!al16(x_bf16) || !al16(weight_bf16) || ((uintptr_t)residual_bf16 & 15) ||
        ((uintptr_t)total_bf16 & 15) || ((uintptr_t)y_bf16 & 15))
        return MOE_EINVAL;
    if (total_bf16 && !residual_bf16) return MOE_EINVAL;
    if (quant != kNone ? !al16(q) || !q_scale || ((uintptr_t)q_scale & (quant == kFp8 ? 3 : 0)) : !y_bf16)
        return MOE_EINVAL;
    const NormArgs a{x_bf16, residual_bf16, weight_bf16, eps, R, H, total_bf16, y_bf16, q, q_scale};
    if (quant == kNone) launch_norm<kNone>(a, (hipStream_t)stream);
    else if (quant == kFp8) launch_norm<kFp8>(a, (hipStream_t)stream);
    else launch_norm<kMxfp4>(a, (hipStream_t)stream);
    return check_launch();
}

extern "C" int moe_rms_norm_grad_workspace(int R, int H, size_t *bytes) {
    if (!row_sizes_ok(R, H) || H > kMaxGradH || !bytes) return MOE_EINVAL;
    *bytes = (size_t)grad_slots(R, H) * H * sizeof(float);
    return MOE_OK;
}

extern "C" int moe_rms_norm_grad(const uint16_t *x_bf16, const uint16_t *weight_bf16,
                                 const uint16_t *dy_bf16, const uint16_t *dtotal_bf16, float eps, int R,
                                 int H, uint16_t *dx_bf16, float *dw, int accumulate, void *ws,
                                 size_t ws_bytes, void *stream) {
    if (!row_sizes_ok(R, H) || H > kMaxGradH || !eps_ok(eps)) return MOE_EINVAL;
    const int slots = grad_slots(R, H);
    if (((uintptr_t)dw & 15) || ((uintptr_t)ws & 15)) return MOE_EINVAL;
    if (dw && R > 0 && (!ws || ws_bytes < (size_t)slots * H * sizeof(float))) return MOE_EINVAL;
    if (R > 0 && (!al16(x_bf16) || !al16(weight_bf16) || !al16(dy_bf16) || !al16(dx_bf16) ||
                  ((uintptr_t)dtotal_bf16 & 15)))
        return MOE_EINVAL;
    hipStream_t s = (hipStream_t)stream;
    if (R > 0) {
        const NormGradArgs a{x_bf16, weight_bf16, dy_bf16, dtotal_bf16, eps, R, H, dx_bf16,
                             dw ? (float *)ws : nullptr, slots};
        const dim3 block(kNormThreads);
        if (H <= 1024) {
            const dim3 grid((unsigned)((slots + 3) / 4));
            if (H <= 512) MOE_LAUNCH(K_NORM_GRAD, (norm_grad_kernel<64, 1>), grid, block, 0, s, a);
            else MOE_LAUNCH(K_NORM_GRAD, (norm_grad_kernel<64, 2>), grid, block, 0, s, a);
        } else {
            const dim3 grid((unsigned)slots);
            if (H <= 2048) MOE_LAUNCH(K_NORM_GRAD, (norm_grad_kernel<256, 1>), grid, block, 0, s, a);
            else if (H <= 4096) MOE_LAUNCH(K_NORM_GRAD, (norm_grad_kernel<256, 2>), grid, block, 0, s, a);
            else if (H <= 8192) MOE_LAUNCH(K_NORM_GRAD, (norm_grad_kernel<256, 4>), grid, block, 0, s, a);
            else MOE_LAUNCH(K_NORM_GRAD, (norm_grad_kernel<256, 8>), grid, block, 0, s, a);
        }
        const int rc = check_launch();
        if (rc != MOE_OK) return rc;
    }
    if (!dw) return MOE_OK;
    MOE_LAUNCH(K_NORM_JOIN, norm_join_kernel, dim3((unsigned)((H + 31) / 32)), dim3(256), 0, s,
               (const float *)ws, R > 0 ? slots : 0, H, accumulate != 0, dw);
    return check_launch();
}

// Sizes of the moves: T tokens of k pairs each.
static bool moves_ok(int T, int k, int H) {
    return T >= 0 && k >= 1 && row_sizes_ok(T, H) && (long)T * k <= kMaxRows;
}

extern "C" int moe_dispatch(const uint16_t *x_bf16, const int32_t *pair_row, int T, int k, int H,
                            uint16_t *out_bf16, int out_n, void *stream) {
    if (!moves_ok(T, k, H) || out_n < 0) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!al16(x_bf16) || !pair_row || (out_n && !al16(out_bf16))) return MOE_EINVAL;
    if (out_n == 0) return MOE_OK;
    const long blocks = ((long)T * (H / 8) + 255) / 256;
    if (!blocks_ok(blocks)) return MOE_EINVAL;
    MOE_LAUNCH(K_DISPATCH, dispatch_kernel, blocks_of(blocks), dim3(256), 0, (hipStream_t)stream, x_bf16,
               pair_row, T, k, H, divisor(H / 8), out_bf16, out_n);
    return check_launch();
}

extern "C" int moe_combine_rows(const void *y, int y_is_fp32, int y_n, const int32_t *pair_row,
                                const float *w, const uint16_t *add_bf16, int T, int k, int H,
                                uint16_t *out_bf16, void *stream) {
    if (!moves_ok(T, k, H) || y_n < 0) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if ((y_n && !al16(y)) || !pair_row || ((uintptr_t)add_bf16 & 15) || !al16(out_bf16)) return MOE_EINVAL;
    const long blocks = ((long)T * (H / 8) + 63) / 64;
    if (!blocks_ok(blocks)) return MOE_EINVAL;
    hipStream_t s = (hipStream_t)stream;
    if (y_n == 0) y = out_bf16, y_is_fp32 = 0;       // (no row exists: any memory of that size is read instead)
#define MOE_CR(F32, KB)                                                                             \
    MOE_LAUNCH(K_COMBINE_ROWS, (combine_rows_kernel<F32, KB>), blocks_of(blocks), dim3(64), 0, s, y, \
               y_n, pair_row, w, add_bf16, T, k, H, divisor(H / 8), out_bf16)
    if (k <= 2) {
        if (y_is_fp32) MOE_CR(true, 2);
        else MOE_CR(false, 2);
    } else {
        if (y_is_fp32) MOE_CR(true, 8);
        else MOE_CR(false, 8);
    }
#undef MOE_CR
    return check_launch();
}

extern "C" int moe_combine_rows_grad(const uint16_t *dout_bf16, const uint16_t *y_bf16, int y_n,
                                     const int32_t *pair_row, const float *w, int T, int k, int H,
                                     uint16_t *dy_bf16, float *dw, void *stream) {
    if (!moves_ok(T, k, H) || y_n < 0) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!al16(dout_bf16) || !pair_row || ((uintptr_t)dy_bf16 & 15) || (!dy_bf16 && !dw && y_n)) return MOE_EINVAL;
    if (dw && y_n && !al16(y_bf16)) return MOE_EINVAL;
    const long pairs = (long)T * k;
    MOE_LAUNCH(K_COMBINE_ROWS_GRAD, combine_rows_grad_kernel, blocks_of((pairs + 3) / 4), dim3(256), 0,
               (hipStream_t)stream, dout_bf16, y_bf16, y_n, pair_row, w, pairs, k, divisor(k), H, dy_bf16,
               dw);
    return check_launch();
}
