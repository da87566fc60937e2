// Matrix products grouped by expert, with ragged row counts:
//   forward  y[i]  = W_e x[r(i)]                    (bf16, or FP8 with a scale per 128)
//   dx       dx[i] = W_e^T dy[r(i)]                 (bf16)
//   dw       dW_e  = sum over the expert's rows i of dy[r(i)] x[r'(i)]^T
// for the rows i of sorted order in [offsets[e], offsets[e+1]), r(i) = i or
// rows[i] / div.
//
// All of them are out[p][q] = sum_c P[p][c] Q[q][c]:
//   forward: p = row, q = n, c = k;  dx: p = row, q = k, c = n;
//   dw: p = n, q = k, c = row.
// An operand is held in memory either with c contiguous (x, dy, W in the
// forward) or with its own index contiguous (W in dx, both operands in dw).
// The first kind enters LDS as rows of 128 bytes of c, the second as 64 rows of
// c; the matrix core wants 8 consecutive c per lane, which the first kind
// gives with one 16-byte read and the second with two transposing reads
// (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 columns and each gets one
// column). Q is the A operand and P the B operand of the 16x16 instruction, so
// a lane ends with 4 consecutive q of one p; the 16 rows of an A tile are
// chosen as q = 16 (r/4) + 4 j + r%4 over four tiles j, which makes them 16
// consecutive q and the stores full lines.
//
// FP8: out[p][q] = sum_b xs[p][b] ws[q/128][b] (sum over 128 columns of block
// b). The inner sum is one 16x16x128 instruction started at zero; a lane's
// four results share one p, so their scale is one number per lane, and
// adding them to the fp32 sums is four multiply-adds.
//
// Rows past an expert's last one read a row that exists and are not stored;
// columns past the end of c read zeros from a zero page (both operands, so
// that no garbage meets a zero).
#include <atomic>

#include "products.hpp"

namespace moe {

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

constexpr int kPThreads = 512;   // 8 wavefronts: 2 along p x 4 along q
constexpr int kBQ = 256;         // q per tile
constexpr int kMaxE = 512;

__device__ const uint32_t g_zero_page[64] = {0};

// XOR key of the 16-byte chunks of an LDS row of c-major data: rows c..c+3 of
// one transposing read (4 pieces of 8 bytes, 32 bytes apart) land in 16
// different chunks of the 256 bytes that the banks span.
__device__ __forceinline__ int t_key(int c) { return (c & 1) | ((c & 2) << 2); }

// Index inside a 64-row block of the p or q that tile j, row r stands for.
__device__ __forceinline__ int perm64(int j, int r) { return 16 * (r >> 2) + 4 * j + (r & 3); }

template <int BP>
struct TileLds {
    char p[2][BP * 128];
    char q[2][kBQ * 128];
    int src[BP];          // source row of each p (forward, dx)
    int dst[BP];          // row of out, or -1
    float xs[2][BP];      // FP8: scales of the p rows, this step and the next
    int rows[2][2][64];   // dw: source rows of dy and x, this step and the next
    int base[kMaxE + 1];  // p tiles before each expert
    int wsum[8];
};

// One tile's place: expert, first p and q.
struct Place {
    int e, p0, q0;
};

template <int MODE, int BP>
__global__ __launch_bounds__(kPThreads) void product_kernel(ProductArgs A) {
    constexpr bool kPT = MODE == kDw, kQT = MODE == kDx || MODE == kDw;
    constexpr int ES = MODE == kFwdFp8 ? 1 : 2;       // bytes of an element
    constexpr int CK = 128 / ES;                       // c per step
    constexpr int WP = BP / 2, NP = WP / 16;           // p of a wavefront, its tiles
    constexpr int DP = BP / 64, DQ = kBQ / 64;         // copies per thread and step
    __shared__ TileLds<BP> L;
    const int t = threadIdx.x, l = lane_id(), w = __builtin_amdgcn_readfirstlane(t / kWave);
    const int wq = w & 3, wp = w >> 2, g = l >> 4, r = l & 15;

    const int Pn = MODE == kDw ? A.N : 0;                        // p count (dw)
    const int Qn = MODE == kFwd || MODE == kFwdFp8 ? A.N : A.K;  // q count
    const int tq = (Qn + kBQ - 1) / kBQ;
    const int tpw = (A.N + BP - 1) / BP;
    const int KB = (A.K + 127) / 128;

    // tiles in expert order
    int total;
    if (MODE == kDw) {
        total = A.E * tpw * tq;
    } else {
        int n = 0;
        if (t < A.E) {
            int lo = 0, cnt = A.R;
            if (A.offsets) {
                const int b = A.offsets[t], f = A.offsets[t + 1];
                lo = b < 0 ? 0 : b > A.R ? A.R : b;
                const int hi = f < 0 ? 0 : f > A.R ? A.R : f;
                cnt = hi > lo ? hi - lo : 0;
            }
            n = (cnt + BP - 1) / BP;
        }
        int incl = n;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (l >= d) incl += o;
        }
        if (l == kWave - 1) L.wsum[w] = incl;
        __syncthreads();
        int before = 0;
        for (int i = 0; i < w; ++i) before += L.wsum[i];
        if (t < A.E) L.base[t + 1] = before + incl;
        if (t == 0) L.base[0] = 0;
        __syncthreads();
        total = L.base[A.E] * tq;
    }

    // workgroup b runs on XCD b % 8; each XCD takes a contiguous range of
    // tiles, so that the tiles of one expert share an L2
    const int nx = gridDim.x >= 8 ? 8 : 1;
    const int xcd = blockIdx.x % nx, per = ((int)gridDim.x - xcd + nx - 1) / nx;
    const int t0 = (int)((long)total * xcd / nx), t1 = (int)((long)total * (xcd + 1) / nx);
    for (int ti = t0 + (int)blockIdx.x / nx; ti < t1; ti += per) {
        Place at;
        int lo, cnt;
        if (MODE == kDw) {
            at.e = ti / (tpw * tq);
            const int li = ti - at.e * tpw * tq;
            at.p0 = (li % tpw) * BP;
            at.q0 = (li / tpw) * kBQ;
            group_of(A, at.e, lo, cnt);
        } else {
            // expert e with base[e] <= m < base[e+1]; q outer, p inner
            int a = 0, b = A.E;
            while (b - a > 1) {
                const int mid = (a + b) >> 1;
                if ((long)L.base[mid] * tq <= ti) a = mid;
                else b = mid;
            }
            at.e = __builtin_amdgcn_readfirstlane(a);
            const int mp = __builtin_amdgcn_readfirstlane(L.base[a + 1] - L.base[a]);
            const int li = ti - __builtin_amdgcn_readfirstlane(L.base[a]) * tq;
            at.p0 = (li % mp) * BP;
            at.q0 = (li / mp) * kBQ;
            group_of(A, at.e, lo, cnt);
        }
        const int C = MODE == kDw ? cnt : MODE == kDx ? A.N : A.K;
        const int steps = (C + CK - 1) / CK;

        __syncthreads();   // the last tile's readers of L are done
        if (MODE != kDw) {
            if (t < BP) {
                const int p = at.p0 + t, i = lo + (p < cnt ? p : at.p0);
                const int s = source_row(A.a, i);
                int d = -1;
                if (p < cnt && s >= 0) {
                    d = A.out_rows ? A.out_rows[i] : i;
                    if (d < 0 || d >= A.out_n) d = -1;
                }
                L.src[t] = s < 0 ? 0 : s;
                L.dst[t] = d;
            }
        } else if (t < 128) {
            const int c = t & 63;
            L.rows[0][t >> 6][c] = c < cnt ? source_row(t < 64 ? A.a : A.b, lo + c) : -1;
        }
        __syncthreads();

        // this thread's copies: 8 rows of 128 bytes (or 2 rows of 512) a
        // wavefront and instruction
        const char *pp[DP];
        const char *qp[DQ];
        const char *const mat = MODE == kDw ? nullptr : mat_of(A, at.e, ES);
        const char *const zero = (const char *)g_zero_page;
        const int chunk = (l & 7) ^ (l >> 3);                 // 16-byte chunk of a 128-byte row
        const int tc = 2 * w + (l >> 5);                      // c of a c-major copy (+ 16 i)
        const int tchunk = (l & 31) ^ t_key(tc);              // its chunk (8 columns)
        const size_t lda = (size_t)(MODE == kFwd || MODE == kFwdFp8 ? A.K : A.N) * ES;
        const size_t ldq = (size_t)A.K * ES;                  // rows of W, x
        if (!kPT) {
#pragma unroll
            for (int i = 0; i < DP; ++i)
                pp[i] = A.a.base + (size_t)L.src[64 * i + 8 * w + (l >> 3)] * lda + 16 * chunk;
        }
        if (!kQT) {
#pragma unroll
            for (int i = 0; i < DQ; ++i) {
                const int rr = 8 * w + (l >> 3);
                int n = at.q0 + 64 * i + perm64(rr >> 4, rr & 15);
                n = n < Qn ? n : Qn - 1;
                qp[i] = mat + (size_t)n * ldq + 16 * chunk;
            }
        } else if (MODE == kDx) {
            int col = at.q0 + 8 * tchunk;
            col = col < Qn ? col : 0;
#pragma unroll
            for (int i = 0; i < DQ; ++i)
                qp[i] = mat + (size_t)(16 * i + tc) * ldq + (size_t)col * 2;
        }
        const float *ws = nullptr;
        const float *xs = nullptr;
        if (MODE == kFwdFp8) {
            const int nb = (at.q0 + 64 * wq) / 128;
            ws = scales_of(A, at.e) + (size_t)(nb < (A.N + 127) / 128 ? nb : 0) * KB;
            if (t < BP) xs = A.a_s + (size_t)L.src[t] * KB;
        }

        // copies of step k into buffer b
        auto fetch = [&](int k, int b) {
            const bool tail = (k + 1) * CK > C;
            if (!kPT) {
                const bool in = !tail || k * CK + chunk * (16 / ES) < C;
#pragma unroll
                for (int i = 0; i < DP; ++i)
                    lds_dma16(in ? pp[i] + (size_t)k * 128 : zero, L.p[b] + (64 * i + 8 * w) * 128);
            } else {
                int col = at.p0 + 8 * tchunk;
                col = col < Pn ? col : 0;
#pragma unroll
                for (int i = 0; i < DQ; ++i) {
                    const int s = L.rows[k & 1][0][16 * i + tc];
                    lds_dma16(s >= 0 ? A.a.base + (size_t)s * lda + (size_t)col * 2 : zero,
                              L.p[b] + (16 * i + 2 * w) * 512);
                }
            }
            if (!kQT) {
                const bool in = !tail || k * CK + chunk * (16 / ES) < C;
#pragma unroll
                for (int i = 0; i < DQ; ++i)
                    lds_dma16(in ? qp[i] + (size_t)k * 128 : zero, L.q[b] + (64 * i + 8 * w) * 128);
            } else if (MODE == kDx) {
#pragma unroll
                for (int i = 0; i < DQ; ++i)
                    lds_dma16(k * CK + 16 * i + tc < C ? qp[i] + (size_t)k * CK * ldq : zero,
                              L.q[b] + (16 * i + 2 * w) * 512);
            } else {
                int col = at.q0 + 8 * tchunk;
                col = col < Qn ? col : 0;
#pragma unroll
                for (int i = 0; i < DQ; ++i) {
                    const int s = L.rows[k & 1][1][16 * i + tc];
                    lds_dma16(s >= 0 ? A.b.base + (size_t)s * ldq + (size_t)col * 2 : zero,
                              L.q[b] + (16 * i + 2 * w) * 512);
                }
            }
            if (MODE == kFwdFp8 && w < BP / kWave) lds_dma4(xs + k, &L.xs[b][64 * w]);
        };

        f32x4 acc[NP][4];
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

        // 8 consecutive c (16 bytes) of the wavefront's tile j of p or q, half s
        auto frag_n = [&](const char *buf, int row, int s) {
            return *(const MOE_LDS u32x4 *)(buf + (row + r) * 128 + (((4 * s + g) ^ (r & 7)) << 4));
        };
        auto frag_t = [&](const char *buf, int blk, int j, int s) {
            const int ci = r >> 2, tt = r & 3;
            const int ch = (8 * blk + 2 * tt + (j >> 1)) ^ t_key(ci);
            const char *a = buf + (32 * s + 8 * g + ci) * 512 + ch * 16 + (j & 1) * 8;
            const s16x4 lo4 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4 *)(a));
            const s16x4 hi4 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4 *)(a + 4 * 512));
            typedef __attribute__((ext_vector_type(8))) short s16x8;
            const s16x8 v = {lo4[0], lo4[1], lo4[2], lo4[3], hi4[0], hi4[1], hi4[2], hi4[3]};
            return __builtin_bit_cast(u32x4, v);
        };

        if (steps > 0) fetch(0, 0);
        for (int k = 0; k < steps; ++k) {
            const int b = k & 1;
            int next_row = 0;
            if (MODE == kDw && t < 128) {
                const int c = (k + 1) * 64 + (t & 63);
                next_row = c < cnt ? source_row(t < 64 ? A.a : A.b, lo + c) : -1;
                L.rows[(k + 1) & 1][t >> 6][t & 63] = next_row;
            }
            wait_vm<0>();
            __syncthreads();
            if (k + 1 < steps) fetch(k + 1, b ^ 1);
            if (MODE == kFwdFp8) {
                const float wsk = as_scalar(ws)[k];
                i32x8 qf[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x4 a0 = frag_n(L.q[b], 64 * wq + 16 * j, 0);
                    const u32x4 a1 = frag_n(L.q[b], 64 * wq + 16 * j, 1);
                    qf[j] = i32x8{(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3],
                                  (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
                }
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const u32x4 b0 = frag_n(L.p[b], WP * wp + 16 * i, 0);
                    const u32x4 b1 = frag_n(L.p[b], WP * wp + 16 * i, 1);
                    const i32x8 pf = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3],
                                      (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
                    const float sc = L.xs[b][WP * wp + 16 * i + r] * wsk;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            qf[j], pf, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[i][j][c] = fmaf(d[c], sc, acc[i][j][c]);
                    }
                }
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    bf16x8 qf[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        qf[j] = as_bf16x8(kQT ? frag_t(L.q[b], wq, j, s)
                                              : frag_n(L.q[b], 64 * wq + 16 * j, s));
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const bf16x8 pf =
                            as_bf16x8(kPT ? frag_t(L.p[b], (WP / 64) * wp + (i >> 2), i & 3, s)
                                          : frag_n(L.p[b], WP * wp + 16 * i, s));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[j], pf,
                                                                                acc[i][j], 0, 0, 0);
                    }
                }
            }
        }

        // lane (g, r): p of tile i, q = 64 wq + 16 g + 4 j + 0..3
        const int q = at.q0 + 64 * wq + 16 * g;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            long row;
            if (MODE == kDw) {
                const int p = at.p0 + WP * wp + (i >> 2) * 64 + perm64(i & 3, r);
                row = p < Pn ? (long)at.e * A.N + p : -1;
            } else {
                row = L.dst[WP * wp + 16 * i + r];
            }
            if (row < 0) continue;
            if (A.out_f32) {
                float *o = (float *)A.out + (size_t)row * Qn + q;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (q + 4 * j < Qn) {
                        f32x4 v = acc[i][j];
                        if (MODE == kDw && A.accumulate) v += *(const MOE_GLOBAL f32x4 *)(o + 4 * j);
                        *(MOE_GLOBAL f32x4 *)(o + 4 * j) = v;
                    }
                }
            } else {
                uint16_t *o = (uint16_t *)A.out + (size_t)row * Qn + q;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (q + 8 * h < Qn) {
                        const f32x4 a0 = acc[i][2 * h], a1 = acc[i][2 * h + 1];
                        *(MOE_GLOBAL u32x4 *)(o + 8 * h) =
                            u32x4{pack_bf16x2(a0[0], a0[1]), pack_bf16x2(a0[2], a0[3]),
                                  pack_bf16x2(a1[0], a1[1]), pack_bf16x2(a1[2], a1[3])};
                    }
                }
            }
        }
    }
}

int compute_units() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
            n = 256;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int MODE>
static void launch_product(const ProductArgs &a, hipStream_t s) {
    const int cu = compute_units();
    constexpr int kid = MODE == kFwd ? K_PROD : MODE == kFwdFp8 ? K_PROD_FP8 : MODE == kDx ? K_PROD_DX : K_PROD_DW;
    // one workgroup a compute unit (its LDS); fewer where there are fewer tiles
    if (MODE == kDw) {
        constexpr int BP = 256;
        const long tiles = (long)a.E * ((a.N + BP - 1) / BP) * ((a.K + kBQ - 1) / kBQ);
        MOE_LAUNCH(kid, (product_kernel<MODE, 256>), dim3((unsigned)(tiles < cu ? tiles : cu)),
                   dim3(kPThreads), 0, s, a);
        return;
    }
    const int Qn = MODE == kDx ? a.K : a.N;
    const long avg = a.R / a.E;
    const int BP = avg > 128 ? 256 : avg > 64 ? 128 : 64;
    const long most = ((a.R + BP - 1) / BP + (a.R < a.E ? a.R : a.E)) * (long)((Qn + kBQ - 1) / kBQ);
    const dim3 grid((unsigned)(most < cu ? most : cu));
    if (BP == 256) MOE_LAUNCH(kid, (product_kernel<MODE, 256>), grid, dim3(kPThreads), 0, s, a);
    else if (BP == 128) MOE_LAUNCH(kid, (product_kernel<MODE, 128>), grid, dim3(kPThreads), 0, s, a);
    else MOE_LAUNCH(kid, (product_kernel<MODE, 64>), grid, dim3(kPThreads), 0, s, a);
}

// Sizes that every product shares; unit: the elements of 16 bytes.
static int check_sizes(int R, int N, int K, int E, const int32_t *offsets, int unit) {
    if (R < 0 || E < 1 || E > kMaxE || N < 8 || K < unit || N % 8 || K % unit) return MOE_EINVAL;
    if (N > (1 << 24) || K > (1 << 24)) return MOE_EINVAL;
    if (!offsets && E != 1) return MOE_EINVAL;
    return MOE_OK;
}

static bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// rows: every row is read in place (n >= R), or through an index
static bool rows_ok(const void *base, const int32_t *idx, int div, int n, int R) {
    return base && aligned16(base) && div >= 1 && n >= (idx ? 1 : R);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_gemm(const uint16_t *x_bf16, const int32_t *x_rows, int x_div, int x_n,
                                const int32_t *offsets, const uint16_t *w_bf16,
                                const moe_expert_w *experts, int mat, int R, int N, int K, int E,
                                void *y, const int32_t *y_rows, int y_n, int y_is_fp32,
                                void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 8);
    if (rc != MOE_OK) return rc;
    if (mat != MOE_MAT_W13 && mat != MOE_MAT_W2) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if ((!w_bf16) == (!experts) || !aligned16(w_bf16) || !y || !aligned16(y)) return MOE_EINVAL;
    if (!rows_ok(x_bf16, x_rows, x_div, x_n, R) || y_n < (y_rows ? 1 : R)) return MOE_EINVAL;
    ProductArgs a{};
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = RowsIn{(const char *)x_bf16, x_rows, x_div, x_n};
    a.m = Mats{(const char *)w_bf16, nullptr, experts, mat};
    a.out = y, a.out_rows = y_rows, a.out_n = y_n, a.out_f32 = y_is_fp32 != 0;
    launch_product<kFwd>(a, (hipStream_t)stream);
    return check_launch();
}

extern "C" int moe_grouped_gemm_fp8(const uint8_t *x_e4m3, const float *x_scale,
                                    const int32_t *x_rows, int x_div, int x_n,
                                    const int32_t *offsets, const uint8_t *w_e4m3,
                                    const float *w_scale, const moe_expert_w *experts, int mat,
                                    int R, int N, int K, int E, void *y, const int32_t *y_rows,
                                    int y_n, int y_is_fp32, void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 16);
    if (rc != MOE_OK) return rc;
    if (mat != MOE_MAT_W13 && mat != MOE_MAT_W2) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if ((!w_e4m3) == (!experts) || (!w_e4m3) != (!w_scale) || !aligned16(w_e4m3) || !y || !aligned16(y))
        return MOE_EINVAL;
    if (!x_scale || !rows_ok(x_e4m3, x_rows, x_div, x_n, R) || y_n < (y_rows ? 1 : R))
        return MOE_EINVAL;
    ProductArgs a{};
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = RowsIn{(const char *)x_e4m3, x_rows, x_div, x_n};
    a.a_s = x_scale;
    a.m = Mats{(const char *)w_e4m3, w_scale, experts, mat};
    a.out = y, a.out_rows = y_rows, a.out_n = y_n, a.out_f32 = y_is_fp32 != 0;
    launch_product<kFwdFp8>(a, (hipStream_t)stream);
    return check_launch();
}

extern "C" int moe_grouped_gemm_dx(const uint16_t *dy_bf16, const int32_t *dy_rows, int dy_div,
                                   int dy_n, const int32_t *offsets, const uint16_t *w_bf16,
                                   const moe_expert_w *experts, int mat, int R, int N, int K,
                                   int E, void *dx, const int32_t *dx_rows, int dx_n,
                                   int dx_is_fp32, void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 8);
    if (rc != MOE_OK) return rc;
    if (mat != MOE_MAT_W13 && mat != MOE_MAT_W2) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if ((!w_bf16) == (!experts) || !aligned16(w_bf16) || !dx || !aligned16(dx)) return MOE_EINVAL;
    if (!rows_ok(dy_bf16, dy_rows, dy_div, dy_n, R) || dx_n < (dx_rows ? 1 : R)) return MOE_EINVAL;
    ProductArgs a{};
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = RowsIn{(const char *)dy_bf16, dy_rows, dy_div, dy_n};
    a.m = Mats{(const char *)w_bf16, nullptr, experts, mat};
    a.out = dx, a.out_rows = dx_rows, a.out_n = dx_n, a.out_f32 = dx_is_fp32 != 0;
    launch_product<kDx>(a, (hipStream_t)stream);
    return check_launch();
}

extern "C" int moe_grouped_gemm_dw(const uint16_t *dy_bf16, const int32_t *dy_rows, int dy_div,
                                   int dy_n, const uint16_t *x_bf16, const int32_t *x_rows,
                                   int x_div, int x_n, const int32_t *offsets, int R, int N, int K,
                                   int E, void *dw, int dw_is_fp32, int accumulate, void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 8);
    if (rc != MOE_OK) return rc;
    if (accumulate && !dw_is_fp32) return MOE_EINVAL;
    if (!dw || !aligned16(dw)) return MOE_EINVAL;
    if (R > 0 && (!rows_ok(dy_bf16, dy_rows, dy_div, dy_n, R) || !rows_ok(x_bf16, x_rows, x_div, x_n, R)))
        return MOE_EINVAL;
    ProductArgs a{};
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = RowsIn{(const char *)dy_bf16, dy_rows, dy_div, dy_n};
    a.b = RowsIn{(const char *)x_bf16, x_rows, x_div, x_n};
    a.out = dw, a.out_n = E * N, a.out_f32 = dw_is_fp32 != 0, a.accumulate = accumulate != 0;
    launch_product<kDw>(a, (hipStream_t)stream);
    return check_launch();
}
