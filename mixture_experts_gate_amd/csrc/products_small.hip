// The products of products.hip in tiles of 128 x 128, for calls in which tiles of
// 256 x 256 are too few to fill the device. Four wavefronts take 64 x 64 each;
// LDS holds four steps, three of them copied ahead, so that a step costs its
// matrix instructions, reads and one barrier (0.8 us) and not a copy's latency.
// Operand layouts as there. Where even these tiles are few and the sums long,
// c is cut into parts that join_kernel adds up.
#include "products.hpp"

namespace moe {

constexpr int kTThreads = 256;
constexpr int kT = 128;          // p and q per tile

constexpr int S = 4;             // steps in LDS

struct SmallLds {
    char p[S][kT * 128];
    char q[S][kT * 128];
    int src[kT];              // source row of each LDS row of p (forward, dx)
    int dst[kT];              // row of out, or -1
    float xs[S][kT];          // FP8: scales of the p rows, by step
    int raw[S + 3][2][64];    // dw: indices of the rows of dy and x, by step,
    int rows[S + 3][2][64];   // and the rows
    int base[kMaxE + 1];  // p tiles before each expert
    int wsum[4];
};

template <int MODE>
__global__ __launch_bounds__(kTThreads) void product_small_kernel(ProductArgs A) {
    constexpr bool kDwMode = MODE == kDw, kQT = MODE == kDx || MODE == kDw;
    constexpr int ES = MODE == kFwdFp8 ? 1 : 2;       // bytes of an element
    constexpr int CK = 128 / ES;                       // c per step
    __shared__ SmallLds L;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l = lane_id(), t = threadIdx.x, g = l >> 4, r = l & 15;
    const int wq = w & 1, wp = w >> 1;

    const int Qn = MODE == kFwd || MODE == kFwdFp8 ? A.N : A.K;  // q count
    const int tq = (Qn + kT - 1) / kT;
    const int tpw = (A.N + kT - 1) / kT;                          // p tiles (dw)
    const int KB = (A.K + 127) / 128;
    const size_t lda = (size_t)(MODE == kFwd || MODE == kFwdFp8 ? A.K : A.N) * ES;
    const size_t ldq = (size_t)A.K * ES;                          // rows of W, x

    int total;
    if (kDwMode) {
        total = A.E * tpw * tq;
    } else {
        total_tiles<kTThreads>(A, kT, L.base, L.wsum);
        total = L.base[A.E] * tq;
    }
    const int ns = A.slices;
    total *= ns;
    const int nx = gridDim.x >= 8 ? 8 : 1;
    const int xcd = blockIdx.x % nx, per = ((int)gridDim.x - xcd + nx - 1) / nx;
    const int t0 = (int)((long)total * xcd / nx), t1 = (int)((long)total * (xcd + 1) / nx);
    for (int si = t0 + (int)blockIdx.x / nx; si < t1; si += per) {
        const int ti = ns > 1 ? si / ns : si, slice = si - ti * ns;     // tile, part of its c
        int e, p0, q0, lo, cnt, half = 64;
        if (kDwMode) {
            e = ti / (tpw * tq);
            place_of(ti - e * tpw * tq, tpw, tq, p0, q0);
            group_of(A, e, lo, cnt);
            p0 *= kT;
        } else {
            // the expert's rows are spread evenly over its tiles, in units of 32
            e = expert_of(L.base, A.E, tq, ti);
            const int mp = __builtin_amdgcn_readfirstlane(L.base[e + 1] - L.base[e]);
            const int li = ti - __builtin_amdgcn_readfirstlane(L.base[e]) * tq;
            group_of(A, e, lo, cnt);
            half = 16 * (int)((cnt + 32u * mp - 1) / (32u * mp));
            half = half < 64 ? half : 64;
            place_of(li, mp, tq, p0, q0);
            p0 *= 2 * half;
        }
        q0 *= kT;
        const int np = half / 16;    // p tiles of a wavefront with work
        const int C = kDwMode ? cnt : MODE == kDx ? A.N : A.K;
        const int steps = (C + CK - 1) / CK;
        const int kb = (int)((long)steps * slice / ns), ke = (int)((long)steps * (slice + 1) / ns);

        __syncthreads();   // the last tile's readers of L are done
        if (!kDwMode) {
            if (t < kT) {
                const int o = t & 63, p = p0 + (t >> 6) * half + o;
                const bool in = o < half && p < cnt;
                const int i = lo + (in ? p : 0);
                const int s = source_row(A.a, i);
                int d = -1;
                if (in && s >= 0) {
                    d = A.out_rows ? A.out_rows[i] : i;
                    d = d < 0 || d >= A.out_n ? -1 : ns > 1 ? i : d;     // (parts keep sorted order)
                }
                L.src[t] = s < 0 ? 0 : s;
                L.dst[t] = d;
            }
        } else if (w < 2 && cnt > 0) {
            const RowsIn &in = w == 0 ? A.a : A.b;
#pragma unroll
            for (int k = kb; k < kb + S + 2; ++k)
                copy_indices(in, 64 * k, lo, cnt, L.raw[k % (S + 3)][w]);
            wait_copies<0>();
#pragma unroll
            for (int k = kb; k < kb + S + 2; ++k)
                rows_from_indices(in, 64 * k, lo, cnt, L.raw[k % (S + 3)][w], L.rows[k % (S + 3)][w]);
        }
        __syncthreads();

        // Copies: 8 rows of 128 bytes an instruction, or 4 rows of 256 (c-major);
        // rows past the end of p or q read one that exists, c past its end
        // becomes zeros.
        const char *pp[4], *qp[4];
        const int chunk = (l & 7) ^ (l >> 3), tchunk = (l & 15) ^ t_key<kDwMode>(l >> 4);
        const int tc = 4 * w + (l >> 4);                      // c of a c-major copy (+ 16 i)
        const char *const mat = kDwMode ? A.b.base : mat_of(A, e, ES);
        const size_t pcol = kDwMode ? 2 * (size_t)(p0 + 8 * tchunk < A.N ? p0 + 8 * tchunk : 0) : 0;
        const size_t qcol = kQT ? 2 * (size_t)(q0 + 8 * tchunk < Qn ? q0 + 8 * tchunk : 0) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!kDwMode) pp[i] = A.a.base + (size_t)L.src[32 * i + 8 * w + (l >> 3)] * lda + 16 * chunk;
            if (!kQT) {
                const int rr = (32 * i + 8 * w + (l >> 3)) & 63;
                int n = q0 + 64 * (i >> 1) + perm64<MODE>(rr >> 4, rr & 15);
                n = n < Qn ? n : Qn - 1;
                qp[i] = mat + (size_t)n * ldq + 16 * chunk;
            } else if (MODE == kDx) {
                qp[i] = mat + (size_t)(16 * i + tc) * ldq + qcol;
            }
        }
        const float *ws = nullptr;
        if (MODE == kFwdFp8) ws = scales_of(A, e) + (size_t)(q0 / 128) * KB;

        auto fetch = [&](int k) {
            char *const P = L.p[k % S], *const Q = L.q[k % S];
            const bool full = (k + 1) * CK <= C;
            if (kDwMode) {
                const size_t first = (size_t)(lo + 64 * k + 4 * w);
                copy_rows<4, 256>(full && !A.a.idx && !A.b.idx,
                                  Rows{A.a, first, lda, (uint32_t)((l >> 4) * lda + pcol), (uint32_t)pcol,
                                       &L.rows[k % (S + 3)][0][tc], P + 4 * w * 256},
                                  Rows{A.b, first, ldq, (uint32_t)((l >> 4) * ldq + qcol), (uint32_t)qcol,
                                       &L.rows[k % (S + 3)][1][tc], Q + 4 * w * 256});
                return;
            }
            if (full) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lds_dma16(pp[i] + (size_t)k * 128, P + (32 * i + 8 * w) * 128);
                    if (MODE == kDx) lds_dma16(qp[i] + (size_t)k * CK * ldq, Q + (16 * i + 4 * w) * 256);
                    else lds_dma16(qp[i] + (size_t)k * 128, Q + (32 * i + 8 * w) * 128);
                }
            } else {
                const bool in = k * CK + chunk * (16 / ES) < C;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    copy_or_zeros(in, pp[i] + (size_t)k * 128, P + (32 * i + 8 * w) * 128);
                    if (MODE == kDx)
                        copy_or_zeros(k * CK + 16 * i + tc < C, qp[i] + (size_t)k * CK * ldq,
                                      Q + (16 * i + 4 * w) * 256);
                    else
                        copy_or_zeros(in, qp[i] + (size_t)k * 128, Q + (32 * i + 8 * w) * 128);
                }
            }
            if (MODE == kFwdFp8 && w < 2)
                lds_dma4(A.a_s + (size_t)L.src[64 * w + l] * KB + k, &L.xs[k % S][64 * w]);
        };

        f32x4 acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < S - 1; ++k)
            if (kb + k < ke) fetch(kb + k);
        for (int k = kb; k < ke; ++k) {
            const char *const bp = L.p[k % S], *const bq = L.q[k % S];
            // the indices of step k + S + 2, which have landed by the wait of step k + 2
            if (kDwMode && w < 2 && k + S + 2 < ke)
                copy_indices(w == 0 ? A.a : A.b, 64 * (k + S + 2), lo, cnt, L.raw[(k + S + 2) % (S + 3)][w]);
            // step k is in LDS (of the S - 2 steps after it, those copied may be in
            // flight), and step k - 1 is read
            const int later = ke - 1 - k < S - 2 ? ke - 1 - k : S - 2;
            if (later >= 2) wait_copies<16>();
            else if (later == 1) wait_copies<8>();
            else wait_copies<0>();
            wait_lds();
            bare_barrier();
            // the rows of step k + S, for the next step's copies
            if (kDwMode && w < 2 && k >= kb + 2 && k + S < ke)
                rows_from_indices(w == 0 ? A.a : A.b, 64 * (k + S), lo, cnt, L.raw[(k + S) % (S + 3)][w],
                                  L.rows[(k + S) % (S + 3)][w]);
            if (k + S - 1 < ke) fetch(k + S - 1);
            const float wsk = MODE == kFwdFp8 ? as_scalar(ws)[k] : 0.0f;
            if (MODE == kFwdFp8) {
                u32x4 qf[4][2];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int s = 0; s < 2; ++s) qf[j][s] = frag_n(bq, 64 * wq + 16 * j, s, g, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= np) continue;
                    const u32x4 a = frag_n(bp, 64 * wp + 16 * i, 0, g, r), b = frag_n(bp, 64 * wp + 16 * i, 1, g, r);
                    const float sc = L.xs[k % S][64 * wp + 16 * i + r] * wsk;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            as_i32x8(qf[j][0], qf[j][1]), as_i32x8(a, b), f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[i][j][c] = fmaf(d[c], sc, acc[i][j][c]);
                    }
                }
            } else {
                u32x4 qf[2][4], pf[2][4];
                uint32_t at[4];
                if (kQT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) at[j] = frag_t_at<kDwMode, 256>(bq, wq, j, g, r);
                    frags_t2<256, 0, 32 * 256>(at, qf[0], qf[1]);
                }
                if (kDwMode) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) at[j] = frag_t_at<kDwMode, 256>(bp, wp, j, g, r);
                    frags_t2<256, 0, 32 * 256>(at, pf[0], pf[1]);
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (!kQT) qf[s][j] = frag_n(bq, 64 * wq + 16 * j, s, g, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i >= np) continue;
                        if (!kDwMode) pf[s][i] = frag_n(bp, 64 * wp + 16 * i, s, g, r);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const bf16x8 p = as_bf16x8(pf[s][i]), q = as_bf16x8(qf[s][j]);
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                q_is_row(MODE) ? q : p, q_is_row(MODE) ? p : q, acc[i][j], 0, 0, 0);
                        }
                    }
                }
            }
        }

        ProductArgs to = A;
        if (ns > 1) {
            to.out = A.part + (size_t)slice * (kDwMode ? (size_t)A.E * A.N : (size_t)A.R) * Qn;
            to.out_f32 = 1, to.accumulate = 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= np) continue;
            store_tile<MODE>(to, q0 + 64 * wq, Qn, g, r, acc[i], [&](int p) -> long {
                if (!kDwMode) return L.dst[64 * wp + 16 * i + p];
                const int n = p0 + 64 * wp + 16 * i + p;
                return n < A.N ? (long)e * A.N + n : -1;
            });
        }
    }
}

// The sum of the parts, in order, to out: 4 q a thread.
template <bool DW>
__global__ __launch_bounds__(256) void join_kernel(ProductArgs A, int Qn) {
    const int per = Qn / 4;
    const long id = (long)blockIdx.x * blockDim.x + threadIdx.x;
    const long row = id / per;
    const int q = (int)(id - row * per) * 4;
    const long rows = DW ? (long)A.E * A.N : A.R;
    if (row >= rows) return;
    long to = row;
    if (!DW) {
        const int i = (int)row;
        if (A.offsets && (i < A.offsets[0] || i >= A.offsets[A.E])) return;
        to = A.out_rows ? A.out_rows[i] : i;
        if (to < 0 || to >= A.out_n || source_row(A.a, i) < 0) return;
    }
    f32x4 v = {0, 0, 0, 0};
    for (int k = 0; k < A.slices; ++k)
        v += *(const MOE_GLOBAL f32x4 *)(A.part + ((size_t)k * rows + row) * Qn + q);
    if (A.out_f32) {
        MOE_GLOBAL f32x4 *const o = (MOE_GLOBAL f32x4 *)((float *)A.out + (size_t)to * Qn + q);
        *o = DW && A.accumulate ? *o + v : v;
    } else {
        typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
        *(MOE_GLOBAL u32x2 *)((uint16_t *)A.out + (size_t)to * Qn + q) =
            u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

static long small_tiles(const ProductArgs &a, int mode) {
    const int Qn = mode == kFwd || mode == kFwdFp8 ? a.N : a.K;
    const long tq = (Qn + kT - 1) / kT;
    return mode == kDw ? (long)a.E * ((a.N + kT - 1) / kT) * tq
                       : (a.R / kT + (a.R < a.E ? a.R : a.E)) * tq;
}

// With few tiles and many steps (64 c, FP8 128) each, c is cut into parts whose
// sums are added afterwards in their order: as many as give every compute unit two
// (dw and dx of 6546 rows, 3320 x 280: 118 us; with one each, 185 us, since 156
// tiles are then not cut at all), of six steps at least. (A step takes 0.8 us, the addition's launch 2
// to 3 us. Forward of 261 rows, K = 3648, N = 112: 48 us whole, 17 us in parts.)
int small_slices(const ProductArgs &a, int mode) {
    const long tiles = small_tiles(a, mode);
    const long c = mode == kDw ? a.R / a.E : mode == kDx ? a.N : a.K;
    const long steps = c / (mode == kFwdFp8 ? 128 : 64);
    long n = 2L * compute_units() / (tiles < 1 ? 1 : tiles);
    n = n < steps / 6 ? n : steps / 6;
    return n < 2 ? 1 : n > 16 ? 16 : (int)n;
}

void launch_product_small(const ProductArgs &a, int mode, hipStream_t s) {
    const int Qn = mode == kFwd || mode == kFwdFp8 ? a.N : a.K;
    const long tiles = small_tiles(a, mode) * a.slices;
    const int cu = compute_units();
    const dim3 grid((unsigned)(tiles < 2L * cu ? tiles : 2L * cu)), block(kTThreads);
    const int kid = kernel_of(mode);
    if (mode == kFwd) MOE_LAUNCH(kid, product_small_kernel<kFwd>, grid, block, 0, s, a);
    else if (mode == kFwdFp8) MOE_LAUNCH(kid, product_small_kernel<kFwdFp8>, grid, block, 0, s, a);
    else if (mode == kDx) MOE_LAUNCH(kid, product_small_kernel<kDx>, grid, block, 0, s, a);
    else MOE_LAUNCH(kid, product_small_kernel<kDw>, grid, block, 0, s, a);
    if (a.slices > 1) {
        const long n = (mode == kDw ? (long)a.E * a.N : (long)a.R) * (Qn / 4);
        const dim3 blocks((unsigned)((n + 255) / 256));
        if (mode == kDw) MOE_LAUNCH(K_PROD_JOIN, join_kernel<true>, blocks, dim3(256), 0, s, a, Qn);
        else MOE_LAUNCH(K_PROD_JOIN, join_kernel<false>, blocks, dim3(256), 0, s, a, Qn);
    }
}

}  // namespace moe
