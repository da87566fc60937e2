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
// column). Which operand is A and which q make a tile goes by the stores (perm64).
//
// FP8: out[p][q] = sum_b xs[p][b] ws[q/128][b] (sum over 128 columns of block
// b). The inner sum is one 16x16x128 instruction started at zero, whose results
// are scaled and added to the fp32 sums. (The instruction adds 8 columns'
// products aligned to the largest, dropping what lies 13 bits below its
// leading bit; across the eights it keeps fp32. Each code was rounded to 2^-4
// before; bf16 instructions on converted codes, which add in fp32, have half
// the rate and were not tried, not in the streaming kernel either, which HBM bounds.)
//
// Rows past an expert's last one read a row that exists and are not stored;
// columns past the end of c are zeros in LDS (both operands, so that no
// garbage meets a zero).
#include <atomic>

#include "products.hpp"

namespace moe {

constexpr int kPThreads = 512;   // 8 wavefronts: 2 along p x 4 along q
constexpr int kBP = 256, kBQ = 256;   // p and q per tile

struct TileLds {
    char p[2][kBP * 128];
    char q[2][kBQ * 128];
    int src[kBP];         // source row of each LDS row of p (forward, dx)
    int dst[kBP];         // row of out, or -1
    float xs[4][kBP];     // FP8: scales of the p rows, by step
    int raw[4][2][64];    // dw: indices of the rows of dy and x, by step,
    int rows[4][2][64];   // and the rows
    int base[kMaxE + 1];  // p tiles before each expert
    int wsum[8];
};

template <int MODE>
__global__ __launch_bounds__(kPThreads) void product_kernel(ProductArgs A) {
    constexpr bool kDwMode = MODE == kDw, kQT = MODE == kDx || MODE == kDw;
    constexpr int ES = MODE == kFwdFp8 ? 1 : 2;       // bytes of an element
    constexpr int CK = 128 / ES;                       // c per step
    __shared__ TileLds L;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wq = w & 3, wp = w >> 2;

    const int Qn = MODE == kFwd || MODE == kFwdFp8 ? A.N : A.K;  // q count
    const int tq = (Qn + kBQ - 1) / kBQ;
    const int tpw = (A.N + kBP - 1) / kBP;                        // p tiles (dw)
    const int KB = (A.K + 127) / 128;

    // tiles in expert order
    int total;
    if (kDwMode) {
        total = A.E * tpw * tq;
    } else {
        total_tiles<kPThreads>(A, kBP, L.base, L.wsum);
        total = L.base[A.E] * tq;
    }

    // workgroup b runs on XCD b % 8; each XCD takes a contiguous range of
    // tiles, so that the tiles of one expert share an L2
    const int nx = gridDim.x >= 8 ? 8 : 1;
    const int xcd = blockIdx.x % nx, per = ((int)gridDim.x - xcd + nx - 1) / nx;
    const int t0 = (int)((long)total * xcd / nx), t1 = (int)((long)total * (xcd + 1) / nx);
    for (int ti = t0 + (int)blockIdx.x / nx; ti < t1; ti += per) {
        // the lane is read anew for every tile, so that what is made of it is
        // not kept in registers from tile to tile
        const int l = fresh_lane(), t = kWave * w + l, g = l >> 4, r = l & 15;
        // expert, first p, p rows of a wavefront row (half the tile's), first q
        int e, p0, q0, lo, cnt, half = 128;
        if (kDwMode) {
            e = ti / (tpw * tq);
            const int li = ti - e * tpw * tq;
            place_of(li, tpw, tq, p0, q0);
            p0 *= kBP;
            group_of(A, e, lo, cnt);
        } else {
            // expert e with base[e] <= m < base[e+1]; q outer, p inner. The
            // expert's rows are spread evenly over its tiles, in units of 64.
            e = expert_of(L.base, A.E, tq, ti);
            const int mp = __builtin_amdgcn_readfirstlane(L.base[e + 1] - L.base[e]);
            const int li = ti - __builtin_amdgcn_readfirstlane(L.base[e]) * tq;
            group_of(A, e, lo, cnt);
            // (cnt + cnt / 4 passes 2^31; more than 128 only where offsets do not ascend)
            half = 32 * (int)((cnt + 64u * mp - 1) / (64u * mp));
            half = half < 128 ? half : 128;
            place_of(li, mp, tq, p0, q0);
            p0 *= 2 * half;
        }
        q0 *= kBQ;
        const int nc = half / 32;    // clusters of 32 rows with work
        const int C = kDwMode ? cnt : MODE == kDx ? A.N : A.K;
        const int steps = (C + CK - 1) / CK;

        __syncthreads();   // the last tile's readers of L are done
        if (!kDwMode) {
            if (t < kBP) {
                const int o = t & 127, p = p0 + (t >> 7) * half + o;
                const bool in = o < half && p < cnt;
                const int i = lo + (in ? p : 0);
                const int s = source_row(A.a, i);
                int d = -1;
                if (in && s >= 0) {
                    d = A.out_rows ? A.out_rows[i] : i;
                    if (d < 0 || d >= A.out_n) d = -1;
                }
                L.src[t] = s < 0 ? 0 : s;
                L.dst[t] = d;
            }
        } else if (w < 2 && cnt > 0) {
            const RowsIn &in = w == 0 ? A.a : A.b;
#pragma unroll
            for (int k = 0; k < 4; ++k) copy_indices(in, 64 * k, lo, cnt, L.raw[k][w]);
            wait_copies<0>();
#pragma unroll
            for (int k = 0; k < 4; ++k) rows_from_indices(in, 64 * k, lo, cnt, L.raw[k][w], L.rows[k][w]);
        }
        __syncthreads();

        // A copy instruction of a wavefront takes 8 rows of 128 bytes, or 2 rows
        // of 512 (c-major). Where nothing has to be cut off, its address is a
        // uniform base and a lane's 32-bit offset, made once per tile (fast);
        // where c or q ends inside the copy or a is beyond 32 bits, it is
        // made anew each time (slow), columns of c past the end becoming zeros.
        const int prow = 128 * wp + 8 * wq;                   // LDS row of a p copy (+ 32 i)
        const size_t lda = (size_t)(MODE == kFwd || MODE == kFwdFp8 ? A.K : A.N) * ES;
        const size_t ldq = (size_t)A.K * ES;                  // rows of W, x
        const char *qb = kDwMode ? A.b.base : mat_of(A, e, ES);
        if (!kQT) qb += (size_t)q0 * ldq;
        const bool easy = kDwMode || (q0 + kBQ <= Qn && (size_t)A.a.n * lda <= 0xFFFFFFFFull);
        uint32_t po[4] = {0, 0, 0, 0}, qo;
        {
            const int chunk = (l & 7) ^ (l >> 3);                 // 16-byte chunk of a 128-byte row
            const int tc = 2 * w + (l >> 5);                      // c of a c-major copy (+ 16 i)
            const int tchunk = (l & 31) ^ t_key<kDwMode>(tc);     // its chunk (8 columns)
            if (!kDwMode) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    po[i] = (uint32_t)(L.src[prow + 32 * i + (l >> 3)] * lda) + 16 * chunk;
            } else {
                po[0] = 2 * (p0 + 8 * tchunk < A.N ? p0 + 8 * tchunk : 0);
            }
            if (!kQT) {
                const int rr = 8 * w + (l >> 3);
                qo = (uint32_t)(perm64<MODE>(rr >> 4, rr & 15) * ldq) + 16 * chunk;
            } else {
                const int col = q0 + 8 * tchunk < Qn ? q0 + 8 * tchunk : 0;
                qo = (MODE == kDx ? (uint32_t)(tc * ldq) : 0) + 2 * col;
            }
            if (kDwMode) po[1] = (uint32_t)((l >> 5) * lda) + po[0], po[2] = (uint32_t)((l >> 5) * ldq) + qo;
        }
        const float *ws = nullptr;
        uint32_t xo = 0;         // this thread's row of the scales of a
        if (MODE == kFwdFp8) {
            const int nb = (q0 + 64 * wq) / 128;
            ws = scales_of(A, e) + (size_t)(nb < (A.N + 127) / 128 ? nb : 0) * KB;
            if (t < kBP) xo = (uint32_t)L.src[t];
        }

        // copy i of 4 of step k, operands P and Q
        auto copy_p = [&](int i, int k, bool fast) {
            char *const to = L.p[k & 1] + (prow + 32 * i) * 128;
            if (fast) {
                lds_dma16(scalar_base(A.a.base + (size_t)k * 128) + here(po[i]), to);
            } else {
                const int fl = fresh_lane(), chunk = (fl & 7) ^ (fl >> 3);
                copy_or_zeros(k * CK + chunk * (16 / ES) < C,
                             A.a.base + (size_t)L.src[prow + 32 * i + (fl >> 3)] * lda +
                                 (size_t)k * 128 + 16 * chunk, to);
            }
        };
        auto copy_q = [&](int i, int k, bool fast) {
            char *const to = L.q[k & 1] + (kQT ? (16 * i + 2 * w) * 512 : (64 * i + 8 * w) * 128);
            if (MODE == kDx) {
                const char *const from = scalar_base(qb + (size_t)(k * CK + 16 * i) * ldq) + here(qo);
                if (fast) lds_dma16(from, to);
                else copy_or_zeros(k * CK + 16 * i + 2 * w + (fresh_lane() >> 5) < C, from, to);
            } else if (fast) {
                lds_dma16(scalar_base(qb + (size_t)i * 64 * ldq + (size_t)k * 128) + here(qo), to);
            } else {
                const int fl = fresh_lane(), chunk = (fl & 7) ^ (fl >> 3), rr = 8 * w + (fl >> 3);
                int n = 64 * i + perm64<MODE>(rr >> 4, rr & 15);
                n = q0 + n < Qn ? n : Qn - 1 - q0;
                copy_or_zeros(k * CK + chunk * (16 / ES) < C, qb + n * ldq + (size_t)k * 128 + 16 * chunk,
                              to);
            }
        };
        // dw: copies i and i + 1 of both
        auto copy_both = [&](int i, int k) {
            const bool in_place = 64 * (k + 1) <= cnt && !A.a.idx && !A.b.idx;
            const int c = 16 * i + 2 * w, fl = fresh_lane();
            const size_t first = (size_t)(lo + 64 * k + c);
            copy_rows<2, 512>(in_place,
                              Rows{A.a, first, lda, po[1], po[0], &L.rows[k & 3][0][c + (fl >> 5)],
                                   L.p[k & 1] + c * 512},
                              Rows{A.b, first, ldq, po[2], qo, &L.rows[k & 3][1][c + (fl >> 5)],
                                   L.q[k & 1] + c * 512});
        };
        auto copy_xs = [&](int k) {
            if (MODE == kFwdFp8 && w < kBP / kWave)
                lds_dma4(A.a_s + (size_t)here(xo) * KB + k, &L.xs[k & 3][64 * w]);
        };

        f32x4 acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

        // A step is two clusters of 32 matrix instructions; cluster 0 / 1 takes
        // the first / second 64 p rows of the wavefront with all of q (dw: all
        // rows with the first / second 32 of c). A cluster is two phases, in
        // each of which the wavefronts of one half of p load (fragments of
        // the next cluster from LDS, copies of later steps) while those of
        // the other half, on the same SIMDs, multiply: the halves run one
        // phase apart, a barrier after every phase.
        //   A buffer is written again two phases after its last reader's load
        // phase began, by copies issued after a barrier that the reads'
        // completion (the wait at the end of every load phase) precedes: the
        // first half of step k + 2 in cluster 1 of step k, its second half in
        // cluster 0 of step k + 1. Each copy is waited for a whole step after its
        // issue, in the load phase before the first one that reads it; the 8
        // copies issued since may stay in flight.
        auto first = [&](int k, bool fast) {      // 6 copies (dw: 4)
            if (kDwMode) {
                copy_both(0, k);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) copy_q(i, k, fast);
                copy_p(0, k, fast), copy_p(1, k, fast);
            }
        };
        auto second = [&](int k, bool fast) {     // 2 copies (dw: 4)
            if (kDwMode) copy_both(2, k);
            else copy_p(2, k, fast), copy_p(3, k, fast);
        };
        auto copy_first = [&](int k) {
            copy_xs(k);
            if (easy && (k + 1) * CK <= C) first(k, true);
            else first(k, false);
        };
        auto copy_second = [&](int k) {
            if (easy && (k + 1) * CK <= C) second(k, true);
            else second(k, false);
        };
        if (steps > 0) {
            copy_first(0);
            copy_second(0);
            if (steps > 1) {
                copy_first(1);
                wait_copies<8>();
            } else {
                wait_copies<0>();
            }
        }
        phase_barrier();
        if (wp == 1) phase_barrier();

        for (int k = 0; k < steps; ++k) {
            const char *const bp = L.p[k & 1], *const bq = L.q[k & 1];
            constexpr int NF = kDwMode ? 8 : 4;      // p fragments of a cluster
            u32x4 qf[2][4], pf[NF][2];
            float sc[4] = {0, 0, 0, 0};
            const float wsk = MODE == kFwdFp8 ? as_scalar(ws)[k] : 0.0f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bool work0 = nc > 2 * c, work1 = nc > 2 * c + 1;   // 32 rows each
                // indices of step k + 4, which land by the next step's first wait, and
                // the rows of step k + 3, for the copies of the next step's cluster 1
                if (kDwMode && w < 2) {
                    const RowsIn &in = w == 0 ? A.a : A.b;
                    if (c == 0 && k + 4 < steps) copy_indices(in, 64 * (k + 4), lo, cnt, L.raw[k & 3][w]);
                    if (c == 1 && k > 0 && k + 3 < steps)
                        rows_from_indices(in, 64 * (k + 3), lo, cnt, L.raw[(k + 3) & 3][w], L.rows[(k + 3) & 3][w]);
                }
                auto read = [&]() {
                    uint32_t qa[4], pa[4];
                    if (kQT && (kDwMode || c == 0))
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            qa[j] = frag_t_at<kDwMode, 512>(bq, wq, j, g, r);
                            if (kDwMode) pa[j] = frag_t_at<kDwMode, 512>(bp, 2 * wp, j, g, r);
                        }
                    if (kDwMode) {
                        u32x4 p0f[4], p1f[4];
                        if (c == 0) {
                            frags_t<512, 0>(qa, qf[0]);
                            frags_t2<512, 0, 128>(pa, p0f, p1f);
                        } else {
                            frags_t<512, 32 * 512>(qa, qf[0]);
                            frags_t2<512, 32 * 512, 32 * 512 + 128>(pa, p0f, p1f);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) pf[i][0] = p0f[i], pf[(4 + i) % NF][0] = p1f[i];
                    } else {
                        if (c == 0) {
                            if (kQT) {
                                frags_t2<512, 0, 32 * 512>(qa, qf[0], qf[1]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 4; ++j)
#pragma unroll
                                    for (int s = 0; s < 2; ++s)
                                        qf[s][j] = frag_n(bq, 64 * wq + 16 * j, s, g, r);
                            }
                        }
                        if (work0) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                pf[i][0] = frag_n(bp, 128 * wp + 64 * c + 16 * i, 0, g, r);
                                pf[i][1] = frag_n(bp, 128 * wp + 64 * c + 16 * i, 1, g, r);
                                if (MODE == kFwdFp8) sc[i] = L.xs[k & 3][128 * wp + 64 * c + 16 * i + r] * wsk;
                            }
                        }
                    }
                };
                // (the transposing reads wait where they stand: the copies go first)
                if (!kQT) read();
                if (c == 0) {
                    if (k + 1 < steps) {
                        copy_second(k + 1);
                        wait_copies<8>();
                    } else {
                        wait_copies<0>();
                    }
                } else {
                    if (k + 2 < steps) {
                        copy_first(k + 2);
                        wait_copies<8>();
                    } else if (k + 1 < steps) {
                        wait_copies<kDwMode ? 4 : 2>();
                    } else {
                        wait_copies<0>();
                    }
                }
                if (kQT) read();
                wait_lds();
                phase_barrier();
                __builtin_amdgcn_s_setprio(1);
                if (kDwMode) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                as_bf16x8(pf[i % NF][0]), as_bf16x8(qf[0][j]), acc[i][j], 0, 0, 0);
                } else {
                    auto multiply = [&](int i0) {     // p tiles i0, i0 + 1 of the cluster
                        if (MODE == kFwdFp8) {
                            f32x4 part[2][4];
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    part[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                        as_i32x8(qf[0][j], qf[1][j]),
                                        as_i32x8(pf[(i0 + i) % NF][0], pf[(i0 + i) % NF][1]),
                                        f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
#pragma unroll
                                    for (int v = 0; v < 4; ++v)
                                        acc[4 * c + i0 + i][j][v] = fmaf(
                                            part[i][j][v], sc[i0 + i], acc[4 * c + i0 + i][j][v]);
                        } else {
#pragma unroll
                            for (int s = 0; s < 2; ++s)
#pragma unroll
                                for (int i = i0; i < i0 + 2; ++i)
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        acc[4 * c + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                            as_bf16x8(q_is_row(MODE) ? qf[s][j] : pf[i % NF][s]),
                                            as_bf16x8(q_is_row(MODE) ? pf[i % NF][s] : qf[s][j]),
                                            acc[4 * c + i][j], 0, 0, 0);
                        }
                    };
                    if (work1) {
                        multiply(0);
                        multiply(2);
                    } else if (work0) {
                        multiply(0);
                    }
                }
                __builtin_amdgcn_s_setprio(0);
                phase_barrier();
            }
        }
        if (wp == 0) phase_barrier();

        const int le = fresh_lane();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= 2 * nc) continue;
            store_tile<MODE>(A, q0 + 64 * wq, Qn, le >> 4, le & 15, acc[i], [&](int p) -> long {
                if (!kDwMode) return L.dst[128 * wp + 16 * i + p];
                const int n = p0 + 128 * wp + 16 * i + p;
                return n < A.N ? (long)e * A.N + n : -1;
            });
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

int kernel_of(int mode) {
    return mode == kFwd ? K_PROD : mode == kFwdFp8 ? K_PROD_FP8 : mode == kDx ? K_PROD_DX : K_PROD_DW;
}

// Whether a product runs in tiles of 128 x 128 rather than 256 x 256: where the
// large ones would leave half of the compute units without one (gradients of
// 301 tokens over 8 experts: 26 against 45 us). With enough of them the large
// tiles win, also at 256 rows per expert (gradients of 4096 tokens: dx 197 against
// 204 us, dw 277 against 296 us).
static bool product_small(const ProductArgs &a, int mode) {
    const int Qn = mode == kFwd || mode == kFwdFp8 ? a.N : a.K;
    const long tq = (Qn + kBQ - 1) / kBQ;
    const long tiles = mode == kDw ? (long)a.E * ((a.N + kBP - 1) / kBP) * tq
                                   : (a.R / kBP + (a.R < a.E ? a.R : a.E)) * tq;
    return 2 * tiles <= compute_units();
}

// Parts that the call cuts c into when it has the workspace for their sums.
static int product_slices(const ProductArgs &a, int mode) {
    const bool forward = mode == kFwd || mode == kFwdFp8;
    if (a.R == 0 || (forward && product_streams(a)) || !product_small(a, mode)) return 1;
    return small_slices(a, mode);
}

static size_t part_bytes(const ProductArgs &a, int mode, int slices) {
    const bool forward = mode == kFwd || mode == kFwdFp8;
    return slices < 2 ? 0 : (size_t)slices * (mode == kDw ? (size_t)a.E * a.N : (size_t)a.R) *
                                (forward ? a.N : a.K) * sizeof(float);
}

template <int MODE>
static void launch_product(ProductArgs &a, void *ws, size_t ws_bytes, hipStream_t s) {
    const int cu = compute_units();
    a.slices = product_slices(a, MODE);
    a.part = (float *)ws;
    if (!ws || ws_bytes < part_bytes(a, MODE, a.slices)) a.slices = 1;
    if ((MODE == kFwd || MODE == kFwdFp8) && product_streams(a)) {
        launch_product_stream(a, MODE == kFwdFp8, s);
        return;
    }
    if (product_small(a, MODE)) {
        launch_product_small(a, MODE, s);
        return;
    }
    // one workgroup a compute unit (its LDS); fewer where there are fewer tiles
    const int Qn = MODE == kFwd || MODE == kFwdFp8 ? a.N : a.K;
    const long tq = (Qn + kBQ - 1) / kBQ;
    const long tiles = MODE == kDw ? (long)a.E * ((a.N + kBP - 1) / kBP) * tq
                                   : (a.R / kBP + (a.R < a.E ? a.R : a.E)) * tq;
    MOE_LAUNCH(kernel_of(MODE), product_kernel<MODE>, dim3((unsigned)(tiles < cu ? tiles : cu)),
               dim3(kPThreads), 0, s, a);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_gemm(const uint16_t *x_bf16, const int32_t *x_rows, int x_div, int x_n,
                                const int32_t *offsets, const uint16_t *w_bf16,
                                const moe_expert_w *experts, int mat, int R, int N, int K, int E,
                                void *y, const int32_t *y_rows, int y_n, int y_is_fp32,
                                void *ws, size_t ws_bytes, void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 8);
    if (rc != MOE_OK) return rc;
    if (mat != MOE_MAT_W13 && mat != MOE_MAT_W2) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if ((!w_bf16) == (!experts) || !aligned16(w_bf16) || !y || !aligned16(y) || !aligned16(ws))
        return MOE_EINVAL;
    if (!rows_ok(x_bf16, x_rows, x_div, x_n, R) || y_n < (y_rows ? 1 : R)) return MOE_EINVAL;
    ProductArgs a{};
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = rows_in(x_bf16, x_rows, x_div, x_n);
    a.m = Mats{(const char *)w_bf16, nullptr, experts, mat};
    a.out = y, a.out_rows = y_rows, a.out_n = y_n, a.out_f32 = y_is_fp32 != 0;
    launch_product<kFwd>(a, ws, ws_bytes, (hipStream_t)stream);
    return check_launch();
}

extern "C" int moe_grouped_gemm_fp8(const uint8_t *x_e4m3, const float *x_scale,
                                    const int32_t *x_rows, int x_div, int x_n,
                                    const int32_t *offsets, const uint8_t *w_e4m3,
                                    const float *w_scale, const moe_expert_w *experts, int mat,
                                    int R, int N, int K, int E, void *y, const int32_t *y_rows,
                                    int y_n, int y_is_fp32, void *ws, size_t ws_bytes,
                                    void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 16);
    if (rc != MOE_OK) return rc;
    if (mat != MOE_MAT_W13 && mat != MOE_MAT_W2) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if ((!w_e4m3) == (!experts) || (!w_e4m3) != (!w_scale) || !aligned16(w_e4m3) || !y || !aligned16(y) ||
        !aligned16(ws))
        return MOE_EINVAL;
    if (!x_scale || !rows_ok(x_e4m3, x_rows, x_div, x_n, R) || y_n < (y_rows ? 1 : R))
        return MOE_EINVAL;
    ProductArgs a{};
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = rows_in(x_e4m3, x_rows, x_div, x_n);
    a.a_s = x_scale;
    a.m = Mats{(const char *)w_e4m3, w_scale, experts, mat};
    a.out = y, a.out_rows = y_rows, a.out_n = y_n, a.out_f32 = y_is_fp32 != 0;
    launch_product<kFwdFp8>(a, ws, ws_bytes, (hipStream_t)stream);
    return check_launch();
}

extern "C" int moe_grouped_gemm_dx(const uint16_t *dy_bf16, const int32_t *dy_rows, int dy_div,
                                   int dy_n, const int32_t *offsets, const uint16_t *w_bf16,
                                   const moe_expert_w *experts, int mat, int R, int N, int K,
                                   int E, void *dx, const int32_t *dx_rows, int dx_n,
                                   int dx_is_fp32, void *ws, size_t ws_bytes, void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 8);
    if (rc != MOE_OK) return rc;
    if (mat != MOE_MAT_W13 && mat != MOE_MAT_W2) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if ((!w_bf16) == (!experts) || !aligned16(w_bf16) || !dx || !aligned16(dx) || !aligned16(ws))
        return MOE_EINVAL;
    if (!rows_ok(dy_bf16, dy_rows, dy_div, dy_n, R) || dx_n < (dx_rows ? 1 : R)) return MOE_EINVAL;
    ProductArgs a{};
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = rows_in(dy_bf16, dy_rows, dy_div, dy_n);
    a.m = Mats{(const char *)w_bf16, nullptr, experts, mat};
    a.out = dx, a.out_rows = dx_rows, a.out_n = dx_n, a.out_f32 = dx_is_fp32 != 0;
    launch_product<kDx>(a, ws, ws_bytes, (hipStream_t)stream);
    return check_launch();
}

extern "C" int moe_grouped_gemm_dw(const uint16_t *dy_bf16, const int32_t *dy_rows, int dy_div,
                                   int dy_n, const uint16_t *x_bf16, const int32_t *x_rows,
                                   int x_div, int x_n, const int32_t *offsets, int R, int N, int K,
                                   int E, void *dw, int dw_is_fp32, int accumulate, void *ws,
                                   size_t ws_bytes, void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 8);
    if (rc != MOE_OK) return rc;
    if (accumulate && !dw_is_fp32) return MOE_EINVAL;
    if (!dw || !aligned16(dw) || !aligned16(ws)) return MOE_EINVAL;
    if (R > 0 && (!rows_ok(dy_bf16, dy_rows, dy_div, dy_n, R) || !rows_ok(x_bf16, x_rows, x_div, x_n, R)))
        return MOE_EINVAL;
    ProductArgs a{};
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = rows_in(dy_bf16, dy_rows, dy_div, dy_n);
    a.b = rows_in(x_bf16, x_rows, x_div, x_n);
    a.out = dw, a.out_n = E * N, a.out_f32 = dw_is_fp32 != 0, a.accumulate = accumulate != 0;
    launch_product<kDw>(a, ws, ws_bytes, (hipStream_t)stream);
    return check_launch();
}

extern "C" int moe_grouped_gemm_workspace(int kind, int R, int N, int K, int E, size_t *bytes) {
    if (kind < kFwd || kind > MOE_GEMM_MXFP4 || !bytes) return MOE_EINVAL;
    const int unit = kind == MOE_GEMM_MXFP4 ? 128 : kind == kFwdFp8 ? 16 : 8;
    const int rc = check_sizes(R, N, K, E, E == 1 ? nullptr : (const int32_t *)16, unit);
    if (rc != MOE_OK) return rc;
    if (kind == MOE_GEMM_MXFP4) {
        if (N % 16) return MOE_EINVAL;
        *bytes = mxfp4_part_bytes(R, N, K, E);
        return MOE_OK;
    }
    ProductArgs a{};
    a.E = E, a.R = R, a.N = N, a.K = K;
    *bytes = part_bytes(a, kind, product_slices(a, kind));
    return MOE_OK;
}
