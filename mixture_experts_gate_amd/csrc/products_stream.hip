// The forward products (bf16, and FP8 with a scale per 128) where experts have
// a handful of rows each: then the cost is reading every touched expert's
// matrix once, and nothing is gained by staging it in LDS.
//
// An entry is up to 16 rows of one expert (an expert with more has several, which
// read its matrix again). A tile is 16 consecutive n of an entry over all of K,
// and one wavefront's: nothing of it is shared, so no barrier holds a
// wavefront up (four wavefronts that split K and met in LDS took 544 against 437 us for
// 64 tokens of the FP8 layer: 2.5 GB of weights, 5.8 TB/s). Its weights go
// straight into LDS, 8 rows x 128 bytes a copy, into the wavefront's ring of four
// stages of 8 KB, three in flight while one is multiplied: 96 KB a compute unit.
// The weights are the A operand; the B operand, the entry's rows of x, is
//   HELD (K up to 32 lines of 128 bytes): in registers while the entry stays the
//     same (256 of them, which the one wavefront of a SIMD has);
//   else: copied along with the weights, half a stage each.
// Wavefronts take consecutive tiles of the entries, whose list each workgroup
// makes from the offsets.
//
// FP8: as in products.hip, one 16x16x128 instruction per block of 128, started
// at zero, its four results per lane scaled by one number.
#include "products.hpp"

namespace moe {

constexpr int kSWaves = 4, kSThreads = kSWaves * kWave;
constexpr int kStages = 4;
constexpr int kHeldLines = 32;    // lines of K (128 bytes) whose part of x fits in registers
constexpr int kEntryRows = 16;
constexpr int kStreamAvg = 16;    // rows per expert on average up to which this kernel runs
constexpr int kEntries = kMaxE + kMaxE * kStreamAvg / kEntryRows;

struct StreamLds {
    char ring[kSWaves][kStages][8192];
    float xs[kSWaves][kStages][kWave];          // FP8, not HELD: scales of the rows of x
    int list[kEntries], lo[kEntries], cnt[kEntries];   // entries: expert, first row, rows
};

// A position in a wavefront's work: the tile (entry, first n), the first line
// of K. e < 0: past the end.
struct Item {
    int tile, e, n0, lo, cnt, c0;
};

template <int LINES>
struct Frags {
    u32x4 v[LINES][2];
    float sc[LINES];       // FP8: scales of this lane's row of x
};

template <bool FP8, bool HELD>
__global__ __launch_bounds__(kSThreads, 1) void product_stream_kernel(ProductArgs A) {
    constexpr int ES = FP8 ? 1 : 2, CK = 128 / ES;     // columns of a line
    constexpr int kLines = HELD ? 4 : 2;                // lines of K in a stage
    constexpr int kHeld = kHeldLines / kLines;
    constexpr int kCopies = HELD || !FP8 ? 8 : 9;       // instructions of a stage's copies
    __shared__ StreamLds L;
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int g = l >> 4, r = l & 15;

    // the entries: every wavefront counts them all, the first writes them
    int entries = 0;
    {
        int lo[kMaxE / kWave], cnt[kMaxE / kWave];
#pragma unroll
        for (int i = 0; i < kMaxE / kWave; ++i) {
            cnt[i] = 0;
            if (i * kWave + l < A.E) group_of_lane(A, i * kWave + l, lo[i], cnt[i]);
        }
#pragma unroll
        for (int i = 0; i < kMaxE / kWave; ++i) {
            if (i * kWave >= A.E) break;
            const int n = (cnt[i] + kEntryRows - 1) / kEntryRows;
            int incl = n;
#pragma unroll
            for (int d = 1; d < kWave; d <<= 1) {
                const int o = __shfl_up(incl, d);
                if (l >= d) incl += o;
            }
            if (w == 0)
                for (int b = 0; b < n; ++b) {
                    const int k = entries + incl - n + b;
                    if (k >= kEntries) break;           // (cannot be: R <= 16 E)
                    L.list[k] = i * kWave + l, L.lo[k] = lo[i] + kEntryRows * b;
                    L.cnt[k] = cnt[i] - kEntryRows * b < kEntryRows ? cnt[i] - kEntryRows * b : kEntryRows;
                }
            entries += __builtin_amdgcn_readlane(incl, kWave - 1);
        }
        entries = entries < kEntries ? entries : kEntries;
    }
    __syncthreads();

    const int nt = (A.N + 15) / 16, nl = (A.K + CK - 1) / CK, KB = (A.K + 127) / 128;
    const int full = A.K / CK;                          // lines without an end inside
    const size_t ld = (size_t)A.K * ES;
    const unsigned tiles = (unsigned)entries * nt;      // at most 2^26
    // (consecutive shares to the wavefronts of a workgroup: they differ by a
    // tile, whole workgroups hardly)
    const unsigned me = blockIdx.x * kSWaves + w, all = kSWaves * gridDim.x;
    const unsigned each = tiles / all, more = tiles % all;
    const int t0 = me * each + me * more / all;
    const int t1 = (me + 1) * each + (me + 1) * more / all;
    if (t0 >= t1) return;

    auto at = [&](int tile) {
        Item i;
        const int ai = (unsigned)tile / (unsigned)nt;
        i.tile = tile;
        i.n0 = (tile - ai * nt) * 16;
        i.e = __builtin_amdgcn_readfirstlane(L.list[ai]);
        i.lo = __builtin_amdgcn_readfirstlane(L.lo[ai]);
        i.cnt = __builtin_amdgcn_readfirstlane(L.cnt[ai]);
        i.c0 = 0;
        return i;
    };
    auto next = [&](Item &i) {
        i.c0 += kLines;
        if (i.c0 < nl) return;
        i.c0 = 0;
        i.tile += 1;
        if (i.tile >= t1) {
            i.e = -1;
            return;
        }
        i.n0 += 16;
        if (i.n0 >= A.N) i = at(i.tile);
    };
    // row `row` of an entry: its row of x (one that exists) and of out (or -1)
    auto rows_of = [&](const Item &i, int row, int &src, int &dst) {
        src = 0, dst = -1;
        if (row < i.cnt) {
            const int s = source_row(A.a, i.lo + row);
            const int d = A.out_rows ? A.out_rows[i.lo + row] : i.lo + row;
            if (s >= 0) src = s, dst = d >= 0 && d < A.out_n ? d : -1;
        }
    };

    // Copies of an item into stage st, kCopies instructions; returns how many
    // certainly are in flight. Rows past N read the last one and are not
    // stored; what lies past the end of K becomes zeros.
    const uint32_t o0 = (uint32_t)((l >> 3) * ld) + 16 * ((l & 7) ^ (l >> 3));
    int xlo = -1;                       // not HELD: whose rows xsrc holds
    int xsrc[2] = {0, 0}, ssrc = 0;     // rows (l / 8) + 8 h of x; row l % 16
    auto copies = [&](const Item &i, int st) {
        if (i.e < 0) return 0;
        char *const to = L.ring[w][st];
        const char *const base = mat_of(A, i.e, ES) + (size_t)i.n0 * ld + (size_t)i.c0 * 128;
        if (HELD && i.c0 + kLines <= full && i.n0 + 16 <= A.N) {
#pragma unroll
            for (int j = 0; j < kLines; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    lds_dma16(scalar_base(base + j * 128 + (size_t)h * 8 * ld) + here(o0),
                              to + j * 2048 + h * 1024);
            return kCopies;
        }
        const int fl = fresh_lane(), chunk = (fl & 7) ^ (fl >> 3);
        if (!HELD && i.lo != xlo) {
            int d;
            rows_of(i, fl >> 3, xsrc[0], d);
            rows_of(i, 8 + (fl >> 3), xsrc[1], d);
            rows_of(i, fl & 15, ssrc, d);
            xlo = i.lo;
        }
#pragma unroll
        for (int j = 0; j < kLines; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 8 * h + (fl >> 3), rows = A.N - i.n0;
                const bool in = (i.c0 + j) * CK + chunk * (16 / ES) < A.K;
                copy_or_zeros(in, base + j * 128 + (size_t)(row < rows ? row : rows - 1) * ld + 16 * chunk,
                              to + j * 2048 + h * 1024);
                if (!HELD)
                    copy_or_zeros(in, A.a.base + (size_t)xsrc[h] * ld + (size_t)(i.c0 + j) * 128 + 16 * chunk,
                                  to + 4096 + j * 2048 + h * 1024);
            }
        if (!HELD && FP8) {
            const int line = i.c0 + (fl >> 4);        // lanes 0..31: line, row
            lds_dma4(A.a_s + (size_t)ssrc * KB + (line < nl ? line : nl - 1), L.xs[w][st]);
        }
        return kCopies;
    };

    const bool four = KB % 4 == 0 && ((uintptr_t)A.a_s & 15) == 0;   // scales by four
    // HELD: the part of row src of x that a stage from line c0 takes. Lanes without
    // a row load nothing: their columns of the product are not stored.
    auto load_x = [&](int src, int c0, Frags<kLines> &x) {
        const char *const xrow = A.a.base + (size_t)src * ld + 16 * g + (size_t)c0 * 128;
        if (c0 + kLines <= full) {
#pragma unroll
            for (int j = 0; j < kLines; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) x.v[j][h] = load16(xrow + j * 128 + 64 * h);
        } else {
#pragma unroll
            for (int j = 0; j < kLines; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool in = (c0 + j) * CK + (64 * h + 16 * g) / ES < A.K;
                    x.v[j][h] = u32x4{0, 0, 0, 0};
                    if (in) x.v[j][h] = load16(xrow + j * 128 + 64 * h);
                }
        }
        if (FP8) {
            const float *const xs = A.a_s + (size_t)src * KB + c0;
            if (HELD && four) {
                const f32x4 v = *(const MOE_GLOBAL f32x4 *)xs;
#pragma unroll
                for (int j = 0; j < kLines; ++j) x.sc[j] = v[j];
            } else {
#pragma unroll
                for (int j = 0; j < kLines; ++j) x.sc[j] = c0 + j < nl ? xs[j] : 0.0f;
            }
        }
    };
    // 16 rows x kLines lines in the matrix core's order
    auto frags = [&](const char *buf, u32x4 (&v)[kLines][2]) {
#pragma unroll
        for (int j = 0; j < kLines; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[j][h] = frag_n(buf + j * 2048, 0, h, g, r);
    };
    auto multiply = [&](const Item &i, const u32x4 (&wv)[kLines][2], const float (&wsc)[kLines],
                        const Frags<kLines> &x, f32x4 &sum) {
#pragma unroll
        for (int j = 0; j < kLines; ++j) {
            if (FP8) {
                if (i.c0 + j >= nl) continue;   // no scale there
                const float sc = x.sc[j] * wsc[j];
                const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    as_i32x8(wv[j][0], wv[j][1]), as_i32x8(x.v[j][0], x.v[j][1]),
                    f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[c] = fmaf(d[c], sc, sum[c]);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        as_bf16x8(wv[j][h]), as_bf16x8(x.v[j][h]), sum, 0, 0, 0);
            }
        }
    };
    // D: lane (g, r) has n 4g .. 4g+3 of row r
    auto store = [&](const Item &i, int dst, const f32x4 &v) {
        const int c = i.n0 + 4 * g;
        if (dst < 0 || c >= A.N) return;
        typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
        if (A.out_f32) *(MOE_GLOBAL f32x4 *)((float *)A.out + (size_t)dst * A.N + c) = v;
        else *(MOE_GLOBAL u32x2 *)((uint16_t *)A.out + (size_t)dst * A.N + c) =
                 u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };

    // The rows of the first entry come before the weights: loads wait in
    // order, so that looked up behind them they would wait for three stages.
    Item i = at(t0);
    Frags<kLines> x[HELD ? kHeld : 1];
    int elo = -1, src = 0, dst = -1;        // whose rows are at hand (by first row)
    auto hold = [&]() {
        rows_of(i, r, src, dst);
        if (HELD && r < i.cnt) {
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (h * kLines < nl) load_x(src, h * kLines, x[HELD ? h : 0]);
        }
        elo = i.lo;
    };
    hold();

    // the ring: `ahead` is three items further than `i`; n0 to n2: copies in
    // flight of the three items after i
    Item ahead = i;
    int n0 = 0, n1 = 0, n2 = 0, st = 0;
    copies(ahead, 0);
    next(ahead), n0 = copies(ahead, 1);
    if (ahead.e >= 0) next(ahead);
    n1 = copies(ahead, 2);
    if (ahead.e >= 0) next(ahead);
    n2 = copies(ahead, 3);
    // (n is 0 or kCopies, and 0 for good from some item on)
    auto arrive = [&]() {
        if (n2) wait_copies<3 * kCopies>();
        else if (n1) wait_copies<2 * kCopies>();
        else if (n0) wait_copies<kCopies>();
        else wait_copies<0>();
    };
    auto leave = [&]() {
        wait_lds();          // the stage is read: its next copies may land
        next(i);
        n0 = n1, n1 = n2;
        if (ahead.e >= 0) next(ahead);
        n2 = copies(ahead, st);
        st = (st + 1) & (kStages - 1);
    };
    auto stage = [&](u32x4 (&wv)[kLines][2], float (&wsc)[kLines]) {
        frags(L.ring[w][st], wv);
#pragma unroll
        for (int j = 0; j < kLines; ++j) {
            wsc[j] = 0.0f;
            if (FP8 && i.c0 + j < nl)
                wsc[j] = as_scalar(scales_of(A, i.e) + (size_t)(i.n0 / 128) * KB)[i.c0 + j];
        }
    };
    u32x4 wv[kLines][2];
    float wsc[kLines];
    while (i.e >= 0) {
        if (i.lo != elo) hold();
        f32x4 sum = {0, 0, 0, 0};
        const Item tile = i;
        if (HELD) {
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (h * kLines < nl) {
                    arrive();
                    stage(wv, wsc);
                    multiply(i, wv, wsc, x[HELD ? h : 0], sum);
                    leave();
                }
        } else {
            for (int c0 = 0; c0 < nl; c0 += kLines) {
                arrive();
                stage(wv, wsc);
                frags(L.ring[w][st] + 4096, x[0].v);
                if (FP8) {
#pragma unroll
                    for (int j = 0; j < kLines; ++j) x[0].sc[j] = L.xs[w][st][16 * j + r];
                }
                multiply(i, wv, wsc, x[0], sum);
                leave();
            }
        }
        store(tile, dst, sum);
    }
}

// Forward products run here up to 16 rows per expert on average. Both sides, us,
// this kernel / tiles, at 4, 8 and 16 rows per expert on average:
//                              even routing                   popularity e^N(0,1)
//   bf16, 128 x 1536 x 2048    143/153  149/154  156/155      131/147  150/147  204/159
//   FP8, 256 x 4096 x 4096     761/812  802/816  848/824      678/717  827/765 1185/830
//   FP8, 64 x 4096 x 7168      356/364  370/362  425/364      332/330  440/336  563/363
// and with all rows on one expert, whose matrix is read again for every 16 of them:
// bf16 28/46, 48/47, 84/47; FP8 (4096 x 4096) 132/64, 247/66, 476/78. Up to 4 rows per
// expert this kernel is the faster one or even unless one expert has nearly all
// rows; at 8 to 16 it loses as routing gets uneven, which the host does not know.
bool product_streams(const ProductArgs &a) {
    return a.R <= (long)kStreamAvg * a.E;
}

void launch_product_stream(const ProductArgs &a, bool fp8, hipStream_t s) {
    const long tiles = (a.R < a.E ? a.R : a.E + a.R / kEntryRows) * (long)((a.N + 15) / 16);
    const long most = compute_units();     // one workgroup a compute unit
    const dim3 grid((unsigned)(tiles < most ? tiles : most)), block(kSThreads);
    const bool held = (long)a.K * (fp8 ? 1 : 2) <= 128L * kHeldLines;
    if (fp8) {
        if (held) MOE_LAUNCH(K_PROD_FP8, (product_stream_kernel<true, true>), grid, block, 0, s, a);
        else MOE_LAUNCH(K_PROD_FP8, (product_stream_kernel<true, false>), grid, block, 0, s, a);
    } else {
        if (held) MOE_LAUNCH(K_PROD, (product_stream_kernel<false, true>), grid, block, 0, s, a);
        else MOE_LAUNCH(K_PROD, (product_stream_kernel<false, false>), grid, block, 0, s, a);
    }
}

}  // namespace moe
