// The forward products (bf16, and FP8 with a scale per 128) where experts have
// a handful of rows each: then the cost is reading every touched expert's
// matrix once, and nothing is gained by staging it in LDS.
//
// A tile is 16 consecutive n of one expert over all of K, and one wavefront's:
// nothing of it is shared, so no barrier holds a wavefront up (four wavefronts
// that split K and met in LDS took TODO). Its weights go straight into LDS, 8 rows x
// 128 bytes a copy, so that neighbouring lanes read neighbouring bytes; loaded
// in the matrix core's order, four lanes of a row 16 apart, a load takes the
// address unit four times as long. The wavefront's ring has four stages of 4 lines (128 bytes of K) x 16
// rows, three in flight while one is multiplied: 96 KB a compute unit. The
// weights are the A operand; the B operand is up to 16 of the expert's rows
// of x, held in registers while the expert stays the same (K up to 32 lines:
// 256 registers, which the one wavefront of a SIMD has); longer or more
// rows are read from the caches with every stage, up to 64 rows to a reading
// of the weights. Wavefronts take consecutive tiles of the experts that have
// rows, whose list each workgroup makes from the offsets.
//
// FP8: as in products.hip, one 16x16x128 instruction per block of 128, started
// at zero, its four results per lane scaled by one number.
#include "products.hpp"

namespace moe {

constexpr int kSWaves = 4, kSThreads = kSWaves * kWave;
constexpr int kLines = 4;     // 128-byte lines of K in a stage
constexpr int kStages = 4;
constexpr int kBlocks = 4;    // blocks of 16 rows that share a read of the weights
constexpr int kHeld = 8;      // stages of a tile whose part of x fits in registers
constexpr int kMaxExperts = 512;

struct StreamLds {
    char ring[kSWaves][kStages][kLines * 2048];
    int list[kMaxExperts];            // experts with rows, ascending,
    int lo[kMaxExperts], cnt[kMaxExperts];   // and their rows
};

// A position in a wavefront's work: the tile (expert, first n), the first of
// up to 64 rows, the first line of K. e < 0: past the end.
struct Item {
    int tile, e, n0, lo, cnt, r0, c0;
};

struct Frags {
    u32x4 v[kLines][2];
    float sc[kLines];      // FP8: scales of this lane's row of x
};

template <bool FP8>
__global__ __launch_bounds__(kSThreads, 1) void product_stream_kernel(ProductArgs A) {
    constexpr int ES = FP8 ? 1 : 2, CK = 128 / ES;     // columns of a line
    __shared__ StreamLds L;
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int g = l >> 4, r = l & 15;

    // the experts with rows: every wavefront counts them all, the first writes
    int active = 0;
    {
        int lo[kMaxExperts / kWave], cnt[kMaxExperts / kWave];
#pragma unroll
        for (int i = 0; i < kMaxExperts / kWave; ++i) {
            cnt[i] = 0;
            if (i * kWave + l < A.E) group_of_lane(A, i * kWave + l, lo[i], cnt[i]);
        }
#pragma unroll
        for (int i = 0; i < kMaxExperts / kWave; ++i) {
            const uint64_t m = __ballot(cnt[i] > 0);
            if (w == 0 && cnt[i] > 0) {
                const int k = active + __popcll(m & lanemask_lt());
                L.list[k] = i * kWave + l, L.lo[k] = lo[i], L.cnt[k] = cnt[i];
            }
            active += __popcll(m);
        }
    }
    __syncthreads();

    const int nt = (A.N + 15) / 16, nl = (A.K + CK - 1) / CK, KB = (A.K + 127) / 128;
    const int full = A.K / CK;                          // lines without an end inside
    const size_t ld = (size_t)A.K * ES;
    const unsigned tiles = (unsigned)active * nt;       // at most 2^25
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
        i.r0 = i.c0 = 0;
        return i;
    };
    auto next = [&](Item &i) {
        i.c0 += kLines;
        if (i.c0 < nl) return;
        i.c0 = 0;
        i.r0 += 16 * kBlocks;
        if (i.r0 < i.cnt) return;
        i.r0 = 0;
        i.tile += 1;
        if (i.tile >= t1) {
            i.e = -1;
            return;
        }
        i.n0 += 16;
        if (i.n0 >= A.N) i = at(i.tile);
    };

    // copies of an item into stage st; returns how many certainly are in
    // flight. Rows past N read the last one and are not stored; what lies
    // past the end of K becomes zeros.
    const uint32_t o0 = (uint32_t)((l >> 3) * ld) + 16 * ((l & 7) ^ (l >> 3));
    auto copies = [&](const Item &i, int st) {
        if (i.e < 0) return 0;
        char *const to = L.ring[w][st];
        const char *const base = mat_of(A, i.e, ES) + (size_t)i.n0 * ld + (size_t)i.c0 * 128;
        if (i.c0 + kLines <= full && i.n0 + 16 <= A.N) {
#pragma unroll
            for (int j = 0; j < kLines; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    lds_dma16(scalar_base(base + j * 128 + (size_t)h * 8 * ld) + here(o0),
                              to + j * 2048 + h * 1024);
            return 2 * kLines;
        }
        const int fl = fresh_lane(), chunk = (fl & 7) ^ (fl >> 3);
#pragma unroll
        for (int j = 0; j < kLines; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 8 * h + (fl >> 3), rows = A.N - i.n0;
                if ((i.c0 + j) * CK + chunk * (16 / ES) < A.K)
                    lds_dma16(base + j * 128 + (size_t)(row < rows ? row : rows - 1) * ld + 16 * chunk,
                              to + j * 2048 + h * 1024);
                else
                    *(MOE_LDS u32x4 *)(to + j * 2048 + h * 1024 + 16 * fl) = u32x4{0, 0, 0, 0};
            }
        return 0;
    };

    const bool four = KB % 4 == 0 && ((uintptr_t)A.a_s & 15) == 0;   // scales by four
    // The part of row src of x that a stage from line c0 takes. Lanes without a
    // row (src < 0) load nothing: their columns of the product are not stored,
    // and every lane costs the address unit its time (16 lanes of one row
    // each: 3 us of a one-token call for K = 4096).
    auto load_x = [&](int src, int c0, Frags &x) {
        if (src < 0) return;
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
            if (four) {
                const f32x4 v = *(const MOE_GLOBAL f32x4 *)xs;
#pragma unroll
                for (int j = 0; j < kLines; ++j) x.sc[j] = v[j];
            } else {
#pragma unroll
                for (int j = 0; j < kLines; ++j) x.sc[j] = c0 + j < nl ? xs[j] : 0.0f;
            }
        }
    };
    // a stage's weights (with their scales) times a block of 16 rows
    struct Weights {
        u32x4 v[kLines][2];
        float sc[kLines];
    };
    auto stage = [&](const Item &i, int st, Weights &wv) {
        const char *const from = L.ring[w][st] + r * 128;
#pragma unroll
        for (int j = 0; j < kLines; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                wv.v[j][h] = *(const MOE_LDS u32x4 *)(from + j * 2048 + (((4 * h + g) ^ (r & 7)) << 4));
            wv.sc[j] = 0.0f;
            if (FP8 && i.c0 + j < nl)
                wv.sc[j] = as_scalar(scales_of(A, i.e) + (size_t)(i.n0 / 128) * KB)[i.c0 + j];
        }
    };
    auto multiply = [&](const Item &i, const Weights &wv, const Frags &x, f32x4 &sum) {
#pragma unroll
        for (int j = 0; j < kLines; ++j) {
            if (FP8) {
                if (i.c0 + j >= nl) continue;   // no scale there
                const float sc = x.sc[j] * wv.sc[j];
                const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    as_i32x8(wv.v[j][0], wv.v[j][1]), as_i32x8(x.v[j][0], x.v[j][1]),
                    f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[c] = fmaf(d[c], sc, sum[c]);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        as_bf16x8(wv.v[j][h]), as_bf16x8(x.v[j][h]), sum, 0, 0, 0);
            }
        }
    };
    // this lane's row (r of block b): its row of x and of out, or -1
    auto rows_of = [&](const Item &i, int b, int &src, int &dst) {
        const int row = i.r0 + 16 * b + r;
        src = dst = -1;
        if (row < i.cnt) {
            const int s = source_row(A.a, i.lo + row);
            const int d = A.out_rows ? A.out_rows[i.lo + row] : i.lo + row;
            if (s >= 0) src = s, dst = d >= 0 && d < A.out_n ? d : -1;
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

    // the ring: `ahead` is three items further than `i`
    Item i = at(t0), ahead = i;
    int n0 = 0, n1 = 0, n2 = 0, st = 0;     // copies in flight of the three items after i
    // The rows of x of the first expert come before the weights: loads wait in
    // order, so that looked up behind them they would wait for three stages.
    Frags x[kHeld];
    int xe = -1, xsrc, xdst;                // whose rows x holds
    auto held = [&](const Item &i) { return i.cnt <= 16 && nl <= kHeld * kLines; };
    auto hold = [&](const Item &i) {
        rows_of(i, 0, xsrc, xdst);
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (h * kLines < nl) load_x(xsrc, h * kLines, x[h]);
        xe = i.e;
    };
    if (held(i)) hold(i);
    copies(ahead, 0);
    next(ahead), n0 = copies(ahead, 1);
    if (ahead.e >= 0) next(ahead);
    n1 = copies(ahead, 2);
    if (ahead.e >= 0) next(ahead);
    n2 = copies(ahead, 3);
    auto arrive = [&]() {
        const int later = n0 + n1 + n2;
        if (later >= 24) wait_copies<24>();
        else if (later >= 16) wait_copies<16>();
        else if (later >= 8) wait_copies<8>();
        else wait_copies<0>();
        wait_lds();          // (zeros written past the end of K)
    };
    auto leave = [&]() {
        wait_lds();          // the stage is read: its next copies may land
        next(i);
        n0 = n1, n1 = n2;
        if (ahead.e >= 0) next(ahead);
        n2 = copies(ahead, st);
        st = (st + 1) & (kStages - 1);
    };
    while (i.e >= 0) {
        if (held(i)) {
            // tiles of one expert, its rows of x in registers
            if (i.e != xe) hold(i);
            while (i.e == xe) {
                f32x4 sum = {0, 0, 0, 0};
                const Item tile = i;
#pragma unroll
                for (int h = 0; h < kHeld; ++h)
                    if (h * kLines < nl) {
                        Weights wv;
                        arrive();
                        stage(i, st, wv);
                        multiply(i, wv, x[h], sum);
                        leave();
                    }
                store(tile, xdst, sum);
            }
        } else {
            const Item tile = i;
            const int nb = (i.cnt - i.r0 + 15) / 16;
            int src[kBlocks], dst[kBlocks];
            f32x4 sum[kBlocks];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                rows_of(i, b, src[b], dst[b]);
                sum[b] = f32x4{0, 0, 0, 0};
            }
            for (int c0 = 0; c0 < nl; c0 += kLines) {
                Weights wv;
                arrive();
                stage(i, st, wv);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
                    if (b < nb) {
                        Frags x;
                        load_x(src[b], c0, x);
                        multiply(i, wv, x, sum[b]);
                    }
                leave();
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                if (b < nb) store(tile, dst[b], sum[b]);
        }
    }
}

// Rows per expert on average up to which the products stream the weights.
bool product_streams(const ProductArgs &a) {
    return a.R <= 16L * a.E;
}

void launch_product_stream(const ProductArgs &a, bool fp8, hipStream_t s) {
    const long tiles = (long)(a.R < a.E ? a.R : a.E) * ((a.N + 15) / 16);
    const long most = compute_units();     // one workgroup a compute unit
    const dim3 grid((unsigned)(tiles < most ? tiles : most));
    if (fp8) MOE_LAUNCH(K_PROD_FP8, product_stream_kernel<true>, grid, dim3(kSThreads), 0, s, a);
    else MOE_LAUNCH(K_PROD, product_stream_kernel<false>, grid, dim3(kSThreads), 0, s, a);
}

}  // namespace moe
