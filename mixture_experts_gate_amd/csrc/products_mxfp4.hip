// The product grouped by expert from MXFP4: rows of x against matrices, both in
// E2M1 codes with a power of two per 32 columns, y[i] = W_e x[r(i)] (products.hip
// has the rows). The matrix core multiplies the scales in, one byte per lane and
// operand, so nothing is left for the vector units inside the sum.
//
// The matrices are in the kernel layout: blocks of 16 rows x 128 columns (a slab of
// K), 1024 bytes in which 16-byte piece 16 g + r holds row r, columns 32 g + 0..31,
// with 64 bytes of scales, byte 16 g + r.
#include "products.hpp"

namespace moe {

struct MxArgs {
    ProductArgs p;             // a: codes of x, m: codes of the matrices
    const uint8_t *xs, *ws;    // scales of x's rows, of the matrices (no table)
};

__device__ __forceinline__ const char *codes_of(const MxArgs &A, int e) {
    const ProductArgs &a = A.p;
    if (a.m.tab) return (const char *)(a.m.mat ? as_scalar(a.m.tab)[e].w2 : as_scalar(a.m.tab)[e].w13);
    return a.m.w + (size_t)e * a.N * (a.K / 2);
}

__device__ __forceinline__ const char *scales_of(const MxArgs &A, int e) {
    const ProductArgs &a = A.p;
    if (a.m.tab) return (const char *)(a.m.mat ? as_scalar(a.m.tab)[e].s2 : as_scalar(a.m.tab)[e].s13);
    return (const char *)A.ws + (size_t)e * a.N * (a.K / 32);
}

template <int V>
struct Const {
    static constexpr int v = V;
};

// Bytes OA and OB of the scale registers scale this lane's 32 codes of a and b.
template <int OA, int OB>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
    const u32x4 z = {0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(as_i32x8(a, z), as_i32x8(b, z), c, 4, 4, OA, (int)sa,
                                                           OB, (int)sb);
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    const u32x4 z = {0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(as_i32x8(a, z), as_i32x8(b, z), c, 4, 4, 0, (int)sa,
                                                            0, (int)sb);
}

// ------------------------------------------------------------------ tiles --
// 128 rows (p) x 256 n (q) a workgroup of eight wavefronts, 32 x 128 each; two
// workgroups a compute unit, so that one multiplies while the other starts or ends a
// tile. A step is a slab; LDS holds three, two of them copied ahead. (With four
// wavefronts of 64 x 128, whose reads of LDS are three fifths of these, nothing runs beside
// a wavefront's reads where a workgroup is alone on its compute unit: 1024 rows of one
// expert of 4096 x 4096 take 30.6 us, 27.0 here, 500 of 1536 x 2048 18.3 and 16.5; more
// slabs in LDS change nothing.)
//
// The middle sizes run here: 64 tokens of 128 experts of 1536 x 2048 45.5 us (about 210
// MB of W, 4.6 TB/s: HBM and the tiles' starts, of few slabs each), 512 rows of one of
// 4096 x 4096 27 us (start, the sum in parts, and their join).
//
// Instruction 32x32x64 with x as A and W as B (16x16x128 has the same rate but
// reads each operand twice as often): a lane (h, b) = (l / 32, l % 32) of result
// register v has row 8 (v / 4) + 4 h + v % 4 and column b. Column b of tile j is q =
// 4 b + j of the wavefront's 128, so that a lane holds four consecutive q of a row
// and 32 lanes store 256 bytes of it. The same order puts the scales of the
// four tiles into the four bytes of one register, which the instruction picks from.
constexpr int kXThreads = 512;
constexpr int kXP = 128, kXQ = 256;
constexpr int kXS = 3;           // slabs in LDS
constexpr int kXCopies = 4;      // copy instructions of a wavefront and slab

// 32 rows of a wavefront's results, four columns from q, to the rows of out in `dst`.
// (The results are pinned to their registers first: the compiler would keep them in the
// order of the stores throughout the sum, and spill 160 registers.)
__device__ __forceinline__ void store_rows(const ProductArgs &A, char *out, bool f32, const int *dst, int q, int h,
                                           f32x16 (&acc)[4]) {
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(acc[j]));
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int to = dst[8 * (v >> 2) + 4 * h + (v & 3)];
        if (to < 0 || q >= A.N) continue;
        const f32x4 y = {acc[0][v], acc[1][v], acc[2][v], acc[3][v]};
        const size_t at = (size_t)to * A.N + q;
        if (f32) *(MOE_GLOBAL f32x4 *)((float *)out + at) = y;
        else *(MOE_GLOBAL u32x2 *)((uint16_t *)out + at) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
    }
}

struct TileLds {
    char p[kXS][kXP * 64];       // rows of 64 bytes, 16-byte pieces XORed with row / 4
    char q[kXS][kXQ * 64];       // blocks as in memory, piece 16 g + r at 16 g + (r ^ block % 4)
    uint32_t xs[kXS][kXP];       // a row's four scales
    char qs[kXS][kXQ * 4];       // blocks' scales as in memory
    int src[kXP], dst[kXP];      // rows of x and of out (-1: none) of the rows in LDS
    int base[kMaxE + 1];         // p tiles before each expert
    int wsum[kXThreads / kWave];
};

__global__ __launch_bounds__(kXThreads, 4) void mxfp4_tile_kernel(MxArgs X) {
    const ProductArgs &A = X.p;
    __shared__ TileLds L;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l = lane_id(), t = threadIdx.x, h = l >> 5, b = l & 31;
    const int wq = w & 1, wp = w >> 1;

    const int tq = (A.N + kXQ - 1) / kXQ, slabs = A.K / 128, blocks = A.N / 16;
    const size_t ldx = (size_t)A.K / 2, lds = (size_t)A.K / 32;
    total_tiles<kXThreads>(A, kXP, L.base, L.wsum);
    const int ns = A.slices, total = L.base[A.E] * tq * ns;
    // workgroup b runs on XCD b % 8 (shifts: with divisions of 64 bits a
    // workgroup starts 1% of a small call later)
    const int lx = gridDim.x >= 8 ? 3 : 0;
    const int xcd = blockIdx.x & ((1 << lx) - 1), per = ((int)gridDim.x - xcd + (1 << lx) - 1) >> lx;
    const int t0 = (int)((long)total * xcd >> lx), t1 = (int)((long)total * (xcd + 1) >> lx);
    for (int si = t0 + ((int)blockIdx.x >> lx); si < t1; si += per) {
        const int ti = ns > 1 ? si / ns : si, slice = si - ti * ns;     // tile, part of its sum
        const int e = expert_of(L.base, A.E, tq, ti);
        const int mp = __builtin_amdgcn_readfirstlane(L.base[e + 1] - L.base[e]);
        const int li = ti - __builtin_amdgcn_readfirstlane(L.base[e]) * tq;
        int p0, q0, lo, cnt;
        group_of(A, e, lo, cnt);
        // the expert's rows are spread evenly over its tiles, in units of 32 (more
        // than four of them only where offsets do not ascend)
        int units = (int)((cnt + 32u * mp - 1) / (32u * mp));
        units = units < 4 ? units : 4;
        place_of(li, mp, tq, p0, q0);
        p0 *= 32 * units, q0 *= kXQ;
        const int kb = slabs * slice / ns, ke = slabs * (slice + 1) / ns;      // (2^13 slabs at most, 16 parts)

        __syncthreads();   // the last tile's readers of L are done
        if (t < kXP) {
            const int u = t >> 5, p = p0 + t;      // (unit u is wavefront row u's)
            const bool in = u < units && p < cnt;
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
        __syncthreads();

        // A wavefront copies 16 rows of x and two blocks of W; blocks past the last one
        // read it and are not stored.
        const char *const pp =
            A.a.base + (size_t)L.src[16 * w + (l >> 2)] * ldx + 16 * ((l & 3) ^ ((l >> 4) & 3));
        const char *const codes = codes_of(X, e), *const scales = scales_of(X, e), *qb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rb = q0 / 16 + 2 * w + i;
            qb[i] = codes + (size_t)(rb < blocks ? rb : blocks - 1) * slabs * 1024;
        }
        const int sb = q0 / 16 + 4 * (w & 3) + (l >> 4);
        const char *const qsp = scales + (size_t)(sb < blocks ? sb : blocks - 1) * slabs * 64 + 4 * (l & 15);
        const char *const xsp = (const char *)X.xs + (size_t)L.src[64 * (w & 1) + l] * lds;
        auto fetch = [&](int k, int st) {
            lds_dma16(pp + (size_t)k * 64, L.p[st] + 16 * w * 64);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                lds_dma16(scalar_base(qb[i] + (size_t)k * 1024) + here(16 * (l ^ ((2 * w + i) & 3))),
                          L.q[st] + (2 * w + i) * 1024);
            // (a row's scales by two wavefronts, so that all count alike)
            if (w < 4) lds_dma4(qsp + (size_t)k * 64, L.qs[st] + 256 * w);
            else lds_dma4(xsp + (size_t)k * 4, &L.xs[st][64 * (w & 1)]);
        };

        f32x16 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[j][v] = 0.0f;
        if (kb < ke) fetch(kb, 0);
        if (kb + 1 < ke) fetch(kb + 1, 1);
        int st = 0;
        const bool work = wp < units;
        for (int k = kb; k < ke; ++k) {
            // slab k is in LDS (the copies of the next one may be in flight), and slab
            // k - 1, whose place slab k + 2 takes, is read
            if (k + 1 < ke) wait_copies<kXCopies>();
            else wait_copies<0>();
            wait_lds();
            bare_barrier();
            if (k + 2 < ke) fetch(k + 2, st == 0 ? 2 : st - 1);
            if (work) {
                const char *const P = L.p[st] + (32 * wp + b) * 64, *const Q = L.q[st] + (8 * wq + (b >> 2)) * 1024;
                const char *const S = L.qs[st] + (8 * wq + (b >> 2)) * 64 + 16 * h + 4 * (b & 3);
                const int key = (b >> 2) & 3;
                u32x4 pf[2], qf[2][4];
                uint32_t qs[2];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    qs[kk] = *(const MOE_LDS uint32_t *)(S + 32 * kk);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        qf[kk][j] = *(const MOE_LDS u32x4 *)(Q + 16 * (32 * kk + 16 * h + 4 * (b & 3) + (j ^ key)));
                    pf[kk] = *(const MOE_LDS u32x4 *)(P + 16 * ((2 * kk + h) ^ key));
                }
                const uint32_t ps = L.xs[st][32 * wp + b] >> (8 * h);
#define MOE_MX(kk, j) acc[j] = mfma32<2 * kk, j>(pf[kk], qf[kk][j], acc[j], ps, qs[kk]);
                MOE_MX(0, 0) MOE_MX(0, 1) MOE_MX(0, 2) MOE_MX(0, 3)
                MOE_MX(1, 0) MOE_MX(1, 1) MOE_MX(1, 2) MOE_MX(1, 3)
#undef MOE_MX
            }
            st = st == 2 ? 0 : st + 1;
        }

        char *const out = ns > 1 ? (char *)(A.part + (size_t)slice * A.R * A.N) : (char *)A.out;
        if (work) store_rows(A, out, ns > 1 || A.out_f32, L.dst + 32 * wp, q0 + 128 * wq + 4 * b, h, acc);
    }
}

// ------------------------------------------------------------ large tiles --
// 256 x 256 a workgroup of eight wavefronts, 64 x 128 each as above, one workgroup a
// compute unit: two thirds of the bytes that tiles of 128 x 256 copy into LDS. The
// wavefronts of a SIMD (w and w + 4) run one phase apart: one reads a slab's fragments
// while the other multiplies, its copies between the matrix instructions; a barrier
// ends each phase. (Four wavefronts of 128 x 128 read a third less from LDS, but one
// that reads, waits or stores leaves its SIMD idle: 8192 rows of 8192 x 8192 take
// 284 us, 257 here.)
//
// What bounds it: power. Matrix instructions alone reach 6.5 PFLOP/s on random codes
// (the limit lowers the clock; on zeros 9.6). One expert of 8192 x 8192 reaches 4.3 at
// 1.6 of 2.4 GHz, the matrix cores 64% busy; one of 4096 x 4096 (4001 rows) 3.2 at 1.5
// GHz, where a fifth of the cycles pass before a workgroup's first slab is there
// (12 thousand of 62: offsets, indices and rows one after another); gate/up of 8192
// tokens of 128 experts (1536 x 2048, 412 GFLOP, 201 MB of results) 2.6 at 1.8 GHz,
// where 40 of 160 us go by while the compute units store together. A slab takes 1500
// cycles of which 1024 multiply: a phase's 512 take about 700 with the copies between
// them, its barriers 120. (LDS is busy for 490 of them: 96 KB of fragments, which it
// gives out at 240 bytes a cycle, and their conflicts.)
//
// LDS holds four slabs, two pairs. The copies run three slabs ahead, and on into the
// next tile, whose rows are looked up during this one's first slabs: only a workgroup's
// first tile waits for its first slab. Scales come a pair at a time (8 bytes a row,
// 128 a block). What a phase may take, the other wavefront's 512 cycles of matrix
// instructions, is about a hundred instructions: hence pairs, whose places in LDS are
// constants, 32-bit offsets from uniform addresses for copies and stores, and no branch
// a row in the stores (rows of none lie outside the buffer's range).
constexpr int kBThreads = 512;
constexpr int kBT = 256;         // rows and n of a tile
constexpr int kBSlabs = 6;       // slabs of K from which this kernel runs, an even number:
                                 // a tile's copies begin three before the end of the last
                                 // tile, which by then has looked up its rows
constexpr uint32_t kBBytes = 0x7FFFFFF0u;    // bytes of out at most; offsets from here on are not stored
constexpr int kBPair = 32768;    // bytes of a pair of slabs of p or q

// Rows p0 on of expert e, whose cnt rows begin at lo, `units` times 32 of them; n from q0.
struct LargeTile {
    int e, lo, cnt, p0, q0, units;
};
constexpr int kBList = 64;       // tiles looked up at a time, one a lane (one after the other
                                 // they took a microsecond each, of ten)

struct LargeLds {
    char p[2][kBPair], q[2][kBPair];             // slabs as in TileLds, 256 rows each
    uint32_t xs[2][kBT][2];                      // rows' scales, of a pair
    char qs[2][8][288];                          // two blocks' scales, of a pair (32 bytes on
                                                 // for every two: 8 blocks in different banks)
    int raw[kBT], rawo[kBT];                     // the next tile's indices into x and out,
    int src[kBT];                                // its rows of x,
    uint32_t to[2][kBT];                         // and the offsets of its rows in out, by tile
    LargeTile list[kBList];                      // the workgroup's next tiles
    int base[kMaxE + 1];                         // p tiles before each expert
    int wsum[kBThreads / kWave];
};

template <int N>
__device__ __forceinline__ void wait_some(int more) {      // until N + more are in flight, more 0, 16 or 32
    if (more == 0) wait_copies<N>();
    else if (more == 16) wait_copies<N + 16>();
    else wait_copies<N + 32>();
}

__global__ __launch_bounds__(kBThreads) void mxfp4_large_kernel(MxArgs X) {
    const ProductArgs &A = X.p;
    __shared__ LargeLds L;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l = lane_id(), h = l >> 5, b = l & 31;
    const int wq = w & 1, wp = w >> 1;
    const int tq = (A.N + kBT - 1) / kBT, slabs = A.K / 128, blocks = A.N / 16;
    total_tiles<kBThreads>(A, kBT, L.base, L.wsum);
    const int total = L.base[A.E] * tq;
    const int lx = gridDim.x >= 8 ? 3 : 0;      // workgroup b runs on XCD b % 8
    const int xcd = blockIdx.x & ((1 << lx) - 1), per = ((int)gridDim.x - xcd + (1 << lx) - 1) >> lx;
    const int t0 = (int)((long)total * xcd >> lx), t1 = (int)((long)total * (xcd + 1) >> lx);
    int si = t0 + ((int)blockIdx.x >> lx);
    if (si >= t1) return;

    // The workgroups that have a tile less than others start later, by up to half of
    // one's time (12 sleeps of 64 cycles a slab, which takes 1500): begun together, all
    // tiles end together, and each end's stores, 32 MB from the device, wait for HBM with
    // nothing to multiply (gate/up of 8192 tokens: 185 -> 171 us).
    const int rank = blockIdx.x >> lx, late = (t1 - t0) % per;
    if (late > 0 && rank >= late)
        for (int i = slabs * 12 * (rank - late) / (per - late); i > 0; --i) __builtin_amdgcn_s_sleep(1);

    using Tile = LargeTile;
    // the workgroup's tiles n, n + 1, ..., by one wavefront
    auto look_up = [&](int n) {
        const long ti = si + (long)(n + l) * per;
        if (ti >= t1) return;
        Tile t;
        int e = 0, end = A.E;
        while (end - e > 1) {
            const int mid = (e + end) >> 1;
            if ((long)L.base[mid] * tq <= ti) e = mid;
            else end = mid;
        }
        const int mp = L.base[e + 1] - L.base[e], li = (int)(ti - (long)L.base[e] * tq);
        t.e = e;
        group_of_lane(A, e, t.lo, t.cnt);
        // rows spread evenly over the expert's tiles, in units of 32 (more than
        // eight only where offsets do not ascend)
        const int units = (int)((t.cnt + 32u * mp - 1) / (32u * mp));
        t.units = units < 8 ? units : 8;
        place_of(li, mp, tq, t.p0, t.q0);
        t.p0 *= 32 * t.units, t.q0 *= kBT;
        L.list[l] = t;
    };
    auto listed = [&](int n) {
        const Tile t = L.list[n % kBList];
        return Tile{__builtin_amdgcn_readfirstlane(t.e),  __builtin_amdgcn_readfirstlane(t.lo),
                    __builtin_amdgcn_readfirstlane(t.cnt), __builtin_amdgcn_readfirstlane(t.p0),
                    __builtin_amdgcn_readfirstlane(t.q0), __builtin_amdgcn_readfirstlane(t.units)};
    };
    // row `row` of LDS: unit u is rows 32 (u / 4) of wavefront row u % 4; -1: past the end
    auto place = [&](const Tile &t, int row) {
        const int u = 4 * ((row >> 5) & 1) + (row >> 6), p = t.p0 + 32 * u + (row & 31);
        return u < t.units && p < t.cnt ? p : -1;
    };
    const uint32_t ldo = (uint32_t)A.N * (A.out_f32 ? 4 : 2);
    auto out_at = [&](const Tile &t, int row, int raw, int rawo) {
        const int p = place(t, row);
        if (p < 0 || (A.a.idx && row_of_index(A.a, raw) < 0)) return kBufOff;
        const int d = A.out_rows ? rawo : t.lo + p;
        return d >= 0 && d < A.out_n ? (uint32_t)d * ldo : kBufOff;
    };
    auto index_at = [&](const Tile &t, int row) {
        const int p = place(t, row);
        return t.lo + (p < 0 ? 0 : p);      // (a row past the end reads the expert's first one)
    };

    if (w == 0) look_up(0);
    __syncthreads();
    const int tiles = (t1 - si + per - 1) / per;
    int n = 0;                           // this tile's number
    Tile cur = listed(0), next = cur;
    // row `row` of a tile from its indices: row of x, offset in out
    auto note_row = [&](const Tile &t, int to, int row, int raw, int rawo) {
        const int r = A.a.idx ? row_of_index(A.a, raw) : index_at(t, row);
        L.src[row] = r < 0 ? 0 : r;
        L.to[to][row] = out_at(t, row, raw, rawo);
    };
    if (threadIdx.x < kBT) {
        const int i = index_at(cur, threadIdx.x);
        note_row(cur, 0, threadIdx.x, A.a.idx ? A.a.idx[i] : 0, A.out_rows ? A.out_rows[i] : 0);
    }
    __syncthreads();

    // Copies: a wavefront takes 32 rows of x, 16 an instruction, and two blocks of W.
    // The lane's offsets into x, its scales and W's, and where the next slab's are.
    uint32_t po[2], xo, so;
    const char *pn, *qn[2], *xn, *sn;
    int ck = 0;                                      // that slab
    auto enter = [&](const Tile &t) {
        const int rb = t.q0 / 16 + 2 * w;
        const char *const codes = codes_of(X, t.e);
        pn = A.a.base, xn = (const char *)X.xs, sn = scales_of(X, t.e);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            po[i] = (uint32_t)L.src[32 * w + 16 * i + (l >> 2)] * (uint32_t)(A.K / 2) + 16 * ((l & 3) ^ ((l >> 4) & 3));
            qn[i] = codes + (size_t)(rb + i < blocks ? rb + i : blocks - 1) * slabs * 1024;
        }
        xo = (uint32_t)L.src[32 * w + (l >> 1)] * (uint32_t)(A.K / 32) + 4 * (l & 1);
        so = (uint32_t)((rb + h < blocks ? rb + h : blocks - 1) * slabs) * 64 + 4 * b;
        ck = 0;
    };
    const uint32_t qo[2] = {16u * (l ^ ((2 * w) & 3)), 16u * (l ^ ((2 * w + 1) & 3))};
    char *const pl = L.p[0] + 32 * w * 64, *const ql = L.q[0] + 2 * w * 1024;
    auto copy_some = [&](int place, auto n) {        // copy n of 4 of that slab
        constexpr int i = decltype(n)::v;
        if constexpr (i == 0) lds_dma16(scalar_base(pn) + here(po[0]), pl + place);
        if constexpr (i == 1) lds_dma16(scalar_base(pn) + here(po[1]), pl + place + 1024);
        if constexpr (i == 2) lds_dma16(scalar_base(qn[0]) + here(qo[0]), ql + place);
        if constexpr (i == 3) {
            lds_dma16(scalar_base(qn[1]) + here(qo[1]), ql + place + 1024);
            pn += 64, qn[0] += 1024, qn[1] += 1024, ++ck;
        }
    };
    auto copy_slab = [&](int place) {
        copy_some(place, Const<0>{}), copy_some(place, Const<1>{}), copy_some(place, Const<2>{}), copy_some(place, Const<3>{});
    };
    auto copy_scales = [&](int u) {                  // 2 copies
        lds_dma4(scalar_base(xn) + here(xo), &L.xs[u][32 * w][0]);
        lds_dma4(scalar_base(sn) + here(so), L.qs[u][w]);
        xn += 8, sn += 128;
    };

    // this lane's places in LDS: x's two pieces of a slab, W's of tile j, and the scales
    const int key = (b >> 2) & 3;
    const char *P[2], *Q[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) P[i] = L.p[0] + (64 * wp + b) * 64 + 16 * ((2 * i + h) ^ key);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        Q[j] = L.q[0] + (8 * wq + (b >> 2)) * 1024 + 16 * (16 * h + 4 * (b & 3) + (j ^ key));
    const char *const S = L.qs[0][4 * wq + (b >> 3)] + 128 * ((b >> 2) & 1) + 16 * h + 4 * (b & 3);
    const char *const XS = (const char *)L.xs[0][64 * wp + b];

    struct Frags {
        u32x4 p[2][2], q[2][4];
    };
    struct Scales {
        uint32_t p[2][2], q[2][2];       // by slab of the pair
    };
    f32x16 acc[2][4];
    enter(cur);
    copy_scales(0), copy_slab(0), copy_slab(kBPair / 2);
    copy_scales(1), copy_slab(kBPair);
    wait_copies<10>();
    bare_barrier();
    if (wp >= 2) bare_barrier();

    int u = 0, db = 0, stores = 0;       // pair in LDS, tile's place in `to`, stores before this tile
    bool work0, work1;
    auto read = [&](Frags &f, int o) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f.q[kk][j] = *(const MOE_LDS u32x4 *)(Q[j] + o + 512 * kk);
            f.p[0][kk] = *(const MOE_LDS u32x4 *)(P[kk] + o);
            f.p[1][kk] = *(const MOE_LDS u32x4 *)(P[kk] + o + 2048);
        }
    };
    auto multiply = [&](const Frags &f, const Scales &c, auto slab, auto copy) {
        constexpr int s = decltype(slab)::v;
        auto between = [&](auto n) {
            __builtin_amdgcn_sched_barrier(0);
            copy(n);
            __builtin_amdgcn_sched_barrier(0);
        };
        wait_lds();
        phase_barrier();
        __builtin_amdgcn_s_setprio(1);
#define MOE_MX(i, kk, j) acc[i][j] = mfma32<2 * kk, j>(f.p[i][kk], f.q[kk][j], acc[i][j], c.p[s][i], c.q[s][kk]);
#define MOE_MX2(i, kk, j) MOE_MX(i, kk, j) MOE_MX(i, kk, j + 1)
        if (work0) {
            MOE_MX2(0, 0, 0)
            between(Const<0>{});
            MOE_MX2(0, 0, 2)
            between(Const<1>{});
            MOE_MX2(0, 1, 0)
            between(Const<2>{});
            MOE_MX2(0, 1, 2)
            between(Const<3>{});
        } else {
            copy(Const<0>{}), copy(Const<1>{}), copy(Const<2>{}), copy(Const<3>{});
        }
        if (work1) {
            MOE_MX2(1, 0, 0) MOE_MX2(1, 0, 2) MOE_MX2(1, 1, 0) MOE_MX2(1, 1, 2)
        }
#undef MOE_MX2
#undef MOE_MX
        __builtin_amdgcn_s_setprio(0);
        phase_barrier();
    };
    auto pair = [&](int k) {
        typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
        // the pair's first slab, and its scales
        Frags f0, f1;
        Scales c;
        read(f0, u * kBPair);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
                c.q[s][kk] = *(const MOE_LDS uint32_t *)(S + u * (int)sizeof(L.qs[0]) + 64 * s + 32 * kk);
        const u32x2 x0 = *(const MOE_LDS u32x2 *)(XS + u * (int)sizeof(L.xs[0]));
        const u32x2 x1 = *(const MOE_LDS u32x2 *)(XS + u * (int)sizeof(L.xs[0]) + 256);
#pragma unroll
        for (int s = 0; s < 2; ++s) c.p[s][0] = x0[s] >> (8 * h), c.p[s][1] = x1[s] >> (8 * h);
        // Slab k + 1 has to be there: of what is in flight, the copies of slab k + 2 with
        // its scales (6) and the last tile's stores are younger. Slab k + 3 goes into the
        // place that slab k - 1, read by all, had.
        wait_some<6>(k == 0 ? stores : 0);
        const int p3 = (u ^ 1) * kBPair + kBPair / 2, p4 = u * kBPair;
        multiply(f0, c, Const<0>{}, [&](auto n) { copy_some(p3, n); });

        // its second slab
        read(f1, u * kBPair + kBPair / 2);
        if (k == 0 && n + 1 < tiles) {
            // the next tile, and the indices of its rows
            next = listed(n + 1);
            const int i = index_at(next, 64 * (w & 3) + l);
            if (w < 4 ? A.a.idx != nullptr : A.out_rows != nullptr)
                lds_dma4((w < 4 ? A.a.idx : A.out_rows) + i, (w < 4 ? L.raw : L.rawo) + 64 * (w & 3));
        }
        if (k == 2 && n + 1 < tiles) {
            const int row = 32 * w + b;      // (this wavefront's copies read these alone)
            note_row(next, db ^ 1, row, L.raw[row], L.rawo[row]);
        }
        if (ck == slabs) {
            // on to the next tile; behind the last one, its last pair once more
            if (n + 1 < tiles) enter(next);
            else pn -= 128, qn[0] -= 2048, qn[1] -= 2048, xn -= 8, sn -= 128, ck -= 2;
        }
        wait_some<4>(k == 0 ? stores : 0);
        multiply(f1, c, Const<1>{}, [&](auto n) {
            if constexpr (decltype(n)::v == 0) copy_scales(u);
            copy_some(p4, n);
        });
        u ^= 1;
    };
    for (;;) {
        work0 = wp < cur.units, work1 = 4 + wp < cur.units;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        for (int k = 0; k < slabs; k += 2) pair(k);
        // A lane stores four columns of 16 rows of each unit.
        const int q = cur.q0 + 128 * wq + 4 * b, bytes = A.out_f32 ? 4 : 2;
        const uint32_t col = q < A.N ? (uint32_t)(q * bytes) : kBBytes;
        const buf_rsrc out = make_rsrc(A.out, (uint32_t)A.out_n * ldo);
        stores = (work0 ? 16 : 0) + (work1 ? 16 : 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (4 * i + wp >= cur.units) continue;
            typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(acc[i][j]));
            u32x4 at[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) at[c] = *(const MOE_LDS u32x4 *)&L.to[db][64 * wp + 32 * i + 8 * c + 4 * h];
            if (A.out_f32) {
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const f32x4 y = {acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), out, at[v >> 2][v & 3] + col, 0, kBufNt);
                }
            } else {
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    __builtin_amdgcn_raw_buffer_store_b64(
                        u32x2{pack_bf16x2(acc[i][0][v], acc[i][1][v]), pack_bf16x2(acc[i][2][v], acc[i][3][v])}, out,
                        at[v >> 2][v & 3] + col, 0, kBufNt);
            }
        }
        if (n + 1 >= tiles) break;
        db ^= 1, ++n, cur = next;
        // (all have read the list's last tile; two barriers come before the next is read)
        if ((n + 1) % kBList == 0 && w == 0) look_up(n + 1);
    }
    wait_copies<0>();       // (copies that nothing reads: LDS is another workgroup's next)
    if (wp < 2) bare_barrier();
}

// -------------------------------------------------------- a handful of rows --
// An entry is up to 16 rows of one expert; a tile is one block row of W (16 n) of an
// entry over all of K, and one wavefront's. Its codes are in the order that the
// matrix core takes them in: they go from memory straight into registers, a
// kilobyte a load, and so do x's, whose rows the caches hold. Chunks of four slabs,
// the next one (of the next tile too) always in flight; 16 wavefronts a compute unit.
// No LDS and no barrier: each wavefront finds its entries by itself, from the
// offsets in its registers. One token of 128 experts of 1536 x 2048 (8 of them, 13.4 MB)
// takes 7.3 us, of which 13.4 MB at HBM's rate are 2: the offsets, the indices and the
// first codes come one after another.
constexpr int kVThreads = 256, kVWaves = kVThreads / kWave;
constexpr int kVRows = 16;       // rows of an entry
constexpr int kVAvg = 16;        // rows per expert on average up to which this kernel runs
                                 // (where large tiles would be few, below)
constexpr int kVChunk = 4;       // slabs of a chunk
constexpr int kVGroups = kMaxE / kWave;

struct Chunk {
    u32x4 w[kVChunk], x[kVChunk];
    uint32_t ws[kVChunk], xs[kVChunk];
};

__global__ __launch_bounds__(kVThreads, 4) void mxfp4_stream_kernel(MxArgs X) {
    const ProductArgs &A = X.p;
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int g = l >> 4, r = l & 15;

    // entries up to and with each expert, lane by lane, 64 experts a group
    int incl[kVGroups], first[kVGroups], count[kVGroups], entries = 0;
#pragma unroll
    for (int i = 0; i < kVGroups; ++i) {
        incl[i] = first[i] = count[i] = 0;
        if (i * kWave + l < A.E) group_of_lane(A, i * kWave + l, first[i], count[i]);
    }
#pragma unroll
    for (int i = 0; i < kVGroups; ++i) {
        if (i * kWave >= A.E) break;
        int n = (count[i] + kVRows - 1) / kVRows;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(n, d);
            if (l >= d) n += o;
        }
        incl[i] = entries + n;
        entries = __builtin_amdgcn_readlane(incl[i], kWave - 1);
    }
    // (no more than ascending offsets can give)
    const int most = A.E + A.R / kVRows;
    entries = entries < most ? entries : most;

    const int blocks = A.N / 16, slabs = A.K / 128, chunks = (slabs + kVChunk - 1) / kVChunk;
    const size_t ldx = (size_t)A.K / 2, lds = (size_t)A.K / 32;
    const unsigned tiles = (unsigned)entries * blocks;          // at most 2^26
    const unsigned me = blockIdx.x * kVWaves + w, all = kVWaves * gridDim.x;
    const unsigned each = tiles / all, more = tiles % all;
    const int t0 = me * each + me * more / all, t1 = (me + 1) * each + (me + 1) * more / all;
    if (t0 >= t1) return;

    // an entry's expert, rows, and this lane's row of x and of out (row r)
    struct Entry {
        int e, lo, src, dst;
    };
    auto entry = [&](int ai) {
        Entry n = {0, 0, 0, -1};
        int cnt = 0;
#pragma unroll
        for (int i = kVGroups - 1; i >= 0; --i) {
            const unsigned long long m = __ballot(incl[i] > ai);
            if (i * kWave >= A.E || !m) continue;
            const int at = __ffsll(m) - 1, c = __builtin_amdgcn_readlane(count[i], at);
            const int skip = kVRows * (ai - __builtin_amdgcn_readlane(incl[i], at) + (c + kVRows - 1) / kVRows);
            n.e = i * kWave + at;
            n.lo = __builtin_amdgcn_readlane(first[i], at) + skip;
            cnt = c - skip;
        }
        // rows past the entry's last one read its first one's and are not stored
        const int i = n.lo + (r < cnt ? r : 0), s = source_row(A.a, i);
        n.src = s < 0 ? 0 : s;
        if (r < cnt && s >= 0) {
            const int d = A.out_rows ? A.out_rows[i] : i;
            n.dst = d >= 0 && d < A.out_n ? d : -1;
        }
        return n;
    };
    // the next chunk to load, and the one to multiply
    int at = t0, ac = 0, ai = t0 / blocks, arb = t0 - ai * blocks;
    Entry ahead = entry(ai), cur = ahead;
    const char *wb = codes_of(X, ahead.e), *sb = scales_of(X, ahead.e);
    auto load = [&](Chunk &c) {
        const char *const wp = wb + (size_t)arb * slabs * 1024 + 16 * l, *const sp = sb + (size_t)arb * slabs * 64 + l;
#pragma unroll
        for (int i = 0; i < kVChunk; ++i) {
            const int s = ac * kVChunk + i < slabs ? ac * kVChunk + i : slabs - 1;
            c.w[i] = load_nt16(wp + (size_t)s * 1024);
            c.ws[i] = load_u8(sp + (size_t)s * 64);
        }
        const char *const xp = A.a.base + (size_t)ahead.src * ldx + 16 * g;
        const char *const yp = (const char *)X.xs + (size_t)ahead.src * lds;
#pragma unroll
        for (int i = 0; i < kVChunk; ++i) {
            const int s = ac * kVChunk + i < slabs ? ac * kVChunk + i : slabs - 1;
            c.x[i] = load16(xp + (size_t)s * 64);
            c.xs[i] = load_u32(yp + (size_t)s * 4);
        }
    };
    auto advance = [&]() {
        if (++ac < chunks) return;
        if (at + 1 >= t1) {
            ac = chunks - 1;     // the last chunk once more, which nothing multiplies
            return;
        }
        ac = 0, ++at;
        if (++arb == blocks) {
            arb = 0;
            ahead = entry(++ai);
            wb = codes_of(X, ahead.e), sb = scales_of(X, ahead.e);
        }
    };
    int ci = ai, crb = arb, cc = 0;
    f32x4 sum = {0, 0, 0, 0};
    auto multiply = [&](const Chunk &c) {
#pragma unroll
        for (int i = 0; i < kVChunk; ++i)
            if (cc * kVChunk + i < slabs) sum = mfma16(c.w[i], c.x[i], sum, c.ws[i], c.xs[i] >> (8 * g));
        if (++cc < chunks) return;
        // lane (g, r) has n 4 g .. 4 g + 3 of row r
        if (cur.dst >= 0) {
            const size_t o = (size_t)cur.dst * A.N + 16 * crb + 4 * g;
            typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
            if (A.out_f32) *(MOE_GLOBAL f32x4 *)((float *)A.out + o) = sum;
            else *(MOE_GLOBAL u32x2 *)((uint16_t *)A.out + o) =
                     u32x2{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
        }
        cc = 0, sum = f32x4{0, 0, 0, 0};
        if (++crb == blocks) crb = 0, ++ci;
        if (ci == ai) cur = ahead;      // (an entry ahead of the one that is multiplied is a whole entry's tiles on)
    };
    Chunk c0, c1;
    load(c0);
    for (int left = (t1 - t0) * chunks;;) {
        advance(), load(c1);
        multiply(c0);
        if (--left == 0) break;
        advance(), load(c0);
        multiply(c1);
        if (--left == 0) break;
    }
}

static long tiles_of(int R, int N, int E, int p, int q) {
    return ((long)R / p + (R < E ? R : E)) * ((N + q - 1) / q);
}

// Which kernel, from the sizes alone. us of a call with uneven routing (popularity
// e^(N(0,1)/4.5 to 2)), streaming / 128 x 256 / 256 x 256 tiles:
//   128 experts of 1536 x 2048, 8 a token: 1, 2, 4, 16, 64, 256, 1024, 4096, 8192 tokens
//     7.3/12.3/13.3  10.3/13.8/14.3  14.7/15.1/15.6  33.7/28.3/29.2  51.0/45.5/45.0
//     -/47.8/46.2  -/58/54  -/112/99  -/194/160
//   256 experts of 4096 x 4096, 6 a token: 1, 2, 8, 32, 256 tokens
//     16.0/18.5/20.1  25.2/22.5/23.2  75/75/72  -/188/184  -/334/327
//   one of 4096 x 4096: 1, 16, 64, 512, 1024, 1536, 2048, 3000, 3800, 4001 rows
//     8.7/12.2/18.2  10.1/13.0/18.3  20.1/15.0/19.0  -/27.8/30.7  -/27.0/30.6  -/27.8/30.7
//     -/29.3/30.8  -/41.5/33.3  -/46.2/37.9  -/47.6/39.6
//   one of 8192 x 8192, 8192 rows -/346/257
// The streaming kernel, which needs no second launch for a sum in parts, wins with few
// tiles; large ones win where rows fill them or the tiles are many. (With one expert
// they win from where the smaller tiles are more than the compute units, 2100 rows of
// the one above, which takes them from 3840 on: 8 us late in between.)
static bool mxfp4_streams(int R, int N, int E) {
    return R <= (long)kVAvg * E && tiles_of(R, N, E, kBT, kBT) <= 128;
}
static bool mxfp4_large(const ProductArgs &a) {
    const size_t out = (size_t)a.out_n * a.N * (a.out_f32 ? 4 : 2);
    if (a.K % 256 || a.K < 128 * kBSlabs || (size_t)a.a.n * (a.K / 2) > 0xFFFFFFFFull || out > kBBytes) return false;
    if ((long)a.N * (a.K / 32) > 0x7FFFFFFFL) return false;
    const long tiles = tiles_of(a.R, a.N, a.E, kBT, kBT);
    return tiles >= compute_units() && (a.R >= 32L * a.E || tiles >= 4L * compute_units());
}

// Parts that the sum of a tile is cut into: where there are fewer tiles than compute
// units, as many as give each one, of eight slabs at least. (4, 8, 16: 64 rows of one
// expert of 4096 x 4096 16.8, 15.0, 17.4 us, 128 rows 22.9, 19.1, 20.1, 256 rows 25.7,
// 24.9, 23.4, 512 rows 28.3, 28.3, 29.4, 500 of 1536 x 2048 17.7, 16.3, 15.8.)
static int mxfp4_slices(int R, int N, int K, int E) {
    if (R == 0 || mxfp4_streams(R, N, E)) return 1;
    const long tiles = tiles_of(R, N, E, kXP, kXQ);
    long n = compute_units() / (tiles < 1 ? 1 : tiles);
    const long steps = K / 128;
    n = n < steps / 8 ? n : steps / 8;
    return n < 2 ? 1 : n > 16 ? 16 : (int)n;
}

size_t mxfp4_part_bytes(int R, int N, int K, int E) {
    const int n = mxfp4_slices(R, N, K, E);
    return n < 2 ? 0 : (size_t)n * R * N * sizeof(float);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_gemm_mxfp4(const uint8_t *x_e2m1, const uint8_t *x_e8m0, const int32_t *x_rows,
                                      int x_div, int x_n, const int32_t *offsets, const uint8_t *w_e2m1,
                                      const uint8_t *w_e8m0, const moe_expert_w *experts, int mat, int R,
                                      int N, int K, int E, void *y, const int32_t *y_rows, int y_n,
                                      int y_is_fp32, void *ws, size_t ws_bytes, void *stream) {
    const int rc = check_sizes(R, N, K, E, offsets, 128);
    if (rc != MOE_OK) return rc;
    if (N % 16 || (mat != MOE_MAT_W13 && mat != MOE_MAT_W2)) return MOE_EINVAL;
    if (R == 0) return MOE_OK;
    if ((!w_e2m1) == (!experts) || (!w_e2m1) != (!w_e8m0) || !aligned16(w_e2m1) || !aligned16(w_e8m0) || !y ||
        !aligned16(y) || !aligned16(ws))
        return MOE_EINVAL;
    if (!x_e8m0 || ((uintptr_t)x_e8m0 & 3) || !rows_ok(x_e2m1, x_rows, x_div, x_n, R) ||
        y_n < (y_rows ? 1 : R))
        return MOE_EINVAL;
    MxArgs m{};
    ProductArgs &a = m.p;
    a.offsets = offsets, a.E = E, a.R = R, a.N = N, a.K = K;
    a.a = rows_in(x_e2m1, x_rows, x_div, x_n);
    a.m = Mats{(const char *)w_e2m1, nullptr, experts, mat};
    a.out = y, a.out_rows = y_rows, a.out_n = y_n, a.out_f32 = y_is_fp32 != 0;
    m.xs = x_e8m0, m.ws = w_e8m0;
    hipStream_t s = (hipStream_t)stream;
    const int cu = compute_units();
    if (mxfp4_streams(R, N, E)) {
        const long tiles = (long)(R < E ? R : E + R / kVRows) * (N / 16), groups = (tiles + kVWaves - 1) / kVWaves;
        MOE_LAUNCH(K_PROD_MXFP4_STREAM, mxfp4_stream_kernel, dim3((unsigned)(groups < 4L * cu ? groups : 4L * cu)),
                   dim3(kVThreads), 0, s, m);
        return check_launch();
    }
    a.slices = mxfp4_slices(R, N, K, E);
    a.part = (float *)ws;
    if (!ws || ws_bytes < mxfp4_part_bytes(R, N, K, E)) a.slices = 1;
    if (mxfp4_large(a)) {
        const long tiles = tiles_of(R, N, E, kBT, kBT);
        MOE_LAUNCH(K_PROD_MXFP4_LARGE, mxfp4_large_kernel, dim3((unsigned)(tiles < cu ? tiles : cu)), dim3(kBThreads), 0,
                   s, m);
        return check_launch();
    }
    const long tiles = tiles_of(R, N, E, kXP, kXQ) * a.slices;
    MOE_LAUNCH(K_PROD_MXFP4, mxfp4_tile_kernel, dim3((unsigned)(tiles < 2L * cu ? tiles : 2L * cu)),
               dim3(kXThreads), 0, s, m);
    if (a.slices > 1) launch_join(a, N, s);
    return check_launch();
}
