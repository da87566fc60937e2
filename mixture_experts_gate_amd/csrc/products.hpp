// Arguments and launch interface of the expert products (products.hip,
// products_stream.hip).
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kMaxE = 512;       // experts of a product
constexpr int kMaxRows = 0x7FFFFF00;    // rows: those of a last tile or workgroup fit an int

// v / div for 0 <= v < 2^31 as (v mul) >> (32 + shift), mul = floor(2^(31 +
// l) / div) + 1 and shift = l - 1 for 2^(l-1) < div <= 2^l: mul exceeds the
// quotient by at most one, which moves v mul by less than 2^31 <= 2^(31 +
// l) / div, one unit of the result over div. mul = 0: div is 1.
struct Divisor {
    uint32_t mul;
    int shift;
};

inline Divisor divisor(int div) {
    if (div <= 1) return Divisor{0, 0};
    int l = 1;
    while ((1LL << l) < div) ++l;
    return Divisor{(uint32_t)((1ULL << (31 + l)) / (uint64_t)div + 1), l - 1};
}

__device__ __forceinline__ uint32_t operator/(uint32_t v, const Divisor &d) {
    return d.mul ? __umulhi(v, d.mul) >> d.shift : v;
}

// A matrix whose rows a product reads: row i of the sorted order is row
// idx[i] / div of the matrix (row i where idx is NULL); n rows exist.
struct RowsIn {
    const char *base;
    const int32_t *idx;
    int n;
    Divisor div;
};

inline RowsIn rows_in(const void *base, const int32_t *idx, int div, int n) {
    return RowsIn{(const char *)base, idx, n, divisor(div)};
}

// The experts' matrices [N][K]: either one array [E][N][K] (tab NULL) or the
// w13 / w2 pointers of a moe_expert_w table.
struct Mats {
    const char *w;
    const float *s;            // FP8: block scales [E][ceil(N/128)][ceil(K/128)]
    const moe_expert_w *tab;
    int mat;
};

struct ProductArgs {
    const int32_t *offsets;    // [E+1]; NULL: one group of R rows
    int E, R, N, K;
    RowsIn a;                  // forward: x; dx, dw: dy
    const float *a_s;          // FP8: scales of a's rows [n][ceil(K/128)]
    RowsIn b;                  // dw: x
    Mats m;
    void *out;
    const int32_t *out_rows;   // NULL: row i of the sorted order is row i of out
    int out_n;
    int out_f32;
    int accumulate;            // dw: add to what is there (fp32)
    float *part;               // sums of `slices` parts of c, [slices][R or E N][q] (slices > 1)
    int slices;
};

enum ProductMode { kFwd = 0, kFwdFp8 = 1, kDx = 2, kDw = 3 };

// Rows of expert e, with offsets kept inside [0, R] whatever they hold.
__device__ __forceinline__ void group_of(const ProductArgs &a, int e, int &lo, int &cnt) {
    if (!a.offsets) {
        lo = 0;
        cnt = a.R;
        return;
    }
    const int b = as_scalar(a.offsets)[e], f = as_scalar(a.offsets)[e + 1];
    lo = b < 0 ? 0 : b > a.R ? a.R : b;
    const int hi = f < 0 ? 0 : f > a.R ? a.R : f;
    cnt = hi > lo ? hi - lo : 0;
}

// The same for an expert of this lane's own.
__device__ __forceinline__ void group_of_lane(const ProductArgs &a, int e, int &lo, int &cnt) {
    lo = 0, cnt = a.R;
    if (!a.offsets) return;
    const int b = a.offsets[e], f = a.offsets[e + 1];
    lo = b < 0 ? 0 : b > a.R ? a.R : b;
    const int hi = f < 0 ? 0 : f > a.R ? a.R : f;
    cnt = hi > lo ? hi - lo : 0;
}

// The row that index v stands for, or -1 where it is not a row of r.
__device__ __forceinline__ int row_of_index(const RowsIn &r, int v) {
    const int q = (int)((uint32_t)v / r.div);
    return v >= 0 && q < r.n ? q : -1;
}

// Source row of sorted row i, or -1.
__device__ __forceinline__ int source_row(const RowsIn &r, int i) {
    return r.idx ? row_of_index(r, r.idx[i]) : i;
}

__device__ __forceinline__ const char *mat_of(const ProductArgs &a, int e, int elem) {
    if (a.m.tab) return (const char *)(a.m.mat ? as_scalar(a.m.tab)[e].w2 : as_scalar(a.m.tab)[e].w13);
    return a.m.w + (size_t)e * a.N * a.K * elem;
}

__device__ __forceinline__ const float *scales_of(const ProductArgs &a, int e) {
    if (a.m.tab)
        return (const float *)(a.m.mat ? as_scalar(a.m.tab)[e].s2 : as_scalar(a.m.tab)[e].s13);
    return a.m.s + (size_t)e * ((a.N + 127) / 128) * ((a.K + 127) / 128);
}

typedef __attribute__((ext_vector_type(8))) int i32x8;

__device__ __forceinline__ i32x8 as_i32x8(u32x4 a, u32x4 b) {
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// 16 bytes a lane from `from`, or zeros. Always one copy instruction, whichever
// lanes are in: the waits count them.
__device__ const uint32_t g_zeros[4] = {0, 0, 0, 0};
__device__ __forceinline__ void copy_or_zeros(bool in, const char *from, char *to) {
    lds_dma16(in ? from : (const char *)g_zeros, to);
}

// A wavefront-uniform address kept in scalar registers: the lanes' offsets are
// added by the load, not kept added to it in vector registers.
__device__ __forceinline__ const char *scalar_base(const char *p) {
    asm volatile("" : "+s"(p));
    return p;
}

// The offset, widened where it is used and not before.
__device__ __forceinline__ uint32_t here(uint32_t o) {
    asm volatile("" : "+v"(o));
    return o;
}

// dw: the indices of 64 rows of sorted order from lo + c, of an expert's cnt, go
// into LDS by a copy (through a register, the wait for one would be a wait for
// every copy issued before it), and a step later one lane a row makes them the
// rows' numbers, -1 past the last one.
__device__ __forceinline__ void copy_indices(const RowsIn &r, int c, int lo, int cnt, int *to) {
    const int i = c + lane_id();
    if (r.idx) lds_dma4(r.idx + lo + (i < cnt ? i : cnt - 1), to);
}

__device__ __forceinline__ void rows_from_indices(const RowsIn &r, int c, int lo, int cnt, const int *raw,
                                                  int *rows) {
    const int l = lane_id();
    const int row = r.idx ? row_of_index(r, raw[l]) : lo + c + l;
    rows[l] = c + l < cnt ? row : -1;
}

// dw: an operand's part in the copies of a step: the row of the first copy where
// rows are in place, bytes of a row, the lane's offset from that row (in place)
// and in a row, the list of rows (first one of this lane), the place in LDS.
struct Rows {
    const RowsIn &r;
    size_t first, ld;
    uint32_t off, col;
    const int *rows;
    char *to;
};

// dw: N copies of each operand, 16 rows of a step apart: rows in place that all
// exist (a uniform base and a lane's offset), or the rows that the lists give. A
// row that is -1 in one list is zeros in both operands: a zero beside a row that
// is read would still give NaN where that one is not finite. One branch for all:
// a branch a copy took as long as the multiplications.
template <int N, int STRIDE>
__device__ __forceinline__ void copy_rows(bool in_place, const Rows &p, const Rows &q) {
    if (in_place) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            lds_dma16(scalar_base(p.r.base + (p.first + 16 * i) * p.ld) + here(p.off), p.to + 16 * i * STRIDE);
#pragma unroll
        for (int i = 0; i < N; ++i)
            lds_dma16(scalar_base(q.r.base + (q.first + 16 * i) * q.ld) + here(q.off), q.to + 16 * i * STRIDE);
    } else {
        int a[N], b[N];
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = p.rows[16 * i], b[i] = q.rows[16 * i];
#pragma unroll
        for (int i = 0; i < N; ++i)
            copy_or_zeros((a[i] | b[i]) >= 0, p.r.base + (size_t)(uint32_t)a[i] * p.ld + p.col,
                          p.to + 16 * i * STRIDE);
#pragma unroll
        for (int i = 0; i < N; ++i)
            copy_or_zeros((a[i] | b[i]) >= 0, q.r.base + (size_t)(uint32_t)b[i] * q.ld + q.col,
                          q.to + 16 * i * STRIDE);
    }
}

// This lane's index, which the compiler takes for a new value.
__device__ __forceinline__ int fresh_lane() {
    int l = lane_id();
    asm volatile("" : "+v"(l));
    return l;
}

// Waits for this wavefront's LDS accesses (lgkmcnt 0, the vector counter as
// it is), or until at most n of its copies and loads are in flight; the
// compiler keeps memory accesses on their side.
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
    asm volatile("" ::: "memory");
}

template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("" ::: "memory");
    wait_vm<N>();
    asm volatile("" ::: "memory");
}

// Barrier without a memory fence (a fenced one would also wait for the loads
// in flight).
__device__ __forceinline__ void bare_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Whether q is the row of the matrix instruction's result (Q its A operand) or
// its column. dx: row, see below; FP8: row, so that a lane's four results share
// one p and one scale (as column, with four scales a lane: 632 against 530 us
// for the FP8 down projection of 4096 tokens).
constexpr bool q_is_row(int mode) { return mode == kDx || mode == kFwdFp8; }

// The 16 q of a matrix instruction's tile j of a 64-column block. Where q is the
// column, four tiles give a lane q = 4 r + 0..3: 16 lanes store 64 consecutive q
// of a row. Where it is the row (and for dx, whose W comes through the
// transposing read, which takes groups of four consecutive columns), q = 16
// (r/4) + 4 j + r%4: a lane has 16 consecutive q.
template <int MODE>
__device__ __forceinline__ int perm64(int j, int r) {
    return q_is_row(MODE) ? 16 * (r >> 2) + 4 * j + (r & 3) : 4 * r + j;
}

// XOR key of the 16-byte chunks of an LDS row of c-major data: what one
// transposing read takes of rows c..c+3 lands in different banks. dw reads 16
// consecutive columns (32 bytes) of each row, dx four times 4 columns 32 bytes
// apart (8 bytes of each of 4 chunks; 16 different chunks of the 256 bytes that the banks span).
template <bool DW>
__device__ __forceinline__ int t_key(int c) {
    return DW ? 2 * (c & 3) : (c & 1) | ((c & 2) << 2);
}

// Tile li of mp x tq: groups of at most 8 p tiles, in a group q outer and p
// inner, so that the 32 tiles an XCD works on at a time are about 8 x 4 of them
// and share their rows of P and Q in its L2 (8192 x 8192 x 8192, bf16: 992 us
// against 1045 us with p inner over all 32 p tiles, whose misses fill the
// bandwidth behind the L2).
__device__ __forceinline__ void place_of(int li, int mp, int tq, int &p, int &q) {
    const int ng = (mp + 7) / 8, gp = (mp + ng - 1) / ng;
    const int gi = li / (gp * tq), rest = li - gi * gp * tq;
    const int gl = mp - gi * gp < gp ? mp - gi * gp : gp;
    q = rest / gl;
    p = gi * gp + rest - q * gl;
}

// Fragments of a matrix instruction from LDS, lane (g, r) = (l / 16, l % 16): 8
// consecutive c (16 bytes), half s of a step.
// Row `row` + r of c-contiguous data (rows of 128 bytes, chunks XORed with the row):
__device__ __forceinline__ u32x4 frag_n(const char *buf, int row, int s, int g, int r) {
    return *(const MOE_LDS u32x4 *)(buf + (row + r) * 128 + (((4 * s + g) ^ (r & 7)) << 4));
}

// Tile j of 64-column block blk of c-major data with rows of STRIDE bytes (dw:
// columns 16 j + 0..15): the address of its first transposing read in half 0; the
// second is 4 rows on, half 1 32 rows, the next block 128 bytes.
template <bool DW, int STRIDE>
__device__ __forceinline__ uint32_t frag_t_at(const char *buf, int blk, int j, int g, int r) {
    const int ci = r >> 2, tt = r & 3;
    const int ch = (DW ? 8 * blk + 2 * j + (tt >> 1) : 8 * blk + 2 * tt + (j >> 1)) ^ t_key<DW>(ci);
    const char *const a = buf + (8 * g + ci) * STRIDE + ch * 16 + (DW ? tt & 1 : j & 1) * 8;
    return (uint32_t)(uintptr_t)(const MOE_LDS char *)a;
}

// The fragments of the four tiles at `at`, OFF bytes on. The reads and their wait
// are one block of assembly: for the builtin the compiler waits until every copy
// into LDS has landed, also those of later steps.
template <int STRIDE, int OFF>
__device__ __forceinline__ void frags_t(const uint32_t (&at)[4], u32x4 (&f)[4]) {
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
    u32x2 a0, a1, b0, b1, c0, c1, d0, d1;
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
        "ds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
        "ds_read_b64_tr_b16 %2, %9 offset:%12\n\t"
        "ds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
        "ds_read_b64_tr_b16 %4, %10 offset:%12\n\t"
        "ds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
        "ds_read_b64_tr_b16 %6, %11 offset:%12\n\t"
        "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a0), "=&v"(a1), "=&v"(b0), "=&v"(b1), "=&v"(c0), "=&v"(c1), "=&v"(d0), "=&v"(d1)
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF), "n"(OFF + 4 * STRIDE)
        : "memory");
    f[0] = u32x4{a0[0], a0[1], a1[0], a1[1]}, f[1] = u32x4{b0[0], b0[1], b1[0], b1[1]};
    f[2] = u32x4{c0[0], c0[1], c1[0], c1[1]}, f[3] = u32x4{d0[0], d0[1], d1[0], d1[1]};
}

// Two such groups (OFF0, OFF1) with one wait.
template <int STRIDE, int OFF0, int OFF1>
__device__ __forceinline__ void frags_t2(const uint32_t (&at)[4], u32x4 (&f)[4], u32x4 (&h)[4]) {
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
    u32x2 v[16];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %16 offset:%20\n\t"
        "ds_read_b64_tr_b16 %1, %16 offset:%21\n\t"
        "ds_read_b64_tr_b16 %2, %17 offset:%20\n\t"
        "ds_read_b64_tr_b16 %3, %17 offset:%21\n\t"
        "ds_read_b64_tr_b16 %4, %18 offset:%20\n\t"
        "ds_read_b64_tr_b16 %5, %18 offset:%21\n\t"
        "ds_read_b64_tr_b16 %6, %19 offset:%20\n\t"
        "ds_read_b64_tr_b16 %7, %19 offset:%21\n\t"
        "ds_read_b64_tr_b16 %8, %16 offset:%22\n\t"
        "ds_read_b64_tr_b16 %9, %16 offset:%23\n\t"
        "ds_read_b64_tr_b16 %10, %17 offset:%22\n\t"
        "ds_read_b64_tr_b16 %11, %17 offset:%23\n\t"
        "ds_read_b64_tr_b16 %12, %18 offset:%22\n\t"
        "ds_read_b64_tr_b16 %13, %18 offset:%23\n\t"
        "ds_read_b64_tr_b16 %14, %19 offset:%22\n\t"
        "ds_read_b64_tr_b16 %15, %19 offset:%23\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]),
          "=&v"(v[7]), "=&v"(v[8]), "=&v"(v[9]), "=&v"(v[10]), "=&v"(v[11]), "=&v"(v[12]), "=&v"(v[13]),
          "=&v"(v[14]), "=&v"(v[15])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF0), "n"(OFF0 + 4 * STRIDE), "n"(OFF1),
          "n"(OFF1 + 4 * STRIDE)
        : "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j] = u32x4{v[2 * j][0], v[2 * j][1], v[2 * j + 1][0], v[2 * j + 1][1]};
        h[j] = u32x4{v[8 + 2 * j][0], v[8 + 2 * j][1], v[9 + 2 * j][0], v[9 + 2 * j][1]};
    }
}

// p tiles before each expert (base[0 .. E]), for tiles of bp rows; by all THREADS
// threads of a workgroup. No more than ascending offsets can give: with others
// the sum could pass 32 bits, and tiles would have rows that do not exist.
template <int THREADS>
__device__ __forceinline__ void total_tiles(const ProductArgs &A, int bp, int *base, int *wsum) {
    const int l = lane_id(), w = threadIdx.x / kWave, most = A.R / bp + A.E;
    int run = 0;
    if (threadIdx.x == 0) base[0] = 0;
    for (int e0 = 0; e0 < A.E; e0 += THREADS) {
        const int e = e0 + threadIdx.x;
        int n = 0;
        if (e < A.E) {
            int lo, cnt;
            group_of_lane(A, e, lo, cnt);
            n = (cnt + bp - 1) / bp;
        }
        int incl = n;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (l >= d) incl += o;
        }
        incl = incl < most ? incl : most;      // (64 of at most 2^24 before)
        if (l == kWave - 1) wsum[w] = incl;
        __syncthreads();
        int before = run, all = run;
        for (int i = 0; i < THREADS / kWave; ++i) {
            before += i < w ? wsum[i] : 0;
            all += wsum[i];
        }
        if (e < A.E) base[e + 1] = before + incl < most ? before + incl : most;
        run = all < most ? all : most;
        __syncthreads();
    }
}

// Expert e with base[e] tq <= ti < base[e+1] tq.
__device__ __forceinline__ int expert_of(const int *base, int E, int tq, int ti) {
    int a = 0, b = E;
    while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if ((long)base[mid] * tq <= ti) a = mid;
        else b = mid;
    }
    return __builtin_amdgcn_readfirstlane(a);
}

// A wavefront's results of p tile i, acc[j][c] for the four q tiles j of its
// 64-column block from q0, to the rows of out that `row` gives for p of the tile (-1: none).
//   dx, FP8: lane (g, r) has q = 16 g + 4 j + c of p = r;
//   forward bf16: q = 4 r + j of p = 4 g + c;  dw: q = 16 j + r of p = 4 g + c.
template <int MODE, class Row>
__device__ __forceinline__ void store_tile(const ProductArgs &A, int q0, int Qn, int g, int r,
                                           const f32x4 (&v)[4], Row row) {
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
    if (q_is_row(MODE)) {
        const long to = row(r);
        const int q = q0 + 16 * g;
        if (to < 0) return;
        if (A.out_f32) {
            float *const o = (float *)A.out + (size_t)to * Qn + q;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (q + 4 * j < Qn) *(MOE_GLOBAL f32x4 *)(o + 4 * j) = v[j];
        } else {
            uint16_t *const o = (uint16_t *)A.out + (size_t)to * Qn + q;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (q + 8 * h < Qn)
                    *(MOE_GLOBAL u32x4 *)(o + 8 * h) =
                        u32x4{pack_bf16x2(v[2 * h][0], v[2 * h][1]), pack_bf16x2(v[2 * h][2], v[2 * h][3]),
                              pack_bf16x2(v[2 * h + 1][0], v[2 * h + 1][1]),
                              pack_bf16x2(v[2 * h + 1][2], v[2 * h + 1][3])};
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const long to = row(4 * g + c);
        if (to < 0) continue;
        if (MODE == kDw) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q = q0 + 16 * j + r;
                if (q >= Qn) continue;
                if (A.out_f32) {
                    MOE_GLOBAL float *const o = (MOE_GLOBAL float *)A.out + (size_t)to * Qn + q;
                    *o = A.accumulate ? *o + v[j][c] : v[j][c];
                } else {
                    ((MOE_GLOBAL uint16_t *)A.out)[(size_t)to * Qn + q] = (uint16_t)f32_to_bf16_bits(v[j][c]);
                }
            }
        } else {
            const int q = q0 + 4 * r;
            if (q >= Qn) continue;
            if (A.out_f32)
                *(MOE_GLOBAL f32x4 *)((float *)A.out + (size_t)to * Qn + q) =
                    f32x4{v[0][c], v[1][c], v[2][c], v[3][c]};
            else
                *(MOE_GLOBAL u32x2 *)((uint16_t *)A.out + (size_t)to * Qn + q) =
                    u32x2{pack_bf16x2(v[0][c], v[1][c]), pack_bf16x2(v[2][c], v[3][c])};
        }
    }
}

// products_stream.hip: the forward products at a handful of rows per expert
bool product_streams(const ProductArgs &a);
void launch_product_stream(const ProductArgs &a, bool fp8, hipStream_t s);

// products_small.hip: any product in tiles of 128 x 128
void launch_product_small(const ProductArgs &a, int mode, hipStream_t s);
int small_slices(const ProductArgs &a, int mode);   // parts that c is worth being cut into

int kernel_of(int mode);   // timing id of a product
int compute_units();   // of the current device (256 on MI355X)

}  // namespace moe
