// Arguments and launch interface of the expert products (products.hip,
// products_stream.hip).
#pragma once

#include "common.hpp"

namespace moe {

// A matrix whose rows a product reads: row i of the sorted order is row
// idx[i] / div of the matrix (row i where idx is NULL); n rows exist.
struct RowsIn {
    const char *base;
    const int32_t *idx;
    int div;
    int n;
};

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

// Source row of sorted row i, or -1 where the index is not a row of r.
__device__ __forceinline__ int source_row(const RowsIn &r, int i) {
    if (!r.idx) return i;
    int v = r.idx[i];
    if (v < 0) return -1;
    v = r.div == 1 ? v : v / r.div;
    return v < r.n ? v : -1;
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

int compute_units();   // of the current device (256 on MI355X)

}  // namespace moe
