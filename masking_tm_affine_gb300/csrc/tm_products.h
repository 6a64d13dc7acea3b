// tm_products.h -- host side of the products on operands of 16 and 8 bits.
#pragma once

#include "tm_host.h"
#include "tm_elem.cuh"

namespace libtm {

enum ProductKind { kProductF16 = 0, kProductBF16 = 1, kProductE4M3 = 2 };

// out[t, f] = sum_r x[t, r] w_e[f, r] (w_mn: w_e[r, f]) for the rows t of each expert e.
struct Product {
    ProductKind kind;
    const void *w;    // [E][F][R], with w_mn [E][R][F]; rows ldw elements apart, matrices rows * ldw
    int64_t ldw;
    bool w_mn;
    const void *x;    // [T][R], rows ldx elements apart
    int64_t ldx;
    void *out;        // [T][F] of otype
    int64_t ldo;
    int32_t otype;
    const int32_t *starts;  // [E + 1] on the device, or nullptr: all rows are expert 0's
    int32_t E;
    int64_t T, F, R;
    // e4m3: sa [T] (group 0) or [T][ceil(R / 128)]; sb [E][ceil(F / 128)][ceil(R / 128)]
    const float *sa, *sb;
    int32_t group;
};

// Row tiles to expect: the experts' borders, which are not known here, cut half a tile each.
inline int64_t tiles_of(const Product &p, int rows) { return (p.T + rows - 1) / rows + (p.E < p.T ? p.E : p.T) / 2; }

// A map of rows of `inner` elements of e bytes in boxes 128 bytes wide and `box` rows high, 128-byte
// swizzle, zeros outside; with E > 0 of E matrices of `rows` rows.
bool rows_map_of(CUtensorMap *m, int e, const void *p, int64_t inner, int64_t rows, int64_t ld, int64_t E, int box);
inline bool rows_map(CUtensorMap *m, ProductKind kind, const void *p, int64_t inner, int64_t rows, int64_t ld, int64_t E, int box)
{
    return rows_map_of(m, kind == kProductE4M3 ? 1 : 2, p, inner, rows, ld, E, box);
}

// The same seen as panels of 64 columns (16-bit; `inner` a multiple of 64): boxes of two panels of
// 64 rows, one behind the other in shared memory, in one copy.  Coordinates: 0, row, panel, matrix.
bool panels_map(CUtensorMap *m, const void *p, int64_t inner, int64_t rows, int64_t ld, int64_t E);

// Few rows an expert: tiles of 128 features and up to 128 rows, split along the sum.
tm_status thin_product(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl);

// 8 bits, many rows an expert: CTA pairs, tiles of 256 by 256.
tm_status wide8_product(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl);

// 16 bits, many rows an expert: CTA pairs, tiles of 256 by 256.
tm_status wide_product(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl);
// dw [E][N][K] of wtype from dy [T][N] and x [T][K].
tm_status wide_weights(ProductKind kind, const void *dy, int64_t lddy, const void *x, int64_t ldx, void *dw, int64_t lddw,
                       int32_t wtype, const int32_t *starts, int32_t E, int64_t T, int64_t N, int64_t K, const DevInfo &dev,
                       cudaStream_t s, bool pdl);

}  // namespace libtm
