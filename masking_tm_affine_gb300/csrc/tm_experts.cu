// tm_experts.cu -- entry points of the products grouped by expert (16 bits) and of the
// 8-bit product: checks of arguments and the choice of kernel.
#include "tm_products.h"

namespace libtm {
namespace {

constexpr int32_t kMostExperts = 1024;

// Extents, experts and their borders.
tm_status check_extents(const int32_t *starts, int32_t E, int64_t T, int64_t N, int64_t K)
{
    if (E < 1 || T < 0 || N < 0 || K < 0 || (E > 1 && starts == nullptr)) return TM_ERR_INVALID_ARG;
    if (E > kMostExperts || T > INT32_MAX - 512 || N > INT32_MAX - 512 || K > INT32_MAX - 512) return TM_ERR_UNSUPPORTED_TILE;
    if (!aligned_to(starts, 4)) return TM_ERR_MISALIGNED;
    return TM_OK;
}

// An operand the copies read: rows on 16-byte boundaries.
bool on_grid(const void *p, int64_t ld, int64_t rows, int64_t inner, int e)
{
    return rows == 0 || inner == 0 || (aligned_to(p, 16) && ld * e % 16 == 0);
}

bool span_fits(int64_t ld, int64_t rows, int e) { return ld < (int64_t(1) << 36) && (rows == 0 || ld <= (int64_t(1) << 56) / rows / e); }

// Whether two sets of rows share a byte: not where both are columns of one tensor, one beside the other.
struct Rows {
    const void *p;
    int64_t ld, rows, cols;
    int e;
};
bool rows_meet(const Rows &a, const Rows &b)
{
    const Span x = span_of(a.p, a.ld, a.rows, a.cols, a.e), y = span_of(b.p, b.ld, b.rows, b.cols, b.e);
    if (!meets(x, y)) return false;
    const int64_t row = a.ld * a.e;
    if (row != b.ld * b.e) return true;
    const int64_t d = x.lo <= y.lo ? (int64_t)(y.lo - x.lo) % row : (row - (int64_t)(x.lo - y.lo) % row) % row;
    return d < a.cols * a.e || d + b.cols * b.e > row;
}

// Nothing of an operand without elements is read, but its map wants an address.
const void *base_of(const void *p, int64_t elements, const void *out)
{
    return elements > 0 ? p : reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(out) & ~uintptr_t(15));
}

// Which kernel.  Tiles of 128 by 32 or 128, whose sums can be cut over a cluster, up to 32 rows an expert
// (where the weights' bytes bound the call), or for long sums while there are so few of those tiles that four CTAs can
// share each sum.
//   64 experts of 2048 x 2048, 16 bits: 32 rows each 105 us either way, 64 rows 119 us thin and 107 wide
//   64 of 2048 x 4096, 8 bits: 32 rows 109 and 129 us, 64 rows 158 and 130
//   sums over four CTAs, one of 512 x 4096, 16 bits: 400 rows 18.5 us thin and 22.6 wide; of 256 x 8192, 8 bits,
//   1000 rows 24.6 and 29.7; over two, of 4096 x 4096, 16 bits, 256 rows: 26.6 and 24.6
//   short ones, 16 bits, 100 rows of 1024 x 1024: 14.3 and 12.3
// The rows of each expert are not known here: where they all go to one of many, tiles of 32 read its matrix once each (2048
// rows, one of 64 experts: of 4096 x 4096 148 us in 16 bits and 124 in 8, alone 48 and 40; of 2048 x 2048 52 and 42, 19 and 17).
bool few_rows(const Product &p, const DevInfo &dev)
{
    if (p.T <= 32 * (int64_t)p.E) return true;
    return tiles_of(p, 128) * ((p.F + 127) / 128) * 4 <= dev.sms && p.R >= 2048;
}

}  // namespace
}  // namespace libtm

using namespace libtm;

extern "C" tm_status tm_gemm_experts(const void *X, int64_t ldx, const void *W, int64_t ldw, void *Y, int64_t ldy,
                                     const int32_t *starts, int32_t E, int64_t T, int64_t N, int64_t K, int32_t xtype,
                                     int32_t ytype, uint32_t flags, tm_stream_t stream)
{
    if ((xtype != TM_F16 && xtype != TM_BF16) || (ytype != xtype && ytype != TM_F32)) return TM_ERR_INVALID_ARG;
    if (flags & ~(uint32_t)TM_PDL) return TM_ERR_INVALID_ARG;
    tm_status st = check_extents(starts, E, T, N, K);
    if (st != TM_OK) return st;
    if (!valid_rows(X, ldx, T, K) || !valid_rows(W, ldw, (int64_t)E * N, K) || !valid_rows(Y, ldy, T, N)) return TM_ERR_INVALID_ARG;
    if (!span_fits(ldx, T, 2) || !span_fits(ldw, (int64_t)E * N, 2)) return TM_ERR_INVALID_ARG;
    const int eo = elem_bytes(ytype);
    if (!on_grid(X, ldx, T, K, 2) || !on_grid(W, ldw, (int64_t)E * N, K, 2) || !aligned_to(Y, (uintptr_t)eo)) return TM_ERR_MISALIGNED;
    const Rows y = {Y, ldy, T, N, eo};
    if (rows_meet(y, {X, ldx, T, K, 2}) || rows_meet(y, {W, ldw, (int64_t)E * N, K, 2}) || rows_meet(y, {starts, E + 1, 1, E + 1, 4}))
        return TM_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return TM_OK;
    const DevInfo *dev;
    if ((st = device_info(&dev)) != TM_OK) return st;
    Product p = {};
    p.kind = xtype == TM_BF16 ? kProductBF16 : kProductF16;
    p.w = base_of(W, K, Y);
    p.ldw = ldw;
    p.x = base_of(X, K, Y);
    p.ldx = ldx;
    p.out = Y;
    p.ldo = ldy;
    p.otype = ytype;
    p.starts = starts;
    p.E = E;
    p.T = T;
    p.F = N;
    p.R = K;
    const bool pdl = (flags & TM_PDL) != 0;
    return few_rows(p, *dev) ? thin_product(p, *dev, as_stream(stream), pdl) : wide_product(p, *dev, as_stream(stream), pdl);
}

extern "C" tm_status tm_gemm_experts_bwd(const void *DY, int64_t lddy, const void *X, int64_t ldx, const void *W, int64_t ldw,
                                         void *DX, int64_t lddx, void *DW, int64_t lddw, const int32_t *starts, int32_t E,
                                         int64_t T, int64_t N, int64_t K, int32_t xtype, int32_t wtype, uint32_t flags,
                                         tm_stream_t stream)
{
    if ((xtype != TM_F16 && xtype != TM_BF16) || (wtype != xtype && wtype != TM_F32)) return TM_ERR_INVALID_ARG;
    if (flags & ~(uint32_t)TM_PDL) return TM_ERR_INVALID_ARG;
    tm_status st = check_extents(starts, E, T, N, K);
    if (st != TM_OK) return st;
    const int64_t EN = (int64_t)E * N;
    const bool rows = DX != nullptr && T > 0 && K > 0, weights = DW != nullptr && N > 0 && K > 0;
    if (!valid_rows(DY, lddy, T, N)) return TM_ERR_INVALID_ARG;
    if (DX != nullptr && (!valid_rows(W, ldw, EN, K) || !valid_rows(DX, lddx, T, K) || !span_fits(ldw, EN, 2))) return TM_ERR_INVALID_ARG;
    if (DW != nullptr && (!valid_rows(X, ldx, T, K) || !valid_rows(DW, lddw, EN, K) || !span_fits(ldx, T, 2))) return TM_ERR_INVALID_ARG;
    if (!span_fits(lddy, T, 2)) return TM_ERR_INVALID_ARG;
    const int ew = elem_bytes(wtype);
    if (!on_grid(DY, lddy, T, N, 2) || (DX != nullptr && (!on_grid(W, ldw, EN, K, 2) || !aligned_to(DX, 2))) ||
        (DW != nullptr && (!on_grid(X, ldx, T, K, 2) || !aligned_to(DW, (uintptr_t)ew))))
        return TM_ERR_MISALIGNED;
    const Rows dx = {DX, lddx, T, K, 2}, dw = {DW, lddw, EN, K, ew};
    const Rows in[] = {{DY, lddy, T, N, 2}, {DW ? X : nullptr, ldx, T, K, 2}, {DX ? W : nullptr, ldw, EN, K, 2}, {starts, E + 1, 1, E + 1, 4}};
    for (const Rows &i : in)
        if (rows_meet(dx, i) || rows_meet(dw, i)) return TM_ERR_INVALID_ARG;
    if (rows_meet(dx, dw)) return TM_ERR_INVALID_ARG;
    if (!rows && !weights) return TM_OK;
    const DevInfo *dev;
    if ((st = device_info(&dev)) != TM_OK) return st;
    const ProductKind kind = xtype == TM_BF16 ? kProductBF16 : kProductF16;
    const bool pdl = (flags & TM_PDL) != 0;
    if (rows) {
        Product p = {};
        p.kind = kind;
        p.w = base_of(W, N, DX);
        p.ldw = ldw;
        p.w_mn = true;
        p.x = base_of(DY, N, DX);
        p.ldx = lddy;
        p.out = DX;
        p.ldo = lddx;
        p.otype = xtype;
        p.starts = starts;
        p.E = E;
        p.T = T;
        p.F = K;
        p.R = N;
        st = few_rows(p, *dev) ? thin_product(p, *dev, as_stream(stream), pdl) : wide_product(p, *dev, as_stream(stream), pdl);
        if (st != TM_OK) return st;
    }
    if (weights)
        st = wide_weights(kind, base_of(DY, T, DW), lddy, base_of(X, T, DW), ldx, DW, lddw, wtype, starts, E, T, N, K, *dev,
                          as_stream(stream), pdl);
    return st;
}

extern "C" tm_status tm_gemm_e4m3(const void *A, int64_t lda, const float *sa, int32_t group, const void *B, int64_t ldb,
                                  const float *sb, void *C, int64_t ldc, const int32_t *starts, int32_t E, int64_t M, int64_t N,
                                  int64_t K, int32_t ctype, uint32_t flags, tm_stream_t stream)
{
    const int ec = elem_bytes(ctype);
    if (ec == 0 || (flags & ~(uint32_t)TM_PDL)) return TM_ERR_INVALID_ARG;
    tm_status st = check_extents(starts, E, M, N, K);
    if (st != TM_OK) return st;
    if (group != 0 && group != 128) return TM_ERR_UNSUPPORTED_TILE;
    const int64_t EN = (int64_t)E * N, KB = (K + 127) / 128, NB = (N + 127) / 128, sacols = group ? KB : 1;
    if (!valid_rows(A, lda, M, K) || !valid_rows(B, ldb, EN, K) || !valid_rows(C, ldc, M, N)) return TM_ERR_INVALID_ARG;
    if (!span_fits(lda, M, 1) || !span_fits(ldb, EN, 1)) return TM_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && K > 0 && (sa == nullptr || sb == nullptr)) return TM_ERR_INVALID_ARG;
    if (!on_grid(A, lda, M, K, 1) || !on_grid(B, ldb, EN, K, 1) || !aligned_to(C, (uintptr_t)ec) || !aligned_to(sa, 4) ||
        !aligned_to(sb, 4))
        return TM_ERR_MISALIGNED;
    const Rows c = {C, ldc, M, N, ec};
    if (rows_meet(c, {A, lda, M, K, 1}) || rows_meet(c, {B, ldb, EN, K, 1}) || rows_meet(c, {sa, sacols, M, sacols, 4}) ||
        rows_meet(c, {sb, NB * KB, E, NB * KB, 4}) || rows_meet(c, {starts, E + 1, 1, E + 1, 4}))
        return TM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TM_OK;
    const DevInfo *dev;
    if ((st = device_info(&dev)) != TM_OK) return st;
    Product p = {};
    p.kind = kProductE4M3;
    p.w = base_of(B, K, C);
    p.ldw = ldb;
    p.x = base_of(A, K, C);
    p.ldx = lda;
    p.out = C;
    p.ldo = ldc;
    p.otype = ctype;
    p.starts = starts;
    p.E = E;
    p.T = M;
    p.F = N;
    p.R = K;
    p.sa = sa;
    p.sb = sb;
    p.group = group;
    const bool pdl = (flags & TM_PDL) != 0;
    return few_rows(p, *dev) ? thin_product(p, *dev, as_stream(stream), pdl) : wide8_product(p, *dev, as_stream(stream), pdl);
}
