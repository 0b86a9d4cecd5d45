// Where the operands of a linear layer's products lie, and which elements a lane
// reads of rows that end anywhere.  Plain arithmetic, for the host and the kernels,
// which a test runs over sizes and layouts without a GPU.
#pragma once

#include <stdint.h>

namespace onebit {

constexpr int64_t kMaxFeatures = (int64_t)1 << 22;  // a tile's rows within 2^31 bytes

constexpr int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }

// An operand: element (i, k) of the product's index i and the summed index k is
// at p[i ld + k] (by rows) or p[k ld + i].  Of a contiguous row `row` elements may be
// read: the matrix's own, or of rows laid out anew also the zeros behind them.  Where
// one operand of a product is the sum of two parts of the same layout, the second
// `rest` bytes behind the first, the sum over k goes over the first parts and then over
// the rest (0 bytes for the other operand).
struct ProductIn {
    const void* p;
    int64_t ld, row;
    int64_t rest;
};

// Of the eight elements of a row from `at` on, those past its end; 8: none is read.
// Otherwise the row's last eight are, from `at` less this number on, so such rows have
// eight elements or more.
constexpr int32_t past_end(int64_t at, int64_t row) {
    return at + 8 <= row ? 0 : at >= row ? 8 : (int32_t)(at + 8 - row);
}

// to[r][c] = from[r][c], columns cols ... padded - 1 are 0 (16-bit elements); rows 0
// for nothing to lay out.
struct PadRows {
    const void* from;
    void* to;
    int64_t ld, padded, rows, cols;
};

// Rows that start and end on 16 bytes, in a buffer whose tiles 32 bits address.
inline bool whole_chunks(const void* p, int64_t ld, int64_t rows, int64_t cols) {
    return (uintptr_t)p % 16 == 0 && cols % 8 == 0 &&
           ((ld % 8 == 0 && ld <= kMaxFeatures) || rows <= 1);
}

// Rows that a product that takes operands anywhere takes as they are.
inline bool any_rows(int64_t ld, int64_t rows, int64_t cols) {
    return cols >= 8 && (ld <= kMaxFeatures || rows <= 1);
}

inline ProductIn as_it_is(const void* p, int64_t ld, int64_t rows, int64_t cols) {
    return ProductIn{p, rows <= 1 ? padded(cols) : ld, cols, 0};
}

// The operand as the product reads it; `anew` says how it is laid out at `room`
// first, if need be, `any` that its rows are not whole chunks.
inline ProductIn operand(const void* p, int64_t ld, int64_t rows, int64_t cols, char* room,
                         bool takes_any, PadRows& anew, bool& any) {
    anew = PadRows{};
    if (rows == 0 || cols == 0 || whole_chunks(p, ld, rows, cols))
        return as_it_is(p, ld, rows, cols);
    if (takes_any && any_rows(ld, rows, cols)) {
        any = true;
        return as_it_is(p, ld, rows, cols);
    }
    anew = PadRows{p, room, ld, padded(cols), rows, cols};
    return ProductIn{room, padded(cols), padded(cols), 0};
}

// What the backward pass's products read: dx from dz and w, dw from dz and x.
struct GradShape {
    const void *dy, *x, *w;
    int64_t M, N, K, ld_dy, ld_x, ld_w;
    bool act, two_parts, want_dx, want_dw;
    bool dx_takes_any, dw_takes_any;
    char *x_room, *w_room, *dz_room;
};

struct GradIn {
    bool dz_anew;  // dz is written to dz_room first (its parts one behind the other)
    ProductIn dz, x, w;
    PadRows x_anew, w_anew;
    bool dx_any, dw_any;
};

inline GradIn grad_operands(const GradShape& s) {
    GradIn g = {};
    // dz is laid out anew for the activation, or where a product does not take it
    const bool chunks = s.M == 0 || s.N == 0 || whole_chunks(s.dy, s.ld_dy, s.M, s.N);
    g.dz_anew = (s.want_dx || s.want_dw) && s.M > 0 && s.N > 0 &&
                (s.act || (!chunks && (!any_rows(s.ld_dy, s.M, s.N) ||
                                       (s.want_dx && !s.dx_takes_any) ||
                                       (s.want_dw && !s.dw_takes_any))));
    const int64_t rest = s.two_parts ? 2 * s.M * padded(s.N) : 0;
    g.dz = g.dz_anew ? ProductIn{s.dz_room, padded(s.N), padded(s.N), rest}
                     : as_it_is(s.dy, s.ld_dy, s.M, s.N);
    g.dx_any = g.dw_any = !g.dz_anew && !chunks;
    if (s.want_dx)
        g.w = operand(s.w, s.ld_w, s.N, s.K, s.w_room, s.dx_takes_any, g.w_anew, g.dx_any);
    if (s.want_dw)
        g.x = operand(s.x, s.ld_x, s.M, s.K, s.x_room, s.dw_takes_any, g.x_anew, g.dw_any);
    return g;
}

}  // namespace onebit
