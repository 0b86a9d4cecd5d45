// Every address that the products of a linear layer read of operands whose rows are
// not whole 16-byte chunks, for small sizes and many layouts: inside the rows of the
// caller's matrix, or of the part of the workspace that the operand is laid out in.
#include <cstdio>
#include <initializer_list>

#include "operands.h"

using namespace onebit;

static long reads = 0, wrong = 0;
static char what[200];
static const int64_t pads[] = {0, 1, 8};

// One operand of `count` by `depth` (the product's index by the summed one), in tiles
// of `tile` by 64, as the kernels' lanes ask for its pieces.
static void walk(const ProductIn& in, bool by_rows, int64_t count, int64_t depth, int tile,
                 int64_t real, const char* room, const char* name) {
    const bool anew = in.p == room;
    const int64_t extent = anew ? padded(real) : real;
    const int64_t rows = by_rows ? count : depth;
    for (int64_t first = 0; first < count; first += tile)
        for (int64_t k0 = 0; k0 < depth + 3 * 64; k0 += 64)
            for (int r = 0; r < (by_rows ? tile : 64); ++r)
                for (int mine = 0; mine < (by_rows ? 64 : tile); mine += 8) {
                    const int64_t row = (by_rows ? first : k0) + r;
                    const int64_t at = (by_rows ? k0 : first) + mine;
                    const int32_t over = past_end(at, in.row);
                    if (over >= 8 || row >= rows) continue;
                    ++reads;
                    const int64_t from = at - over;
                    if (from >= 0 && from + 8 <= extent && (rows <= 1 || in.ld >= extent)) continue;
                    if (wrong++ == 0)
                        printf("%s: %s row %ld elements %ld ... %ld of %ld\n", what, name, (long)row,
                               (long)from, (long)from + 7, (long)extent);
                }
}

int main() {
    static char rooms[3][1 << 16];
    static char mem[3][1 << 16];
    auto on16 = [](char* p) { return p + (16 - (uintptr_t)p % 16) % 16; };
    char *xr = on16(rooms[0]), *wr = on16(rooms[1]), *zr = on16(rooms[2]);
    long taken = 0;
    for (int64_t M : {1, 8, 33, 70})
        for (int64_t N = 1; N <= 29; ++N)
            for (int64_t K : {1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 24, 29})
                for (int layout = 0; layout < 27; ++layout)
                    for (int how = 0; how < 32; ++how) {
                        const int d = layout % 3, a = layout / 3 % 3, b = layout / 9;
                        // what is padded by one starts on no 16 bytes
                        GradShape s = {on16(mem[0]) + 2 * (d == 1), on16(mem[1]) + 2 * (a == 1),
                                       on16(mem[2]) + 2 * (b == 1), M, N, K, N + pads[d],
                                       K + pads[a], K + pads[b], (how & 1) != 0, false, (how & 2) != 0, (how & 4) != 0,
                                       (how & 8) != 0, (how & 16) != 0, xr, wr, zr};
                        const GradIn g = grad_operands(s);
                        snprintf(what, sizeof(what), "M %ld N %ld K %ld layout %d how %d", (long)M,
                                 (long)N, (long)K, layout, how);
                        if (s.want_dx && g.dx_any) {
                            ++taken;
                            walk(g.dz, true, M, N, 64, N, zr, "dx dz");
                            walk(g.w, false, K, N, 128, K, wr, "dx w");
                        }
                        if (s.want_dw && g.dw_any) {
                            ++taken;
                            walk(g.dz, false, N, M, 128, N, zr, "dw dz");
                            walk(g.x, false, K, M, 128, K, xr, "dw x");
                        }
                        // operands that are read by whole chunks
                        for (const ProductIn* in : {&g.dz, &g.w, &g.x}) {
                            const bool dx = s.want_dx && !g.dx_any && in != &g.x;
                            const bool dw = s.want_dw && !g.dw_any && in != &g.w;
                            if (!dx && !dw) continue;
                            if ((uintptr_t)in->p % 16 || in->ld % 8)
                                if (wrong++ == 0) printf("%s: not whole chunks\n", what);
                        }
                    }
    // the forward product: both operands by rows
    for (int64_t M : {33, 64, 70})
        for (int64_t N = 1; N <= 29; N += 7)
            for (int64_t K = 1; K <= 140; ++K)
                for (int layout = 0; layout < 9; ++layout)
                    for (bool takes : {false, true}) {
                        const int a = layout % 3, b = layout / 3;
                        PadRows anew;
                        bool any = false;
                        const ProductIn x = operand(on16(mem[1]) + 2 * (a == 1), K + pads[a], M, K,
                                                    xr, takes, anew, any);
                        const ProductIn w = operand(on16(mem[2]) + 2 * (b == 1), K + pads[b], N, K,
                                                    wr, takes, anew, any);
                        snprintf(what, sizeof(what), "forward M %ld N %ld K %ld layout %d", (long)M,
                                 (long)N, (long)K, layout);
                        if (!any) continue;
                        ++taken;
                        walk(x, true, M, K, 64, K, xr, "x");
                        walk(w, true, N, K, 128, K, wr, "w");
                    }
    printf("%ld products, %ld reads, %ld outside\n", taken, reads, wrong);
    return wrong ? 1 : taken && reads ? 0 : 2;
}
