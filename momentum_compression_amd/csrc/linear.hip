// Matrix products of 16-bit elements with an epilogue, on the matrix cores.
//
// out[r][c] = sum over k of R(r, k) C(c, k).  The columns' operand C is the
// matrix instruction's A, so that a lane's registers hold eight consecutive
// columns of one row of the result (16 bytes of it) when A's rows are read in
// perm_row() order.  Each operand comes with k contiguous (read as rows of the
// tile in LDS) or with its own index contiguous (read by transposing LDS reads),
// so the product of a layer and both of its gradients need no transposed copies.
#include "activation.h"
#include "attention.h"

namespace onebit {
namespace {

constexpr int kDeep = 64;  // of the summed index a tile

// Eight values of a row of the result, `n` of them inside.
template <typename S>
__device__ __forceinline__ void load_row8(float out[8], const S* p, int64_t n) {
    const Vec8<S> x = n >= 8 ? load8(p) : load_tail(p, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = (float)x.v[e];
}

template <typename S>
__device__ __forceinline__ void store_row8(S* p, const float v[8], int64_t n) {
    if (n >= 8) {
        Vec8<S> x;
#pragma unroll
        for (int e = 0; e < 8; ++e) x.v[e] = (S)v[e];
        *reinterpret_cast<Vec8<S>*>(p) = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) p[e] = (S)v[e];
}

// The epilogue for columns c ... c + 7 of row r.
template <typename S, typename T>
__device__ __forceinline__ void emit8(const ProductOut& o, int64_t r, int64_t c, float z[8]) {
    const int64_t n = o.cols - c;
    if (n <= 0) return;
    if (o.bias) {
        float b[8];
        if (o.bias_wide) load_row8(b, (const float*)o.bias + c, n);
        else load_row8(b, (const T*)o.bias + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += b[e];
    }
    if (o.pre) store_row8((S*)o.pre + r * o.ld_pre + c, z, n);
    if (o.act != ONEBIT_NONE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = activate(z[e], o.act);
    }
    if (o.residual) {
        float v[8];
        load_row8(v, (const S*)o.residual + r * o.ld_r + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += v[e];
    }
    S* to = (S*)o.out + r * o.ld + c;
    if (o.accumulate) {
        float v[8];
        load_row8(v, (const S*)to, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += v[e];
    }
    store_row8(to, z, n);
}

// One operand's tiles, memory to LDS without registers between.  By rows: TILE
// rows of kDeep elements, laid out as tile_at<64>; otherwise kDeep rows of TILE
// elements, with the 16-byte chunks of a row xored as in tile_at<128>.  What lies
// past the matrix reads as 0: such chunks get an offset past the buffer's end.
template <typename T, bool ROWS, int TILE, int WAVES>
struct Operand {
    static constexpr int kChunks = ROWS ? kDeep / 8 : TILE / 8;  // of a row in LDS
    static constexpr int kRowsAtOnce = 64 / kChunks * WAVES;
    static constexpr int kPer = TILE * kDeep * 2 / (1024 * WAVES);
    static constexpr int kBytes = TILE * kDeep * 2;
    const char* base;
    uint32_t stride, at;  // in bytes
    int32_t count;        // rows (by rows), else columns from `first` on
    int32_t mine;         // by rows: the lane's first k in a tile

    static __device__ __forceinline__ int swizzled(int row, int chunk) {
        return ROWS ? chunk ^ swizzle<64>(row)
                    : TILE == 64 ? chunk ^ swizzle<64>(row) : chunk ^ swizzle<128>(row);
    }
    __device__ __forceinline__ Operand(const ProductIn& in, int64_t first, int64_t extent, int wave,
                                       int lane) {
        const int row = wave * (64 / kChunks) + lane / kChunks;
        const int chunk = swizzled(row, lane % kChunks);  // the same kRowsAtOnce rows on
        stride = (uint32_t)in.ld * 2;
        const int64_t left = extent - first;
        count = left < TILE ? (int32_t)left : TILE;
        base = (const char*)in.p + (ROWS ? first * in.ld * 2 : first * 2);
        at = (uint32_t)row * stride + 16 * chunk;
        mine = 8 * chunk;
        if (!ROWS && 8 * chunk >= count) at = 0x80000000u;
    }
    __device__ __forceinline__ void load(char* tile, int64_t k0, int64_t depth, int wave) const {
        const int64_t left = depth - k0;
        const char* from = base + (ROWS ? k0 * 2 : k0 * stride);
        const int32_t deep = left < kDeep ? (int32_t)left : kDeep;
        // rows are made of whole chunks
        const uint32_t bytes =
            deep <= 0 ? 0u
            : ROWS    ? (uint32_t)(count - 1) * stride + (uint32_t)((deep + 7) & ~7) * 2
                      : (uint32_t)(deep - 1) * stride + (uint32_t)((count + 7) & ~7) * 2;
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc((void*)from, 0, (int)bytes, 0x00027000);
        const uint32_t off = ROWS && mine >= deep ? 0x80000000u : at;
#pragma unroll
        for (int x = 0; x < kPer; ++x)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc,
                (__attribute__((address_space(3))) void*)(tile + (x * WAVES + wave) * 1024), 16,
                (int)(off + (uint32_t)(x * kRowsAtOnce) * stride), 0, 0, 0);
    }
    // 32 of the operand's index from `first` on, k from 16 kc on; PERM: the
    // order of perm_row().
    template <bool PERM>
    static __device__ __forceinline__ typename Mma<T>::x8 frag(const char* tile, int first, int kc,
                                                               int lane) {
        if (ROWS) {
            const int row = first + (PERM ? perm_row(lane & 31) : lane & 31);
            return *reinterpret_cast<const typename Mma<T>::x8*>(
                tile + row * (kDeep * 2) + (swizzled(row, 2 * kc + (lane >> 5)) << 4));
        }
        // of 16 lanes, lane i reads four elements of k row i / 4; swapping the
        // middle two groups of four permutes what the lanes get
        const int i = lane & 15;
        const int group = PERM ? ((i & 1) << 1) | ((i >> 1) & 1) : i & 3;
        const int row = 16 * kc + 8 * (lane >> 5) + (i >> 2);
        const int chunk = first / 8 + 2 * ((lane >> 4) & 1) + (group >> 1);
        const auto lo = read_tr<T>(tile + row * (TILE * 2) + (swizzled(row, chunk) << 4) +
                                   8 * (group & 1));
        const auto hi = read_tr<T>(tile + (row + 4) * (TILE * 2) + (swizzled(row + 4, chunk) << 4) +
                                   8 * (group & 1));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

struct ProductArgs {
    ProductIn a, b;       // columns' and rows' operand
    ProductOut out;
    float* parts;         // [splits][rows][cols padded] of a divided sum, or nullptr
    int64_t depth, padded;
    int32_t tiles_a, tiles_b, splits;
};

// WA x WB waves of TILE x TILE results.
template <typename T, typename S, bool A_ROWS, bool B_ROWS, int TILE, int WA, int WB>
__global__ __launch_bounds__(64 * WA * WB) void product_kernel(ProductArgs p) {
    constexpr int waves = WA * WB, na = TILE / WA / 32, nb = TILE / WB / 32;
    using A = Operand<T, A_ROWS, TILE, waves>;
    using B = Operand<T, B_ROWS, TILE, waves>;
    extern __shared__ __align__(16) char lds[];
    const int wave = wave_id(), lane = lane_id();
    const int wa = wave % WA, wb = wave / WA;
    const uint32_t tiles = (uint32_t)p.tiles_a * p.tiles_b;
    const uint32_t tile = blockIdx.x % tiles, split = blockIdx.x / tiles;
    const int64_t a0 = (int64_t)(tile % p.tiles_a) * TILE, b0 = (int64_t)(tile / p.tiles_a) * TILE;
    const int64_t steps = (p.depth + kDeep - 1) / kDeep;
    const int64_t first = steps * split / p.splits, last = steps * (split + 1) / p.splits;
    const A as(p.a, a0, p.out.cols, wave, lane);
    const B bs(p.b, b0, p.out.rows, wave, lane);
    f32x16 acc[na][nb];
#pragma unroll
    for (int i = 0; i < na; ++i)
#pragma unroll
        for (int j = 0; j < nb; ++j) acc[i][j] = f32x16{};
    if (first < last) {
        as.load(lds, first * kDeep, p.depth, wave);
        bs.load(lds + A::kBytes, first * kDeep, p.depth, wave);
    }
    int buf = 0;
    for (int64_t s = first; s < last; ++s, buf ^= 1) {
        const char* at = lds + buf * (A::kBytes + B::kBytes);
        const char* bt = at + A::kBytes;
        tiles_barrier();  // this tile is there, and the other buffer is read
        if (s + 1 < last) {
            char* next = lds + (buf ^ 1) * (A::kBytes + B::kBytes);
            as.load(next, (s + 1) * kDeep, p.depth, wave);
            bs.load(next + A::kBytes, (s + 1) * kDeep, p.depth, wave);
        }
#pragma unroll
        for (int kc = 0; kc < kDeep / 16; ++kc) {
            typename Mma<T>::x8 af[na], bf[nb];
#pragma unroll
            for (int i = 0; i < na; ++i)
                af[i] = A::template frag<true>(at, wa * (TILE / WA) + 32 * i, kc, lane);
#pragma unroll
            for (int j = 0; j < nb; ++j)
                bf[j] = B::template frag<false>(bt, wb * (TILE / WB) + 32 * j, kc, lane);
#pragma unroll
            for (int i = 0; i < na; ++i)
#pragma unroll
                for (int j = 0; j < nb; ++j) acc[i][j] = Mma<T>::mul(af[i], bf[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int j = 0; j < nb; ++j) {
        const int64_t r = b0 + wb * (TILE / WB) + 32 * j + (lane & 31);
        if (r >= p.out.rows) continue;
#pragma unroll
        for (int i = 0; i < na; ++i)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int64_t c = a0 + wa * (TILE / WA) + 32 * i + 16 * g + 8 * (lane >> 5);
                if (c >= p.out.cols) continue;
                float z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = acc[i][j][8 * g + e];
                if (!p.parts) {
                    emit8<S, T>(p.out, r, c, z);
                } else {
                    float* to = p.parts + ((int64_t)split * p.out.rows + r) * p.padded + c;
                    *reinterpret_cast<f4*>(to) = f4{z[0], z[1], z[2], z[3]};
                    *reinterpret_cast<f4*>(to + 4) = f4{z[4], z[5], z[6], z[7]};
                }
            }
    }
}

// Adds the parts of a divided sum in their order and finishes.
template <typename T, typename S>
__global__ __launch_bounds__(kThreads) void product_join_kernel(ProductArgs p) {
    const int64_t groups = p.padded / 8;
    const int64_t all = p.out.rows * groups, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += step) {
        const int64_t r = i / groups, c = (i % groups) * 8;
        float z[8] = {};
        for (int32_t s = 0; s < p.splits; ++s) {
            const float* from = p.parts + ((int64_t)s * p.out.rows + r) * p.padded + c;
            const f4 lo = *reinterpret_cast<const f4*>(from);
            const f4 hi = *reinterpret_cast<const f4*>(from + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[e] += lo[e];
                z[4 + e] += hi[e];
            }
        }
        emit8<S, T>(p.out, r, c, z);
    }
}

// ---------------------------------------------------------------- operands laid out anew
__global__ __launch_bounds__(kThreads) void pad_rows_kernel(const uint16_t* from, int64_t ld,
                                                            uint16_t* to, int64_t padded,
                                                            int64_t rows, int64_t cols) {
    const int64_t groups = padded / 8, all = rows * groups;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / groups, c = (i % groups) * 8;
        const uint16_t* p = from + r * ld + c;
        const Vec8<uint16_t> x = c + 8 <= cols ? load8(p) : load_tail(p, cols - c);
        *reinterpret_cast<Vec8<uint16_t>*>(to + r * padded + c) = x;
    }
}

// ---------------------------------------------------------------- the activation's slope
// A thread has eight columns of a part of the rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void slope_kernel(SlopeArgs a, int64_t groups,
                                                         int64_t rows_of_part) {
    const int64_t strips = (groups + kThreads - 1) / kThreads;
    const int64_t c = 8 * ((int64_t)(blockIdx.x % strips) * kThreads + threadIdx.x);
    const int64_t part = blockIdx.x / strips, n = a.cols - c;
    if (n <= 0) return;
    const int64_t end = (part + 1) * rows_of_part < a.rows ? (part + 1) * rows_of_part : a.rows;
    float sums[8] = {};
    for (int64_t r = part * rows_of_part; r < end; ++r) {
        float d[8];
        load_row8(d, (const T*)a.dy + r * a.ld_dy + c, n);
        if (a.act != ONEBIT_NONE) {
            float z[8];
            load_row8(z, (const T*)a.pre + r * a.ld_pre + c, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = d[e] * slope(z[e], a.act);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[e] += d[e];
        if (a.dz) {
            // the rest of the last group is zeros
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = e < n ? d[e] : 0.0f;
            store_row8((T*)a.dz + r * a.padded + c, d, 8);
        }
    }
    if (!a.partials) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) a.partials[part * a.cols + c + e] = sums[e];
}

constexpr int kTileBig = 256, kTileSmall = 128;

template <typename T, typename S, bool A_ROWS, bool B_ROWS>
void launch_tiles(const ProductArgs& p, int32_t tile, hipStream_t st) {
    const unsigned grid = (unsigned)((int64_t)p.tiles_a * p.tiles_b * p.splits);
    if (tile == kTileBig)
        hipLaunchKernelGGL((product_kernel<T, S, A_ROWS, B_ROWS, kTileBig, 2, 4>), dim3(grid),
                           dim3(512), 4 * kTileBig * kDeep * 2, st, p);
    else
        hipLaunchKernelGGL((product_kernel<T, S, A_ROWS, B_ROWS, kTileSmall, 2, 2>), dim3(grid),
                           dim3(256), 4 * kTileSmall * kDeep * 2, st, p);
    if (p.parts) {
        const int64_t groups = (p.out.rows * (p.padded / 8) + kThreads - 1) / kThreads;
        hipLaunchKernelGGL((product_join_kernel<T, S>), dim3((unsigned)(groups < 4096 ? groups : 4096)),
                           dim3(kThreads), 0, st, p);
    }
}

template <typename T, typename S>
void launch_operands(const ProductArgs& p, bool a_rows, bool b_rows, int32_t tile,
                     hipStream_t st) {
    if (a_rows) launch_tiles<T, S, true, true>(p, tile, st);
    else if (b_rows) launch_tiles<T, S, false, true>(p, tile, st);
    else launch_tiles<T, S, false, false>(p, tile, st);
}

template <typename T>
void launch_typed(const ProductArgs& p, bool a_rows, bool b_rows, int32_t tile, hipStream_t st) {
    if (p.out.type == ONEBIT_F32) launch_operands<T, float>(p, a_rows, b_rows, tile, st);
    else launch_operands<T, T>(p, a_rows, b_rows, tile, st);
}

int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

}  // namespace

ProductPlan product_plan(int64_t rows, int64_t cols, int64_t depth) {
    ProductPlan plan;
    const int64_t big = tiles_of(rows, kTileBig) * tiles_of(cols, kTileBig);
    plan.tile = big >= 256 ? kTileBig : kTileSmall;
    const int64_t tiles = tiles_of(rows, plan.tile) * tiles_of(cols, plan.tile);
    const int64_t steps = tiles_of(depth, kDeep);
    int64_t splits = tiles > 0 ? 256 / tiles : 1;
    if (splits > steps / 4) splits = steps / 4;
    plan.splits = (int32_t)(splits < 1 ? 1 : splits);
    plan.bytes = plan.splits > 1
                     ? (size_t)plan.splits * rows * ((cols + 7) / 8 * 8) * sizeof(float)
                     : 0;
    return plan;
}

hipError_t launch_product(int32_t dtype, const ProductIn& cols_in, bool cols_by_rows,
                          const ProductIn& rows_in, bool rows_by_rows, int64_t depth,
                          const ProductOut& out, float* parts, hipStream_t st) {
    if (out.rows == 0 || out.cols == 0) return hipSuccess;
    const ProductPlan plan = product_plan(out.rows, out.cols, depth);
    ProductArgs p = {};
    p.a = cols_in;
    p.b = rows_in;
    p.out = out;
    p.parts = plan.splits > 1 ? parts : nullptr;
    p.depth = depth;
    p.padded = (out.cols + 7) / 8 * 8;
    p.tiles_a = (int32_t)tiles_of(out.cols, plan.tile);
    p.tiles_b = (int32_t)tiles_of(out.rows, plan.tile);
    p.splits = plan.splits;
    if (dtype == ONEBIT_BF16) launch_typed<bf16>(p, cols_by_rows, rows_by_rows, plan.tile, st);
    else launch_typed<f16>(p, cols_by_rows, rows_by_rows, plan.tile, st);
    return hipGetLastError();
}

hipError_t launch_pad_rows(const void* from, int64_t ld, void* to, int64_t padded, int64_t rows,
                           int64_t cols, hipStream_t st) {
    const int64_t groups = (rows * (padded / 8) + kThreads - 1) / kThreads;
    if (groups == 0) return hipSuccess;
    hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)(groups < 8192 ? groups : 8192)),
                       dim3(kThreads), 0, st, (const uint16_t*)from, ld, (uint16_t*)to, padded,
                       rows, cols);
    return hipGetLastError();
}

int64_t slope_parts(int64_t rows, int64_t cols) {
    const int64_t strips = tiles_of(tiles_of(cols, 8), kThreads);
    int64_t parts = strips > 0 ? 2048 / strips : 1;
    if (parts > tiles_of(rows, 4)) parts = tiles_of(rows, 4);
    return parts < 1 ? 1 : parts;
}

hipError_t launch_slope(const SlopeArgs& a, hipStream_t st) {
    const int64_t groups = tiles_of(a.cols, 8), strips = tiles_of(groups, kThreads);
    const int64_t parts = slope_parts(a.rows, a.cols);
    const dim3 grid((unsigned)(strips * parts)), block(kThreads);
    const int64_t rows_of_part = tiles_of(a.rows, parts);
    if (a.dtype == ONEBIT_BF16)
        hipLaunchKernelGGL((slope_kernel<bf16>), grid, block, 0, st, a, groups, rows_of_part);
    else
        hipLaunchKernelGGL((slope_kernel<f16>), grid, block, 0, st, a, groups, rows_of_part);
    return hipGetLastError();
}

}  // namespace onebit
