// Element types, unaligned vectors and the row-group split shared by the
// kernels that work beside the optimizer (dropout, position bias, attention).
#pragma once

#include "common.h"
#include "operands.h"

namespace onebit {

using bf16 = __bf16;
using f16 = _Float16;

// Eight consecutive elements, loaded and stored whole at any element address
// (global memory takes a 16-byte access at any alignment).
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Vec8 {
    T v[8];
};

template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
    return *reinterpret_cast<const Vec8<T>*>(p);
}

// The first n < 8 of eight elements; the others 0.
template <typename T>
__device__ __forceinline__ Vec8<T> load_tail(const T* p, int64_t n) {
    Vec8<T> x = {};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) x.v[e] = p[e];
    return x;
}

// Whole 32-bit words go out: stores of single elements would be merged with
// those of a partial group and split the access.  Past the caches: what a pass
// over a tensor writes is not read by it (dropout with a residual over 16384 x
// 4096 bf16: 74 -> 57 us; loads stay cached, past the caches 65).
template <typename T>
__device__ __forceinline__ void store8(T* p, const float in[8]) {
    constexpr int words = 8 * sizeof(T) / 4;
    typedef uint32_t Words __attribute__((ext_vector_type(words), aligned(sizeof(T))));
    T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (T)in[e];
    __builtin_nontemporal_store(__builtin_bit_cast(Words, x), reinterpret_cast<Words*>(p));
}

// Division of a 32-bit number by one fixed divisor: a multiplication's high
// half and two shifts (the round-up reciprocal with its 33rd bit implied).
struct FastDiv {
    uint32_t d, mul, s1, s2;
    explicit FastDiv(uint32_t div = 1) : d(div) {
        uint32_t l = 0;
        while (l < 32 && ((uint64_t)1 << l) < div) ++l;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - div)) / div + 1);
        s1 = l < 1 ? l : 1;
        s2 = l < 1 ? 0 : l - 1;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        const uint32_t t = __umulhi(n, mul);
        return (t + ((n - t) >> s1)) >> s2;
    }
};

// Largest distance that keeps a bias value of its own.
constexpr int32_t kMaxRadius = 1024;
constexpr int32_t kMaxBuckets = 1024;

hipError_t launch_dropout(const void* x, const void* residual, void* y, int32_t dtype, int64_t rows,
                          int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_y, int64_t row0,
                          float p, uint64_t seed, uint32_t step, const uint32_t* step_dev,
                          hipStream_t st);

struct RelBias {
    const float* table;    // [n_buckets][H]
    const int32_t* map;    // [2 radius + 1]
    int32_t n_buckets, radius, H;
};

hipError_t launch_rel_bias(const RelBias& b, void* out, int32_t dtype, int32_t Tq, int32_t Tk,
                           int32_t q_pos, hipStream_t st);

// Bias gradient: workgroups of a head (their partial sums are the workspace).
struct BiasGradPlan {
    int32_t row_blocks;   // blocks of rows of the score map
    int32_t rows;         // rows of a block
    int32_t col_blocks;   // segments of columns
    int32_t batches;      // sequences of one workgroup
    int32_t batch_blocks;
    int64_t parts() const { return (int64_t)row_blocks * col_blocks * batch_blocks; }
};
BiasGradPlan bias_grad_plan(int32_t B, int32_t H, int32_t Tq, int32_t Tk, int32_t dtype);

hipError_t launch_rel_bias_grad(const void* ds, int32_t dtype, const int32_t* map, float* dtable,
                                int32_t B, int32_t H, int32_t n_buckets, int32_t radius,
                                int32_t Tq, int32_t Tk, int32_t q_pos, bool accumulate,
                                float* partials, hipStream_t st);

// Joins per-workgroup distance sums [H][parts][2 radius + 1] into the table's
// gradient.
hipError_t launch_bias_join(const float* partials, const int32_t* map, float* dtable, int32_t H,
                            int64_t parts, int32_t n_buckets, int32_t radius, bool accumulate,
                            hipStream_t st);

// ---------------------------------------------------------------- layer norm
struct NormArgs {
    const void *x, *dy;
    void *y, *dx;            // dx may be nullptr
    const void *weight, *bias;  // or nullptr
    float *mean, *rstd;      // [rows]; outputs of the forward pass, or nullptr
    float* partials;         // [norm_parts][2][cols] of the backward pass, or nullptr
    int64_t rows, cols, ld_x, ld_y, ld_dy, ld_dx;
    float eps;
    int32_t dtype;
    bool w_wide;             // weight and bias are binary32
};

// Workgroups whose sums over rows the backward pass joins.
int64_t norm_parts(int64_t rows, int64_t cols);

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st);
hipError_t launch_layer_norm_grad(const NormArgs& a, float* dweight, float* dbias, bool accumulate,
                                  hipStream_t st);

// Sums partials [parts][n] over the parts; the first `cols` columns go to out0,
// the others to out1 (either may be nullptr).
hipError_t launch_column_join(const float* partials, int64_t parts, int64_t n, int64_t cols,
                              float* out0, float* out1, bool accumulate, hipStream_t st);

// ---------------------------------------------------------------- AdamW
// Elements of a workgroup (2048, 4096, 8192: 302 tensors in 8 bits 894, 925, 953 us).
constexpr int64_t kAdamWTile = 2048;
constexpr int64_t kStateBlock = 256;  // elements that share a scale of the 8-bit states

// A tensor in the plan that the kernel reads.
struct AdamWTensor {
    float* x;
    const void* g;
    void* copy;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    int64_t first_tile;
    float lr_scale, weight_decay;
};

struct AdamWArgs {
    const AdamWTensor* tensors;
    const int32_t* tensor_of;   // [tiles]
    int64_t tiles;
    const float* g_scale;       // or nullptr
    float lr, beta1, beta2, eps;
    float rate, root;           // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    uint32_t k0, k1, step;      // of the rounding draws
};

hipError_t launch_adamw(const AdamWArgs& a, int32_t state_bits, int32_t g_dtype, int32_t copy_dtype,
                        hipStream_t st);

// ---------------------------------------------------------------- matrix products
// Where a product's sums go: [rows][cols] of `type`, through
//   z = sum + bias[col];  pre = z;  out = (accumulate ? out : 0) + act(z) + residual
struct ProductOut {
    void* out;
    const void *bias, *residual;  // or nullptr
    void* pre;                    // or nullptr
    int64_t rows, cols, ld, ld_r, ld_pre;
    int32_t type;                 // of out, residual and pre
    int32_t act;
    bool bias_wide;               // bias is binary32
    bool accumulate;
};

// How a product is divided: tiles of tile_a columns by tile_b rows of the result,
// the sum over `splits` parts.
struct ProductPlan {
    int32_t tile_a, tile_b;
    int32_t splits;
    size_t bytes;  // workspace of the parts
};
ProductPlan product_plan(int64_t rows, int64_t cols, int64_t depth, bool cols_by_rows,
                         bool rows_by_rows);

// The summed index's extent with an operand of two parts.
int64_t product_depth(int64_t depth, bool two);

// Whether the division's kernels take operands that lie anywhere; the larger tiles,
// whose work is worth a copy of the operands, take rows of whole 16-byte chunks.
bool product_any(const ProductPlan& plan);

// out[r][c] = sum over k < depth of rows_in(r, k) cols_in(c, k).  The operand
// types: by_rows says whether k is the contiguous index.  (cols_in, rows_in) is
// (true, true), (false, true) or (false, false).  Contiguous indices and strides
// are multiples of 8 and the addresses of 16 bytes; with `any` (product_any)
// contiguous rows have 8 elements or more, and others are refused.
hipError_t launch_product(int32_t dtype, const ProductIn& cols_in, bool cols_by_rows,
                          const ProductIn& rows_in, bool rows_by_rows, int64_t depth,
                          const ProductOut& out, bool any, float* parts, hipStream_t st);

// Whether a product of both operands by rows goes by launch_product_few, for which
// they may lie anywhere.
bool product_few(int64_t rows);
hipError_t launch_product_few(int32_t dtype, const ProductIn& cols_in, const ProductIn& rows_in,
                              int64_t depth, const ProductOut& out, hipStream_t st);

// Two matrices in one launch.
hipError_t launch_pad_rows(const PadRows& one, const PadRows& two, hipStream_t st);

// Whether dz is a number of the element type.
constexpr bool slope_exact(int32_t act) { return act == ONEBIT_NONE || act == ONEBIT_RELU; }

// dz = dy act'(pre) into `dz` (rows of `padded` elements, zeros at their end) where
// given, rounded to the element type or, with `rest` bytes to the second, in two parts
// of it, and its unrounded sums over parts of the rows into partials
// [slope_parts][cols] where given.
struct SlopeArgs {
    const void *dy, *pre;
    void* dz;
    float* partials;
    int64_t rows, cols, ld_dy, ld_pre, padded, rest;
    int32_t act, dtype;
};
int64_t slope_parts(int64_t rows, int64_t cols);
hipError_t launch_slope(const SlopeArgs& a, hipStream_t st);

}  // namespace onebit
