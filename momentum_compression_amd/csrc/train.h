// Element types, unaligned vectors and the row-group split shared by the
// kernels that work beside the optimizer (dropout, position bias, attention).
#pragma once

#include "common.h"

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

}  // namespace onebit
