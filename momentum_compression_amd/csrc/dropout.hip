// Dropout whose mask is never stored: y = [residual +] (kept ? x * s : 0),
// with the mask of element (row, column) drawn from its own counter, so the
// backward pass (the same map applied to the gradient) draws it again.
//
// Bound by memory: 2 or 3 passes over the tensor.  A generator call is about 20
// wide multiplications for 8 elements, hidden behind the loads at 16 bits a
// draw (the same time with and without draws at 16384 x 4096).
//
// One lane takes 8 consecutive columns of a 2-byte type: one generator call,
// one 16-byte load and store.  Of binary32 a pair of lanes takes the 8 columns
// of two groups, each one half of both, so that an access of the wave is still
// one run; each draws for one group and they exchange half of their draws
// (16411 x 4099, three tensors in turn: 92 us, 5.8 TB/s; the same tensor over and
// over, part of which stays in the last cache, 79, with 8 columns a lane 93).
// With a residual, bf16, the same tensors over and over: 8192 x 1024 7.7 us (9.1
// in turn), 65536 x 4096 259 us (6.2 TB/s); two groups a lane took 7.3 and 278.
#include "philox.h"
#include "train.h"

namespace onebit {

namespace {

template <typename T, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const T* x, const T* r, T* y,
                                                          uint32_t groups, FastDiv per_row,
                                                          int64_t cols, int64_t ld_x, int64_t ld_r,
                                                          int64_t ld_y, uint64_t row0, DropArgs d) {
    const uint32_t step = d.step + (d.step_dev ? *d.step_dev : 0u);
    const uint32_t g = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
    if (g >= groups) return;
    const uint32_t row = per_row.div(g), cg = g - row * per_row.d;
    const int64_t c = 8 * (int64_t)cg;
    const bool whole = c + 8 <= cols;
    const T* xp = x + (int64_t)row * ld_x + c;
    const T* rp = RES ? r + (int64_t)row * ld_r + c : nullptr;
    Vec8<T> xv, rv = {};
    if (whole) {
        xv = load8(xp);
        if (RES) rv = load8(rp);
    } else {
        xv = load_tail(xp, cols - c);
        if (RES) rv = load_tail(rp, cols - c);
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (d.threshold != kDropAll) drop_draws(w, cg, row0 + row, step, d.k0, d.k1);
    float out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // a dropped element is 0 whatever it held (a select, not a product)
        const float k = drop_keep(w, e, d.threshold) ? (float)xv.v[e] * d.scale : 0.0f;
        out[e] = RES ? (float)rv.v[e] + k : k;
    }
    T* yp = y + (int64_t)row * ld_y + c;
    if (whole) {
        store8(yp, out);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (c + e < cols) yp[e] = (T)out[e];
    }
}

using f4u = float __attribute__((ext_vector_type(4), aligned(4)));

// The lane's neighbour's value (lanes 2 k and 2 k + 1).
__device__ __forceinline__ uint32_t pair_swap(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // [1,0,3,2]
}

template <bool RES>
__global__ __launch_bounds__(kThreads) void dropout_f32_kernel(
    const float* x, const float* r, float* y, uint32_t groups, FastDiv per_row, int64_t cols,
    int64_t ld_x, int64_t ld_r, int64_t ld_y, uint64_t row0, DropArgs d) {
    const uint32_t step = d.step + (d.step_dev ? *d.step_dev : 0u);
    const uint32_t odd = threadIdx.x & 1;
    f4 xv[2], rv[2];
    uint32_t row[2], cg[2];
    bool ok[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint32_t g = blockIdx.x * (uint32_t)kThreads + u * (kThreads / 2) + (threadIdx.x >> 1);
        ok[u] = g < groups;
        row[u] = per_row.div(g);
        cg[u] = g - row[u] * per_row.d;
        xv[u] = rv[u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        if (!ok[u]) continue;
        const int64_t c = 8 * (int64_t)cg[u] + 4 * odd;
        const float* xp = x + (int64_t)row[u] * ld_x + c;
        const float* rp = RES ? r + (int64_t)row[u] * ld_r + c : nullptr;
        if (c + 4 <= cols) {
            xv[u] = *reinterpret_cast<const f4u*>(xp);
            if (RES) rv[u] = *reinterpret_cast<const f4u*>(rp);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                if (c + e < cols) {
                    xv[u][e] = xp[e];
                    if (RES) rv[u][e] = rp[e];
                }
            }
        }
    }
    // every lane draws (past the last group too: its neighbour may not be)
    uint32_t w[4] = {0u, 0u, 0u, 0u}, got[2];
    if (d.threshold != kDropAll)
        drop_draws(w, odd ? cg[1] : cg[0], row0 + (odd ? row[1] : row[0]), step, d.k0, d.k1);
    got[0] = pair_swap(odd ? w[0] : w[2]);
    got[1] = pair_swap(odd ? w[1] : w[3]);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (!ok[u]) break;
        // the draws of this half: the group's own words, or the neighbour's
        const bool own = odd == (uint32_t)u;
        const uint32_t half[4] = {own ? w[2 * u] : got[0], own ? w[2 * u + 1] : got[1], 0u, 0u};
        f4 out;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float k = drop_keep(half, e, d.threshold) ? xv[u][e] * d.scale : 0.0f;
            out[e] = RES ? rv[u][e] + k : k;
        }
        const int64_t c = 8 * (int64_t)cg[u] + 4 * odd;
        float* yp = y + (int64_t)row[u] * ld_y + c;
        if (c + 4 <= cols) {
            __builtin_nontemporal_store(out, reinterpret_cast<f4u*>(yp));
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (c + e < cols) yp[e] = out[e];
        }
    }
}

template <bool RES>
void launch(const void* x, const void* r, void* y, int32_t dtype, uint32_t groups,
            const FastDiv& div, int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_y,
            uint64_t row0, const DropArgs& d, hipStream_t st) {
    const dim3 grid((groups + (uint32_t)kThreads - 1) / (uint32_t)kThreads);
    if (dtype == ONEBIT_F32)
        hipLaunchKernelGGL((dropout_f32_kernel<RES>), grid, dim3(kThreads), 0, st, (const float*)x,
                           (const float*)r, (float*)y, groups, div, cols, ld_x, ld_r, ld_y, row0,
                           d);
    else if (dtype == ONEBIT_BF16)
        hipLaunchKernelGGL((dropout_kernel<bf16, RES>), grid, dim3(kThreads), 0, st,
                           (const bf16*)x, (const bf16*)r, (bf16*)y, groups, div, cols, ld_x, ld_r,
                           ld_y, row0, d);
    else
        hipLaunchKernelGGL((dropout_kernel<f16, RES>), grid, dim3(kThreads), 0, st, (const f16*)x,
                           (const f16*)r, (f16*)y, groups, div, cols, ld_x, ld_r, ld_y, row0, d);
}

}  // namespace

hipError_t launch_dropout(const void* x, const void* residual, void* y, int32_t dtype, int64_t rows,
                          int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_y, int64_t row0,
                          float p, uint64_t seed, uint32_t step, const uint32_t* step_dev,
                          hipStream_t st) {
    const DropArgs d = drop_args(p, seed, step, step_dev);
    const int64_t per_row = (cols + 7) / 8;
    const uint32_t groups = (uint32_t)(rows * per_row);
    const FastDiv div((uint32_t)per_row);
    if (residual)
        launch<true>(x, residual, y, dtype, groups, div, cols, ld_x, ld_r, ld_y, (uint64_t)row0, d,
                     st);
    else
        launch<false>(x, nullptr, y, dtype, groups, div, cols, ld_x, 0, ld_y, (uint64_t)row0, d,
                      st);
    return hipGetLastError();
}

}  // namespace onebit
