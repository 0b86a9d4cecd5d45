// Dropout whose mask is never stored: y = [residual +] (kept ? x * s : 0),
// with the mask of element (row, column) drawn from its own counter, so the
// backward pass (the same map applied to the gradient) draws it again.
//
// One lane takes 8 consecutive columns: one generator call, one 16-byte load
// and store of 2-byte types.  Bound by memory: 2 or 3 passes over the tensor.
// A generator call is about 20 wide multiplications for 8 elements, which at
// 2 bytes an element is close to what the same time moves (16-bit draws keep
// it below).
#include "philox.h"
#include "train.h"

namespace onebit {

namespace {

constexpr int kGroups = 2;  // groups of 8 columns per lane, loads first

template <typename T, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const T* x, const T* r, T* y,
                                                          uint32_t groups, FastDiv per_row,
                                                          int64_t cols, int64_t ld_x, int64_t ld_r,
                                                          int64_t ld_y, uint64_t row0, DropArgs d) {
    const uint32_t step = d.step + (d.step_dev ? *d.step_dev : 0u);
    const uint32_t first = blockIdx.x * (uint32_t)(kThreads * kGroups) + threadIdx.x;
    Vec8<T> xv[kGroups], rv[kGroups];
    uint32_t row[kGroups], cg[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        const uint32_t g = first + (uint32_t)(u * kThreads);
        row[u] = cg[u] = 0;
        xv[u] = rv[u] = Vec8<T>{};
        if (g >= groups) continue;
        row[u] = per_row.div(g);
        cg[u] = g - row[u] * per_row.d;
        const int64_t c = 8 * (int64_t)cg[u];
        const T* xp = x + (int64_t)row[u] * ld_x + c;
        const T* rp = RES ? r + (int64_t)row[u] * ld_r + c : nullptr;
        if (c + 8 <= cols) {
            xv[u] = load8(xp);
            if (RES) rv[u] = load8(rp);
        } else {
            xv[u] = load_tail(xp, cols - c);
            if (RES) rv[u] = load_tail(rp, cols - c);
        }
    }
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        const uint32_t g = first + (uint32_t)(u * kThreads);
        if (g >= groups) break;
        float out[8];
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (d.threshold != kDropAll) drop_draws(w, cg[u], row0 + row[u], step, d.k0, d.k1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // a dropped element is 0 whatever it held (a select, not a product)
            const float k = drop_keep(w, e, d.threshold) ? (float)xv[u].v[e] * d.scale : 0.0f;
            out[e] = RES ? (float)rv[u].v[e] + k : k;
        }
        const int64_t c = 8 * (int64_t)cg[u];
        T* yp = y + (int64_t)row[u] * ld_y + c;
        if (c + 8 <= cols) {
            store8(yp, out);
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (c + e < cols) yp[e] = (T)out[e];
        }
    }
}

template <typename T>
hipError_t launch(const void* x, const void* r, void* y, int64_t rows, int64_t cols, int64_t ld_x,
                  int64_t ld_r, int64_t ld_y, int64_t row0, const DropArgs& d, hipStream_t st) {
    const int64_t per_row = (cols + 7) / 8;
    const uint32_t groups = (uint32_t)(rows * per_row);
    const dim3 grid((groups + (uint32_t)(kThreads * kGroups) - 1) / (uint32_t)(kThreads * kGroups));
    const FastDiv div((uint32_t)per_row);
    if (r)
        hipLaunchKernelGGL((dropout_kernel<T, true>), grid, dim3(kThreads), 0, st, (const T*)x,
                           (const T*)r, (T*)y, groups, div, cols, ld_x, ld_r, ld_y, (uint64_t)row0,
                           d);
    else
        hipLaunchKernelGGL((dropout_kernel<T, false>), grid, dim3(kThreads), 0, st, (const T*)x,
                           (const T*)nullptr, (T*)y, groups, div, cols, ld_x, (int64_t)0, ld_y,
                           (uint64_t)row0, d);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, const void* residual, void* y, int32_t dtype, int64_t rows,
                          int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_y, int64_t row0,
                          float p, uint64_t seed, uint32_t step, const uint32_t* step_dev,
                          hipStream_t st) {
    const DropArgs d = drop_args(p, seed, step, step_dev);
    switch (dtype) {
        case ONEBIT_F32:
            return launch<float>(x, residual, y, rows, cols, ld_x, ld_r, ld_y, row0, d, st);
        case ONEBIT_BF16:
            return launch<bf16>(x, residual, y, rows, cols, ld_x, ld_r, ld_y, row0, d, st);
        case ONEBIT_F16:
            return launch<f16>(x, residual, y, rows, cols, ld_x, ld_r, ld_y, row0, d, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace onebit
