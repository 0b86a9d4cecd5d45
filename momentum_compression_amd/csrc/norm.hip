// Layer norm over the rows of a matrix, forward and backward.
//
// A row lies in the registers of `G` lanes, V groups of eight columns a lane
// (group j of lane l: columns 8 (l + G j) ... + 7), so memory is read once and
// written once: the kernels are bound by those bytes.  A workgroup takes rows in
// turn and keeps what belongs to its columns in registers: the weights, and in
// the backward pass the sums over rows.  Rows of more columns
// than that holds are read again for each pass.
//
// Measured: forward 8192 x 1024 bf16 10.1 us (33.6 MB, 3.3 TB/s: two rounds of loads
// and their latency), backward 16384 x 2048 bf16 44 us and 5 for the join (201 MB),
// 16411 x 1003 float32 41 and 4.7 (198 MB): 4.6 to 4.8 TB/s.
#include <type_traits>

#include "train.h"

namespace onebit {
namespace {

// Sum over the lane's group of G lanes (a power of two up to 64), in every lane.
template <int G>
__device__ __forceinline__ float lanes_sum(float x) {
    auto dpp = [](float v, auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp(
            (int)__float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    if (G >= 2) x += dpp(x, std::integral_constant<int, 0xB1>{});    // lane ^ 1
    if (G >= 4) x += dpp(x, std::integral_constant<int, 0x4E>{});    // lane ^ 2
    if (G >= 8) x += dpp(x, std::integral_constant<int, 0x141>{});   // the other four of eight
    if (G >= 16) x += dpp(x, std::integral_constant<int, 0x140>{});  // the other eight of 16
    if (G >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x),
                                                        false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if (G >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x),
                                                        false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return x;
}

// Sums of two values over the G threads of a row.  With more than a wave to a
// row, every thread of the workgroup comes here, and `lds` (2 x 16 floats) is
// another one at the next call.
template <int G>
__device__ __forceinline__ void row_sums(float& a, float& b, float2* lds) {
    constexpr int lanes = G < 64 ? G : 64;
    a = lanes_sum<lanes>(a);
    b = lanes_sum<lanes>(b);
    if (G > 64) {
        constexpr int waves = G / 64;
        const int wave = threadIdx.x >> 6;
        if (lane_id() == 0) lds[wave] = float2{a, b};
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < waves; ++w) {
            a += lds[w].x;
            b += lds[w].y;
        }
    }
}

// The group of lanes that the thread is in; a wave's or more as a scalar, so that
// rows' addresses are.
template <int G>
__device__ __forceinline__ int group_id() {
    return G >= 64 ? __builtin_amdgcn_readfirstlane((int)(threadIdx.x / G)) : (int)threadIdx.x / G;
}

template <int G>
constexpr int norm_threads() {
    return G > 256 ? G : 256;
}

// Eight parameters from column c on, `n` of them there.
__device__ __forceinline__ void load_params(float out[8], const void* p, bool wide, int32_t dtype,
                                            int64_t c, int64_t n, float otherwise) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = otherwise;
    if (!p || n <= 0) return;
    if (wide) {
        const auto x = n >= 8 ? load8((const float*)p + c) : load_tail((const float*)p + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = x.v[e];
    } else if (dtype == ONEBIT_BF16) {
        const auto x = n >= 8 ? load8((const bf16*)p + c) : load_tail((const bf16*)p + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = (float)x.v[e];
    } else {
        const auto x = n >= 8 ? load8((const f16*)p + c) : load_tail((const f16*)p + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = (float)x.v[e];
    }
}

// Eight elements of a row in whole 32-bit words: as single elements the compiler
// gives each a register of its own.
template <typename T>
struct Part {
    typedef uint32_t Words __attribute__((ext_vector_type(2 * sizeof(T))));
    Words w;
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        else return (float)__builtin_bit_cast(T, (uint16_t)(w[e >> 1] >> (16 * (e & 1))));
    }
    // The same bits, of which the compiler knows nothing.
    __device__ __forceinline__ void hide() {
#pragma unroll
        for (unsigned k = 0; k < 2 * sizeof(T); ++k) {
            uint32_t x = w[k];
            asm volatile("" : "+v"(x));
            w[k] = x;
        }
    }
};

template <typename T>
__device__ __forceinline__ Part<T> load_whole(const T* p) {
    typedef typename Part<T>::Words Any __attribute__((aligned(sizeof(T))));
    return Part<T>{*reinterpret_cast<const Any*>(p)};
}

template <typename T>
__device__ __forceinline__ Part<T> load_part(const T* row, int64_t c, int64_t cols) {
    if (c + 8 <= cols) return load_whole(row + c);
    Part<T> x;
    x.w = 0;
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (c + e < cols) {
            if constexpr (sizeof(T) == 4) x.w[e] = __float_as_uint(row[c + e]);
            else x.w[e >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, row[c + e]) << (16 * (e & 1));
        }
    return x;
}

template <typename T>
__device__ __forceinline__ void store_part(T* row, int64_t c, int64_t cols, const float v[8]) {
    if (c + 8 <= cols) {
        store8(row + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (c + e < cols) row[c + e] = (T)v[e];
    }
}

// ---------------------------------------------------------------- forward
// The mean in two steps: d = x - m1 with m1 the mean as binary32 sums leave it,
// then what m1 is off, the mean of d.  A common offset of the row costs y
// nothing then, and the variance is that of small numbers.
struct Moments {
    float shift, rest, rstd;  // mean = shift + rest
};

__device__ __forceinline__ Moments moments(float shift, float sum, float squares, float inv,
                                           float eps) {
    const float rest = sum * inv;
    const float var = __builtin_fmaf(-rest, rest, squares * inv);
    return Moments{shift, rest, 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps)};
}

template <typename T, int G, int V>
__global__ __launch_bounds__(norm_threads<G>()) void layer_norm_kernel(NormArgs a) {
    constexpr int per_block = norm_threads<G>() / G;
    __shared__ float2 lds[3][16];
    const int part = threadIdx.x % G;
    const int cols = (int)a.cols;
    const int64_t step = (int64_t)gridDim.x * per_block;
    const float inv = 1.0f / (float)cols;
    // the next row is on its way while one is computed
    Part<T> next[V];
    auto fetch = [&](int64_t row) {
        const T* x = (const T*)a.x + row * a.ld_x;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = 8 * (part + G * j);
            next[j].w = 0;
            if (row < a.rows && c < cols) next[j] = load_part(x, c, cols);
        }
    };
    fetch((int64_t)blockIdx.x * per_block + group_id<G>());
    for (int64_t r0 = (int64_t)blockIdx.x * per_block; r0 < a.rows; r0 += step) {
        const int64_t row = r0 + group_id<G>();
        const bool ok = row < a.rows;
        float d[V][8];
        float sum = 0.0f, zero = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) d[j][e] = next[j][e];
            sum += ((d[j][0] + d[j][1]) + (d[j][2] + d[j][3])) +
                   ((d[j][4] + d[j][5]) + (d[j][6] + d[j][7]));
        }
        fetch(row + step);
        row_sums<G>(sum, zero, lds[0]);
        const float shift = sum * inv;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = 8 * (part + G * j);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                d[j][e] = c + e < cols ? d[j][e] - shift : 0.0f;
                s1 += d[j][e];
                s2 = __builtin_fmaf(d[j][e], d[j][e], s2);
            }
        }
        row_sums<G>(s1, s2, lds[1]);
        const Moments m = moments(shift, s1, s2, inv, a.eps);
        if (ok && part == 0) {
            if (a.mean) a.mean[row] = m.shift + m.rest;
            if (a.rstd) a.rstd[row] = m.rstd;
        }
        T* y = (T*)a.y + row * a.ld_y;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = 8 * (part + G * j);
            if (!ok || c >= cols) continue;
            // from the caches for each row: in registers they would halve the
            // rows under way
            float w[8], b[8], o[8];
            load_params(w, a.weight, a.w_wide, a.dtype, c, cols - c, 1.0f);
            load_params(b, a.bias, a.w_wide, a.dtype, c, cols - c, 0.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = __builtin_fmaf((d[j][e] - m.rest) * m.rstd, w[e], b[e]);
            store_part(y, c, cols, o);
        }
        if (G > 64) __syncthreads();  // lds is read
    }
}

// Rows of any length: a workgroup a row, three passes over it.
constexpr int kLong = 1024;

template <typename T>
__global__ __launch_bounds__(kLong) void layer_norm_long_kernel(NormArgs a) {
    __shared__ float2 lds[2][16];
    const int64_t cols = a.cols;
    const float inv = 1.0f / (float)cols;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = (const T*)a.x + row * a.ld_x;
        T* y = (T*)a.y + row * a.ld_y;
        float sum = 0.0f, zero = 0.0f;
        for (int64_t c = 8 * threadIdx.x; c < cols; c += 8 * kLong) {
            const Part<T> v = load_part(x, c, cols);
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[e];
            sum += s;
        }
        row_sums<kLong>(sum, zero, lds[0]);
        const float shift = sum * inv;
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = 8 * threadIdx.x; c < cols; c += 8 * kLong) {
            const Part<T> v = load_part(x, c, cols);
            float p = 0.0f, q = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = c + e < cols ? v[e] - shift : 0.0f;
                p += d;
                q = __builtin_fmaf(d, d, q);
            }
            s1 += p;
            s2 += q;
        }
        row_sums<kLong>(s1, s2, lds[1]);
        const Moments m = moments(shift, s1, s2, inv, a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = m.shift + m.rest;
            if (a.rstd) a.rstd[row] = m.rstd;
        }
        for (int64_t c = 8 * threadIdx.x; c < cols; c += 8 * kLong) {
            const Part<T> v = load_part(x, c, cols);
            float w[8], b[8], o[8];
            load_params(w, a.weight, a.w_wide, a.dtype, c, cols - c, 1.0f);
            load_params(b, a.bias, a.w_wide, a.dtype, c, cols - c, 0.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = __builtin_fmaf(((v[e] - m.shift) - m.rest) * m.rstd, w[e], b[e]);
            store_part(y, c, cols, o);
        }
        __syncthreads();  // lds is read
    }
}

// ---------------------------------------------------------------- backward
// dx = rstd (u - mean(u) - h mean(u h)) with u = dy w, h = (x - mean) rstd, and
// the sums of dy h and dy over the workgroup's rows, kept by columns.  Groups of
// lanes that hold the same columns are added at the end, in their order.
//
// Where a row ends inside a lane's eight columns, the lane reads the row's last
// eight, and those that belong to the lane before it have weight 0 here (no
// branches to load single elements, which cost 40 registers for every eight
// columns).
template <typename T, int G, int V>
__global__ __launch_bounds__(norm_threads<G>(), 2) void layer_norm_grad_kernel(NormArgs a) {
    constexpr int threads = norm_threads<G>(), per_block = threads / G;
    __shared__ float2 lds[16];
    __shared__ float share[per_block > 1 ? threads * 8 * V : 1];
    const int part = threadIdx.x % G, cols = (int)a.cols;
    const int64_t step = (int64_t)gridDim.x * per_block;
    const float inv = 1.0f / (float)cols;
    int at[V], low[V], high[V];  // the lane's columns at + low ... at + high - 1
    float w[V][8], dw[V][8] = {}, db[V][8] = {};
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = 8 * (part + G * j);
        at[j] = G > 1 && c + 8 > cols ? cols - 8 : c;
        low[j] = c - at[j];
        high[j] = c >= cols ? 0 : G > 1 ? 8 : cols;
        load_params(w[j], a.weight, a.w_wide, a.dtype, at[j], high[j], 1.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[j][e] = e >= low[j] && e < high[j] ? w[j][e] : 0.0f;
    }
    // the next row is on its way while one is computed, where there is room for it
    constexpr bool ahead = V * sizeof(T) <= 8;
    Part<T> xv[V], gv[V], xn[V], gn[V];
    float mean = 0.0f, rstd = 0.0f, mean_next = 0.0f, rstd_next = 0.0f;
    auto fetch = [&](int64_t row, Part<T>(&xs)[V], Part<T>(&gs)[V], float& m, float& r) {
        const bool ok = row < a.rows;
        const T* x = (const T*)a.x + row * a.ld_x;
        const T* dy = (const T*)a.dy + row * a.ld_dy;
        m = ok ? a.mean[row] : 0.0f;
        r = ok ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            xs[j].w = gs[j].w = 0;
            if (ok && high[j] > 0) {
                xs[j] = G > 1 ? load_whole(x + at[j]) : load_part(x, 0, cols);
                gs[j] = G > 1 ? load_whole(dy + at[j]) : load_part(dy, 0, cols);
            }
        }
    };
    if (ahead)
        fetch((int64_t)blockIdx.x * per_block + group_id<G>(), xn, gn, mean_next, rstd_next);
    for (int64_t r0 = (int64_t)blockIdx.x * per_block; r0 < a.rows; r0 += step) {
        const int64_t row = r0 + group_id<G>();
        const bool ok = row < a.rows;
        if (ahead) {
            mean = mean_next;
            rstd = rstd_next;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xv[j] = xn[j];
                gv[j] = gn[j];
            }
            fetch(row + step, xn, gn, mean_next, rstd_next);
        } else {
            fetch(row, xv, gv, mean, rstd);
        }
        float su = 0.0f, suh = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = (xv[j][e] - mean) * rstd, g = gv[j][e], u = g * w[j][e];
                dw[j][e] = __builtin_fmaf(g, h, dw[j][e]);
                db[j][e] += g;
                su += u;
                suh = __builtin_fmaf(u, h, suh);
            }
            __builtin_amdgcn_sched_barrier(0);  // one group's values at a time
        }
        if (!a.dx) continue;  // the same for all
        row_sums<G>(su, suh, lds);
        su *= inv;
        suh *= inv;
        T* dx = (T*)a.dx + row * a.ld_dx;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (!ok || high[j] == 0) continue;
            // what the first pass made of them is not kept: registers are rows
            // under way
            xv[j].hide();
            gv[j].hide();
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = (xv[j][e] - mean) * rstd, u = gv[j][e] * w[j][e];
                o[e] = rstd * __builtin_fmaf(-h, suh, u - su);
            }
            if (low[j] == 0 && high[j] == 8) {
                store8(dx + at[j], o);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= low[j] && e < high[j]) dx[at[j] + e] = (T)o[e];
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (G > 64) __syncthreads();  // lds is read
    }
    if (!a.partials) return;
    float* to = a.partials + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (s && per_block > 1) __syncthreads();  // the first sums are read
        float* out = per_block > 1 ? share + (group_id<G>()) * (8 * G * V) : to + s * cols;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= low[j] && e < high[j]) out[at[j] + e] = s ? db[j][e] : dw[j][e];
        if (per_block == 1) continue;
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += threads) {
            float t = 0.0f;
            for (int p = 0; p < per_block; ++p) t += share[p * (8 * G * V) + c];
            to[s * cols + c] = t;
        }
    }
}

// Rows of any length: first the sums over rows, a workgroup for 2048 columns of
// a part of the rows, then dx with a workgroup a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void layer_norm_grad_cols_kernel(NormArgs a, int64_t strips,
                                                                        int64_t parts,
                                                                        int64_t rows_of_part) {
    const int64_t cols = a.cols;
    for (int64_t block = blockIdx.x; block < strips * parts; block += gridDim.x) {
        const int64_t c = 8 * (block % strips * kThreads + threadIdx.x), part = block / strips;
        if (c >= cols) continue;
        const int64_t end = (part + 1) * rows_of_part < a.rows ? (part + 1) * rows_of_part : a.rows;
        float dw[8] = {}, db[8] = {};
        for (int64_t row = part * rows_of_part; row < end; ++row) {
            const Part<T> xv = load_part((const T*)a.x + row * a.ld_x, c, cols);
            const Part<T> gv = load_part((const T*)a.dy + row * a.ld_dy, c, cols);
            const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = gv[e];
                dw[e] = __builtin_fmaf(g, (xv[e] - mean) * rstd, dw[e]);
                db[e] += g;
            }
        }
        float* to = a.partials + part * 2 * cols;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c + e >= cols) break;
            to[c + e] = dw[e];
            to[cols + c + e] = db[e];
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kLong) void layer_norm_grad_rows_kernel(NormArgs a) {
    __shared__ float2 lds[16];
    const int64_t cols = a.cols;
    const float inv = 1.0f / (float)cols;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = (const T*)a.x + row * a.ld_x;
        const T* dy = (const T*)a.dy + row * a.ld_dy;
        T* dx = (T*)a.dx + row * a.ld_dx;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float su = 0.0f, suh = 0.0f;
        for (int64_t c = 8 * threadIdx.x; c < cols; c += 8 * kLong) {
            const Part<T> xv = load_part(x, c, cols), gv = load_part(dy, c, cols);
            float w[8], p = 0.0f, q = 0.0f;
            load_params(w, a.weight, a.w_wide, a.dtype, c, cols - c, 1.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = c + e < cols ? (xv[e] - mean) * rstd : 0.0f;
                const float u = gv[e] * w[e];
                p += u;
                q = __builtin_fmaf(u, h, q);
            }
            su += p;
            suh += q;
        }
        row_sums<kLong>(su, suh, lds);
        su *= inv;
        suh *= inv;
        for (int64_t c = 8 * threadIdx.x; c < cols; c += 8 * kLong) {
            const Part<T> xv = load_part(x, c, cols), gv = load_part(dy, c, cols);
            float w[8], o[8];
            load_params(w, a.weight, a.w_wide, a.dtype, c, cols - c, 1.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = (xv[e] - mean) * rstd;
                o[e] = rstd * __builtin_fmaf(-h, suh, gv[e] * w[e] - su);
            }
            store_part(dx, c, cols, o);
        }
        __syncthreads();  // lds is read
    }
}

// Joins the workgroups' sums [parts][n] over their n columns in a fixed order,
// in binary64, 64 columns to a workgroup, its 16 waves taking parts in turn.  The
// first `cols` of the n go to out0, the others to out1.
__global__ __launch_bounds__(1024) void column_join_kernel(const float* partials, int64_t parts,
                                                           int64_t n, int64_t cols, float* out0,
                                                           float* out1, bool accumulate) {
    __shared__ double sums[16][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < n; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        double t = 0.0;
        if (c < n) {
            int64_t p = wave;
            for (; p + 7 * 16 < parts; p += 8 * 16) {  // eight loads at once
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = partials[(p + 16 * k) * n + c];
#pragma unroll
                for (int k = 0; k < 8; ++k) t += v[k];
            }
            for (; p < parts; p += 16) t += partials[p * n + c];
        }
        sums[wave][lane] = t;
        __syncthreads();
        float* out = c < cols ? out0 : out1;
        if (wave == 0 && c < n && out) {
            for (int w = 1; w < 16; ++w) t += sums[w][lane];
            const int64_t at = c < cols ? c : c - cols;
            out[at] = (float)(accumulate ? (double)out[at] + t : t);
        }
        __syncthreads();  // the sums are read
    }
}

template <typename F>
hipError_t with_type(int32_t dtype, F&& f) {
    if (dtype == ONEBIT_F32) f(float{});
    else if (dtype == ONEBIT_BF16) f(bf16{});
    else f(f16{});
    return hipGetLastError();
}

// The lanes of a row and its groups of columns a lane; {0, 0}: a row that is read
// again for each pass.  The fewer groups the more rows are under way; the backward
// pass keeps 24 registers a group for its sums and weights, and with 1024 lanes of
// two groups (not enough registers) takes 122 us where reading again takes 90
// (2048 x 16384 bf16).
struct Shape {
    int G, V;
};

Shape shape_of(int64_t rows, int64_t cols, bool grad) {
    if (cols <= 8) return {1, 1};
    if (cols <= 32) return {4, 1};
    if (cols <= 128) return {16, 1};
    if (cols <= 512) return {64, 1};
    // few rows: a workgroup each
    if (!grad && rows <= 1024 && cols <= 2048) return {256, 1};
    if (cols <= 1024) return {64, 2};
    if (cols <= 2048) return grad ? Shape{256, 1} : Shape{64, 4};
    if (cols <= 4096) return {256, 2};
    if (cols <= 8192) return grad ? Shape{1024, 1} : Shape{256, 4};
    if (cols <= 16384 && !grad) return {1024, 2};
    return {0, 0};
}

// Workgroups at most.  The backward pass's sums are joined: with 512, 1024 and 2048
// of them 16384 x 2048 takes 49, 53 and 64 us.
constexpr int64_t kForwardBlocks = 4096, kNormBlocks = 512;
constexpr int64_t kLongParts = 64;        // parts of the rows, at most
// a launch holds fewer than 2^32 threads, of 1024 a workgroup at most
constexpr int64_t kMostBlocks = (int64_t)1 << 21;

// f with a shape that shape_of gives for the pass.
template <bool GRAD, typename F>
void with_shape(const Shape& s, F&& f) {
    auto is = [&](int G, int V) { return s.G == G && s.V == V; };
#define ONEBIT_SHAPE(G, V) \
    if (is(G, V)) return f(std::integral_constant<int, G>{}, std::integral_constant<int, V>{})
    ONEBIT_SHAPE(1, 1);
    ONEBIT_SHAPE(4, 1);
    ONEBIT_SHAPE(16, 1);
    ONEBIT_SHAPE(64, 1);
    ONEBIT_SHAPE(64, 2);
    ONEBIT_SHAPE(256, 1);
    ONEBIT_SHAPE(256, 2);
    if constexpr (GRAD) {
        ONEBIT_SHAPE(1024, 1);
    } else {
        ONEBIT_SHAPE(64, 4);
        ONEBIT_SHAPE(256, 4);
        ONEBIT_SHAPE(1024, 2);
    }
#undef ONEBIT_SHAPE
}

int64_t row_blocks(const Shape& s, int64_t rows, int64_t most) {
    const int64_t per = s.G ? (s.G > 256 ? 1 : 256 / s.G) : 1;
    const int64_t need = (rows + per - 1) / per;
    return need < most ? need : most;
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t cols) {
    const Shape s = shape_of(rows, cols, true);
    if (s.G) return row_blocks(s, rows, kNormBlocks);
    return rows < kLongParts ? rows : kLongParts;
}

hipError_t launch_column_join(const float* partials, int64_t parts, int64_t n, int64_t cols,
                              float* out0, float* out1, bool accumulate, hipStream_t st) {
    const int64_t groups = (n + 63) / 64;
    hipLaunchKernelGGL(column_join_kernel, dim3((unsigned)(groups < kMostBlocks ? groups : kMostBlocks)),
                       dim3(1024), 0, st, partials, parts, n, cols, out0, out1, accumulate);
    return hipGetLastError();
}

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st) {
    const Shape s = shape_of(a.rows, a.cols, false);
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        if (!s.G) {
            hipLaunchKernelGGL((layer_norm_long_kernel<T>),
                               dim3((unsigned)(a.rows < 4096 ? a.rows : 4096)), dim3(kLong), 0, st,
                               a);
            return;
        }
        with_shape<false>(s, [&](auto G, auto V) {
            hipLaunchKernelGGL((layer_norm_kernel<T, G.value, V.value>),
                               dim3((unsigned)row_blocks(s, a.rows, kForwardBlocks)),
                               dim3(norm_threads<G.value>()), 0, st, a);
        });
    });
}

hipError_t launch_layer_norm_grad(const NormArgs& a, float* dweight, float* dbias, bool accumulate,
                                  hipStream_t st) {
    const Shape s = shape_of(a.rows, a.cols, true);
    const int64_t parts = norm_parts(a.rows, a.cols);
    hipError_t e = hipSuccess;
    if (a.rows > 0)
        e = with_type(a.dtype, [&](auto t) {
            using T = decltype(t);
            if (s.G) {
                with_shape<true>(s, [&](auto G, auto V) {
                    hipLaunchKernelGGL((layer_norm_grad_kernel<T, G.value, V.value>),
                                       dim3((unsigned)parts), dim3(norm_threads<G.value>()), 0, st,
                                       a);
                });
                return;
            }
            if (a.partials) {
                const int64_t strips = (a.cols + 8 * kThreads - 1) / (8 * kThreads);
                const int64_t rows_of_part = (a.rows + parts - 1) / parts;
                const int64_t blocks = strips * parts;
                hipLaunchKernelGGL((layer_norm_grad_cols_kernel<T>),
                                   dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)),
                                   dim3(kThreads), 0, st, a, strips, parts, rows_of_part);
            }
            if (a.dx)
                hipLaunchKernelGGL((layer_norm_grad_rows_kernel<T>),
                                   dim3((unsigned)(a.rows < 4096 ? a.rows : 4096)), dim3(kLong), 0,
                                   st, a);
        });
    if (e != hipSuccess || !a.partials) return e;
    return launch_column_join(a.partials, parts, 2 * a.cols, a.cols, dweight, dbias, accumulate, st);
}

}  // namespace onebit
