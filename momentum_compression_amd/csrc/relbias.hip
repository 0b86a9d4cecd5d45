// A relative position bias learned per (bucket, head), written out as a map,
// and its gradient.
//
//   out[h][i][j]    = table[map[clamp(d, -R, R) + R]][h],  d = j - (i + q_pos)
//   dtable[b][h] (+)= sum of ds[.][h][i][j] over every (i, j) of bucket b
//
// The map from distances to buckets is whole numbers made once by the caller,
// so no logarithm decides a bucket on the device.  A map entry outside the
// table counts as no bias.
#include "train.h"

namespace onebit {

namespace {

__device__ __forceinline__ float bias_value(const RelBias& b, int x, int h) {
    const int m = b.map[x];
    return (uint32_t)m < (uint32_t)b.n_buckets ? b.table[(int64_t)m * b.H + h] : 0.0f;
}

// LDS slot of a distance: one word of padding after eight, so that lanes that
// are eight distances apart read different banks.
__device__ __forceinline__ int slot(int x) { return x + (x >> 3); }

constexpr int kExpandGroups = 4;  // groups of 8 columns per lane

template <typename T>
__global__ __launch_bounds__(kThreads) void rel_bias_kernel(RelBias b, T* __restrict__ out,
                                                           uint32_t groups, FastDiv per_row,
                                                           int32_t Tq, int32_t Tk, int32_t q_pos) {
    __shared__ float vals[2 * kMaxRadius + 1 + (2 * kMaxRadius + 1) / 8 + 1];
    const int h = blockIdx.y, R = b.radius;
    for (int x = threadIdx.x; x <= 2 * R; x += kThreads) vals[slot(x)] = bias_value(b, x, h);
    __syncthreads();
    T* head = out + (int64_t)h * Tq * Tk;
#pragma unroll
    for (int u = 0; u < kExpandGroups; ++u) {
        const uint32_t g = (blockIdx.x * kExpandGroups + u) * (uint32_t)kThreads + threadIdx.x;
        if (g >= groups) break;
        const uint32_t i = per_row.div(g);
        const int32_t c = 8 * (int32_t)(g - i * per_row.d);
        const int32_t d = c - (int32_t)i - q_pos;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int32_t x = d + e < -R ? -R : (d + e > R ? R : d + e);
            v[e] = vals[slot(x + R)];
        }
        T* p = head + (int64_t)i * Tk + c;
        if (c + 8 <= Tk) {
            store8(p, v);
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (c + e < Tk) p[e] = (T)v[e];
        }
    }
}

// Gradient.  One pass over ds.  A wave holds 8 rows of C * W columns: a lane has
// C columns (16 bytes) of each row, whose values fall on C + 7 diagonals, so it
// keeps that many sums in registers over all its sequences.  Neighbouring
// lanes' diagonals overlap by 7 and are joined by 7 shuffles; what is left are
// C distances a lane, added to the wave's own bins in LDS without atomics (no
// two lanes own the same distance), so the result does not depend on timing.
// Narrow maps give the other 64 / W parts of the wave other sequences.
constexpr int kGradWaves = 8;
constexpr int kGradThreads = 64 * kGradWaves;

// 16 bytes of consecutive elements, and the first n of them (the others 0).
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Piece {
    static constexpr int kCols = 16 / sizeof(T);
    T v[kCols];
    __device__ __forceinline__ static Piece load(const T* p) {
        return *reinterpret_cast<const Piece*>(p);
    }
    __device__ __forceinline__ static Piece tail(const T* p, int n) {
        Piece x = {};
#pragma unroll
        for (int e = 0; e < kCols - 1; ++e)
            if (e < n) x.v[e] = p[e];
        return x;
    }
};

template <typename T, int W>
__global__ __launch_bounds__(kGradThreads) void bias_grad_kernel(const T* __restrict__ ds,
                                                            float* __restrict__ partials,
                                                            BiasGradPlan plan, int32_t B, int32_t H,
                                                            int32_t radius, int32_t Tq, int32_t Tk,
                                                            int32_t q_pos) {
    extern __shared__ float lds[];  // [waves][2 radius + 1]
    constexpr int C = Piece<T>::kCols;
    const int R = radius, bins_n = 2 * R + 1;
    const int wave = threadIdx.x >> 6, lane = lane_id();
    const int col = lane % W, sub = lane / W;
    constexpr int subs = 64 / W;
    float* bins = lds + wave * bins_n;
    for (int x = lane; x < bins_n; x += 64) bins[x] = 0.0f;
    const int h = blockIdx.y;
    int64_t part = blockIdx.x;
    const int bb = (int)(part % plan.batch_blocks);
    part /= plan.batch_blocks;
    const int cb = (int)(part % plan.col_blocks);
    const int rb = (int)(part / plan.col_blocks);
    const int32_t c0 = cb * (C * W) + C * col;
    // unsigned: up to a part and a step past the last sequence, below 2^32
    const uint32_t b0 = (uint32_t)bb * (uint32_t)plan.batches;
    const uint32_t stop = b0 + (uint32_t)plan.batches;
    const uint32_t b1 = stop < (uint32_t)B ? stop : (uint32_t)B;
    const bool whole = c0 + C <= Tk;
    float far_lo = 0.0f, far_hi = 0.0f;
    for (int32_t i0 = rb * plan.rows + 8 * wave; i0 < Tq && i0 < (rb + 1) * plan.rows;
         i0 += 8 * kGradWaves) {
        float acc[C + 7];
#pragma unroll
        for (int k = 0; k < C + 7; ++k) acc[k] = 0.0f;
        for (uint32_t b = b0 + sub; b < b1; b += subs) {
            const T* p = ds + (((int64_t)b * H + h) * Tq + i0) * (int64_t)Tk + c0;
            Piece<T> v[8];
            if (whole && i0 + 8 <= Tq) {
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = Piece<T>::load(p + (int64_t)r * Tk);
            } else {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    v[r] = Piece<T>{};
                    if (i0 + r >= Tq) continue;
                    v[r] = whole ? Piece<T>::load(p + (int64_t)r * Tk)
                                 : Piece<T>::tail(p + (int64_t)r * Tk, Tk - c0);
                }
            }
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int e = 0; e < C; ++e) acc[e - r + 7] += (float)v[r].v[e];
        }
#pragma unroll
        for (int off = W; off < 64; off <<= 1)
#pragma unroll
            for (int k = 0; k < C + 7; ++k) acc[k] += __shfl_xor(acc[k], off, 64);
        // the next lane's sum k is this lane's k + C; ascending, so that what a
        // sum takes in is passed on with it where C < 7
#pragma unroll
        for (int k = 0; k < 7; ++k) {
            const float next = __shfl_down(acc[k], 1, 64);
            if (col + 1 < W) acc[k + C] += next;
        }
        // acc[k] is the sum of distance d0 + k
        const int32_t d0 = c0 - i0 - q_pos - 7;
        if (sub == 0) {
#pragma unroll
            for (int k = 0; k < C + 7; ++k) {
                if (k < 7 && col != 0) continue;
                const int32_t d = d0 + k;
                if (d <= -R) far_lo += acc[k];
                else if (d >= R) far_hi += acc[k];
                else bins[d + R] += acc[k];
            }
        }
        // the next rows' distances lie with other lanes
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    for (int off = 32; off > 0; off >>= 1) {
        far_lo += __shfl_xor(far_lo, off, 64);
        far_hi += __shfl_xor(far_hi, off, 64);
    }
    if (lane == 0) {
        bins[0] += far_lo;
        bins[2 * R] += far_hi;
    }
    __syncthreads();
    float* to = partials + ((int64_t)h * gridDim.x + blockIdx.x) * bins_n;
    for (int x = threadIdx.x; x < bins_n; x += kGradThreads) {
        float v = lds[x];
#pragma unroll
        for (int w = 1; w < kGradWaves; ++w) v += lds[w * bins_n + x];
        to[x] = v;
    }
}

constexpr int kJoinThreads = 1024;

// One workgroup per (bucket, head): the bucket's distances are listed in
// order, then its threads take (part, distance) pairs in turn, neighbouring
// threads neighbouring distances, and their binary64 sums are added in a fixed
// order.
__global__ __launch_bounds__(kJoinThreads) void bias_join_kernel(const float* __restrict__ partials,
                                                            const int32_t* __restrict__ map,
                                                            float* __restrict__ dtable, int32_t H,
                                                            int32_t parts, int32_t radius,
                                                            int32_t accumulate) {
    __shared__ double sums[kJoinThreads / 64];
    __shared__ int16_t list[2 * kMaxRadius + 1];
    __shared__ int32_t found[kJoinThreads / 64];
    const int b = blockIdx.x, h = blockIdx.y, n = 2 * radius + 1;
    const int wave = threadIdx.x >> 6, lane = lane_id();
    int m = 0;
    for (int x0 = 0; x0 < n; x0 += kJoinThreads) {
        const int x = x0 + (int)threadIdx.x;
        const bool mine = x < n && map[x] == b;
        const uint64_t lanes = __ballot(mine);
        if (lane == 0) found[wave] = __builtin_popcountll(lanes);
        __syncthreads();
        int at = m + __builtin_popcountll(lanes & (((uint64_t)1 << lane) - 1));
        for (int w = 0; w < kJoinThreads / 64; ++w) {
            if (w < wave) at += found[w];
            m += found[w];
        }
        if (mine) list[at] = (int16_t)x;
        __syncthreads();
    }
    const float* from = partials + (int64_t)h * parts * n;
    double v = 0.0;
    if (m > 0) {
        const int dq = kJoinThreads / m, de = kJoinThreads % m;  // a thread's next pair
        int q = (int)threadIdx.x / m, e = (int)threadIdx.x % m;
        while (q < parts) {
            float x[8];  // eight loads in flight
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[k] = q < parts ? from[(int64_t)q * n + list[e]] : 0.0f;
                q += dq;
                e += de;
                if (e >= m) {
                    e -= m;
                    ++q;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) v += (double)x[k];
        }
    }
    v = wave_sum(v);
    if (lane == 0) sums[wave] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kJoinThreads / 64; ++w) v += sums[w];
        float* to = dtable + (int64_t)b * H + h;
        *to = accumulate ? (float)((double)*to + v) : (float)v;
    }
}

template <typename T, int W>
void grad_w(const void* ds, float* partials, const BiasGradPlan& plan, int32_t B, int32_t H,
            int32_t radius, int32_t Tq, int32_t Tk, int32_t q_pos, hipStream_t st) {
    const dim3 grid((unsigned)plan.parts(), (unsigned)H);
    const size_t lds = kGradWaves * (2 * (size_t)radius + 1) * sizeof(float);
    hipLaunchKernelGGL((bias_grad_kernel<T, W>), grid, dim3(kGradThreads), lds, st, (const T*)ds,
                       partials, plan, B, H, radius, Tq, Tk, q_pos);
}

// Lanes that span the columns of a row: the smallest power of two that does.
int32_t grad_lanes(int32_t Tk, int32_t cols) {
    int32_t w = 8;
    while (w < 64 && cols * w < Tk) w *= 2;
    return w;
}

template <typename T>
void grad_t(const void* ds, float* partials, const BiasGradPlan& plan, int32_t B, int32_t H,
            int32_t radius, int32_t Tq, int32_t Tk, int32_t q_pos, hipStream_t st) {
    switch (grad_lanes(Tk, Piece<T>::kCols)) {
        case 8: return grad_w<T, 8>(ds, partials, plan, B, H, radius, Tq, Tk, q_pos, st);
        case 16: return grad_w<T, 16>(ds, partials, plan, B, H, radius, Tq, Tk, q_pos, st);
        case 32: return grad_w<T, 32>(ds, partials, plan, B, H, radius, Tq, Tk, q_pos, st);
        default: return grad_w<T, 64>(ds, partials, plan, B, H, radius, Tq, Tk, q_pos, st);
    }
}

}  // namespace

hipError_t launch_rel_bias(const RelBias& b, void* out, int32_t dtype, int32_t Tq, int32_t Tk,
                           int32_t q_pos, hipStream_t st) {
    const uint32_t per_row = ((uint32_t)Tk + 7) / 8;
    const uint32_t groups = per_row * (uint32_t)Tq;
    const uint32_t span = kThreads * kExpandGroups;
    const dim3 grid((groups + span - 1) / span, (unsigned)b.H);
    const FastDiv div(per_row);
    switch (dtype) {
        case ONEBIT_F32:
            hipLaunchKernelGGL((rel_bias_kernel<float>), grid, dim3(kThreads), 0, st, b,
                               (float*)out, groups, div, Tq, Tk, q_pos);
            break;
        case ONEBIT_BF16:
            hipLaunchKernelGGL((rel_bias_kernel<bf16>), grid, dim3(kThreads), 0, st, b,
                               (bf16*)out, groups, div, Tq, Tk, q_pos);
            break;
        case ONEBIT_F16:
            hipLaunchKernelGGL((rel_bias_kernel<f16>), grid, dim3(kThreads), 0, st, b, (f16*)out,
                               groups, div, Tq, Tk, q_pos);
            break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// Rows and sequences of a workgroup: the split whose rounds of 512 workgroups
// (two a CU at a time) take the fewest row visits, each workgroup's bins and
// its part of the join counted as 24 rows.  A map of 16 x 16 heads and 512 x 512
// takes 28 us with 512 workgroups, against 31 with 1024 and 36 with 2048; an odd
// binary32 one of 3 x 7 and 1021 x 2053 34 us with the 504 that this picks.
BiasGradPlan bias_grad_plan(int32_t B, int32_t H, int32_t Tq, int32_t Tk, int32_t dtype) {
    constexpr int64_t kResident = 512;
    BiasGradPlan best = {};
    const int32_t cols = dtype == ONEBIT_F32 ? 4 : 8;
    const int32_t wide = cols * grad_lanes(Tk, cols);
    const int32_t col_blocks = (Tk + wide - 1) / wide;
    int64_t least = INT64_MAX;
    for (int32_t rows = 8 * kGradWaves; rows <= 1024; rows *= 2) {
        const int32_t row_blocks = (Tq + rows - 1) / rows;
        for (int64_t split = 1; split <= B; split = split < 4 ? split + 1 : split + split / 2) {
            BiasGradPlan p;
            p.rows = rows;
            p.row_blocks = row_blocks;
            p.col_blocks = col_blocks;
            p.batches = (int32_t)((B + split - 1) / split);
            p.batch_blocks = (int32_t)(((int64_t)B + p.batches - 1) / p.batches);
            const int64_t groups = p.parts() * H;
            const int64_t visits = (int64_t)(rows < Tq ? rows : Tq) * p.batches + 24;
            const int64_t cost = (groups + kResident - 1) / kResident * visits;
            if (cost < least || (cost == least && groups < best.parts() * H)) {
                least = cost;
                best = p;
            }
        }
        if (row_blocks == 1) break;
    }
    return best;
}

hipError_t launch_bias_join(const float* partials, const int32_t* map, float* dtable, int32_t H,
                            int64_t parts, int32_t n_buckets, int32_t radius, bool accumulate,
                            hipStream_t st) {
    hipLaunchKernelGGL(bias_join_kernel, dim3((unsigned)n_buckets, (unsigned)H),
                       dim3(kJoinThreads), 0,
                       st, partials, map, dtable, H, (int32_t)parts, radius, accumulate ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_rel_bias_grad(const void* ds, int32_t dtype, const int32_t* map, float* dtable,
                                int32_t B, int32_t H, int32_t n_buckets, int32_t radius,
                                int32_t Tq, int32_t Tk, int32_t q_pos, bool accumulate,
                                float* partials, hipStream_t st) {
    const BiasGradPlan plan = bias_grad_plan(B, H, Tq, Tk, dtype);
    switch (dtype) {
        case ONEBIT_F32: grad_t<float>(ds, partials, plan, B, H, radius, Tq, Tk, q_pos, st); break;
        case ONEBIT_BF16: grad_t<bf16>(ds, partials, plan, B, H, radius, Tq, Tk, q_pos, st); break;
        case ONEBIT_F16: grad_t<f16>(ds, partials, plan, B, H, radius, Tq, Tk, q_pos, st); break;
        default: return hipErrorInvalidValue;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_bias_join(partials, map, dtable, H, plan.parts(), n_buckets, radius, accumulate,
                            st);
}

}  // namespace onebit
