// What the attention kernels share: arguments, the tile layout in LDS, matrix
// instruction wrappers, the bias window and the launchers.
//
// Layouts.  v_mfma_f32_32x32x16 takes A[row = lane & 31][k] and
// B[k][col = lane & 31] with k = 8 (lane >> 5) + 0 ... 7, and leaves
// C[row = 8 (r >> 2) + 4 (lane >> 5) + (r & 3)][col = lane & 31] in register r.
// Reading the rows of A in the order perm_row() makes register r of a lane
// hold row 16 (r >> 3) + 8 (lane >> 5) + (r & 7) instead: eight consecutive
// rows to a lane, which is exactly the B operand of the next product (no
// exchange between lanes) and exactly one group of eight dropout draws.
#pragma once

#include "philox.h"
#include "train.h"

namespace onebit {

constexpr int kRows = 32;           // rows of a wave (columns of its products)
constexpr int kWaves = 4;
constexpr int kTileRows = kRows * kWaves;
constexpr int kStep = 64;           // rows of the other side per staged tile
constexpr int kPad = 96;            // distances past the radius that a wave's tile can reach
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

using f32x16 = float __attribute__((ext_vector_type(16)));

struct Strides {
    int64_t b, t, h;  // elements between sequences, tokens, heads
};

struct AttnArgs {
    const void *q, *k, *v, *d_o;
    const void* o_in;
    void *o, *dq, *dk, *dv;
    Strides sq, sk, sv, so, sdo, sdq, sdk, sdv;
    float* lse;           // [B][H][Tq] natural logarithm, or nullptr
    float* delta;         // [B][H][Tq] row sums of P dP, without the kept share's scale
    float* norm;          // [B][H][Tq] rows with a base: log2 of the sum above it
    float* partials;      // distance sums [H][parts][2 radius + 1]
    float* split_o;       // [rows][splits][D] of a split forward
    f4* split_ml;         // [rows][splits] base, reference and sum
    const int32_t* q_pos_dev;
    const int32_t* k_len;
    RelBias bias;         // radius 0: none
    DropArgs drop;
    int32_t B, H, Hkv, Tq, Tk, D;
    int32_t q_pos, causal;
    bool few;                     // attn_few_kernel
    int32_t splits, split_tiles;  // key tiles of one split
    float scale;
};

// ---------------------------------------------------------------- element types
template <typename T>
struct Mma;

template <>
struct Mma<bf16> {
    using x8 = __bf16 __attribute__((ext_vector_type(8)));
    using x4 = __bf16 __attribute__((ext_vector_type(4)));
    static __device__ __forceinline__ f32x16 mul(x8 a, x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Mma<f16> {
    using x8 = _Float16 __attribute__((ext_vector_type(8)));
    using x4 = _Float16 __attribute__((ext_vector_type(4)));
    static __device__ __forceinline__ f32x16 mul(x8 a, x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// Transposing read: of each 16 lanes, lane i asks for 8 bytes at p (row i / 4,
// four columns from 4 (i % 4)) and gets column i of the four rows.
template <typename T>
__device__ __forceinline__ typename Mma<T>::x4 read_tr(const char* p) {
    using s4 = short __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(typename Mma<T>::x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                       (__attribute__((address_space(3))) s4*)p));
}

// Matrix row that lane row m of the A operand reads (see the top).
__device__ __forceinline__ int perm_row(int m) {
    return (m & 16) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3);
}

// A tile of kStep rows of DP elements in LDS: 16-byte chunks, the chunk number
// xored with a function of the row.  LDS serves 256 bytes a cycle: a row read
// takes 16 lanes at a time (16 rows, one chunk number), a transposing read 32
// lanes (4 consecutive rows of 4 consecutive chunks).  Row bits go where both
// meet every bank once: the low bits of the row move whole groups of four
// chunks, the next ones the chunks of a group (with 128-byte rows the lowest
// row bit already selects half of the banks).  Measured: 4 and 2 cycles a
// read, no conflicts.
template <int DP>
__device__ __forceinline__ int swizzle(int row) {
    return DP == 64 ? (((row >> 1) & 1) << 2) | (((row >> 2) & 1) << 1) | ((row >> 3) & 1)
                    : ((row & 3) << 2) | ((row >> 2) & 3);
}

template <int DP>
__device__ __forceinline__ int tile_at(int row, int chunk) {
    return row * (DP * 2) + ((chunk ^ swizzle<DP>(row)) << 4);
}

template <int DP>
constexpr int tile_bytes() {
    return kStep * DP * 2;
}

// Fills tiles with global rows, memory to LDS without registers between: a
// lane's 16 bytes land beside its neighbours', so the lane asks for the chunk
// that the swizzle puts there.  Rows past the last one and columns from D on
// lie past the buffer's end, which reads as 0.  What is under way is there for
// the workgroup when every wave that issued a part of it has passed
// tiles_barrier(): a __syncthreads() alone does not wait for it.
template <typename T, int DP>
struct Feed {
    static constexpr int kChunks = DP / 8;
    static constexpr int kPer = kStep * kChunks / kThreads;  // loads a lane and tile
    const T* base;
    uint32_t stride, row_bytes, at;  // in bytes

    __device__ __forceinline__ Feed(const T* from, int64_t token_stride, int32_t D, int wave,
                                    int lane)
        : base(from), stride((uint32_t)token_stride * 2), row_bytes((uint32_t)D * 2) {
        const int row = wave * (64 / kChunks) + lane / kChunks;
        const int chunk = (lane % kChunks) ^ swizzle<DP>(row);  // the same kStep / kPer rows on
        at = 8 * chunk < D ? (uint32_t)row * stride + 16 * chunk : 0x80000000u;
    }
    // rows first ... first + kStep - 1, those below `end`
    __device__ __forceinline__ void load(char* tile, int32_t first, int32_t end, int wave) const {
        const int32_t rows = end - first < kStep ? end - first : kStep;
        const uint32_t bytes = rows > 0 ? (uint32_t)(rows - 1) * stride + row_bytes : 0u;
        const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(
            (void*)((const char*)base + (int64_t)first * stride), 0, (int)bytes, 0x00027000);
#pragma unroll
        for (int x = 0; x < kPer; ++x)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                from,
                (__attribute__((address_space(3))) void*)(tile + (x * kWaves + wave) * 1024), 16,
                (int)(at + (uint32_t)x * (kStep / kPer) * stride), 0, 0, 0);
    }
};

// A barrier that shows all waves the tiles whose loads they issued before it.
// Each wave waits for its own loads first (vmcnt 0, the other counters left).
__device__ __forceinline__ void tiles_barrier() {
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
}

// A operand: 32 rows (in perm_row order) of the tile from `row0`, columns
// 16 kc ... 16 kc + 15.
template <typename T, int DP>
__device__ __forceinline__ typename Mma<T>::x8 row_frag(const char* tile, int row0, int kc,
                                                        int lane) {
    const int row = row0 + perm_row(lane & 31);
    return *reinterpret_cast<const typename Mma<T>::x8*>(tile +
                                                         tile_at<DP>(row, 2 * kc + (lane >> 5)));
}

// A operand of the transposed tile: rows are the tile's columns 32 db ... + 31,
// k its rows row0 ... row0 + 15.  Sixteen lanes read four rows of 16 elements
// and lane i gets column i of them.
template <typename T, int DP>
__device__ __forceinline__ typename Mma<T>::x8 col_frag(const char* tile, int row0, int db,
                                                        int lane) {
    const int i = lane & 15;
    const int row = row0 + 8 * (lane >> 5) + (i >> 2);
    const int chunk = 4 * db + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
    const auto lo = read_tr<T>(tile + tile_at<DP>(row, chunk) + 8 * (i & 1));
    const auto hi = read_tr<T>(tile + tile_at<DP>(row + 4, chunk) + 8 * (i & 1));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Order of the LDS reads and matrix instructions of a block: AHEAD reads first,
// then after each matrix instruction the reads of a later one.  Left alone they
// come one or two instructions before their use, and a wave that has its SIMD
// to itself waits out the LDS latency at every one.  The compiler follows it
// for the row reads and, in the key pass for heads of 128, for the transposing
// ones; with heads of 64 those products still wait for their own two reads.
template <int READS_PER_MMA, int MMAS, int AHEAD>
__device__ __forceinline__ void read_ahead() {
    constexpr int kRead = 0x100, kMma = 0x8;
    constexpr int later = (READS_PER_MMA * MMAS - AHEAD) / READS_PER_MMA;
    static_assert(AHEAD % READS_PER_MMA == 0 && later >= 0, "whole instructions");
    __builtin_amdgcn_sched_group_barrier(kRead, AHEAD, 0);
#pragma unroll
    for (int i = 0; i < later; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kRead, READS_PER_MMA, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMma, MMAS - later, 0);
}

// B operand straight from memory: row `row` of `base` (0 where not ok),
// columns 16 kc + 8 (lane >> 5) ... + 7.
template <typename T, int DP>
__device__ __forceinline__ void load_frags(typename Mma<T>::x8 (&f)[DP / 16], const T* base,
                                           int64_t stride, int32_t row, bool ok, int32_t D,
                                           int lane) {
#pragma unroll
    for (int kc = 0; kc < DP / 16; ++kc) {
        const int c = 16 * kc + 8 * (lane >> 5);
        f[kc] = typename Mma<T>::x8{};
        if (ok && c < D)
            f[kc] = *reinterpret_cast<const typename Mma<T>::x8*>(base + (int64_t)row * stride + c);
    }
}

template <typename T>
__device__ __forceinline__ typename Mma<T>::x8 pack8(const float* p) {
    typename Mma<T>::x8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (T)p[e];
    return r;
}

// The wave's number as a scalar, so that what follows from it branches as one.
__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// The value the other half of the wave holds for the same column.
__device__ __forceinline__ float other_half(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return __uint_as_float((lane_id() < 32) ? r[1] : r[0]);
}

// ---------------------------------------------------------------- bias window
// One head's bias, divided by the scale, over the distances -radius - kPad ...
// radius + kPad, so that a tile that reaches past the radius needs no clamp:
// the products of a tile start from it, and one scale serves both.
__device__ __forceinline__ int window_floats(int radius) { return 2 * radius + 1 + 2 * kPad; }

//
// A table value of -2^40 or less counts as -infinity, and so does one that
// leaves binary32 here.
__device__ __forceinline__ float low_value(float t) { return t <= -0x1p40f ? -INFINITY : t; }

__device__ __forceinline__ void fill_window(float* w, const RelBias& b, int h, float scale) {
    const int R = b.radius;
    const float inv_scale = 1.0f / scale;
    for (int x = threadIdx.x; x < window_floats(R); x += kThreads) {
        int i = x - kPad;
        i = i < 0 ? 0 : (i > 2 * R ? 2 * R : i);
        const int m = b.map[i];
        w[x] = (uint32_t)m < (uint32_t)b.n_buckets
                   ? low_value(b.table[(int64_t)m * b.H + h]) * inv_scale
                   : 0.0f;
    }
}

// An exponential's argument is one fused multiplication and addition of the
// score and the row's reference, which leaves up to half a step of the
// reference in it, in the backward pass a few (lse is a product and its base-2
// form another): an exponent of 64 at 2^30.  From 2^10 on (base 2; half a step of
// 2^-14) a row gets a base near its reference that is taken off its scores
// before the products are added, so that scores and reference are small again.
__device__ __forceinline__ bool is_large(float reference) {
    const float r = __builtin_fabsf(reference);
    return r >= 0x1p10f && r < INFINITY;
}

// Where the 32 x 32 scores of queries from i0 and keys from j0 lie against the
// radius: -1 all at or before -radius, 1 all at or past it, 0 otherwise.
__device__ __forceinline__ int side_of(int32_t j0, int32_t i0, int32_t pos, int32_t R) {
    const int32_t d = j0 - i0 - pos;
    return d + 31 <= -R ? -1 : (d - 31 >= R ? 1 : 0);
}

// The backward pass's base of a row of large lse.
__device__ __forceinline__ float large_base(float lse, float scale) { return lse / scale; }

// A row's normaliser in base 2; one that empties a row without keys.
__device__ __forceinline__ float base2_lse(float lse) {
    return lse == -INFINITY ? INFINITY : lse * kLog2e;
}

// ---------------------------------------------------------------- per sequence
__device__ __forceinline__ int32_t query_position(const AttnArgs& a, int b) {
    if (!a.q_pos_dev) return a.q_pos;
    constexpr int32_t far = 1 << 29;  // as the host checks the number
    const int32_t p = __builtin_amdgcn_readfirstlane(a.q_pos_dev[b]);
    return p < -far ? -far : (p > far ? far : p);
}

// Keys that some query sees: the others are not read, whatever lies there.
__device__ __forceinline__ int32_t key_count(const AttnArgs& a, int b, int32_t pos) {
    int32_t n = a.Tk;
    if (a.k_len) {
        n = __builtin_amdgcn_readfirstlane(a.k_len[b]);
        n = n > a.Tk ? a.Tk : n;
    }
    if (a.causal && a.Tq + pos < n) n = a.Tq + pos;
    return n < 0 ? 0 : n;
}

// Workgroups go to the 8 XCDs in turn.  The workgroups of one group (a
// sequence's head) read the same rows, so they get numbers of one XCD and share
// its L2; successive groups go to successive XCDs, which spreads sequences of
// different lengths.  Items of one size go group by group; items of falling
// size (a causal mask) go size by size, the largest first.
enum WorkOrder {
    kEven,       // one size
    kFalling,    // one workgroup a CU at a time: who is done takes the next size
    kFallingTwo  // two or more at a time: every second 32 (an XCD's CUs) in
                 // reverse, so that a large one has a small one beside it (a
                 // prompt of 4093 tokens and 16 heads: 99 us, kFalling 101,
                 // kEven 124)
};
// False for a number past the work.
__device__ __forceinline__ bool xcd_work(uint32_t groups, uint32_t per_group, WorkOrder order,
                                         uint32_t& group, uint32_t& item) {
    const uint32_t x = blockIdx.x & 7;
    uint32_t s = blockIdx.x >> 3;
    if (order == kEven) {
        group = (s / per_group) * 8 + x;
        item = s % per_group;
        return group < groups;
    }
    const uint32_t mine = (groups + 7 - x) / 8;  // groups of this XCD
    if (s >= mine * per_group) return false;
    if (order == kFallingTwo && (s & 32) && (s | 31) < mine * per_group) s ^= 31;
    item = s / mine;
    group = (s % mine) * 8 + x;
    return true;
}
inline unsigned xcd_grid(int64_t groups, int64_t per_group) {
    return (unsigned)((groups + 7) / 8 * 8 * per_group);
}

inline int32_t attn_tiles(int32_t T) { return (T + kTileRows - 1) / kTileRows; }

// ---------------------------------------------------------------- results
// A query's row from the accumulators (column 32 d + 8 (r >> 2) + 4 half +
// (r & 3) in register r of block d), its reference (the base, m above it in base
// 2) and sum l.  Bases are scores before the scale; of the kernel for few
// queries, base-2 ones.
template <typename T, int DP>
__device__ __forceinline__ void write_rows(const AttnArgs& a, const f32x16 (&acc)[DP / 32], int b,
                                           int h, int32_t i, int64_t row, float base, float m,
                                           float l, int half) {
    // no key seen: l is 0 and so is the row (a NaN goes through)
    const float inv = l == 0.0f ? 0.0f : a.drop.scale / l;
    T* to = (T*)a.o + b * a.so.b + i * a.so.t + h * a.so.h;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * d + 8 * g + 4 * half;
            if (c >= a.D) continue;
            typename Mma<T>::x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (T)(acc[d][4 * g + e] * inv);
            *reinterpret_cast<typename Mma<T>::x4*>(to + c) = v;
        }
    if (a.lse && half == 0)
        a.lse[row] = l == 0.0f
                         ? -INFINITY
                         : base * (a.few ? kLn2 : a.scale) + (m * kLn2 + __logf(l));
}

// The same of one split, to be joined.
template <int DP>
__device__ __forceinline__ void write_split(const AttnArgs& a, const f32x16 (&acc)[DP / 32],
                                            int64_t row, int split, float base, float m, float l,
                                            int half) {
    float* to = a.split_o + (row * a.splits + split) * a.D;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * d + 8 * g + 4 * half;
            if (c < a.D)
                *reinterpret_cast<f4*>(to + c) = f4{acc[d][4 * g], acc[d][4 * g + 1],
                                                    acc[d][4 * g + 2], acc[d][4 * g + 3]};
        }
    if (half == 0) a.split_ml[row * a.splits + split] = f4{base, m, l, 0.0f};
}

// ---------------------------------------------------------------- launchers
// How a forward call divides its work: by the kernel for few queries or the one
// for many, and the keys over this many workgroups.
struct AttnSplits {
    bool few;
    int32_t splits;
};
AttnSplits attn_splits(int32_t B, int32_t H, int32_t Hkv, int32_t Tq, int32_t Tk);

hipError_t launch_attn_few(const AttnArgs& a, int32_t dtype, hipStream_t st);
hipError_t launch_attn_forward(const AttnArgs& a, int32_t dtype, hipStream_t st);
hipError_t launch_attn_backward(const AttnArgs& a, int32_t dtype, float* dtable, bool accumulate,
                                hipStream_t st);

}  // namespace onebit
