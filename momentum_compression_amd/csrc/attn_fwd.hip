// Attention with a relative position bias and dropout, forward:
//
//   s_ij = scale q_i . k_j + bias(j - i - pos),  P = softmax over the seen keys
//   o_i  = sum_j P_ij keep_ij v_j / (kept share),   lse_i = log sum_j exp s_ij
//
// One pass over the keys with the running maximum and sum; scores and weights
// stay in registers.  A wave has 32 queries as the columns of
// S^T = K Q^T, so a query's whole softmax lies in one lane and its other half,
// and the rounded weights are the B operand of O^T += V^T P^T as they are.
#include "attention.h"

namespace onebit {

namespace {

// Tile type of the bias for one wave: the whole tile before or past the
// radius has one value.
enum BiasKind { kNoBias, kBelow, kAbove, kWindow };

// Heads of 64 run four workgroups a CU, which leaves 128 registers; with three
// and 168 the same times (with bias and dropout 16 sequences of 128 ... 512 tokens
// and 16 heads 37.5 us, without a bias 8 of 512 24.6).
template <typename T, int DP, bool BIAS, bool DROP, bool SPLIT>
__global__ __launch_bounds__(kThreads, DP == 64 ? 4 : 2) void attn_fwd_kernel(AttnArgs a) {
    extern __shared__ __align__(16) char lds[];
    using x8 = typename Mma<T>::x8;
    constexpr int kc_n = DP / 16, db_n = DP / 32;
    const uint32_t tiles_q = (a.Tq + kTileRows - 1) / kTileRows;
    uint32_t bh, item;
    if (!xcd_work((uint32_t)a.B * a.H, tiles_q * a.splits, a.causal ? kFallingTwo : kEven, bh,
                  item)) return;
    // under a causal mask the last queries have the most keys: first
    const int qt = (int)(tiles_q - 1 - item / a.splits);
    const int split = (int)(item % a.splits);
    const int h = (int)(bh % a.H), b = (int)(bh / a.H);
    const int lane = lane_id(), wave = wave_id(), half = lane >> 5;
    const int32_t pos = query_position(a, b), n_keys = key_count(a, b, pos);
    const int32_t iw = qt * kTileRows + wave * kRows;  // the wave's first query
    const int32_t i = iw + (lane & 31);
    const int R = a.bias.radius;

    float* window = reinterpret_cast<float*>(lds + 4 * tile_bytes<DP>());

    const T* kp = (const T*)a.k + b * a.sk.b + (int64_t)(h / (a.H / a.Hkv)) * a.sk.h;
    const T* vp = (const T*)a.v + b * a.sv.b + (int64_t)(h / (a.H / a.Hkv)) * a.sv.h;
    x8 qf[kc_n];
    load_frags<T, DP>(qf, (const T*)a.q + b * a.sq.b + h * a.sq.h, a.sq.t, i, i < a.Tq, a.D, lane);

    // keys this workgroup goes over, and the last one each query sees
    int32_t first = 0, end = n_keys;
    const int32_t last_q = (qt + 1) * kTileRows < a.Tq ? (qt + 1) * kTileRows - 1 : a.Tq - 1;
    if (a.causal && last_q + pos + 1 < end) end = last_q + pos + 1;
    if (SPLIT) {
        first = split * a.split_tiles * kStep;
        const int32_t stop = first + a.split_tiles * kStep;
        if (stop < end) end = stop;
    }
    const int32_t limit = a.causal && i + pos < n_keys - 1 ? i + pos : n_keys - 1;
    const int32_t limit_lo = a.causal && iw + pos < n_keys - 1 ? iw + pos : n_keys - 1;
    const int32_t limit_hi = a.causal && iw + 31 + pos < n_keys - 1 ? iw + 31 + pos : n_keys - 1;

    f32x16 acc[db_n];
#pragma unroll
    for (int d = 0; d < db_n; ++d) acc[d] = f32x16{};
    float m = -INFINITY, l = 0.0f;
    const float scale2 = a.scale * kLog2e;
    const uint64_t drop_row = ((uint64_t)b * a.H + h) * (uint64_t)a.Tq + (uint64_t)i;
    const uint32_t step = DROP ? a.drop.step + (a.drop.step_dev ? *a.drop.step_dev : 0u) : 0u;

    const Feed<T, DP> ks(kp, a.sk.t, a.D, wave, lane), vs(vp, a.sv.t, a.D, wave, lane);
    if (first < end) {
        ks.load(lds, first, n_keys, wave);
        vs.load(lds + tile_bytes<DP>(), first, n_keys, wave);
    }
    if (BIAS) fill_window(window, a.bias, h, a.scale);
    int buf = 0;
    for (int32_t j0 = first; j0 < end; j0 += kStep, buf ^= 1) {
        char* kt = lds + buf * 2 * tile_bytes<DP>();
        char* vt = kt + tile_bytes<DP>();
        // this tile (and the window) is there, and the other buffer is read
        tiles_barrier();
        if (j0 + kStep < end) {
            char* next = lds + (buf ^ 1) * 2 * tile_bytes<DP>();
            ks.load(next, j0 + kStep, n_keys, wave);
            vs.load(next + tile_bytes<DP>(), j0 + kStep, n_keys, wave);
        }
        if (j0 > limit_hi) continue;

        // the products start from the bias; where the tile has one value of it
        // that is added in the exponential's argument
        int kind = kNoBias;
        const int32_t d_lo = j0 - (iw + 31) - pos, d_hi = j0 + kStep - 1 - iw - pos;
        if (BIAS) kind = d_hi <= -R ? kBelow : (d_lo >= R ? kAbove : kWindow);
        f32x16 s[2] = {};
        float add = 0.0f;
        if (BIAS && kind == kWindow) {
            const float* at = window + (j0 + 8 * half - i - pos + R + kPad);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[u][r] = at[32 * u + 16 * (r >> 3) + (r & 7)];
        } else if (BIAS) {
            add = window[kind == kBelow ? 0 : 2 * R + 2 * kPad] * scale2;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int kc = 0; kc < kc_n; ++kc)
                s[u] = Mma<T>::mul(row_frag<T, DP>(kt, 32 * u, kc, lane), qf[kc], s[u]);
        }
        if (j0 + kStep - 1 > limit_lo) {
            const int32_t seen = limit - j0 - 8 * half;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (32 * u + 16 * (r >> 3) + (r & 7) > seen) s[u][r] = -INFINITY;
        }
        float mx = s[0][0];
#pragma unroll
        for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[0][r]);
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[1][r]);
        mx = __builtin_fmaf(fmaxf(mx, other_half(mx)), scale2, add);
        // The reference value m follows the maximum only when that is more
        // than 2^8 above it: weights up to 256 lose nothing, and most tiles
        // leave the sums as they are.
        if (__any(mx > m + 8.0f)) {
            const float m_new = fmaxf(m, mx);
            const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - m_new);
            // sums from a large reference far below may not be numbers: gone,
            // not multiplied (a NaN of a score stays in l)
            const bool gone = alpha == 0.0f && is_large(m);
            if (__builtin_expect(__any(gone), 0)) {
                if (gone && l == l) l = 0.0f;
#pragma unroll
                for (int d = 0; d < db_n; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[d][r] = gone ? 0.0f : acc[d][r];
            }
            l *= alpha;
#pragma unroll
            for (int d = 0; d < db_n; ++d) acc[d] *= alpha;
            m = m_new;
        }
        add -= m == -INFINITY ? 0.0f : m;  // no key seen yet
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][8 * c + e], scale2, add));
                }
                l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
                if (DROP) {
                    uint32_t wd[4];
                    drop_draws(wd, (uint32_t)(j0 + 32 * u + 16 * c + 8 * half) >> 3, drop_row, step,
                               a.drop.k0, a.drop.k1);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (!drop_keep(wd, e, a.drop.threshold)) p[e] = 0.0f;
                }
                // weights rounded to the element type for the product, as the
                // values they meet are: relative to 1, half a step
                const x8 pb = pack8<T>(p);
#pragma unroll
                for (int d = 0; d < db_n; ++d)
                    acc[d] = Mma<T>::mul(col_frag<T, DP>(vt, 32 * u + 16 * c, d, lane), pb, acc[d]);
            }
        }
    }

    l += other_half(l);
    const int64_t row = ((int64_t)b * a.H + h) * a.Tq + i;
    bool again = is_large(m);
    if (SPLIT && BIAS && __builtin_expect(__any(again), 0)) {
        // A split of keys with a low bias alone: the row's nearest key, in some
        // split, may lie so far above that these have no weight.
        const int32_t j = i + pos < limit ? (i + pos > 0 ? i + pos : 0) : (limit > 0 ? limit : 0);
        x8 kf[kc_n];
        load_frags<T, DP>(kf, kp, a.sk.t, j, true, a.D, lane);
        float near = 0.0f;
#pragma unroll
        for (int kc = 0; kc < kc_n; ++kc)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                near = __builtin_fmaf((float)qf[kc][e], (float)kf[kc][e], near);
        near += other_half(near);
        int32_t d = j - i - pos;
        d = d < -R ? -R : (d > R ? R : d);
        near = (near + window[d + R + kPad]) * scale2;
        if (again && near > m + 256.0f) {
            again = false;
            m = -INFINITY;
            if (l == l) l = 0.0f;
#pragma unroll
            for (int x = 0; x < db_n; ++x) acc[x] = f32x16{};
        }
    }
    if (i < a.Tq && !again) {
        if (SPLIT) write_split<DP>(a, acc, row, split, 0.0f, m, l, half);
        else write_rows<T, DP>(a, acc, b, h, i, row, 0.0f, m, l, half);
    }

    // Rows of large references once more: the reference is what holds of them,
    // and becomes the base.  Scores are rounded before the maximum comes off, so
    // that no weight passes 1.  32 keys at a time, a tile after the other.
    __shared__ uint32_t waves_large[kWaves];
    if (lane == 0) waves_large[wave] = __any(again);
    __syncthreads();  // the tiles are read, too
    const bool none = !(waves_large[0] | waves_large[1] | waves_large[2] | waves_large[3]);
    if (__builtin_expect(none, 1)) return;
    // The generator's keys, and below the lane's addresses, anew: kept through
    // the first pass for this one they would go to memory (with that, launches
    // take up to 5 us longer).
    uint32_t k0 = a.drop.k0, k1 = a.drop.k1;
    asm volatile("" : "+s"(k0), "+s"(k1));
    const float base = again ? m / scale2 : 0.0f;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < db_n; ++d) acc[d] = f32x16{};
    for (int32_t j0 = first; j0 < end; j0 += kStep) {
        ks.load(lds, j0, n_keys, wave);
        vs.load(lds + tile_bytes<DP>(), j0, n_keys, wave);
        tiles_barrier();
#pragma unroll 1
        for (int u = 0; u < kStep; u += 32) {
            const int32_t js = j0 + u;
            if (js > limit_hi) break;
            int lane_now = lane;
            asm volatile("" : "+v"(lane_now));
            const int lane = lane_now, half = lane >> 5;
            const int side = BIAS ? side_of(js, iw, pos, R) : 0;
            f32x16 s = {};
            float flat = 0.0f;
            if (BIAS && side == 0) {
                const float* at = window + (js + 8 * half - i - pos + R + kPad);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = at[16 * (r >> 3) + (r & 7)] - base;
            } else {
                if (BIAS) flat = window[side < 0 ? 0 : 2 * R + 2 * kPad];
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = flat - base;
            }
#pragma unroll
            for (int kc = 0; kc < kc_n; ++kc)
                s = Mma<T>::mul(row_frag<T, DP>(lds, u, kc, lane), qf[kc], s);
            const int32_t seen = limit - js - 8 * half;
            float mx = -INFINITY;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[r] = 16 * (r >> 3) + (r & 7) > seen ? -INFINITY : s[r] * scale2;
                mx = fmaxf(mx, s[r]);
            }
            const float m_new = fmaxf(m, fmaxf(mx, other_half(mx)));
            const float m_use = m_new == -INFINITY ? 0.0f : m_new;
            const float alpha = __builtin_amdgcn_exp2f(m - m_use);
            l *= alpha;
#pragma unroll
            for (int d = 0; d < db_n; ++d) acc[d] *= alpha;
            m = m_new;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(s[8 * c + e] - m_use);
                l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
                if (DROP) {
                    uint32_t wd[4];
                    drop_draws(wd, (uint32_t)(js + 16 * c + 8 * half) >> 3, drop_row, step,
                               k0, k1);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (!drop_keep(wd, e, a.drop.threshold)) p[e] = 0.0f;
                }
                const x8 pb = pack8<T>(p);
#pragma unroll
                for (int d = 0; d < db_n; ++d)
                    acc[d] = Mma<T>::mul(
                        col_frag<T, DP>(lds + tile_bytes<DP>(), u + 16 * c, d, lane), pb, acc[d]);
            }
        }
        __syncthreads();  // this tile is read
    }
    l += other_half(l);
    if (i >= a.Tq || !again) return;
    if (SPLIT) write_split<DP>(a, acc, row, split, base, m, l, half);
    else write_rows<T, DP>(a, acc, b, h, i, row, base, m, l, half);
}

// Joins the splits of a row (at most 64, one a lane for their weights), two
// columns a lane.  WAVES waves share a row's splits where there are many: one
// wave would take 14 us for 32 of them, a load after the other.
template <typename T, int WAVES>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a) {
    __shared__ float2 sums[kWaves][64];
    const int64_t rows = (int64_t)a.B * a.H * a.Tq;
    const int wave = wave_id(), lane = lane_id();
    const int64_t row = (int64_t)blockIdx.x * (kWaves / WAVES) + wave / WAVES;
    const bool ok = row < rows;
    float base = 0.0f, m = -INFINITY, l = 0.0f;
    if (ok && lane < a.splits) {
        const f4 x = a.split_ml[row * a.splits + lane];
        base = x[0];
        m = x[1];
        l = x[2];
    }
    const float unit = a.few ? 1.0f : a.scale * kLog2e;  // of the bases
    float origin = 0.0f, top = m;
    if (__any(base != 0.0f)) {
        // all to one split's base: the highest's, as far as a first one shows
        for (int k = 0; k < 2; ++k) {
            const float above = m == -INFINITY ? m : (base - origin) * unit + m;
            float most = above;
            for (int off = 32; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
            const uint64_t at = __ballot(above == most);
            if (at) origin = __shfl(base, __builtin_ctzll(at), 64);
        }
        if (m != -INFINITY) m += (base - origin) * unit;
        top = m;
    }
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    const float weight = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
    l *= weight;
    for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off, 64);
    const int c = 2 * lane;
    float2 o = {0.0f, 0.0f};
    // Every lane goes through the loop, those without a column too: they hold
    // splits' weights for the others.
    const bool mine = ok && c < a.D;
    const float* from = a.split_o + (mine ? row * a.splits * (int64_t)a.D + c : 0);
    for (int s0 = wave % WAVES; s0 < a.splits; s0 += 8 * WAVES) {
        float2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = s0 + k * WAVES;
            v[k] = mine && s < a.splits
                       ? *reinterpret_cast<const float2*>(from + (int64_t)s * a.D)
                       : float2{0.0f, 0.0f};
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float w = __uint_as_float(__builtin_amdgcn_readlane(
                __float_as_uint(weight), (s0 + k * WAVES) & 63));
            o.x = __builtin_fmaf(w, v[k].x, o.x);
            o.y = __builtin_fmaf(w, v[k].y, o.y);
        }
    }
    if (WAVES > 1) {
        sums[wave][lane] = o;
        __syncthreads();
        if (wave % WAVES) return;
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            o.x += sums[wave + w][lane].x;
            o.y += sums[wave + w][lane].y;
        }
    }
    if (!ok) return;
    const float inv = l == 0.0f ? 0.0f : a.drop.scale / l;
    const int i = (int)(row % a.Tq);
    const int64_t bh = row / a.Tq;
    T* to = (T*)a.o + (bh / a.H) * a.so.b + i * a.so.t + (bh % a.H) * a.so.h;
    if (c < a.D) {
        to[c] = (T)(o.x * inv);
        to[c + 1] = (T)(o.y * inv);
    }
    if (a.lse && lane == 0)
        a.lse[row] = l == 0.0f
                         ? -INFINITY
                         : origin * (a.few ? kLn2 : a.scale) + (top * kLn2 + __logf(l));
}

template <typename T, int DP, bool BIAS, bool DROP>
void run(const AttnArgs& a, hipStream_t st) {
    const size_t lds = 4 * tile_bytes<DP>() +
                       (BIAS ? (2 * (size_t)a.bias.radius + 1 + 2 * kPad) * sizeof(float) : 0);
    const dim3 grid(xcd_grid((int64_t)a.B * a.H, (int64_t)attn_tiles(a.Tq) * a.splits));
    if (a.splits > 1)
        hipLaunchKernelGGL((attn_fwd_kernel<T, DP, BIAS, DROP, true>), grid, dim3(kThreads), lds,
                           st, a);
    else
        hipLaunchKernelGGL((attn_fwd_kernel<T, DP, BIAS, DROP, false>), grid, dim3(kThreads), lds,
                           st, a);
}

template <typename T, int DP>
void run_d(const AttnArgs& a, hipStream_t st) {
    const bool bias = a.bias.radius > 0, drop = a.drop.threshold != kDropAll;
    if (bias && drop) run<T, DP, true, true>(a, st);
    else if (bias) run<T, DP, true, false>(a, st);
    else if (drop) run<T, DP, false, true>(a, st);
    else run<T, DP, false, false>(a, st);
}

template <typename T>
hipError_t run_t(const AttnArgs& a, int32_t dtype, hipStream_t st) {
    hipError_t e;
    if (a.few) {
        e = launch_attn_few(a, dtype, st);
    } else {
        if (a.D <= 64) run_d<T, 64>(a, st);
        else run_d<T, 128>(a, st);
        e = hipGetLastError();
    }
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t rows = (int64_t)a.B * a.H * a.Tq;
    if (a.splits > 8)
        hipLaunchKernelGGL((attn_join_kernel<T, kWaves>), dim3((unsigned)rows), dim3(kThreads), 0,
                           st, a);
    else
        hipLaunchKernelGGL((attn_join_kernel<T, 1>), dim3((unsigned)((rows + kWaves - 1) / kWaves)),
                           dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace

AttnSplits attn_splits(int32_t B, int32_t H, int32_t Hkv, int32_t Tq, int32_t Tk) {
    AttnSplits p = {false, 1};
    if (B == 0 || Tq == 0) return p;
    // all queries of a key head in one wave's columns
    p.few = (int64_t)Tq * (H / Hkv) <= kRows;
    const int64_t work = p.few ? (int64_t)B * Hkv : (int64_t)B * H * attn_tiles(Tq);
    // two workgroups a CU; few: a wave with two tiles of 32 keys at least,
    // otherwise four tiles of 64.  Twice as many workgroups even out lengths but
    // start and end twice (few, 32 sequences and 4 key heads: 97 -> 100 us of
    // 8192 keys, 70 -> 72 of a quarter to all; 64, 8 and 1024 keys 50 -> 60)
    const int64_t want = 512;
    const int64_t most = (Tk + (p.few ? 2 * kWaves * kRows : 4 * kStep) - 1) /
                         (p.few ? 2 * kWaves * kRows : 4 * kStep);
    int64_t n = (want + work - 1) / work;
    if (n > most) n = most;
    if (n > 64) n = 64;
    p.splits = n < 1 ? 1 : (int32_t)n;
    return p;
}

hipError_t launch_attn_forward(const AttnArgs& a, int32_t dtype, hipStream_t st) {
    return dtype == ONEBIT_BF16 ? run_t<bf16>(a, dtype, st) : run_t<f16>(a, dtype, st);
}

}  // namespace onebit
