// Attention with a relative position bias and dropout, backward.  With keep_ij
// (0 or 1 / kept share), P from the scores and the forward's lse:
//
//   dP_ij = keep_ij (dO_i . v_j),   delta_i = sum_j P_ij dP_ij = dO_i . o_i
//   dS_ij = P_ij (dP_ij - delta_i)
//   dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i
//   dv_j = sum_i keep_ij P_ij dO_i, dtable[b][h] = sum of dS over bucket b
//
// Two passes compute the scores again, one with the queries and one with the
// keys as a wave's columns, so that each gradient is summed by one workgroup
// in a fixed order: no atomics, the same bits on every run.
#include <type_traits>

#include "attention.h"

namespace onebit {

namespace {

// Up to kShort queries and keys (the call's lengths, padding included) the
// products take P and dS as a rounded part and the rounded rest, twice the
// products of these.  The roundings of P and dS add to the result's own, each as
// large: measured error of dq, dk and dv over a plain form's that rounds only
// results 1.4 without the rest, whatever the lengths (heads of 8 ... 128, rows of
// 2 ... 600 keys), and 1.0 with it.  A few short sequences are as fast with it
// (2 of 37 tokens, backward 25.7 us, 25.1 without), many nearly (64 of 64
// tokens, 16 heads of 64: 54.6 and 53.3); at longer ones the products count.
constexpr int kShort = 64;

// What rounding left of eight values.
template <typename T>
__device__ __forceinline__ typename Mma<T>::x8 pack_rest(const float* p,
                                                         typename Mma<T>::x8 rounded) {
    typename Mma<T>::x8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (T)(p[e] - (float)rounded[e]);
    return r;
}

// Queries as columns: dq and, for the second pass, delta in binary32.  With any value
// delta' near it, delta = delta' + sum P (dP - delta') / sum P; the sum of dS comes
// beside dS, and the sum of P is 1 but for the roundings of lse: 5 times 2^-24 of it,
// 2^-12 at the largest that rows without a base have, of a correction that is itself
// 2^-8 of delta (summed and divided by, it took 3 % longer).  dq itself takes delta' =
// dO . o of the rounded output, which is there before the pass: off by half a step of
// the element type times the row's output.  That is small beside what dS is rounded by
// where many keys share the weight, but not where few do, so workgroups with at most
// kTwice keys make the pass twice, the first time for the sums alone and from the first
// key's dP: a query that sees one key then has delta = dP to the bit, and dS = 0 in
// both passes over the scores.  (Over more keys a query whose weight lies on one of
// them by its scores keeps the half step times that key in dq, where dk and dtable have
// the exact delta.)  Measured error of dq against 64 bits, in units of the output's own
// rounding, with one pass and with two: 37 keys 1.51 and 1.41, 256 keys 1.47 and 1.43,
// fp16 rows of at most 5 keys 2.9 and 1.4; with one pass 512 keys 1.46, 1000 keys 1.44.
// Two passes up to 512 keys would take 69 instead of 50 us for 16 sequences of up to
// 512 keys and 16 heads of 64; one pass always, 46.
//
// The kept share's scale is common to all dP: dS here is P (keep dP' - delta')
// with dP' and delta' before it, and it enters once, with the result's scale.
constexpr int kTwice = 256;

template <typename T, int DP, bool BIAS, bool DROP, bool SHORT>
__global__ __launch_bounds__(kThreads, DP == 64 && !SHORT ? 3 : 2) void attn_dq_kernel(AttnArgs a) {
    extern __shared__ __align__(16) char lds[];
    using x8 = typename Mma<T>::x8;
    constexpr int kc_n = DP / 16, db_n = DP / 32;
    const uint32_t tiles_q = (a.Tq + kTileRows - 1) / kTileRows;
    uint32_t bh, item;
    if (!xcd_work((uint32_t)a.B * a.H, tiles_q, a.causal ? kFallingTwo : kEven, bh, item)) return;
    const int qt = (int)(tiles_q - 1 - item);
    const int h = (int)(bh % a.H), b = (int)(bh / a.H);
    const int lane = lane_id(), wave = wave_id(), half = lane >> 5;
    const int32_t pos = query_position(a, b), n_keys = key_count(a, b, pos);
    const int32_t iw = qt * kTileRows + wave * kRows;
    const int32_t i = iw + (lane & 31);
    const int R = a.bias.radius;

    float* window = reinterpret_cast<float*>(lds + 4 * tile_bytes<DP>());

    const int hk = h / (a.H / a.Hkv);
    const T* kp = (const T*)a.k + b * a.sk.b + hk * a.sk.h;
    const T* vp = (const T*)a.v + b * a.sv.b + hk * a.sv.h;
    x8 qf[kc_n], gf[kc_n];
    load_frags<T, DP>(qf, (const T*)a.q + b * a.sq.b + h * a.sq.h, a.sq.t, i, i < a.Tq, a.D, lane);
    load_frags<T, DP>(gf, (const T*)a.d_o + b * a.sdo.b + h * a.sdo.h, a.sdo.t, i, i < a.Tq, a.D,
                      lane);
    const int64_t row = ((int64_t)b * a.H + h) * a.Tq + i;
    const float lse2 = i < a.Tq ? base2_lse(a.lse[row]) : INFINITY;
    float delta = 0.0f;
    {
        x8 of[kc_n];
        load_frags<T, DP>(of, (const T*)a.o_in + b * a.so.b + h * a.so.h, a.so.t, i, i < a.Tq, a.D,
                          lane);
#pragma unroll
        for (int kc = 0; kc < kc_n; ++kc)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                delta = __builtin_fmaf((float)of[kc][e], (float)gf[kc][e], delta);
    }
    delta += other_half(delta);
    if (DROP) delta /= a.drop.scale;

    int32_t end = n_keys;
    const int32_t last_q = (qt + 1) * kTileRows < a.Tq ? (qt + 1) * kTileRows - 1 : a.Tq - 1;
    if (a.causal && last_q + pos + 1 < end) end = last_q + pos + 1;
    const int32_t limit = a.causal && i + pos < n_keys - 1 ? i + pos : n_keys - 1;
    const int32_t limit_lo = a.causal && iw + pos < n_keys - 1 ? iw + pos : n_keys - 1;
    const int32_t limit_hi = a.causal && iw + 31 + pos < n_keys - 1 ? iw + 31 + pos : n_keys - 1;

    f32x16 acc[db_n];
#pragma unroll
    for (int d = 0; d < db_n; ++d) acc[d] = f32x16{};
    float sum = 0.0f;  // of P (dP - delta) over the row
    const float scale2 = a.scale * kLog2e;
    const uint64_t drop_row = (uint64_t)row;
    const uint32_t step = DROP ? a.drop.step + (a.drop.step_dev ? *a.drop.step_dev : 0u) : 0u;

    const Feed<T, DP> ks(kp, a.sk.t, a.D, wave, lane), vs(vp, a.sv.t, a.D, wave, lane);
    if (BIAS) fill_window(window, a.bias, h, a.scale);
    for (int pass = end <= kTwice ? 0 : 1; pass < 2; ++pass) {
        if (end > 0) {
            ks.load(lds, 0, n_keys, wave);
            vs.load(lds + tile_bytes<DP>(), 0, n_keys, wave);
        }
        int buf = 0;
        for (int32_t j0 = 0; j0 < end; j0 += kStep, buf ^= 1) {
            char* kt = lds + buf * 2 * tile_bytes<DP>();
            char* vt = kt + tile_bytes<DP>();
            // this tile (and the window) is there, and the other buffer is read
            tiles_barrier();
            if (j0 + kStep < end) {
                char* next = lds + (buf ^ 1) * 2 * tile_bytes<DP>();
                ks.load(next, j0 + kStep, n_keys, wave);
                vs.load(next + tile_bytes<DP>(), j0 + kStep, n_keys, wave);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int32_t js = j0 + 32 * u;
                if (js > limit_hi) continue;
                const int side = BIAS ? side_of(js, iw, pos, R) : 0;
                f32x16 s = {}, dp = {};
                float add = -lse2;
                if (BIAS && side == 0) {
                    const float* at = window + (js + 8 * half - i - pos + R + kPad);
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = at[16 * (r >> 3) + (r & 7)];
                } else if (BIAS) {
                    add = __builtin_fmaf(window[side < 0 ? 0 : 2 * R + 2 * kPad], scale2, -lse2);
                }
#pragma unroll
                for (int kc = 0; kc < kc_n; ++kc)
                    s = Mma<T>::mul(row_frag<T, DP>(kt, 32 * u, kc, lane), qf[kc], s);
#pragma unroll
                for (int kc = 0; kc < kc_n; ++kc)
                    dp = Mma<T>::mul(row_frag<T, DP>(vt, 32 * u, kc, lane), gf[kc], dp);
                read_ahead<1, 2 * kc_n, 4>();
                const int32_t seen = limit - js - 8 * half;
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], scale2, add));
                if (js + 31 > limit_lo) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (16 * (r >> 3) + (r & 7) > seen) s[r] = 0.0f;
                }
                if (DROP) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t wd[4];
                        drop_draws(wd, (uint32_t)(js + 16 * c + 8 * half) >> 3, drop_row, step,
                                   a.drop.k0, a.drop.k1);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (!drop_keep(wd, e, a.drop.threshold)) dp[8 * c + e] = 0.0f;
                    }
                }
                if (pass == 0 && js == 0) {  // the first key's dP, whichever half has it
                    const float other = other_half(dp[0]);
                    delta = half ? other : dp[0];
                }
                float ds[16], part[2] = {0.0f, 0.0f};
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    ds[r] = s[r] * (dp[r] - delta);
                    part[r & 1] += ds[r];
                }
                sum += part[0] + part[1];
                if (pass == 0) continue;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const x8 db = pack8<T>(ds + 8 * c);
                    const x8 dr = SHORT ? pack_rest<T>(ds + 8 * c, db) : x8{};
#pragma unroll
                    for (int d = 0; d < db_n; ++d) {
                        const x8 kd = col_frag<T, DP>(kt, 32 * u + 16 * c, d, lane);
                        acc[d] = Mma<T>::mul(kd, db, acc[d]);
                        if (SHORT) acc[d] = Mma<T>::mul(kd, dr, acc[d]);
                    }
                }
                if (!SHORT) read_ahead<2, 2 * db_n, 4>();
            }
        }
        delta += sum + other_half(sum);
        sum = 0.0f;
        if (pass == 0) __syncthreads();  // the tiles are read
    }

    const auto write = [&]() __attribute__((always_inline)) {
        if (half == 0) a.delta[row] = delta;
        const float out = DROP ? a.scale * a.drop.scale : a.scale;
        T* to = (T*)a.dq + b * a.sdq.b + i * a.sdq.t + h * a.sdq.h;
#pragma unroll
        for (int d = 0; d < db_n; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = 32 * d + 8 * g + 4 * half;
                if (c >= a.D) continue;
                typename Mma<T>::x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = (T)(acc[d][4 * g + e] * out);
                *reinterpret_cast<typename Mma<T>::x4*>(to + c) = v;
            }
    };
    const bool again = is_large(lse2);
    if (i < a.Tq && !again) write();

    // Rows of large references once more, from their bases and with the
    // normaliser above the base, which lse has lost: it is summed first, then
    // delta from the first key's dP, then dq.  32 keys at a time, a tile after
    // the other.
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
    const float base = again ? large_base(a.lse[i < a.Tq ? row : 0], a.scale) : 0.0f;
    float m = -INFINITY, l = 0.0f, norm = 0.0f;
    delta = sum = 0.0f;
    const auto sweep = [&](auto which) __attribute__((always_inline)) {
        constexpr int pass = decltype(which)::value;
        for (int32_t j0 = 0; j0 < end; j0 += kStep) {
            char* vt = lds + tile_bytes<DP>();
            ks.load(lds, j0, n_keys, wave);
            vs.load(vt, j0, n_keys, wave);
            tiles_barrier();
#pragma unroll 1
            for (int u = 0; u < kStep; u += 32) {
                const int32_t js = j0 + u;
                if (js > limit_hi) break;
                int lane_now = lane;
                asm volatile("" : "+v"(lane_now));
                const int lane = lane_now, half = lane >> 5;
                const int side = BIAS ? side_of(js, iw, pos, R) : 0;
                f32x16 s = {}, dp = {};
                if (BIAS && side == 0) {
                    const float* at = window + (js + 8 * half - i - pos + R + kPad);
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = at[16 * (r >> 3) + (r & 7)] - base;
                } else {
                    const float flat = BIAS ? window[side < 0 ? 0 : 2 * R + 2 * kPad] : 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = flat - base;
                }
#pragma unroll
                for (int kc = 0; kc < kc_n; ++kc)
                    s = Mma<T>::mul(row_frag<T, DP>(lds, u, kc, lane), qf[kc], s);
                read_ahead<1, kc_n, 2>();
                const int32_t seen = limit - js - 8 * half;
                if (pass == 0) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        s[r] = 16 * (r >> 3) + (r & 7) > seen ? -INFINITY : s[r] * scale2;
                        mx = fmaxf(mx, s[r]);
                    }
                    const float m_new = fmaxf(m, fmaxf(mx, other_half(mx)));
                    const float m_use = m_new == -INFINITY ? 0.0f : m_new;
                    l *= __builtin_amdgcn_exp2f(m - m_use);
                    m = m_new;
#pragma unroll
                    for (int r = 0; r < 16; ++r) l += __builtin_amdgcn_exp2f(s[r] - m_use);
                    continue;
                }
#pragma unroll
                for (int kc = 0; kc < kc_n; ++kc)
                    dp = Mma<T>::mul(row_frag<T, DP>(vt, u, kc, lane), gf[kc], dp);
                read_ahead<1, kc_n, 2>();
                if (DROP) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t wd[4];
                        drop_draws(wd, (uint32_t)(js + 16 * c + 8 * half) >> 3, drop_row, step,
                                   k0, k1);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (!drop_keep(wd, e, a.drop.threshold)) dp[8 * c + e] = 0.0f;
                    }
                }
                if (pass == 1 && js == 0) {
                    const float other = other_half(dp[0]);
                    delta = half ? other : dp[0];
                }
                float ds[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], scale2, -norm));
                    ds[r] = 16 * (r >> 3) + (r & 7) > seen ? 0.0f : p * (dp[r] - delta);
                    sum += ds[r];
                }
                if (pass == 1) continue;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const x8 db = pack8<T>(ds + 8 * c), dr = pack_rest<T>(ds + 8 * c, db);
#pragma unroll
                    for (int d = 0; d < db_n; ++d) {
                        const x8 kd = col_frag<T, DP>(lds, u + 16 * c, d, lane);
                        acc[d] = Mma<T>::mul(kd, db, acc[d]);
                        acc[d] = Mma<T>::mul(kd, dr, acc[d]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            __syncthreads();  // this tile is read
        }
        if (pass == 0) norm = m + __log2f(l + other_half(l));
        delta += sum + other_half(sum);
        sum = 0.0f;
    };
    sweep(std::integral_constant<int, 0>());
    sweep(std::integral_constant<int, 1>());
#pragma unroll
    for (int d = 0; d < db_n; ++d) acc[d] = f32x16{};
    sweep(std::integral_constant<int, 2>());
    if (i >= a.Tq || !again) return;
    if (half == 0) a.norm[row] = norm;
    write();
}

// Sums down the diagonals of the 32 x 32 scores' gradients of a wave (queries
// as rows, eight consecutive ones to a lane), added to the wave's bins.  The
// values go through LDS of the wave's own: a query's 32 keys, then 32 zeros
// that stay.  Lane x sums the diagonal x - 31: it reads word q + x - 31 of each
// query's row, which past either end of the keys lies among zeros (its own
// row's or the one's before), so there is nothing to select.  No two lanes own
// the same diagonal: no atomics.  `first` is the distance of lane 31's.
constexpr int kSkewRow = 64;
constexpr int kSkewFloats = 32 + 32 * kSkewRow;  // zeros before the first row

__device__ __forceinline__ void add_diagonals(const float (&ds)[16], float* skew, float* bins,
                                              int32_t first, int R, float& below, float& above,
                                              int lane) {
    const int half = lane >> 5;
    float* to = skew + 32 + 8 * half * kSkewRow + (lane & 31);
#pragma unroll
    for (int r = 0; r < 16; ++r) to[(16 * (r >> 3) + (r & 7)) * kSkewRow] = ds[r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const float* from = skew + 1 + lane;  // 32 + q (kSkewRow + 1) + lane - 31
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 32; ++q) v[q & 3] += from[q * (kSkewRow + 1)];
    const float sum = (v[0] + v[1]) + (v[2] + v[3]);
    const int32_t d = first + lane - 31;
    if (d <= -R) below += sum;
    else if (d >= R) above += sum;
    else if (lane < 63) bins[d + R] += sum;  // lane 63's diagonal is empty
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

constexpr int kRowFloats = 384;  // a query tile's rows in LDS, two buffers

// Keys as columns: dk and dv of 128 keys of one key head, over every query of
// the heads that share it, in order; with TABLE the sums of dS (from the exact
// delta, unrounded) for each distance, one part a workgroup and head.
template <typename T, int DP, bool BIAS, bool DROP, bool TABLE, bool SHORT>
__global__ __launch_bounds__(kThreads, DP == 64 ? 2 : 1) void attn_dkv_kernel(AttnArgs a) {
    extern __shared__ __align__(16) char lds[];
    using x8 = typename Mma<T>::x8;
    constexpr int kc_n = DP / 16, db_n = DP / 32, kUnroll = TABLE && DP == 128 ? 1 : 2;
    const uint32_t tiles_k = (a.Tk + kTileRows - 1) / kTileRows;
    uint32_t bh, item;
    const WorkOrder order = !a.causal ? kEven : (DP == 64 ? kFallingTwo : kFalling);
    if (!xcd_work((uint32_t)a.B * a.Hkv, tiles_k, order, bh, item)) return;
    // under a causal mask the first keys have the most queries: first
    const int kt_i = (int)item;
    const int hk = (int)(bh % a.Hkv), b = (int)(bh / a.Hkv);
    const int lane = lane_id(), wave = wave_id(), half = lane >> 5;
    const int32_t pos = query_position(a, b), n_keys = key_count(a, b, pos);
    const int32_t jw = kt_i * kTileRows + wave * kRows;
    const int32_t j = jw + (lane & 31);
    const int R = a.bias.radius, group = a.H / a.Hkv, bins_n = 2 * R + 1;

    // negative normaliser and delta of a tile's queries, and bases where one
    // has any; two buffers
    float* rows_lds = reinterpret_cast<float*>(lds + 4 * tile_bytes<DP>());
    uint32_t* kept_lds = reinterpret_cast<uint32_t*>(rows_lds + kRowFloats) + wave * 32;
    float* skew =
        rows_lds + kRowFloats + (DROP ? kWaves * 32 : 0) + (TABLE ? wave * kSkewFloats : 0);
    float* window =
        rows_lds + kRowFloats + (DROP ? kWaves * 32 : 0) + (TABLE ? kWaves * kSkewFloats : 0);
    float* all_bins = window + window_floats(R);
    float* bins = all_bins + wave * bins_n;
    float below = 0.0f, above = 0.0f;  // dS at or past the radius

    x8 kf[kc_n], vf[kc_n];
    load_frags<T, DP>(kf, (const T*)a.k + b * a.sk.b + hk * a.sk.h, a.sk.t, j, j < n_keys, a.D,
                      lane);
    load_frags<T, DP>(vf, (const T*)a.v + b * a.sv.b + hk * a.sv.h, a.sv.t, j, j < n_keys, a.D,
                      lane);
    f32x16 dk[db_n], dv[db_n];
#pragma unroll
    for (int d = 0; d < db_n; ++d) dk[d] = dv[d] = f32x16{};
    const float scale2 = a.scale * kLog2e;
    const uint32_t step = DROP ? a.drop.step + (a.drop.step_dev ? *a.drop.step_dev : 0u) : 0u;
    const int key_bit = drop_bit(lane & 31);

    // queries that see a key of the tile, for each head of the group in turn
    int32_t first = a.causal ? kt_i * kTileRows - pos : 0;
    first = first < 0 ? 0 : first / kStep * kStep;
    const int32_t per_head =
        kt_i * kTileRows < n_keys && first < a.Tq ? (a.Tq - first + kStep - 1) / kStep : 0;
    const uint32_t total = (uint32_t)per_head * (uint32_t)group;

    float row_lse = 0.0f, row_delta = 0.0f;
    bool large = false;  // the tile has a row with a base
    int32_t head = hk * group, i0 = first;  // of the tile to load next
    Feed<T, DP> qs((const T*)a.q + b * a.sq.b + head * a.sq.h, a.sq.t, a.D, wave, lane);
    Feed<T, DP> gs((const T*)a.d_o + b * a.sdo.b + head * a.sdo.h, a.sdo.t, a.D, wave, lane);
    int64_t head_row = ((int64_t)b * a.H + head) * a.Tq;
    const auto load = [&](int to) {
        const int32_t i = i0 + lane;
        const int64_t row = head_row + i;
        row_lse = i < a.Tq ? a.lse[row] : -INFINITY;
        if (wave == 1) row_delta = i < a.Tq ? a.delta[row] : 0.0f;
        char* tile = lds + to * 2 * tile_bytes<DP>();
        qs.load(tile, i0, a.Tq, wave);
        gs.load(tile + tile_bytes<DP>(), i0, a.Tq, wave);
    };
    const auto keep_rows = [&](int to) {
        float value = -base2_lse(row_lse);
        const bool far = is_large(value);
        large = __any(far);
        if (wave == 0) {
            if (large) {
                if (far) value = -a.norm[head_row + i0 + lane];
                rows_lds[256 + to * 64 + lane] = far ? large_base(row_lse, a.scale) : 0.0f;
            }
            rows_lds[to * 128 + lane] = value;
        } else if (wave == 1) {
            rows_lds[to * 128 + 64 + lane] = -row_delta;
        }
    };
    // one head's sums to its part; its bins are complete
    const auto flush = [&](int h) {
        for (int off = 32; off > 0; off >>= 1) {
            below += __shfl_xor(below, off, 64);
            above += __shfl_xor(above, off, 64);
        }
        if (lane == 0) {
            bins[0] = below;
            bins[2 * R] = above;
        }
        below = above = 0.0f;
        __syncthreads();
        const int64_t part = (int64_t)b * tiles_k + kt_i, parts = (int64_t)a.B * tiles_k;
        float* to = a.partials + ((int64_t)h * parts + part) * bins_n;
        for (int x = threadIdx.x; x < bins_n; x += kThreads) {
            const float v = (all_bins[x] + all_bins[bins_n + x]) +
                            (all_bins[2 * bins_n + x] + all_bins[3 * bins_n + x]);
            to[x] = DROP ? v * a.drop.scale : v;
        }
        __syncthreads();
        for (int x = lane; x < bins_n; x += 64) bins[x] = 0.0f;
    };
    if (TABLE) {
        for (int x = lane; x < bins_n; x += 64) bins[x] = 0.0f;
        for (int x = lane; x < kSkewFloats; x += 64) skew[x] = 0.0f;
    }
    if (total > 0) {
        load(0);
        keep_rows(0);
    }
    int buf = 0, filled = -1;
    for (uint32_t t = 0; t < total; ++t, buf ^= 1) {
        const int32_t h = head, it = i0;  // this tile
        char* qt = lds + buf * 2 * tile_bytes<DP>();
        char* gt = qt + tile_bytes<DP>();
        const float* lse2 = rows_lds + buf * 128;
        const float* delta = lse2 + 64;
        const float* bases = rows_lds + 256 + buf * 64;
        if (BIAS && filled != h) {
            __syncthreads();  // the other head's window is read
            if (TABLE && filled >= 0) flush(filled);
            fill_window(window, a.bias, h, a.scale);
            filled = h;
        }
        tiles_barrier();  // this tile is there, and the other buffer is read
        const bool more = t + 1 < total;
        if (more) {
            i0 += kStep;
            if (i0 >= a.Tq) {
                i0 = first;
                ++head;
                qs.base += a.sq.h;
                gs.base += a.sdo.h;
                head_row += a.Tq;
            }
            load(buf ^ 1);
        }
        // One after the other in code too where that is large enough.  Backward
        // call of 2 x 2048 tokens and 16 heads of 128, causal: with the table 202
        // us, unrolled 205; without it unrolled 174, not 180.  Heads of 64 with
        // the table unrolled: with dropout (16 sequences of 128 ... 512 tokens)
        // 144 us, not 146; causal without (2 x 2048) 134, not 131.
#pragma unroll(kUnroll)
        for (int u = 0; u < 2; ++u) {
            const int32_t is = it + 32 * u;
            if (is >= a.Tq || (a.causal && is + 31 + pos < jw) || jw >= n_keys) continue;
            const float* lse_at = lse2 + 32 * u + 8 * half;
            const float* delta_at = delta + 32 * u + 8 * half;
            // the scores start from the bias.  dP starts from 0 as in the query
            // pass, so that both have the same bits and dS sums to 0 over a
            // row: started from -delta, the matrix instructions' rounding
            // showed in the far buckets of dtable (1.7e-6 of the table, at
            // 1000 keys)
            f32x16 s = {}, dp = {};
            const int side = BIAS ? side_of(jw, is, pos, R) : 0;
            if (BIAS && side == 0) {
                const float* at = window + (j - is - 8 * half - pos + R + kPad);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = at[-16 * (r >> 3) - (r & 7)];
            } else if (BIAS) {
                const float c = window[side < 0 ? 0 : 2 * R + 2 * kPad];
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = c;
            }
            if (large) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[r] -= bases[32 * u + 8 * half + 16 * (r >> 3) + (r & 7)];
            }
#pragma unroll
            for (int kc = 0; kc < kc_n; ++kc)
                s = Mma<T>::mul(row_frag<T, DP>(qt, 32 * u, kc, lane), kf[kc], s);
#pragma unroll
            for (int kc = 0; kc < kc_n; ++kc)
                dp = Mma<T>::mul(row_frag<T, DP>(gt, 32 * u, kc, lane), vf[kc], dp);
            read_ahead<1, 2 * kc_n, 6>();
#pragma unroll
            for (int r = 0; r < 16; ++r)
                s[r] = __builtin_amdgcn_exp2f(
                    __builtin_fmaf(s[r], scale2, lse_at[16 * (r >> 3) + (r & 7)]));
            if ((a.causal && is + pos < jw + 31) || jw + 31 >= n_keys) {
                // a key past the sequence is seen by no query
                const int32_t from = j >= n_keys ? 64 : (a.causal ? j - pos - is - 8 * half : 0);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (16 * (r >> 3) + (r & 7) < from) s[r] = 0.0f;
            }
            if (DROP) {
                // lane (query q, half) draws the keys 16 half ... + 15 of its
                // query; a query's 32 decisions go to LDS as a word, bit
                // drop_bit(key)
                const uint64_t row = ((uint64_t)b * a.H + h) * (uint64_t)a.Tq +
                                     (uint64_t)(is + (lane & 31));
                uint32_t dropped = 0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t wd[4];
                    drop_draws(wd, (uint32_t)(jw + 16 * half + 8 * c) >> 3, row, step, a.drop.k0,
                               a.drop.k1);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        dropped |= drop_pair(wd[k], a.drop.threshold) << (4 * c + k);
                }
                dropped <<= 8 * half;
                dropped |= __float_as_uint(other_half(__uint_as_float(dropped)));
                if (half == 0) kept_lds[lane] = ~dropped;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
            float ds[16], p[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int q = 16 * (r >> 3) + (r & 7);
                p[r] = s[r];
                float g = dp[r];
                if (DROP) {
                    const int m = __builtin_amdgcn_sbfe((int)kept_lds[q + 8 * half], key_bit, 1);
                    p[r] = __int_as_float(__float_as_int(p[r]) & m);
                    g = __int_as_float(__float_as_int(g) & m);
                }
                ds[r] = s[r] * (g + delta_at[q]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const x8 pb = pack8<T>(p + 8 * c), db = pack8<T>(ds + 8 * c);
                const x8 pr = SHORT ? pack_rest<T>(p + 8 * c, pb) : x8{};
                const x8 dr = SHORT ? pack_rest<T>(ds + 8 * c, db) : x8{};
#pragma unroll
                for (int d = 0; d < db_n; ++d) {
                    const x8 gd = col_frag<T, DP>(gt, 32 * u + 16 * c, d, lane);
                    dv[d] = Mma<T>::mul(gd, pb, dv[d]);
                    if (SHORT) dv[d] = Mma<T>::mul(gd, pr, dv[d]);
                    const x8 qd = col_frag<T, DP>(qt, 32 * u + 16 * c, d, lane);
                    dk[d] = Mma<T>::mul(qd, db, dk[d]);
                    if (SHORT) dk[d] = Mma<T>::mul(qd, dr, dk[d]);
                }
            }
            if (!SHORT) read_ahead<2, 4 * db_n, 8>();
            if (DROP) {  // the words are read before the next ones are written
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
            if (TABLE) {
                if (side == 0) {
                    add_diagonals(ds, skew, bins, jw - is - pos, R, below, above, lane);
                } else {
                    float v = 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) v += ds[r];
                    if (side < 0) below += v;
                    else above += v;
                }
            }
        }
        if (more) keep_rows(buf ^ 1);
    }
    if (TABLE) {
        // the last head's part, and those of a group that saw no query
        __syncthreads();
        if (filled >= 0) flush(filled);
        else
            for (int h = hk * group; h < (hk + 1) * group; ++h) flush(h);
    }
    if (j >= a.Tk) return;
    const float out_v = DROP ? a.drop.scale : 1.0f, out_k = a.scale * out_v;
    T* to_k = (T*)a.dk + b * a.sdk.b + (int64_t)j * a.sdk.t + hk * a.sdk.h;
    T* to_v = (T*)a.dv + b * a.sdv.b + (int64_t)j * a.sdv.t + hk * a.sdv.h;
#pragma unroll
    for (int d = 0; d < db_n; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * d + 8 * g + 4 * half;
            if (c >= a.D) continue;
            typename Mma<T>::x4 x, y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = (T)(dk[d][4 * g + e] * out_k);
                y[e] = (T)(dv[d][4 * g + e] * out_v);
            }
            *reinterpret_cast<typename Mma<T>::x4*>(to_k + c) = x;
            *reinterpret_cast<typename Mma<T>::x4*>(to_v + c) = y;
        }
}

template <typename T, int DP, bool BIAS, bool DROP, bool TABLE, bool SHORT>
hipError_t run(const AttnArgs& a, hipStream_t st) {
    const size_t window = (2 * (size_t)a.bias.radius + 1 + 2 * kPad) * sizeof(float);
    const size_t tiles = 4 * tile_bytes<DP>();
    if ((int64_t)a.B * a.Tq > 0)
        hipLaunchKernelGGL((attn_dq_kernel<T, DP, BIAS, DROP, SHORT>),
                           dim3(xcd_grid((int64_t)a.B * a.H, attn_tiles(a.Tq))), dim3(kThreads),
                           tiles + (BIAS ? window : 0), st, a);
    if ((int64_t)a.B * a.Tk > 0) {
        size_t lds =
            tiles + (kRowFloats + (DROP ? kWaves * 32 : 0)) * sizeof(float) + (BIAS ? window : 0);
        if (TABLE)
            lds += kWaves * (kSkewFloats + 2 * (size_t)a.bias.radius + 1) * sizeof(float);
        hipLaunchKernelGGL((attn_dkv_kernel<T, DP, BIAS, DROP, TABLE, SHORT>),
                           dim3(xcd_grid((int64_t)a.B * a.Hkv, attn_tiles(a.Tk))), dim3(kThreads),
                           lds, st, a);
    }
    return hipGetLastError();
}

template <typename T, int DP, bool SHORT>
hipError_t run_s(const AttnArgs& a, bool table, hipStream_t st) {
    const bool bias = a.bias.radius > 0, drop = a.drop.threshold != kDropAll;
    if (table)
        return drop ? run<T, DP, true, true, true, SHORT>(a, st)
                    : run<T, DP, true, false, true, SHORT>(a, st);
    if (bias)
        return drop ? run<T, DP, true, true, false, SHORT>(a, st)
                    : run<T, DP, true, false, false, SHORT>(a, st);
    return drop ? run<T, DP, false, true, false, SHORT>(a, st)
                : run<T, DP, false, false, false, SHORT>(a, st);
}

template <typename T, int DP>
hipError_t run_d(const AttnArgs& a, bool table, hipStream_t st) {
    return a.Tq <= kShort && a.Tk <= kShort ? run_s<T, DP, true>(a, table, st)
                                            : run_s<T, DP, false>(a, table, st);
}

}  // namespace

hipError_t launch_attn_backward(const AttnArgs& a, int32_t dtype, float* dtable, bool accumulate,
                                hipStream_t st) {
    hipError_t e;
    if (dtype == ONEBIT_BF16)
        e = a.D <= 64 ? run_d<bf16, 64>(a, dtable, st) : run_d<bf16, 128>(a, dtable, st);
    else
        e = a.D <= 64 ? run_d<f16, 64>(a, dtable, st) : run_d<f16, 128>(a, dtable, st);
    if (e != hipSuccess || !dtable) return e;
    return launch_bias_join(a.partials, a.bias.map, dtable, a.H,
                            (int64_t)a.B * attn_tiles(a.Tk), a.bias.n_buckets, a.bias.radius,
                            accumulate, st);
}

}  // namespace onebit
