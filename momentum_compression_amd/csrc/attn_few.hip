// Attention forward for few queries over many keys: single tokens over a
// cache, where all that counts is to read the keys and values once.
//
// The queries of all heads that share a key head (at most 32 together) are the
// columns of the products, so a key is read once for all of them.  The keys of
// a sequence are split over workgroups and over their waves; a wave goes
// through its part alone, 32 keys at a time, without barriers: whole rows come
// in, through LDS of its own they become operands, the next 32 on their way
// while these are used.  The waves of a workgroup are joined in LDS, the
// workgroups by attn_join.
//
// Bound by memory: 32 sequences of 8192 keys, 4 key heads of 128 and 16 query heads
// take 93 us without a bias (5.8 TB/s) and 97 with one, of 2048 ... 8192 keys 71 us
// with one (4.7 TB/s; the short sequences' workgroups end first).  Loads past the
// caches, as each key is read once (113 and 79 us with a bias through them).  One
// token of one sequence over 16384 keys takes 22 us, most of it the latencies of
// two launches.
#include <type_traits>

#include "attention.h"

namespace onebit {

namespace {

template <typename T, int DP, bool BIAS, bool DROP>
__global__ __launch_bounds__(kThreads, 2) void attn_few_kernel(AttnArgs a) {
    using x8 = typename Mma<T>::x8;
    constexpr int kc_n = DP / 16, db_n = DP / 32;
    constexpr int chunks = DP / 8, v_n = kRows * chunks / 64;  // 16-byte pieces a lane
    // the waves' key and value tiles; afterwards the joined rows of two waves
    __shared__ __align__(16) char tiles[2 * kWaves * kRows * DP * 2];
    __shared__ float2 stats[kWaves][kRows];
    __shared__ float bases[kWaves][kRows];

    uint32_t bh, part;
    if (!xcd_work((uint32_t)a.B * a.Hkv, (uint32_t)a.splits, kEven, bh, part)) return;
    const int hk = (int)(bh % a.Hkv), b = (int)(bh / a.Hkv);
    const int lane = lane_id(), wave = wave_id();
    const int32_t pos = query_position(a, b), n_keys = key_count(a, b, pos);
    const int group = a.H / a.Hkv, R = a.bias.radius;
    // The query of a lane's column.  The lane number comes anew for each use: what
    // follows from it, kept through the keys, would go to memory (with that a
    // bias costs 6 to 10 us).
    struct Place {
        int half, col, h;
        int32_t i;
        bool mine;
    };
    const auto place = [&](int n) {
        asm volatile("" : "+v"(n));
        const int col = n & 31;
        const bool mine = col < group * a.Tq;
        return Place{n >> 5, col, hk * group + (mine ? col % group : 0), mine ? col / group : 0,
                     mine};
    };

    const T* kp = (const T*)a.k + b * a.sk.b + hk * a.sk.h;
    const T* vp = (const T*)a.v + b * a.sv.b + hk * a.sv.h;
    const int32_t n_tiles = (n_keys + kRows - 1) / kRows;
    // every waves-th tile: neighbouring waves read neighbouring rows, and the
    // few tiles near the queries, whose bias is gathered, go to different waves
    const int32_t waves = a.splits * kWaves;
    const int32_t limit_lo = a.causal && pos < n_keys - 1 ? pos : n_keys - 1;

    const float scale2 = a.scale * kLog2e, inv_scale = 1.0f / a.scale;
    const auto bias_at = [&](int32_t d, int h) {
        d = d < -R ? -R : (d > R ? R : d);
        const int m = a.bias.map[d + R];
        // divided by the scale and multiplied again, so that the values too low
        // for the other kernels' windows are too low here
        return (uint32_t)m < (uint32_t)a.bias.n_buckets
                   ? low_value(a.bias.table[(int64_t)m * a.H + h]) * inv_scale * scale2
                   : 0.0f;
    };
    const float below = BIAS ? bias_at(-R, place(lane).h) : 0.0f;
    const float above = BIAS ? bias_at(R, place(lane).h) : 0.0f;
    const uint32_t step = DROP ? a.drop.step + (a.drop.step_dev ? *a.drop.step_dev : 0u) : 0u;

    char* kt = tiles + 2 * wave * (kRows * DP * 2);
    char* vt = kt + kRows * DP * 2;
    x8 kr[v_n], vr[v_n];
    const auto load = [&](x8 (&to)[v_n], const T* base, int64_t stride, int32_t tile, int lane) {
#pragma unroll
        for (int x = 0; x < v_n; ++x) {
            const int32_t j = tile * kRows + (x * 64 + lane) / chunks;
            const int c = 8 * (lane % chunks);
            to[x] = x8{};
            if (j < n_keys && c < a.D)
                to[x] = __builtin_nontemporal_load(
                    reinterpret_cast<const x8*>(base + (int64_t)j * stride + c));
        }
    };
    const auto store = [&](char* tile, const x8 (&from)[v_n], int lane) {
#pragma unroll
        for (int x = 0; x < v_n; ++x)
            *reinterpret_cast<x8*>(tile + tile_at<DP>((x * 64 + lane) / chunks, lane % chunks)) =
                from[x];
    };

    f32x16 acc[db_n];
    float base = 0.0f, m = -INFINITY, l;
    // The wave's keys; BASED: once more, from the rows' bases.
    const auto pass = [&](auto based) __attribute__((always_inline)) {
        constexpr bool BASED = decltype(based)::value;
        const float from = BASED ? base : 0.0f;
        uint32_t k0 = a.drop.k0, k1 = a.drop.k1;  // not the first pass's schedule
        if (BASED) asm volatile("" : "+s"(k0), "+s"(k1));
        int32_t t = (int)part * kWaves + wave;
        const Place q = place(lane);
        const int h = q.h;
        const int32_t i = q.i;
        const int32_t limit = a.causal && i + pos < n_keys - 1 ? i + pos : n_keys - 1;
        const uint64_t drop_row = ((uint64_t)b * a.H + h) * (uint64_t)a.Tq + (uint64_t)i;
        x8 qf[kc_n];
        load_frags<T, DP>(qf, (const T*)a.q + b * a.sq.b + h * a.sq.h, a.sq.t, i, q.mine, a.D,
                          lane);
#pragma unroll
        for (int d = 0; d < db_n; ++d) acc[d] = f32x16{};
        l = 0.0f;
        if (!BASED && t < n_tiles) {
            load(kr, kp, a.sk.t, t, lane);
            load(vr, vp, a.sv.t, t, lane);
        }
        for (; t < n_tiles; t += waves) {
            const int32_t j0 = t * kRows;
            int lane_now = lane;  // the second pass reads nothing ahead, too
            if (BASED) asm volatile("" : "+v"(lane_now));
            const int lane = lane_now, half = lane >> 5;
            if (BASED) load(kr, kp, a.sk.t, t, lane);
            store(kt, kr, lane);
            if (!BASED && t + waves < n_tiles) load(kr, kp, a.sk.t, t + waves, lane);
            if (BASED) load(vr, vp, a.sv.t, t, lane);
            store(vt, vr, lane);
            if (!BASED && t + waves < n_tiles) load(vr, vp, a.sv.t, t + waves, lane);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the tiles are written
            __builtin_amdgcn_wave_barrier();
            f32x16 s = {};
#pragma unroll
            for (int kc = 0; kc < kc_n; ++kc)
                s = Mma<T>::mul(row_frag<T, DP>(kt, 0, kc, lane), qf[kc], s);
            // base-2 scores; the queries of the columns stand at pos ... pos + Tq - 1
            if (BIAS && j0 + 31 - pos > -R && j0 - (pos + a.Tq - 1) < R) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[r] = __builtin_fmaf(s[r], scale2,
                                          bias_at(j0 + 16 * (r >> 3) + 8 * half + (r & 7) - i - pos,
                                                  h) -
                                              from);
            } else {
                const float c = (!BIAS ? 0.0f : (j0 < pos ? below : above)) - from;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], scale2, c);
            }
            if (j0 + 31 > limit_lo) {
                const int32_t seen = limit - j0 - 8 * half;
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (16 * (r >> 3) + (r & 7) > seen) s[r] = -INFINITY;
            }
            float mx = s[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[r]);
            mx = fmaxf(mx, other_half(mx));
            if (__any(mx > m + 8.0f)) {  // as in the forward pass for many queries
                const float m_new = fmaxf(m, mx);
                const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - m_new);
                l *= alpha;
#pragma unroll
                for (int d = 0; d < db_n; ++d) acc[d] *= alpha;
                m = m_new;
            }
            const float m_use = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(s[8 * c + e] - m_use);
                l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
                if (DROP) {
                    uint32_t wd[4];
                    drop_draws(wd, (uint32_t)(j0 + 16 * c + 8 * half) >> 3, drop_row, step, k0, k1);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (!drop_keep(wd, e, a.drop.threshold)) p[e] = 0.0f;
                }
                const x8 pb = pack8<T>(p);
#pragma unroll
                for (int d = 0; d < db_n; ++d)
                    acc[d] = Mma<T>::mul(col_frag<T, DP>(vt, 16 * c, d, lane), pb, acc[d]);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // ... and read
            __builtin_amdgcn_wave_barrier();
        }
    };
    pass(std::false_type());

    // Large references become the rows' bases, and the wave goes through its keys
    // once more: what the products add to scores of that size is lost.  (Not
    // where the wave has keys of a low bias alone, but the row's nearest key has
    // another: they hardly count then, and their weights are right as they are.)
    if (__builtin_expect(__any(is_large(m)), 0)) {
        bool far = is_large(m);
        if (BIAS && m < 0.0f) {
            const Place q = place(lane);
            const int32_t at = q.i + pos, last = n_keys - 1;
            if (!is_large(bias_at(at < 0 ? -at : (at > last ? last - at : 0), q.h))) far = false;
        }
        if (__any(far)) {
            base = far ? m : 0.0f;
            m = -INFINITY;
            pass(std::true_type());
        }
    }

    // the waves' references and sums, then their rows, two waves at a time
    l += other_half(l);
    const Place q = place(lane);
    const int half = q.half, col = q.col;
    if (half == 0) {
        stats[wave][col] = float2{m, l};
        bases[wave][col] = base;
    }
    __syncthreads();
    // all to one wave's base: the highest's, as far as a first one shows
    float origin = 0.0f;
    const auto reach = [&](int w) {
        const float m_w = stats[w][col].x;
        return m_w == -INFINITY ? m_w : (bases[w][col] - origin) + m_w;
    };
    const bool any = bases[0][col] != 0.0f || bases[1][col] != 0.0f || bases[2][col] != 0.0f ||
                     bases[3][col] != 0.0f;
    if (__builtin_expect(__any(any), 0)) {
        for (int k = 0; k < 2; ++k) {
            int best = 0;
            for (int w = 1; w < kWaves; ++w)
                if (reach(w) > reach(best)) best = w;
            origin = bases[best][col];
        }
    }
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, reach(w));
    const float m_use = m == -INFINITY ? 0.0f : m;
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        l += __builtin_amdgcn_exp2f(reach(w) - m_use) * stats[w][col].y;
    const float weight = __builtin_amdgcn_exp2f(reach(wave) - m_use);
#pragma unroll
    for (int d = 0; d < db_n; ++d) acc[d] *= weight;
    float* rows = reinterpret_cast<float*>(tiles);
#pragma unroll
    for (int left = 2; left >= 1; left >>= 1) {  // waves that take in another's
        float* at = rows + (wave % left) * (kRows * DP) + half * 4 * kRows + col;
        if (wave >= left && wave < 2 * left) {
#pragma unroll
            for (int d = 0; d < db_n; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    at[(32 * d + 8 * (r >> 2) + (r & 3)) * kRows] = acc[d][r];
        }
        __syncthreads();
        if (wave < left) {
#pragma unroll
            for (int d = 0; d < db_n; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[d][r] += at[(32 * d + 8 * (r >> 2) + (r & 3)) * kRows];
        }
        __syncthreads();
    }
    if (wave != 0 || !q.mine) return;
    const int64_t row = ((int64_t)b * a.H + q.h) * a.Tq + q.i;
    if (a.splits > 1)
        write_split<DP>(a, acc, row, (int)part, origin, m, l, half);
    else
        write_rows<T, DP>(a, acc, b, q.h, q.i, row, origin, m, l, half);
}

template <typename T, int DP>
void run_d(const AttnArgs& a, hipStream_t st) {
    const bool bias = a.bias.radius > 0, drop = a.drop.threshold != kDropAll;
    const dim3 grid(xcd_grid((int64_t)a.B * a.Hkv, a.splits));
    if (bias && drop)
        hipLaunchKernelGGL((attn_few_kernel<T, DP, true, true>), grid, dim3(kThreads), 0, st, a);
    else if (bias)
        hipLaunchKernelGGL((attn_few_kernel<T, DP, true, false>), grid, dim3(kThreads), 0, st, a);
    else if (drop)
        hipLaunchKernelGGL((attn_few_kernel<T, DP, false, true>), grid, dim3(kThreads), 0, st, a);
    else
        hipLaunchKernelGGL((attn_few_kernel<T, DP, false, false>), grid, dim3(kThreads), 0, st, a);
}

}  // namespace

hipError_t launch_attn_few(const AttnArgs& a, int32_t dtype, hipStream_t st) {
    if (dtype == ONEBIT_BF16) {
        if (a.D <= 64) run_d<bf16, 64>(a, st);
        else run_d<bf16, 128>(a, st);
    } else {
        if (a.D <= 64) run_d<f16, 64>(a, st);
        else run_d<f16, 128>(a, st);
    }
    return hipGetLastError();
}

}  // namespace onebit
