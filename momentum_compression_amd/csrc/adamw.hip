// The AdamW step over many tensors in one launch, states in 32 or in 8 bits.
//
// A workgroup takes kAdamWTile elements of one tensor, which a table by
// workgroup names (one scalar load; a search over the tensors' offsets would be
// nine in a row).  A wave has two blocks of 256 elements at a time, a lane four
// consecutive elements of each.  The kernel
// moves what the step cannot do without, 24 + g + copy bytes an element with
// 32-bit states and 12 + g + copy with 8-bit ones, and is bound by them: 302 tensors
// of 336 million elements in 1484 to 1671 us (9.41 GB, 5.6 to 6.3 TB/s, one GPU or
// another), with 8-bit states in 868 to 893 (5.40 GB, 6.0 to 6.2 TB/s).
//
// 8-bit states.  256 consecutive elements share a power of two; over it, m is an
// e4m3 number and v an e5m2 one (v spans the square of what m does: two bits of
// mantissa give sqrt(v) the steps that three give m).  Values are rounded up or
// down with the probabilities that keep their mean: with rounding to nearest a
// state that decays by 1 - beta2 = 0.001 a step would stay where it is for good.
// The conversion adds the draw below the kept bits and cuts the rest off, which is
// exact for every binade and below the normal numbers.
#include <type_traits>

#include "philox.h"
#include "train.h"

namespace onebit {
namespace {

constexpr uint32_t kTag = 0x41444D57u;
constexpr uint32_t kInfinite = 0x7F800000u;

typedef uint32_t u32_any __attribute__((aligned(1)));

// Maximum over the wave, which holds a block.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    auto step = [](uint32_t v, auto ctrl) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, decltype(ctrl)::value, 0xF,
                                                              0xF, true);
        return v > o ? v : o;
    };
    x = step(x, std::integral_constant<int, 0xB1>{});
    x = step(x, std::integral_constant<int, 0x4E>{});
    x = step(x, std::integral_constant<int, 0x141>{});
    x = step(x, std::integral_constant<int, 0x140>{});
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = r[0] > r[1] ? r[0] : r[1];
    const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return h[0] > h[1] ? h[0] : h[1];
}

// Exponent (with the bias of binary32) of a block's power of two, which puts the
// pattern of its largest finite magnitude into [2^TOP, 2^(TOP + 1)).
constexpr uint32_t kTopM = 7, kTopV = 14;
template <uint32_t TOP>
__device__ __forceinline__ uint32_t scale_exponent(uint32_t most) {
    const uint32_t e = most >> 23;
    return (e > TOP + 1 ? e : TOP + 1) - TOP;
}

__device__ __forceinline__ float power_of_two(uint32_t e) { return __uint_as_float(e << 23); }

// The values of four codes.
template <bool M>
__device__ __forceinline__ void decode4(float out[4], uint32_t codes, float scale) {
    const auto lo = M ? __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false)
                      : __builtin_amdgcn_cvt_pk_f32_bf8((int)codes, false);
    const auto hi = M ? __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true)
                      : __builtin_amdgcn_cvt_pk_f32_bf8((int)codes, true);
    out[0] = lo[0] * scale;
    out[1] = lo[1] * scale;
    out[2] = hi[0] * scale;
    out[3] = hi[1] * scale;
}

// Square root of a number within 2^-100 ... 2^60, correctly rounded: one correction
// from the exact remainder (compared with sqrtf for every mantissa of both
// parities of the exponent, over that range).  Eight issue slots to its twenty.
__device__ __forceinline__ float root_of(float v) {
    const float y = __builtin_amdgcn_rsqf(v), s = v * y;
    return __builtin_fmaf(__builtin_fmaf(-s, s, v), 0.5f * y, s);
}

// m / d, correctly rounded, where neither they nor the quotient come near the ends
// of the range.  The reciprocal is brought to half a step or so by one step of Newton's
// iteration, and the quotient by two corrections with its exact remainder (Markstein's
// method of division by fused multiply-adds).  With the remainder's sign the other way
// round a quotient of -0 stays one.
__device__ __forceinline__ float quotient_of(float m, float d) {
    const float y0 = __builtin_amdgcn_rcpf(d);
    const float y = __builtin_fmaf(__builtin_fmaf(-d, y0, 1.0f), y0, y0);
    float q = m * y;
    q = __builtin_fmaf(-__builtin_fmaf(d, q, -m), y, q);
    return __builtin_fmaf(-__builtin_fmaf(d, q, -m), y, q);
}

// Four consecutive elements at any element address, `n` of them there.  Past the
// caches, as a step reads everything once (302 tensors with 32-bit states 1543 ->
// 1484 us, with 8-bit ones 893 -> 868; 8-bit codes past the caches 900).
template <typename T>
__device__ __forceinline__ void load4(float out[4], const T* p, int64_t n) {
    T x[4] = {};
    if (n >= 4) {
        typedef uint32_t Words __attribute__((ext_vector_type(sizeof(T)), aligned(sizeof(T))));
        const Words w = __builtin_nontemporal_load(reinterpret_cast<const Words*>(p));
        __builtin_memcpy(x, &w, sizeof(x));
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) x[e] = p[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = (float)x[e];
}

// Past the caches: a step does not read again what it writes.
template <typename T>
__device__ __forceinline__ void store4(T* p, const float v[4], int64_t n) {
    if (n >= 4) {
        typedef uint32_t Words __attribute__((ext_vector_type(sizeof(T)), aligned(sizeof(T))));
        T x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (T)v[e];
        __builtin_nontemporal_store(__builtin_bit_cast(Words, x), reinterpret_cast<Words*>(p));
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < n) p[e] = (T)v[e];
}

__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t n) {
    if (n >= 4) return *reinterpret_cast<const u32_any*>(p);
    uint32_t x = 0;
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < n) x |= (uint32_t)p[e] << (8 * e);
    return x;
}

__device__ __forceinline__ void store_codes(uint8_t* p, uint32_t x, int64_t n) {
    if (n >= 4) {
        *reinterpret_cast<u32_any*>(p) = x;  // a store past the caches would go by bytes
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < n) p[e] = (uint8_t)(x >> (8 * e));
}

__device__ __forceinline__ uint32_t other_of_pair(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true);
}

// C: type of the 16-bit copy of the parameters, float for none.
template <typename G, typename C, bool EIGHT>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamWArgs a) {
    const int32_t which = a.tensor_of[blockIdx.x];
    const AdamWTensor t = a.tensors[which];
    const float omb1 = 1.0f - a.beta1, omb2 = 1.0f - a.beta2;
    const float lr = a.lr * t.lr_scale;
    const float decay = 1.0f - lr * t.weight_decay, rate = lr * a.rate;
    const float g_scale = a.g_scale ? *a.g_scale : 1.0f;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = lane_id();
    constexpr int kSets = 2;  // blocks of a wave
    static_assert(kAdamWTile == kSets * kStateBlock * (kThreads / 64), "a workgroup's blocks");
    const int64_t base = ((int64_t)blockIdx.x - t.first_tile) * kAdamWTile +
                         wave * (kSets * kStateBlock);
    if (base >= t.n) return;  // the same for the wave
    float x[kSets][4], g[kSets][4], m[kSets][4], v[kSets][4];
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
        const int64_t first = base + s * kStateBlock, at = first + 4 * lane, n = t.n - at;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[s][e] = g[s][e] = m[s][e] = v[s][e] = 0.0f;
        if (n <= 0) continue;
        load4(x[s], t.x + at, n);
        load4(g[s], (const G*)t.g + at, n);
        if (EIGHT) {
            const float ms = t.m_scale[first / kStateBlock], vs = t.v_scale[first / kStateBlock];
            decode4<true>(m[s], load_codes((const uint8_t*)t.m + at, n), ms);
            decode4<false>(v[s], load_codes((const uint8_t*)t.v + at, n), vs);
        } else {
            load4(m[s], (const float*)t.m + at, n);
            load4(v[s], (const float*)t.v + at, n);
        }
    }
    float m_most[kSets], v_most[kSets];  // of the lane, NaN left out
    uint32_t m_least = ~0u, v_least = ~0u, v_last = 0u;  // patterns; zeros of m left out
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (a.g_scale) g[s][e] = g[s][e] * g_scale;
            m[s][e] = a.beta1 * m[s][e] + omb1 * g[s][e];
            v[s][e] = a.beta2 * v[s][e] + omb2 * (g[s][e] * g[s][e]);
            const uint32_t mb = (__float_as_uint(m[s][e]) & 0x7FFFFFFFu) - 1u;
            const uint32_t vb = __float_as_uint(v[s][e]);
            m_least = mb < m_least ? mb : m_least;
            v_least = vb < v_least ? vb : v_least;
            v_last = vb > v_last ? vb : v_last;
        }
        m_most[s] = fmaxf(fmaxf(__builtin_fabsf(m[s][0]), __builtin_fabsf(m[s][1])),
                          fmaxf(__builtin_fabsf(m[s][2]), __builtin_fabsf(m[s][3])));
        v_most[s] = fmaxf(fmaxf(v[s][0], v[s][1]), fmaxf(v[s][2], v[s][3]));
    }
    // m of 2^-60 ... 2^60 or 0, v of 2^-100 ... 2^60, a divisor of 2^-50 ... 2^43
    const bool usual = m_least >= (67u << 23) - 1u && fmaxf(m_most[0], m_most[1]) <= 0x1p60f &&
                       v_least >= 27u << 23 && v_last <= 187u << 23 && a.eps <= 1.0f;
    if (__all(usual)) {
#pragma unroll
        for (int s = 0; s < kSets; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[s][e] = x[s][e] * decay -
                          rate * quotient_of(m[s][e], root_of(v[s][e]) * a.root + a.eps);
    } else {
#pragma unroll
        for (int s = 0; s < kSets; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[s][e] = x[s][e] * decay - rate * (m[s][e] / (sqrtf(v[s][e]) * a.root + a.eps));
    }
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
        const int64_t at = base + s * kStateBlock + 4 * lane, n = t.n - at;
        if (n <= 0) continue;
        store4(t.x + at, x[s], n);
        if (sizeof(C) == 2) store4((C*)t.copy + at, x[s], n);
        if (!EIGHT) {
            store4((float*)t.m + at, m[s], n);
            store4((float*)t.v + at, v[s], n);
        }
    }
    if (!EIGHT) return;
    // A group of eight draws serves a pair of lanes: the even lane makes the
    // first block's, the odd lane the second's, and they exchange halves.
    const int odd = lane & 1;
    uint32_t w[4] = {(uint32_t)(base >> 3) + (uint32_t)(odd * (kStateBlock / 8) + (lane >> 1)),
                     (uint32_t)which, 0u, a.step};
    philox10(w[0], w[1], w[2], w[3], a.k0, a.k1);
    uint32_t draws[kSets][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t got = other_of_pair(odd ? w[h] : w[2 + h]);
        draws[0][h] = odd ? got : w[h];
        draws[1][h] = odd ? w[2 + h] : got;
    }
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
        const int64_t first = base + s * kStateBlock, at = first + 4 * lane, n = t.n - at;
        if (first >= t.n) continue;  // the same for the wave
        // elements past the tensor's end are 0 and count for nothing
        uint32_t mm = block_max(__float_as_uint(m_most[s]));
        uint32_t vm = block_max(__float_as_uint(v_most[s]));
        if (__builtin_expect(mm >= kInfinite || vm >= kInfinite, 0)) {
            // infinities count for nothing either
            mm = vm = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t mb = __float_as_uint(m[s][e]) & 0x7FFFFFFFu;
                const uint32_t vb = __float_as_uint(v[s][e]) & 0x7FFFFFFFu;
                mm = mb < kInfinite && mb > mm ? mb : mm;
                vm = vb < kInfinite && vb > vm ? vb : vm;
            }
            mm = block_max(mm);
            vm = block_max(vm);
        }
        const uint32_t me = scale_exponent<kTopM>(mm), ve = scale_exponent<kTopV>(vm);
        const float m_inv = power_of_two(254 - me), v_inv = power_of_two(254 - ve);
        int mc = 0, vc = 0;
        auto encode = [&](auto at_byte) {
            constexpr int e = decltype(at_byte)::value;
            // one draw for both states: each alone keeps its mean.  Half a
            // draw's step is added, so that 0 and 65535 are alike.
            const uint32_t word = draws[s][e >> 1];
            const uint32_t noise = ((e & 1) ? word & 0xFFFF0000u : word << 16) | 0x8000u;
            mc = __builtin_amdgcn_cvt_sr_fp8_f32(m[s][e] * m_inv, noise, mc, e);
            // a variance above 0 stays above 0, or its element's next step
            // would be divided by eps alone
            const float y = v[s][e] * v_inv;
            vc = __builtin_amdgcn_cvt_sr_bf8_f32(
                v[s][e] > 0.0f && y < 0x1p-16f ? 0x1p-16f : y, noise, vc, e);
        };
        encode(std::integral_constant<int, 0>{});
        encode(std::integral_constant<int, 1>{});
        encode(std::integral_constant<int, 2>{});
        encode(std::integral_constant<int, 3>{});
        if (n > 0) {
            store_codes((uint8_t*)t.m + at, (uint32_t)mc, n);
            store_codes((uint8_t*)t.v + at, (uint32_t)vc, n);
        }
        if (lane == 0) {
            t.m_scale[first / kStateBlock] = power_of_two(me);
            t.v_scale[first / kStateBlock] = power_of_two(ve);
        }
    }
}

template <typename G, typename C>
void launch_bits(const AdamWArgs& a, bool eight, hipStream_t st) {
    const dim3 grid((unsigned)a.tiles), block(kThreads);
    if (eight) hipLaunchKernelGGL((adamw_kernel<G, C, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((adamw_kernel<G, C, false>), grid, block, 0, st, a);
}

template <typename G>
void launch_copy(const AdamWArgs& a, bool eight, int32_t copy_dtype, hipStream_t st) {
    if (copy_dtype == ONEBIT_BF16) launch_bits<G, bf16>(a, eight, st);
    else if (copy_dtype == ONEBIT_F16) launch_bits<G, f16>(a, eight, st);
    else launch_bits<G, float>(a, eight, st);
}

}  // namespace

hipError_t launch_adamw(const AdamWArgs& args, int32_t state_bits, int32_t g_dtype,
                        int32_t copy_dtype, hipStream_t st) {
    AdamWArgs a = args;
    a.k1 ^= kTag;
    const bool eight = state_bits == 8;
    if (g_dtype == ONEBIT_F32) launch_copy<float>(a, eight, copy_dtype, st);
    else if (g_dtype == ONEBIT_BF16) launch_copy<bf16>(a, eight, copy_dtype, st);
    else launch_copy<f16>(a, eight, copy_dtype, st);
    return hipGetLastError();
}

}  // namespace onebit
