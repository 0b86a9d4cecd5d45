// The AdamW step over many tensors in one launch, states in 32 or in 8 bits.
//
// A workgroup takes kAdamWTile elements of one tensor, which a table by
// workgroup names (one scalar load; a search over the tensors' offsets would be
// nine in a row).  A wave has two blocks of 256 elements at a time, a lane four
// consecutive elements of each.  The kernel
// moves what the step cannot do without, 28 + g + copy bytes an element with
// 32-bit states and 12 + g + copy with 8-bit ones, and is bound by them.
//
// 8-bit states.  256 consecutive elements share a power of two; over it, m is an
// e4m3 number and v an e5m2 one (v spans the square of what m does: two bits of
// mantissa give sqrt(v) the steps that three give m).  Values are rounded up or
// down with the probabilities that keep their mean: with rounding to nearest a
// state that decays by 1 - beta2 = 0.001 a step would stay where it is for good.
// The draw is added below the kept bits of the binary32 pattern and the rest cut
// off, which is exact for every binade.
#include <type_traits>

#include "philox.h"
#include "train.h"

namespace onebit {
namespace {

constexpr uint32_t kTag = 0x41444D57u;

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

// A format's codes: normal values from 2^kLeast on, kDigits bits of mantissa, the
// block's largest value in [2^kTop, 2^(kTop + 1)).
template <int TOP, int LEAST, int DIGITS>
struct Code {
    static constexpr int kDrop = 23 - DIGITS;
    static constexpr uint32_t kNan = DIGITS == 3 ? 0x7F : 0x7E;

    // Exponent of the block's power of two (with the bias of binary32), from the
    // pattern of its largest finite magnitude.
    static __device__ __forceinline__ uint32_t scale_exponent(uint32_t most) {
        const uint32_t e = most >> 23;
        return (e > TOP + 1 ? e : TOP + 1) - TOP;
    }
    // y >= 0, below 2^(TOP + 1); 16 bits of draw
    static __device__ __forceinline__ uint32_t encode(float y, uint32_t draw) {
        const bool tiny = y < __uint_as_float((uint32_t)(127 + LEAST) << 23);
        // below the normal values the grid is that of the first binade: there the
        // sum's pattern counts it
        const float z = tiny ? y + __uint_as_float((uint32_t)(127 + LEAST) << 23) : y;
        const uint32_t noise = (draw << (kDrop - 16)) + (1u << (kDrop - 17)) -
                               ((uint32_t)(126 + LEAST) << 23);
        return ((__float_as_uint(z) + noise) >> kDrop) - (tiny ? 1u << DIGITS : 0u);
    }
    static __device__ __forceinline__ float decode(uint32_t code) {
        const uint32_t at = code & 0x7F;
        const float y = __uint_as_float(at << kDrop) *
                        __uint_as_float((uint32_t)(253 + LEAST) << 23);
        const float s = __uint_as_float(__float_as_uint(y) | (code & 0x80) << 24);
        return DIGITS == 3 ? (at == 0x7F ? __builtin_nanf("") : s)
                           : (at >= 0x7C ? (at == 0x7C ? INFINITY : __builtin_nanf("")) : s);
    }
};
using CodeM = Code<7, -6, 3>;
using CodeV = Code<14, -14, 2>;

__device__ __forceinline__ bool finite(uint32_t magnitude) { return magnitude < 0x7F800000u; }

// Four consecutive elements at any element address, `n` of them there.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Four {
    T v[4];
};

template <typename T>
__device__ __forceinline__ void load4(float out[4], const T* p, int64_t n) {
    Four<T> x = {};
    if (n >= 4) {
        x = *reinterpret_cast<const Four<T>*>(p);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) x.v[e] = p[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = (float)x.v[e];
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
        __builtin_nontemporal_store(x, reinterpret_cast<u32_any*>(p));
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
    const int64_t begin = ((int64_t)blockIdx.x - t.first_tile) * kAdamWTile;
    const float omb1 = 1.0f - a.beta1, omb2 = 1.0f - a.beta2;
    const float lr = a.lr * t.lr_scale;
    const float decay = 1.0f - lr * t.weight_decay, rate = lr * a.rate;
    const float g_scale = a.g_scale ? *a.g_scale : 1.0f;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = lane_id();
    constexpr int kSets = 2;  // blocks of a wave at a time
    constexpr int kRounds = kAdamWTile / (kSets * kStateBlock * kThreads / 64);
#pragma unroll 1
    for (int k = 0; k < kRounds; ++k) {
        const int64_t base = begin + (int64_t)(k * (kThreads / 64) + wave) * kSets * kStateBlock;
        if (base >= t.n) break;  // the same for the wave
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
                const uint32_t mc = load_codes((const uint8_t*)t.m + at, n);
                const uint32_t vc = load_codes((const uint8_t*)t.v + at, n);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    m[s][e] = CodeM::decode(mc >> (8 * e) & 0xFF) * ms;
                    v[s][e] = CodeV::decode(vc >> (8 * e) & 0xFF) * vs;
                }
            } else {
                load4(m[s], (const float*)t.m + at, n);
                load4(v[s], (const float*)t.v + at, n);
            }
        }
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            const int64_t at = base + s * kStateBlock + 4 * lane, n = t.n - at;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (a.g_scale) g[s][e] = g[s][e] * g_scale;
                m[s][e] = a.beta1 * m[s][e] + omb1 * g[s][e];
                v[s][e] = a.beta2 * v[s][e] + omb2 * (g[s][e] * g[s][e]);
                x[s][e] = x[s][e] * decay - rate * (m[s][e] / (sqrtf(v[s][e]) * a.root + a.eps));
            }
            if (n <= 0) continue;
            store4(t.x + at, x[s], n);
            if (sizeof(C) == 2) store4((C*)t.copy + at, x[s], n);
            if (!EIGHT) {
                store4((float*)t.m + at, m[s], n);
                store4((float*)t.v + at, v[s], n);
            }
        }
        if (!EIGHT) continue;
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
            uint32_t m_most = 0, v_most = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t mb = __float_as_uint(m[s][e]) & 0x7FFFFFFFu;
                const uint32_t vb = __float_as_uint(v[s][e]) & 0x7FFFFFFFu;
                m_most = finite(mb) && mb > m_most ? mb : m_most;
                v_most = finite(vb) && vb > v_most ? vb : v_most;
            }
            const uint32_t me = CodeM::scale_exponent(block_max(m_most));
            const uint32_t ve = CodeV::scale_exponent(block_max(v_most));
            const float m_inv = __uint_as_float((254 - me) << 23);
            const float v_inv = __uint_as_float((254 - ve) << 23);
            uint32_t mc = 0, vc = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // one draw for both states: each alone keeps its mean
                const uint32_t word = draws[s][e >> 1];
                const uint32_t draw = (e & 1) ? word >> 16 : word & 0xFFFFu;
                const uint32_t bits = __float_as_uint(m[s][e]);
                uint32_t c = finite(bits & 0x7FFFFFFFu)
                                 ? CodeM::encode(__uint_as_float(bits & 0x7FFFFFFFu) * m_inv, draw)
                                 : CodeM::kNan;
                c |= (bits >> 24) & 0x80;
                mc |= c << (8 * e);
                // a variance above 0 stays above 0, or its element's next step
                // would be divided by eps alone
                uint32_t d = CodeV::encode(v[s][e] * v_inv, draw);
                d = v[s][e] > 0.0f && d == 0u ? 1u : d;
                d = finite(__float_as_uint(v[s][e])) ? d : CodeV::kNan;
                vc |= d << (8 * e);
            }
            if (n > 0) {
                store_codes((uint8_t*)t.m + at, mc, n);
                store_codes((uint8_t*)t.v + at, vc, n);
            }
            if (lane == 0) {
                t.m_scale[first / kStateBlock] = __uint_as_float(me << 23);
                t.v_scale[first / kStateBlock] = __uint_as_float(ve << 23);
            }
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
