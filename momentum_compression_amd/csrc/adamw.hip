// The AdamW step over many tensors in one launch, states in 32 or in 8 bits.
//
// A workgroup takes kAdamWTile elements of one tensor, which a table by
// workgroup names (one scalar load; a search over the tensors' offsets would be
// nine in a row).  A lane has eight consecutive elements at a time: 32 bytes of
// the parameter and of each binary32 state, 8 bytes of an 8-bit one.  The kernel
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

using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// Maximum over the 32 lanes that hold a block.
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
    return r[0] > r[1] ? r[0] : r[1];
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

template <typename T>
__device__ __forceinline__ void load_some(float out[8], const T* p, int64_t n) {
    const Vec8<T> x = n >= 8 ? load8(p) : load_tail(p, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = (float)x.v[e];
}

template <typename T>
__device__ __forceinline__ void store_some(T* p, const float v[8], int64_t n) {
    if (n >= 8) {
        store8(p, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) p[e] = (T)v[e];
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int64_t n) {
    if (n >= 8) return *reinterpret_cast<const u32x2_any*>(p);
    u32x2 x = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) x[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
    return x;
}

__device__ __forceinline__ void store_codes(uint8_t* p, u32x2 x, int64_t n) {
    if (n >= 8) {
        *reinterpret_cast<u32x2_any*>(p) = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) p[e] = (uint8_t)(x[e >> 2] >> (8 * (e & 3)));
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
    constexpr int kRounds = kAdamWTile / (8 * kThreads);
#pragma unroll 1
    for (int k = 0; k < kRounds; ++k) {
        const int64_t at = begin + ((int64_t)k * kThreads + threadIdx.x) * 8;
        const int64_t n = t.n - at;  // elements from here on
        // a block's lanes stay together: they need each other for its maximum
        if ((at & ~(kStateBlock - 1)) >= t.n) break;
        float x[8] = {}, g[8] = {}, m[8] = {}, v[8] = {};
        if (n > 0) {
            load_some(x, t.x + at, n);
            load_some(g, (const G*)t.g + at, n);
            if (EIGHT) {
                const int64_t block = at / kStateBlock;
                const float ms = t.m_scale[block], vs = t.v_scale[block];
                const u32x2 mc = load_codes((const uint8_t*)t.m + at, n);
                const u32x2 vc = load_codes((const uint8_t*)t.v + at, n);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    m[e] = CodeM::decode(mc[e >> 2] >> (8 * (e & 3)) & 0xFF) * ms;
                    v[e] = CodeV::decode(vc[e >> 2] >> (8 * (e & 3)) & 0xFF) * vs;
                }
            } else {
                load_some(m, (const float*)t.m + at, n);
                load_some(v, (const float*)t.v + at, n);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (a.g_scale) g[e] = g[e] * g_scale;
            m[e] = a.beta1 * m[e] + omb1 * g[e];
            v[e] = a.beta2 * v[e] + omb2 * (g[e] * g[e]);
            x[e] = x[e] * decay - rate * (m[e] / (sqrtf(v[e]) * a.root + a.eps));
        }
        if (n > 0) {
            store_some(t.x + at, x, n);
            if (sizeof(C) == 2) store_some((C*)t.copy + at, x, n);
        }
        if (!EIGHT) {
            if (n > 0) {
                store_some((float*)t.m + at, m, n);
                store_some((float*)t.v + at, v, n);
            }
            continue;
        }
        // elements past the tensor's end are 0 and count for nothing
        uint32_t m_most = 0, v_most = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t mb = __float_as_uint(m[e]) & 0x7FFFFFFFu;
            const uint32_t vb = __float_as_uint(v[e]) & 0x7FFFFFFFu;
            m_most = finite(mb) && mb > m_most ? mb : m_most;
            v_most = finite(vb) && vb > v_most ? vb : v_most;
        }
        const uint32_t me = CodeM::scale_exponent(block_max(m_most));
        const uint32_t ve = CodeV::scale_exponent(block_max(v_most));
        const float m_inv = __uint_as_float((254 - me) << 23);
        const float v_inv = __uint_as_float((254 - ve) << 23);
        uint32_t w[4] = {(uint32_t)(at >> 3), (uint32_t)which, 0u, a.step};
        philox10(w[0], w[1], w[2], w[3], a.k0, a.k1);
        u32x2 mc = {0u, 0u}, vc = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // one draw for both states: each alone keeps its mean
            const uint32_t draw = (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
            const uint32_t bits = __float_as_uint(m[e]);
            uint32_t c = finite(bits & 0x7FFFFFFFu)
                             ? CodeM::encode(__uint_as_float(bits & 0x7FFFFFFFu) * m_inv, draw)
                             : CodeM::kNan;
            c |= (bits >> 24) & 0x80;
            mc[e >> 2] |= c << (8 * (e & 3));
            // a variance above 0 stays above 0, or its element's next step would
            // be divided by eps alone
            uint32_t d = CodeV::encode(v[e] * v_inv, draw);
            d = v[e] > 0.0f && d == 0u ? 1u : d;
            d = finite(__float_as_uint(v[e])) ? d : CodeV::kNan;
            vc[e >> 2] |= d << (8 * (e & 3));
        }
        if (n > 0) {
            store_codes((uint8_t*)t.m + at, mc, n);
            store_codes((uint8_t*)t.v + at, vc, n);
            if ((at & (kStateBlock - 1)) == 0) {
                t.m_scale[at / kStateBlock] = __uint_as_float(me << 23);
                t.v_scale[at / kStateBlock] = __uint_as_float(ve << 23);
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
