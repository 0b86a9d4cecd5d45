// Philox4x32-10, the counter-based generator of the INT8 rounding and of the
// dropout masks.
//
// The SC'11 construction: per round two 32x32->64 multiplies of counter words
// 0 and 2, xor of the high halves with the other words and the round key; key
// bumped by the two Weyl constants.
#pragma once

#include "common.h"

namespace onebit {

__device__ __forceinline__ void philox_round(uint32_t& c0, uint32_t& c1, uint32_t& c2,
                                             uint32_t& c3, uint32_t k0, uint32_t k1) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0;
    const uint64_t p1 = (uint64_t)0xCD9E8D57u * c2;
    // three-way exclusive or in one instruction (0x96 is its truth table)
    const uint32_t n0 = __builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), c1, k0, 0x96);
    const uint32_t n1 = (uint32_t)p1;
    const uint32_t n2 = __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), c3, k1, 0x96);
    const uint32_t n3 = (uint32_t)p0;
    c0 = n0;
    c1 = n1;
    c2 = n2;
    c3 = n3;
}

__device__ __forceinline__ void philox10(uint32_t& c0, uint32_t& c1, uint32_t& c2, uint32_t& c3,
                                         uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        philox_round(c0, c1, c2, c3, k0, k1);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// ---------------------------------------------------------------- dropout draws
// The draws of an element (row, column): the 16-bit half word (column & 7) of
// the call on counter (column / 8, row low, row high, step), low half of a
// word first.  A key tweak keeps them apart from the INT8 rounding's draws
// under the same seed.  An element is kept where its draw is below
// threshold = round((1 - p) 65536): sixteen bits give p to 2^-17 at half the
// generator's work of 32-bit draws, and the kept share threshold / 65536 is
// exact, so the scale 65536 / threshold leaves the mean as it was.
constexpr uint32_t kDropTag = 0x44524F50u;
constexpr uint32_t kDropAll = 65536u;  // threshold that keeps every element

struct DropArgs {
    uint32_t k0, k1;           // seed words, the second with the tweak
    uint32_t step;             // added to *step_dev where that is given
    const uint32_t* step_dev;  // device word or nullptr
    uint32_t threshold;        // kDropAll: no draws
    float scale;               // 65536 / threshold
};

inline DropArgs drop_args(float p, uint64_t seed, uint32_t step, const uint32_t* step_dev) {
    DropArgs d;
    d.k0 = (uint32_t)seed;
    d.k1 = (uint32_t)(seed >> 32) ^ kDropTag;
    d.step = step;
    d.step_dev = step_dev;
    const double kept = (1.0 - (double)p) * 65536.0 + 0.5;  // p in [0, 1)
    d.threshold = kept < 1.0 ? 1u : (uint32_t)kept;
    d.scale = (float)(65536.0 / (double)d.threshold);
    return d;
}

// The eight draws of one group, packed two to a word.
__device__ __forceinline__ void drop_draws(uint32_t w[4], uint32_t group, uint64_t row,
                                           uint32_t step, uint32_t k0, uint32_t k1) {
    w[0] = group;
    w[1] = (uint32_t)row;
    w[2] = (uint32_t)(row >> 32);
    w[3] = step;
    philox10(w[0], w[1], w[2], w[3], k0, k1);
}

__device__ __forceinline__ bool drop_keep(const uint32_t w[4], int e, uint32_t threshold) {
    const uint32_t u = (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
    return u < threshold;
}

// The two decisions of one word at once: bit 0 and bit 16 set where the low
// and the high draw drop their element (saturating 16-bit arithmetic).
__device__ __forceinline__ uint32_t drop_pair(uint32_t w, uint32_t threshold) {
    using u16x2 = uint16_t __attribute__((ext_vector_type(2)));
    const uint16_t t = (uint16_t)(threshold - 1);
    const u16x2 over = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, w), u16x2{t, t});
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(over, u16x2{1, 1}));
}

// Where 32 columns' decisions lie when drop_pair's words of their four groups
// are gathered, word k of group g shifted by 4 g + k: even columns in the low
// half, odd ones in the high half.
__device__ __forceinline__ int drop_bit(int column) {
    return 16 * (column & 1) + 4 * (column >> 3) + ((column >> 1) & 3);
}

}  // namespace onebit
