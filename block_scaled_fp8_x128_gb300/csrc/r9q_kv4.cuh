// The paged 4-bit key-value cache: its layout, the quantiser that writes it and
// the read-back.  Shared by the kernels that write the cache
// (r9q_rope.cu) and by the attention that reads it (r9q_kv4_attention.cu).
//
// One bf16 pair (step, lowest) and D codes of 4 bits per token and head, K and
// V apart; code c stands for lowest + step * c.  The group is the whole head
// vector (64 or 128 elements), so the pair can be applied to a score, or folded
// into an attention weight, and never touches the inner products.
//   k  [pages][heads][page][D/2]: byte i of a token holds element 2i in its low
//      nibble and 2i+1 in its high one.
//   v  [pages][heads][page/16][D/64][8 r][4 j][4 m][4 b]: token t of a group of
//      16 has j = (t % 8) / 2, b = 2 (t % 2) + t / 8, and element
//      d = 64 c + 16 m + 8 n + r sits in nibble n (0 low) of byte [c][r][j][m][b].
//   kp, vp [pages][heads][page]: step in bits 0..15, lowest in bits 16..31.
// The V order is that of the A fragment of a 16x8x16 matrix product whose rows
// are elements and whose inner index is tokens: lane 4r + j loads 16 bytes that
// hold its fragments of four element tiles, with every byte owned by one token,
// so tokens are written without touching their neighbours.  K needs no
// reordering: there the tokens are the rows and a lane's 16 bytes of one token
// are its fragments.
#pragma once

#include "r9q_device.cuh"
#include "r9q_kernels.h"

namespace r9q {

// The quotient of 0 <= n < 2^31 by a divisor prepared on the host.
__device__ __forceinline__ int operator/(int n, const FastDiv& d) {
    return (int)(__umulhi((uint32_t)n * 2u, d.m) >> d.l);
}
inline FastDiv fast_div(int d) {
    int l = 0;
    while ((1ll << l) < d) ++l;
    return {(uint32_t)(((1ull << (31 + l)) + d - 1) / d), l, d};
}

__host__ __device__ __forceinline__ int64_t kv4_head_bytes(int page, int D) { return (int64_t)page * (D / 2); }

// Byte of token t (0..15) inside a group's [j][m][b] block, m = 0.
__device__ __forceinline__ int kv4_v_token_byte(int t) { return ((t & 7) >> 1) * 16 + 2 * (t & 1) + (t >> 3); }

// Reductions over the NL lanes that hold one head vector.
template <int NL>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = NL / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int NL>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = NL / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The largest of three; NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Quantises a head vector held by NL = D/8 adjacent lanes, 8 elements each.
// lowest = bf16(min), step = bf16((max - min) fl32(1/15)), both rounded to nearest (a
// 16-bit pair keeps the cost at 4 bytes a vector, and codes are taken against
// the rounded pair, so its rounding only moves the grid by a fraction of a
// step); code = clamp(rint((x - lowest) / step), 0, 15) with the IEEE fp32
// quotient (quot_exact, or the division where the step is tiny).  A constant
// vector has step 0 and codes 0.  A vector with a NaN or an infinity, or a range
// over fp32's, gets a NaN pair: it reads back as NaN.  Returns the lane's 8
// codes, element i in bits 4i..4i+3.
template <int NL>
__device__ __forceinline__ uint32_t kv4_quantise(const float (&x)[8], uint32_t& pair) {
    float hi = max3_nan(max3_nan(max3_nan(x[0], x[1], x[2]), x[3], x[4]), max3_nan(x[5], x[6], x[7]), x[0]);
    float lo = max3_nan(max3_nan(max3_nan(-x[0], -x[1], -x[2]), -x[3], -x[4]), max3_nan(-x[5], -x[6], -x[7]), -x[0]);
#pragma unroll
    for (int o = NL / 2; o > 0; o >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
        hi = max3_nan(hi, h, h);
        lo = max3_nan(lo, l, l);
    }
    lo = -lo;
    const float range = hi - lo;
    if (!(range < __int_as_float(0x7F800000))) {         // a NaN, an infinity, or no range that fp32 holds
        pair = 0x7FC07FC0u;
        return 0u;
    }
    const float low = bf16_round(lo), step = bf16_round(__fmul_rn(range, 1.0f / 15.0f));
    pair = pack_bf16x2(step, low);
    if (!(step > 0.0f)) return 0u;
    float q[8];
    const bool small = step < kQuotExactMinScale;
    const float r = __frcp_rn(step);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = x[i] - low;
        const float t = small ? __fdiv_rn(d, step) : quot_exact(d, step, r);
        // 2^23 + t rounds t to the nearest even integer
        q[i] = __fadd_rn(__fadd_rn(fminf(fmaxf(t, 0.0f), 15.0f), 8388608.0f), -8388608.0f);
    }
    // four codes make an integer below 2^16, exactly; adding 2^23 leaves it in the low bits
    const float a = fmaf(fmaf(fmaf(q[3], 16.0f, q[2]), 16.0f, q[1]), 16.0f, q[0]) + 8388608.0f;
    const float b = fmaf(fmaf(fmaf(q[7], 16.0f, q[6]), 16.0f, q[5]), 16.0f, q[4]) + 8388608.0f;
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
}

// Stores the codes of a head vector, lane l of NL = D/8 holding elements 8l..8l+7.
__device__ __forceinline__ void kv4_store_k(uint8_t* row, int l, uint32_t codes) {
    reinterpret_cast<uint32_t*>(row)[l] = codes;
}
// `group`: the 16-token group's first byte, t the token in it.  Lanes 2i and 2i+1 hold
// element tile i (its low- and high-nibble halves): they swap and store four bytes each.
__device__ __forceinline__ void kv4_store_v(uint8_t* group, int t, int l, uint32_t codes) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, codes, 1);
    if (!group) return;
    const int odd = l & 1, m = l >> 1;
    const uint32_t lo = (odd ? other : codes) >> (16 * odd), hi = (odd ? codes : other) >> (16 * odd);
    uint8_t* p = group + (m >> 2) * 512 + (m & 3) * 4 + kv4_v_token_byte(t) + odd * 256;
#pragma unroll
    for (int i = 0; i < 4; ++i)                                  // r = 4 odd + i
        p[i * 64] = (uint8_t)(((lo >> (4 * i)) & 15u) | (((hi >> (4 * i)) & 15u) << 4));
}

__device__ __forceinline__ uint32_t kv4_load_k(const uint8_t* row, int l) {
    return reinterpret_cast<const uint32_t*>(row)[l];
}
__device__ __forceinline__ uint32_t kv4_load_v(const uint8_t* group, int t, int l) {
    const int odd = l & 1, m = l >> 1;
    uint32_t mine = 0;
    if (group) {
        const uint8_t* p = group + (m >> 2) * 512 + (m & 3) * 4 + kv4_v_token_byte(t) + odd * 256;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine |= (uint32_t)p[i * 64] << (8 * i);
    }
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
    const uint32_t r03 = odd ? other : mine, r47 = odd ? mine : other;   // bytes r = 0..3 and 4..7
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        codes |= ((r03 >> (8 * i + 4 * odd)) & 15u) << (4 * i);
        codes |= ((r47 >> (8 * i + 4 * odd)) & 15u) << (16 + 4 * i);
    }
    return codes;
}

}  // namespace r9q
