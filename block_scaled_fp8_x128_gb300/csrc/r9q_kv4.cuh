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

// Launches a kernel of the attention block so that its CTAs may be set up while the
// kernel before it in the stream ends.  Each of these kernels begins with
// begin_chained(): the next one may be set up from then on, and nothing is read or
// written before all that came before is complete and visible.
template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                           const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Arrival of a CTA at a counter, by one thread after a barrier: releases what the CTA's
// threads wrote before the barrier, and for the last to arrive acquires what the others
// released.  Returns the arrivals before it.
__device__ __forceinline__ int arrive(int* counter) {
    int n;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
    return n;
}
__device__ __forceinline__ void begin_chained() {
    pdl_trigger();
    pdl_wait();
}

__host__ __device__ __forceinline__ int64_t kv4_head_bytes(int page, int D) { return (int64_t)page * (D / 2); }

// Byte of token t (0..15) inside a group's [j][m][b] block, m = 0.
__device__ __forceinline__ int kv4_v_token_byte(int t) { return ((t & 7) >> 1) * 16 + 2 * (t & 1) + (t >> 3); }

// ---- packed pairs of fp32 ----
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 parts_of(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Eight elements as four pairs.
struct Eight {
    uint64_t v[4];
};
__device__ __forceinline__ Eight unpack(const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = pair_of(bf16_lo(w[i]), bf16_hi(w[i]));
    return r;
}
__device__ __forceinline__ uint4 pack(const Eight& x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = parts_of(x.v[i]);
        w[i] = pack_bf16x2(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float dot(const Eight& a, const Eight& b) {
    uint64_t s = mul2(a.v[0], b.v[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = fma2(a.v[i], b.v[i], s);
    const float2 f = parts_of(s);
    return f.x + f.y;
}
__device__ __forceinline__ void spread(const Eight& x, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = parts_of(x.v[i]);
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
    }
}
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
// quotient.  A constant
// vector has step 0 and codes 0.  A vector with a NaN or an infinity, or a range
// over fp32's, gets a NaN pair: it reads back as NaN.  Returns the lane's 8
// codes, element i in bits 4i..4i+3.
template <int NL>
__device__ __forceinline__ uint32_t kv4_quantise(const Eight& v, uint32_t& pair) {
    float x[8];
    spread(v, x);
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
    float low = bf16_round(lo), step = bf16_round(__fmul_rn(range, 1.0f / 15.0f));
    pair = pack_bf16x2(step, low);
    if (!(range < __int_as_float(0x7F800000))) pair = 0x7FC07FC0u;   // a NaN, an infinity, or no range that fp32 holds
    // The quotient by quot_exact's steps, two at a time (low - x instead of x - low: the same, negated).  A step that
    // is too small for it is taken 2^100 times as large, and so are the differences: both exactly.
    const float up = step < kQuotExactMinScale ? 0x1p100f : 1.0f;
    step *= up;
    const float r = step > 0.0f ? __frcp_rn(step) : 0.0f;             // step 0: all codes 0
    const uint64_t one = pair_of(-1.0f, -1.0f), low2 = pair_of(low, low), step2 = pair_of(step, step),
                   up2 = pair_of(up, up), minus_r = pair_of(-r, -r), magic = pair_of(8388608.0f, 8388608.0f),
                   back = pair_of(-8388608.0f, -8388608.0f);
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t d = mul2(fma2(v.v[i], one, low2), up2);        // low - x
        const uint64_t y = mul2(d, minus_r), e = fma2(step2, y, d);
        const float2 f = parts_of(fma2(e, minus_r, y));
        // 2^23 + t rounds t to the nearest even integer
        const uint64_t k = pair_of(fminf(fmaxf(f.x, 0.0f), 15.0f), fminf(fmaxf(f.y, 0.0f), 15.0f));
        const float2 g = parts_of(add2(add2(k, magic), back));
        q[2 * i] = g.x;
        q[2 * i + 1] = g.y;
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

// ---- a whole group of 16 tokens of one head, two tokens (or more) a round ----
// With NV = 32 / NL tokens at a time, round i holds token NV i + sub in the lanes sub NL .. sub NL + NL - 1.
// Lane (sub, l): bytes r = 4 odd .. 4 odd + 3 (odd = l & 1) of element tile m = l >> 1 of every token it holds.

// Four nibbles to the low nibbles of four bytes.
__device__ __forceinline__ uint32_t nibbles_to_bytes(uint32_t n) {
    n = (n | (n << 8)) & 0x00FF00FFu;
    return (n | (n << 4)) & 0x0F0F0F0Fu;
}
__device__ __forceinline__ uint32_t bytes_to_nibbles(uint32_t b) {       // (bits 4..7 of each are 0)
    b = (b | (b >> 4)) & 0x00FF00FFu;
    return (b | (b >> 8)) & 0x0000FFFFu;
}
// The lane's four bytes of a token's element tile, from the tokens' codes (lane l: elements 8l .. 8l+7), and back.
__device__ __forceinline__ uint32_t kv4_tile_bytes(uint32_t codes, int l) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, codes, 1);
    const int odd = l & 1;
    const uint32_t lo = (odd ? other : codes) >> (16 * odd), hi = (odd ? codes : other) >> (16 * odd);
    return nibbles_to_bytes(lo & 0xFFFFu) | (nibbles_to_bytes(hi & 0xFFFFu) << 4);
}
__device__ __forceinline__ uint32_t kv4_tile_codes(uint32_t bytes, int l) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, bytes, 1);
    const int odd = l & 1;
    const uint32_t first = (odd ? other : bytes) >> (4 * odd), second = (odd ? bytes : other) >> (4 * odd);
    return bytes_to_nibbles(first & 0x0F0F0F0Fu) | (bytes_to_nibbles(second & 0x0F0F0F0Fu) << 16);
}

// D = 128 (two tokens a round, eight rounds): the even tokens are in lanes 0..15, the odd ones in 16..31.  A word of
// the group is {t = 2j, 2j + 8, 2j + 1, 2j + 9}: two bytes of either half, which swap so that a lane has rows
// 4 odd + 2 sub and the next of all four j.
// D = 64 (four tokens a round, four rounds): token 4i + sub; a word's bytes lie in lanes sub = 2 (j & 1) + (t & 1) of
// rounds j >> 1 and (j >> 1) + 2.
template <int D>
__device__ __forceinline__ void kv4_store_v_group(uint8_t* group, int lane, const uint32_t* bytes) {
    constexpr int NL = D / 8;
    const int l = lane & (NL - 1), sub = lane / NL, odd = l & 1, m = l >> 1;
    const int half = D == 128 ? sub : sub & 1;             // which bytes of a word the lane has: tokens of even or odd t
    uint8_t* p = group + (m >> 2) * 512 + (m & 3) * 4 + (4 * odd + 2 * half) * 64;
#pragma unroll
    for (int i = 0; i < (D == 128 ? 4 : 2); ++i) {
        const uint32_t a = bytes[i], b = bytes[i + (D == 128 ? 4 : 2)];
        const uint32_t r01 = __byte_perm(a, b, 0x5140), r23 = __byte_perm(a, b, 0x7362);
        const uint32_t got = __shfl_xor_sync(0xffffffffu, half ? r01 : r23, NL);
        const uint32_t even = half ? got : r01, odds = half ? r23 : got;
        const int j = D == 128 ? i : 2 * i + (sub >> 1);
        *reinterpret_cast<uint32_t*>(p + j * 16) = __byte_perm(even, odds, 0x5410);
        *reinterpret_cast<uint32_t*>(p + j * 16 + 64) = __byte_perm(even, odds, 0x7632);
    }
}
template <int D>
__device__ __forceinline__ void kv4_load_v_group(const uint8_t* group, int lane, uint32_t* bytes) {
    constexpr int NL = D / 8;
    const int l = lane & (NL - 1), sub = lane / NL, odd = l & 1, m = l >> 1;
    const int half = D == 128 ? sub : sub & 1;
    const uint8_t* p = group + (m >> 2) * 512 + (m & 3) * 4 + (4 * odd + 2 * half) * 64;
    uint32_t w[D / 32][2];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const int j = D == 128 ? i : 2 * i + (sub >> 1);
        w[i][0] = *reinterpret_cast<const uint32_t*>(p + j * 16);
        w[i][1] = *reinterpret_cast<const uint32_t*>(p + j * 16 + 64);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint32_t even = __byte_perm(w[i][0], w[i][1], 0x5410), odds = __byte_perm(w[i][0], w[i][1], 0x7632);
        const uint32_t got = __shfl_xor_sync(0xffffffffu, half ? even : odds, NL);
        const uint32_t r01 = half ? got : even, r23 = half ? odds : got;
        bytes[i] = __byte_perm(r01, r23, 0x6420);
        bytes[i + D / 32] = __byte_perm(r01, r23, 0x7531);
    }
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
