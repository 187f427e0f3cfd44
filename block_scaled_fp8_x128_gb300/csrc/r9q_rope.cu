// RMS norm of query and key heads with the position rotation in the same pass,
// its gradient, and the forms that write the paged 4-bit cache.
//
// A head vector x[D] with weight w: y = w x r, r = (mean(x^2) + eps)^-1/2; then
// each pair (a, b) of the first `rot` elements turns by its position's angle to
// (a cos - b sin, b cos + a sin).  Both are linear in x once r is known, so with
// x' the pair's other element
//   out = r (x (w c) + x' (w' s')),   s' = -sin for a, +sin for b,
// and w c, w' s' depend on the token and the element only: a warp forms them
// once and uses them for all its heads of the token.
//
// HBM bound: each input and output once (8192 tokens of 32 + 32 heads of 128: 43.4 us,
// 6.3 TB/s, 92 % of the copy rate; of 32 + 8: 32.8 us, 5.2 TB/s; eight tokens: 2.2 us,
// the launch).  A head vector takes D/8 lanes, 16 bytes
// each.  Where the whole vector turns in pairs (i, i + D/2), the common case, a lane
// takes four elements of either half (two 8-byte accesses), so that it holds both of
// each pair; otherwise it takes eight in a row and x' comes from the lane that holds
// it, by a shuffle of the packed input (adjacent pairs: from the same register).  A
// warp takes kUnroll x (32 / (D/8)) heads of one token at a time, all their loads in
// flight; warps of a block share a token where they can, so that the rows of the cos
// and sin tables come from L1 after the first.  Elements are worked on two at a time
// (packed fp32, two IEEE results an instruction).
#include <type_traits>

#include "r9q_kv4.cuh"

namespace r9q {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                   // 8192 tokens of 32 + 32 heads of 128: 43.4 us, with two 48.5 (32 + 8: 32.8/34.7)
// A warp takes up to so many rounds of heads of its token, which share its set-up, as long as that leaves
// kEnoughWarps.  Us, one round / always four / this rule, 32 + 32 heads of 128: 512 tokens 3.5/6.6/3.5, 1024 5.4/8.1/5.4,
// 2048 13.1/10.3/10.3, 4096 26.0/22.3/22.3, 8192 48.5/43.4/43.4; 32 + 8: 1024 4.5/6.0/4.5, 2048 7.5/7.2/7.2, 4096
// 16.6/15.9/15.9, 8192 32.3/32.8/32.8.
constexpr int kMaxRounds = 4;
constexpr int64_t kEnoughWarps = 152 * 24;
// Tokens from which a warp takes a head of 16 tokens at a time, which it can where they fill a group of the cache,
// instead of a token's heads.  8 heads of 128 (writes: and 32 query heads), us, by tokens / by groups / by groups where the
// call's windows of 16 tokens lie across two groups each, which then go token by token: writing 1024 tokens 8.7/8.2/11.4,
// 2048 13.8/12.4/14.7, 4096 27.0/20.6/22.7, 8192 49.5/37.3/40.4; appending 1024 4.7/7.1/12.4, 2048 6.4/7.1/10.2, 4096
// 9.9/8.6/12.3, 8192 18.6/15.3/19.5; reading 4096 5.4/5.9/9.6, 8192 9.6/8.0/13.6.
constexpr int kGroupTokens = 1024;
constexpr int kAppendGroupTokens = 4096;
constexpr int kGatherGroupTokens = 8192;

template <int D>
constexpr int heads_a_round() { return kUnroll * (256 / D); }

// The lane's elements of a head vector: the first four at first(l), the others at
// second(l).  SPLIT: four of either half, else eight in a row.
template <int D, bool SPLIT>
__device__ __forceinline__ int first(int l) { return SPLIT ? 4 * l : 8 * l; }
template <int D, bool SPLIT>
__device__ __forceinline__ int second(int l) { return SPLIT ? D / 2 + 4 * l : 8 * l + 4; }

template <int D, bool SPLIT>
__device__ __forceinline__ uint4 load_bf16(const uint16_t* head, int l) {
    if (!SPLIT) return *reinterpret_cast<const uint4*>(head + 8 * l);
    const uint2 a = *reinterpret_cast<const uint2*>(head + first<D, SPLIT>(l));
    const uint2 b = *reinterpret_cast<const uint2*>(head + second<D, SPLIT>(l));
    return make_uint4(a.x, a.y, b.x, b.y);
}
template <int D, bool SPLIT>
__device__ __forceinline__ void store_bf16(uint16_t* head, int l, const uint4& v) {
    if (SPLIT) {
        *reinterpret_cast<uint2*>(head + first<D, SPLIT>(l)) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2*>(head + second<D, SPLIT>(l)) = make_uint2(v.z, v.w);
    } else {
        *reinterpret_cast<uint4*>(head + 8 * l) = v;
    }
}
// Four floats at p, on a 16-byte boundary or not.
__device__ __forceinline__ float4 load4(const float* p, bool wide) {
    return wide ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ Eight eight_of(const float4& a, const float4& b) {
    return {{pair_of(a.x, a.y), pair_of(a.z, a.w), pair_of(b.x, b.y), pair_of(b.z, b.w)}};
}
template <int D, bool SPLIT>
__device__ __forceinline__ Eight load_weight(const float* w, int l) {
    const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
    return eight_of(load4(w + first<D, SPLIT>(l), wide), load4(w + second<D, SPLIT>(l), wide));
}

// A lane's part of the rotation: its eight cos and signed sin (-sin for the first
// element of a pair), and without SPLIT the lane that holds its pairs' other elements.
struct Turn {
    int src;
    Eight c, s;
};
constexpr uint64_t kSigns = 0x8000000080000000ull;

// (0 where nothing turns: pos may be NULL then)
__device__ __forceinline__ int64_t load_pos(const RopeParams& p, int t) { return p.rot > 0 ? p.pos[t] : 0; }

template <int D, bool SPLIT>
__device__ __forceinline__ Turn load_turn(const RopeParams& p, int64_t pos, int lane) {
    const int l = lane & (D / 8 - 1), d0 = 8 * l, half = p.rot / 2;
    Turn u;
    u.src = lane;
    if (!SPLIT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u.c.v[i] = pair_of(1.0f, 1.0f), u.s.v[i] = 0;
        if (p.rot == 0) return u;
    }
    if (pos < 0 || pos >= p.npos) {
        if (lane == 0) record_error(p.err, kErrArg);
        const float nan = __int_as_float(0x7FC00000);
#pragma unroll
        for (int i = 0; i < 4; ++i) u.c.v[i] = u.s.v[i] = pair_of(nan, nan);
        return u;
    }
    const float* cs = p.cos + pos * half;
    const float* sn = p.sin + pos * half;
    if (SPLIT) {
        const float4 c = load4(cs + 4 * l, true), s = load4(sn + 4 * l, true);
        u.c = eight_of(c, c);
        u.s = eight_of(s, s);
        u.s.v[0] ^= kSigns;
        u.s.v[1] ^= kSigns;
        return u;
    }
    if (d0 >= p.rot) return u;
    if (p.interleaved) {
        const float4 a = load4(cs + d0 / 2, true), b = load4(sn + d0 / 2, true);
        const float c4[4] = {a.x, a.y, a.z, a.w}, s4[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u.c.v[i] = pair_of(c4[i], c4[i]);
            u.s.v[i] = pair_of(-s4[i], s4[i]);
        }
    } else {
        const bool upper = d0 >= half;
        const int at = upper ? d0 - half : d0;
        u.src = upper ? lane - half / 8 : lane + half / 8;
        u.c = eight_of(load4(cs + at, true), load4(cs + at + 4, true));
        u.s = eight_of(load4(sn + at, true), load4(sn + at + 4, true));
        if (!upper) {
#pragma unroll
            for (int i = 0; i < 4; ++i) u.s.v[i] ^= kSigns;
        }
    }
    return u;
}

// What load_turn() reads, to be loaded ahead: nothing without SPLIT, where turn_of() loads.
struct Angles {
    float4 c, s;
};
template <int D, bool SPLIT>
__device__ __forceinline__ Angles load_angles(const RopeParams& p, int64_t pos, int l, int lane) {
    Angles x = {};
    if (!SPLIT) return x;
    if (pos < 0 || pos >= p.npos) {
        if (lane == 0) record_error(p.err, kErrArg);
        const float nan = __int_as_float(0x7FC00000);
        x.c = x.s = make_float4(nan, nan, nan, nan);
        return x;
    }
    x.c = load4(p.cos + pos * (D / 2) + 4 * l, true);
    x.s = load4(p.sin + pos * (D / 2) + 4 * l, true);
    return x;
}
template <int D, bool SPLIT>
__device__ __forceinline__ Turn turn_of(const RopeParams& p, const Angles& x, int64_t pos, int lane) {
    if (!SPLIT) return load_turn<D, SPLIT>(p, pos, lane);
    Turn u;
    u.src = lane;
    u.c = eight_of(x.c, x.c);
    u.s = eight_of(x.s, x.s);
    u.s.v[0] ^= kSigns;
    u.s.v[1] ^= kSigns;
    return u;
}

// The other elements of the lane's pairs; `raw` the lane's elements as packed bf16, x unpacked.
template <bool SPLIT>
__device__ __forceinline__ Eight partner(const uint4& v, const Eight& x, const Turn& u, int interleaved) {
    if (SPLIT) return {{x.v[2], x.v[3], x.v[0], x.v[1]}};
    if (interleaved)
        return unpack(make_uint4(__byte_perm(v.x, 0, 0x1032), __byte_perm(v.y, 0, 0x1032),
                                 __byte_perm(v.z, 0, 0x1032), __byte_perm(v.w, 0, 0x1032)));
    return unpack(make_uint4(__shfl_sync(0xffffffffu, v.x, u.src), __shfl_sync(0xffffffffu, v.y, u.src),
                             __shfl_sync(0xffffffffu, v.z, u.src), __shfl_sync(0xffffffffu, v.w, u.src)));
}
// w c and w' s' for the lane's elements, in place of c and s.
template <int D, bool SPLIT>
__device__ __forceinline__ void fold_weight(Turn& u, const float* w, int lane, int interleaved) {
    const Eight own = load_weight<D, SPLIT>(w, lane & (D / 8 - 1));
    const Eight other = SPLIT ? Eight{{own.v[2], own.v[3], own.v[0], own.v[1]}}
                        : interleaved ? own : load_weight<D, SPLIT>(w, u.src & (D / 8 - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u.c.v[i] = mul2(u.c.v[i], own.v[i]);
        const float2 o = parts_of(other.v[i]);
        u.s.v[i] = mul2(u.s.v[i], !SPLIT && interleaved ? pair_of(o.y, o.x) : other.v[i]);
    }
}
__device__ __forceinline__ float inverse_root(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Sum of the squares of a head vector in a fixed order, one rounding a step: 32
// partial sums of every 32nd square, in their order, then a binary tree over
// neighbouring partial sums.  The lanes that hold a partial sum's terms exchange
// them so that each forms its share of the partial sums.
template <int NL, bool SPLIT>
__device__ __forceinline__ float sum_squares_in_order(const float (&x)[8], int l) {
    float q[8], s;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(x[i], x[i]);
    if constexpr (SPLIT && NL == 8) {                     // a lane has four partial sums
        s = __fadd_rn(__fadd_rn(__fadd_rn(q[0], q[4]), __fadd_rn(q[1], q[5])),
                      __fadd_rn(__fadd_rn(q[2], q[6]), __fadd_rn(q[3], q[7])));
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 1));
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 2));
        return __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 4));
    } else if constexpr (SPLIT) {                         // lanes l, l ^ 8: two partial sums each, two terms of four
        const bool up = l & 8;
        float p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float a = __shfl_xor_sync(0xffffffffu, up ? q[i] : q[2 + i], 8);
            const float b = __shfl_xor_sync(0xffffffffu, up ? q[4 + i] : q[6 + i], 8);
            const float c = up ? q[2 + i] : q[i], d = up ? q[6 + i] : q[4 + i];
            p[i] = __fadd_rn(__fadd_rn(__fadd_rn(up ? a : c, up ? c : a), up ? b : d), up ? d : b);
        }
        s = __fadd_rn(p[0], p[1]);
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 8));
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 1));
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 2));
        return __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 4));
    } else if constexpr (NL == 8) {                       // lanes l, l ^ 4: four partial sums each, two terms
        const bool up = l & 4;
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? q[i] : q[4 + i], 4);
            p[i] = __fadd_rn(up ? q[4 + i] : q[i], other);
        }
        s = __fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3]));
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 4));
    } else {                                              // lanes l, l ^ 4, l ^ 8, l ^ 12: two partial sums, four terms
        const bool hi = l & 8, lo = l & 4;
        float a[4], b[4];                                 // elements 4 hi .. 4 hi + 3 of this lane and of l ^ 8
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = hi ? q[4 + i] : q[i];
            b[i] = __shfl_xor_sync(0xffffffffu, hi ? q[i] : q[4 + i], 8);
        }
        float p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float a1 = __shfl_xor_sync(0xffffffffu, lo ? a[i] : a[2 + i], 4);
            const float b1 = __shfl_xor_sync(0xffffffffu, lo ? b[i] : b[2 + i], 4);
            const float a0 = lo ? a[2 + i] : a[i], b0 = lo ? b[2 + i] : b[i];
            // the terms by their lanes: l & 3, + 4, + 8, + 12
            const float t0 = hi ? (lo ? b1 : b0) : (lo ? a1 : a0), t1 = hi ? (lo ? b0 : b1) : (lo ? a0 : a1);
            const float t2 = hi ? (lo ? a1 : a0) : (lo ? b1 : b0), t3 = hi ? (lo ? a0 : a1) : (lo ? b0 : b1);
            p[i] = __fadd_rn(__fadd_rn(__fadd_rn(t0, t1), t2), t3);
        }
        s = __fadd_rn(p[0], p[1]);                        // partial sums 8 (l & 3) + 4 hi + 2 lo, and the next
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 4));
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 8));
    }
    s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 1));
    return __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 2));
}

// A key on its way to 4 bits.  A code flips where its value lies within an fp32
// rounding of the middle between two codes, so the keys' value is fixed to the
// last bit: (x r) w, the two products of the rotation and their sum each round
// once, and the sum of squares has sum_squares_in_order's order.  An evaluation in
// fp32 in that order gives the same codes; another order would do as well, but moves
// about one code in a million.
template <int NL, bool SPLIT>
__device__ __forceinline__ Eight norm_rope_in_order(const Eight& x, const Eight& weight, const Turn& u, int lane,
                                                    const RopeParams& p) {
    float y[8], w[8], cs[8], sn[8];
    spread(x, y);
    spread(weight, w);
    spread(u.c, cs);
    spread(u.s, sn);
    const float mean = __fmul_rn(sum_squares_in_order<NL, SPLIT>(y, lane & (NL - 1)), 1.0f / (8 * NL));
    const float r = inverse_root(__fadd_rn(mean, p.eps));
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(__fmul_rn(y[e], r), w[e]);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = SPLIT ? y[e ^ 4] : p.interleaved ? y[e ^ 1] : __shfl_sync(0xffffffffu, y[e], u.src);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __fadd_rn(__fmul_rn(y[e], cs[e]), __fmul_rn(z[e], sn[e]));
    return {{pair_of(y[0], y[1]), pair_of(y[2], y[3]), pair_of(y[4], y[5]), pair_of(y[6], y[7])}};
}

enum Pass { kRope, kRopeCache, kAppend };

struct ForwardArgs {
    HeadsIn q, k, v;
    HeadsOut qo, ko;
    RopeParams rope;
    Kv4Cache c;
    const int64_t* slots;
    int64_t T;
    int rounds;              // of heads a warp takes
    int nq, nk;              // warps that a token's query and key heads take
    FastDiv parts;           // and all its heads
    // the launch by whole groups of tokens
    int windows;             // of 16 tokens
    uint32_t cache_share;    // of its blocks that are the cache's, in 2^-32
    FastDiv v_heads, k_parts;
};

// Where a token goes: its page and place, or page -1 for padding and for a slot
// outside the cache (an error).
struct Place {
    int64_t page;
    int at;
};
__device__ __forceinline__ int64_t page_of(const Kv4Cache& c, int64_t slot) {      // slot >= 0
    return slot >> 32 ? slot / c.page : (int64_t)((uint32_t)slot / (uint32_t)c.page);
}
__device__ __forceinline__ Place find_slot(const Kv4Cache& c, int64_t slot, int lane, int* err) {
    Place r = {-1, 0};
    if (slot >= 0) {
        const int64_t page = page_of(c, slot);
        if (page < c.pages) {
            r.page = page;
            r.at = (int)(slot - page * c.page);
        } else if (lane == 0) {
            record_error(err, kErrArg);
        }
    }
    return r;
}

// A warp's share of a token's key or value heads h, h + NV, ... below `end`, into the cache:
// keys normalised and turned (`turned`) or as they are, values as they are.
template <int D, bool SPLIT>
__device__ __forceinline__ void write_heads(const ForwardArgs& a, const HeadsIn& in, bool key, bool turned, int t, int h,
                                            int end, int lane) {
    constexpr int NL = D / 8, NV = 32 / NL, HR = heads_a_round<D>();
    const int l = lane & (NL - 1), sub = lane / NL;
    const uint16_t* src = in.p + t * in.ts + h * in.hs;
    uint4 x[kUnroll];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (h + i * NV < end) x[i] = turned ? load_bf16<D, SPLIT>(src, l) : load_bf16<D, false>(src, l);
            src += NV * in.hs;
        }
    };
    load(h);                                             // (on its way first)
    const Place place = find_slot(a.c, a.slots[t], lane, a.rope.err);
    Turn u;
    Eight w;
    if (turned) {
        u = load_turn<D, SPLIT>(a.rope, load_pos(a.rope, t), lane);
        w = load_weight<D, SPLIT>(a.rope.wk, l);
    }
    for (; h - sub < end; h += HR) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (h - sub + i * NV >= end) break;          // the same for the whole warp
            Eight z = unpack(x[i]);
            if (turned) z = norm_rope_in_order<NL, SPLIT>(z, w, u, lane, a.rope);
            uint32_t pair;
            const uint32_t codes = kv4_quantise<NL>(z, pair);
            const bool live = h + i * NV < end && place.page >= 0;
            const int64_t head = place.page * a.c.heads + h + i * NV;
            if (key) {
                if (live) {
                    uint8_t* row = a.c.k + head * kv4_head_bytes(a.c.page, D) + (int64_t)place.at * (D / 2);
                    if (turned && SPLIT) {               // elements 2i and 2i + 1 share byte i
                        *reinterpret_cast<uint16_t*>(row + 2 * l) = (uint16_t)codes;
                        *reinterpret_cast<uint16_t*>(row + D / 4 + 2 * l) = (uint16_t)(codes >> 16);
                    } else {
                        kv4_store_k(row, l, codes);
                    }
                    if (l == 0) a.c.kp[head * a.c.page + place.at] = pair;
                }
            } else {
                kv4_store_v(live ? a.c.v + head * kv4_head_bytes(a.c.page, D) + (int64_t)(place.at >> 4) * (8 * D)
                                 : nullptr,
                            place.at & 15, l, codes);
                if (live && l == 0) a.c.vp[head * a.c.page + place.at] = pair;
            }
        }
        if (h - sub + HR < end) load(h + HR);
    }
}

// A warp's share of a token's query or key heads h, h + NV, ... below `end`: normalised and turned, as bf16.
template <int D, bool SPLIT>
__device__ __forceinline__ void turn_heads(const RopeParams& p, const HeadsIn& in, const HeadsOut& out,
                                           const float* weight, int t, int h, int end, int lane) {
    constexpr int NL = D / 8, NV = 32 / NL, HR = heads_a_round<D>();
    const int l = lane & (NL - 1), sub = lane / NL;
    const uint16_t* src = in.p + t * in.ts + h * in.hs;
    uint16_t* dst = out.p + t * out.ts + h * out.hs;
    Turn u;
    bool ready = false;
    for (; h - sub < end; h += HR) {
        uint4 x[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            x[i] = h + i * NV < end ? load_bf16<D, SPLIT>(src, l) : make_uint4(0u, 0u, 0u, 0u);
            src += NV * in.hs;
        }
        if (!ready) {                                    // (after the loads are on their way)
            u = load_turn<D, SPLIT>(p, load_pos(p, t), lane);
            fold_weight<D, SPLIT>(u, weight, lane, p.interleaved);
            ready = true;
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            Eight y = unpack(x[i]);
            const Eight xp = partner<SPLIT>(x[i], y, u, p.interleaved);
            const float r = inverse_root(fmaf(group_sum<NL>(dot(y, y)), 1.0f / D, p.eps));
            const uint64_t rr = pair_of(r, r);
            Eight z;
#pragma unroll
            for (int e = 0; e < 4; ++e) z.v[e] = mul2(rr, fma2(y.v[e], u.c.v[e], mul2(xp.v[e], u.s.v[e])));
            if (h + i * NV < end) store_bf16<D, SPLIT>(dst, l, pack(z));
            dst += NV * out.hs;
        }
    }
}

// One launch over tokens, their query, key and value heads side by side.
template <int D, int PASS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, PASS == kRope && SPLIT ? 4 : 3) forward_kernel(const ForwardArgs a) {
    begin_chained();
    constexpr int NL = D / 8, HR = heads_a_round<D>();
    const int lane = threadIdx.x & 31, sub = lane / NL;
    const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = unit / a.parts;
    if (t >= a.T) return;
    int part = unit - t * a.parts.d;
    int kind = 0;                                        // 0 query, 1 key, 2 value
    if (part >= a.nq) {
        part -= a.nq;
        kind = 1;
        if (part >= a.nk) {
            part -= a.nk;
            kind = 2;
        }
    }
    const HeadsIn& in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int h = part * a.rounds * HR + sub;            // the lane's first head
    const int end = min(in.heads, part * a.rounds * HR + a.rounds * HR);
    if (PASS == kRope || (PASS == kRopeCache && kind == 0))
        turn_heads<D, SPLIT>(a.rope, in, kind == 0 ? a.qo : a.ko, kind == 0 ? a.rope.wq : a.rope.wk, t, h, end, lane);
    else
        write_heads<D, SPLIT>(a, in, kind == 1, PASS != kAppend && kind < 2, t, h, end, lane);
}

// The 16 tokens of a window, if they are a whole group of the cache in order: the group's place, else page -1.
__device__ __forceinline__ Place group_of(const Kv4Cache& c, const int64_t* slots, int64_t t0, int64_t T, int lane) {
    Place r = {-1, 0};
    if (t0 + 16 > T) return r;
    const int64_t slot = slots[t0 + (lane & 15)], first = __shfl_sync(0xffffffffu, slot, 0);
    const bool group = first >= 0 && first % 16 == 0 && slot == first + (lane & 15);
    if (!__all_sync(0xffffffffu, group)) return r;
    const int64_t page = page_of(c, first);
    if (page >= c.pages) return r;                       // (the tokens, one by one, record the error)
    r.page = page;
    r.at = (int)(first - page * c.page);
    return r;
}

// Many tokens into the cache.  Value warps take one head of 16 tokens of the call at a time: where these are a group of
// the cache they put whole words together and store those, not a byte at a time (8192 tokens of 8 heads: 4.2 M partial
// sectors written become 0.3 M).  That holds for a prompt whose first token in the call begins a group; one that begins
// elsewhere, or after others in the call whose lengths are no multiples of 16, goes token by token here (kGroupTokens has
// the times).  Key warps as above.  The query heads, which HBM bounds, and the quantising are blocks of one grid in
// turn, so that an SM has both.  8192 tokens of 32 + 8 + 8 heads of 128: 37.3 us; its bytes alone would take 26.  63 % of
// the issue slots, and the 44 % of the warps that registers leave wait for loads most.
template <int D, bool TURNED, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 4) prompt_kernel(const ForwardArgs a) {
    begin_chained();
    constexpr int NL = D / 8, NV = 32 / NL, HR = heads_a_round<D>(), ROUNDS = 16 / NV;
    const int lane = threadIdx.x & 31, l = lane & (NL - 1), sub = lane / NL, warp = threadIdx.x >> 5;
    // of every grid / cache_blocks blocks one is the cache's
    const uint32_t before = __umulhi(blockIdx.x, a.cache_share), upto = __umulhi(blockIdx.x + 1, a.cache_share);
    if (TURNED && upto == before) {
        const int unit = (blockIdx.x - before) * (kThreads / 32) + warp, t = unit / a.parts;
        if (t >= a.T) return;
        const int h = (unit - t * a.parts.d) * a.rounds * HR;
        turn_heads<D, SPLIT>(a.rope, a.q, a.qo, a.rope.wq, t, h + sub, min(a.q.heads, h + a.rounds * HR), lane);
        return;
    }
    int unit = (TURNED ? before : blockIdx.x) * (kThreads / 32) + warp;
    if (unit >= a.windows * a.v_heads.d) {
        unit -= a.windows * a.v_heads.d;
        const int t = unit / a.k_parts;
        if (t >= a.T) return;
        const int h = (unit - t * a.k_parts.d) * HR;
        write_heads<D, SPLIT>(a, a.k, true, TURNED, t, h + sub, min(a.k.heads, h + HR), lane);
        return;
    }
    const int window = unit / a.v_heads, h = unit - window * a.v_heads.d;
    const int64_t t0 = (int64_t)window * 16;
    uint4 x[ROUNDS];
    const uint16_t* src = a.v.p + (t0 + sub) * a.v.ts + h * a.v.hs + 8 * l;
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i)
        x[i] = t0 + i * NV + sub < a.T ? *reinterpret_cast<const uint4*>(src + i * NV * a.v.ts)
                                       : make_uint4(0u, 0u, 0u, 0u);
    const Place place = group_of(a.c, a.slots, t0, a.T, lane);
    uint32_t codes[ROUNDS], pairs[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) codes[i] = kv4_quantise<NL>(unpack(x[i]), pairs[i]);
    if (place.page >= 0) {
        const int64_t head = place.page * a.c.heads + h;
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) codes[i] = kv4_tile_bytes(codes[i], l);
        kv4_store_v_group<D>(a.c.v + head * kv4_head_bytes(a.c.page, D) + (int64_t)place.at * (D / 2), lane, codes);
        uint32_t pair = pairs[0];
#pragma unroll
        for (int i = 1; i < ROUNDS; ++i) pair = l == i ? pairs[i] : pair;
        if (l < ROUNDS) a.c.vp[head * a.c.page + place.at + l * NV + sub] = pair;
        return;
    }
#pragma unroll 1
    for (int i = 0; i < ROUNDS; ++i) {                   // token by token
        uint32_t code = codes[0], pair = pairs[0];
#pragma unroll
        for (int k = 1; k < ROUNDS; ++k) {
            code = i == k ? codes[k] : code;
            pair = i == k ? pairs[k] : pair;
        }
        const int64_t t = t0 + i * NV + sub;
        Place one = {-1, 0};
        if (t < a.T) one = find_slot(a.c, a.slots[t], l, a.rope.err);
        const bool live = one.page >= 0;
        const int64_t head = one.page * a.c.heads + h;
        kv4_store_v(live ? a.c.v + head * kv4_head_bytes(a.c.page, D) + (int64_t)(one.at >> 4) * (8 * D) : nullptr,
                    one.at & 15, l, code);
        if (live && l == 0) a.c.vp[head * a.c.page + one.at] = pair;
    }
}

template <int D, int PASS>
cudaError_t launch_forward(ForwardArgs a, cudaStream_t st) {
    constexpr int HR = heads_a_round<D>();
    const bool split = PASS != kAppend && a.rope.rot == D && !a.rope.interleaved;
    auto warps = [&](int heads) { return (heads + a.rounds * HR - 1) / (a.rounds * HR); };
    auto blocks_of = [](int64_t n) { return (n + kThreads / 32 - 1) / (kThreads / 32); };
    // (kMaxRounds, kEnoughWarps)
    const bool groups = PASS != kRope && a.T >= (PASS == kAppend ? kAppendGroupTokens : kGroupTokens);
    for (a.rounds = kMaxRounds;; a.rounds /= 2) {
        a.nq = PASS == kAppend ? 0 : warps(a.q.heads);
        a.nk = groups ? 0 : warps(a.k.heads);
        const int parts = a.nq + a.nk + (PASS == kRope || groups ? 0 : warps(a.v.heads));
        a.parts = fast_div(parts > 0 ? parts : 1);
        if (a.rounds == 1 || a.T * parts >= kEnoughWarps) break;
    }
    const int64_t most = INT32_MAX / (kThreads / 32);
    int64_t blocks = blocks_of(a.T * a.parts.d);
    if (blocks > most) return cudaErrorInvalidValue;
    if constexpr (PASS != kRope) {
        if (groups) {
            a.windows = (int)((a.T + 15) / 16);
            a.v_heads = fast_div(a.v.heads);
            a.k_parts = fast_div((a.k.heads + HR - 1) / HR);
            const int64_t cache = blocks_of((int64_t)a.windows * a.v.heads + a.T * a.k_parts.d);
            if (PASS == kAppend) blocks = 0;
            blocks += cache;
            if (blocks > most) return cudaErrorInvalidValue;
            a.cache_share = (uint32_t)((((uint64_t)cache << 32) + blocks - 1) / blocks);       // (rounded up: all of them)
            auto kernel = split ? prompt_kernel<D, PASS == kRopeCache, PASS == kRopeCache>
                                : prompt_kernel<D, PASS == kRopeCache, false>;
            return launch_chained(kernel, (unsigned)blocks, kThreads, 0, st, a);
        }
    }
    return launch_chained(split ? forward_kernel<D, PASS, PASS != kAppend> : forward_kernel<D, PASS, false>,
                          (unsigned)blocks, kThreads, 0, st, a);
}

template <int PASS>
cudaError_t launch_forward_d(int D, const ForwardArgs& a, cudaStream_t st) {
    return D == 64 ? launch_forward<64, PASS>(a, st) : launch_forward<128, PASS>(a, st);
}

// ------------------------------------------------------------- read-back --

// bf16(lowest + step * code).
__device__ __forceinline__ uint4 kv4_values(uint32_t codes, uint32_t pair) {
    const uint64_t step = pair_of(bf16_lo(pair), bf16_lo(pair)), low = pair_of(bf16_hi(pair), bf16_hi(pair));
    Eight y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // 2^23 + code, as its bits, less 2^23
        const uint32_t a = 0x4B000000u | (codes >> (8 * i) & 15u), b = 0x4B000000u | (codes >> (8 * i + 4) & 15u);
        const uint64_t c = add2(pair_of(__uint_as_float(a), __uint_as_float(b)), pair_of(-8388608.0f, -8388608.0f));
        y.v[i] = fma2(step, c, low);
    }
    return pack(y);
}

// The tokens at `slots`, zeros for padding: a warp takes NV heads of one token, or (gather_groups_kernel) a head of 16
// tokens where they are a group of the cache.  8192 tokens of 8 heads of 128, 42 MB: 8.0 us, where the bytes would take
// 6.2; a warp loads, converts and stores once, and nothing of its own overlaps its wait.
template <int D>
__device__ __forceinline__ void gather_token(const Kv4Cache& c, const Place& place, int64_t t, int h, bool mine, int l,
                                             uint16_t* k, uint16_t* v) {
    const bool live = place.page >= 0 && mine;
    const int64_t head = place.page * c.heads + h;
    uint32_t codes = 0, pair[2] = {0, 0};
    if (live) {
        codes = kv4_load_k(c.k + head * kv4_head_bytes(c.page, D) + (int64_t)place.at * (D / 2), l);
        pair[0] = c.kp[head * c.page + place.at];
        pair[1] = c.vp[head * c.page + place.at];
    }
    const uint32_t vcodes = kv4_load_v(
        live ? c.v + head * kv4_head_bytes(c.page, D) + (int64_t)(place.at >> 4) * (8 * D) : nullptr, place.at & 15, l);
    if (!mine) return;
    *reinterpret_cast<uint4*>(k + (t * c.heads + h) * D + 8 * l) = kv4_values(codes, pair[0]);
    *reinterpret_cast<uint4*>(v + (t * c.heads + h) * D + 8 * l) = kv4_values(vcodes, pair[1]);
}
template <int D>
__global__ void __launch_bounds__(kThreads) gather_kernel(const Kv4Cache c, const int64_t* slots, int64_t T,
                                                          const FastDiv parts, uint16_t* k, uint16_t* v, int* err) {
    begin_chained();
    constexpr int NL = D / 8, NV = 32 / NL;
    const int lane = threadIdx.x & 31, l = lane & (NL - 1), sub = lane / NL;
    const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = unit / parts;
    if (t >= T) return;
    const int h = (unit - t * parts.d) * NV + sub;
    gather_token<D>(c, find_slot(c, slots[t], lane, err), t, h, h < c.heads, l, k, v);
}

// Many tokens: a warp takes one head of 16 of them, word by word where they are a group of the cache.
template <int D>
__global__ void __launch_bounds__(kThreads) gather_groups_kernel(const Kv4Cache c, const int64_t* slots, int64_t T,
                                                                 const FastDiv heads, uint16_t* k, uint16_t* v,
                                                                 int* err) {
    begin_chained();
    constexpr int NL = D / 8, NV = 32 / NL, ROUNDS = 16 / NV;
    const int lane = threadIdx.x & 31, l = lane & (NL - 1), sub = lane / NL;
    const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int window = unit / heads, h = unit - window * heads.d;
    const int64_t t0 = (int64_t)window * 16;
    if (t0 >= T) return;
    const Place place = group_of(c, slots, t0, T, lane);
    if (place.page < 0) {
#pragma unroll 1
        for (int i = 0; i < ROUNDS; ++i) {
            const int64_t t = t0 + i * NV + sub;
            Place one = {-1, 0};
            if (t < T) one = find_slot(c, slots[t], l, err);
            gather_token<D>(c, one, t, h, t < T, l, k, v);
        }
        return;
    }
    const int64_t head = place.page * c.heads + h;
    const uint8_t* rows = c.k + head * kv4_head_bytes(c.page, D) + (int64_t)place.at * (D / 2);
    uint32_t codes[ROUNDS], bytes[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) codes[i] = kv4_load_k(rows + (i * NV + sub) * (D / 2), l);
    kv4_load_v_group<D>(c.v + head * kv4_head_bytes(c.page, D) + (int64_t)place.at * (D / 2), lane, bytes);
    const uint32_t kp = c.kp[head * c.page + place.at + (lane & 15)], vp = c.vp[head * c.page + place.at + (lane & 15)];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
        const int64_t at = ((t0 + i * NV + sub) * c.heads + h) * D + 8 * l;
        *reinterpret_cast<uint4*>(k + at) = kv4_values(codes[i], __shfl_sync(0xffffffffu, kp, i * NV + sub));
        *reinterpret_cast<uint4*>(v + at) =
            kv4_values(kv4_tile_codes(bytes[i], l), __shfl_sync(0xffffffffu, vp, i * NV + sub));
    }
}

// -------------------------------------------------------------- gradient --

// With g = R^T dy (the turn by the opposite angle) and xh = x r:
//   dw = sum over tokens and heads of g xh,
//   dx = r (w g - xh mean(w g xh)).
// xh is of the order of one whatever x is, and r goes in once and last, so that inputs of
// any size are in range whose mean square is (a form with r^3 is not from an rms of 1e14).
// r is computed again from x: that reads nothing that dx does not need.  A unit is a
// token's query or key heads, kBwdUnroll loads of a warp at a time; the warps of one
// block an SM take equal, contiguous ranges of all units, so that a token's angles are
// loaded once, and ahead.  The projection takes a second reduction after r; in whole units the
// first ones of all vectors overlap (4096 tokens 24.0 us; one vector after another 26.7, 16,384
// 80.0 and 84.4).  A warp copies its next unit's dy and x to shared memory while it works
// on one, and each lane sums its elements' dw in 32 bits; a block's sums go to `part`,
// and the block that finishes last adds the blocks' sums in their order, all loads in
// flight, so dw does not depend on timing.
//
// Bound: HBM, once the batch is long.  12 warps have 168 registers each, which lets
// the four vectors' reductions overlap.  32 + 8 heads of 128 (us, 12 warps / 16): 256
// tokens 5.5/5.8, 1024 8.6/9.8, 4096 24.0/25.4, 16384 80.0/87.5 (the bytes alone: 75);
// with few heads 16 are a little faster (8192 tokens of 14 + 2 heads of 64 16.9/16.1).
// Of the 24, about 5 are the launch, the first loads and the last block's sums.
struct BackwardArgs {
    HeadsIn dqo, dko, q, k;
    RopeParams rope;
    HeadsOut dq, dk;
    float *dwq, *dwk, *part;
    int* done;
    FastDiv parts;               // units of a token: those of its query heads, then of its key heads
    int q_parts, per_warp, more; // a warp has per_warp units, the first `more` warps one more
};
constexpr int kBwdThreads = 384;
constexpr int kBwdUnroll = 4;
constexpr int kBwdStages = 2;
constexpr int kBwdStage = kBwdUnroll * 1024;                 // bytes: the warp's parts of dy and x
constexpr int kBwdSmem = kBwdThreads / 32 * kBwdStages * kBwdStage;
static_assert(kBwdSmem >= kBwdThreads / 32 * 256 * 4 && kBwdSmem >= kBwdThreads * 16, "room for the sums");

// 16 bytes of each to shared memory, zeros where not `live`.
__device__ __forceinline__ void copy16(bool live, uint32_t g_dst, const void* g, uint32_t x_dst, const void* x) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %4;\n\tcp.async.cg.shared.global [%2], [%3], 16, %4;" ::"r"(
                     g_dst),
                 "l"(g), "r"(x_dst), "l"(x), "r"(live ? 16 : 0)
                 : "memory");
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads, 1) backward_kernel(const BackwardArgs a) {
    begin_chained();
    constexpr int NL = D / 8, NV = 32 / NL, HR = kBwdUnroll * NV, NW = kBwdThreads / 32;
    extern __shared__ __align__(16) uint8_t smem[];          // the ring; at the end the warps' sums, then four a thread
    float* sums = reinterpret_cast<float*>(smem);
    const RopeParams& p = a.rope;
    const int lane = threadIdx.x & 31, l = lane & (NL - 1), sub = lane / NL, warp = threadIdx.x >> 5;
    const int id = blockIdx.x * NW + warp, begin = id * a.per_warp + min(id, a.more),
              end = begin + a.per_warp + (id < a.more ? 1 : 0);
    Eight dw = {{0, 0, 0, 0}}, dw_other = dw;                // of the unit's kind, and of the other
    int kind = 0;
    if (begin < end) {
        int t = begin / a.parts, part = begin - t * a.parts.d;
        // the ring: kBwdStages units of the warp, [g, x][i][lane] 16 bytes each
        const uint32_t ring = smem_u32(smem) + warp * (kBwdStages * kBwdStage) + lane * 16;
        int t_ahead = t, part_ahead = part, ahead = begin, fill = 0;
        auto issue = [&] {
            if (ahead < end) {
                const bool key = part_ahead >= a.q_parts;
                const HeadsIn& gin = key ? a.dko : a.dqo;
                const HeadsIn& xin = key ? a.k : a.q;
                const int h = (key ? part_ahead - a.q_parts : part_ahead) * HR + sub;
                const uint16_t* gp = gin.p + t_ahead * gin.ts + h * gin.hs + 8 * l;
                const uint16_t* xp = xin.p + t_ahead * xin.ts + h * xin.hs + 8 * l;
                const uint32_t to = ring + fill * kBwdStage;
#pragma unroll
                for (int i = 0; i < kBwdUnroll; ++i) {
                    copy16(h + i * NV < xin.heads, to + i * 512, gp, to + (kBwdUnroll + i) * 512, xp);
                    gp += NV * gin.hs;
                    xp += NV * xin.hs;
                }
                ++ahead;
                fill = fill == kBwdStages - 1 ? 0 : fill + 1;
                if (++part_ahead == a.parts.d) {
                    part_ahead = 0;
                    ++t_ahead;
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < kBwdStages - 1; ++i) issue();
        const uint8_t* stage = smem + warp * (kBwdStages * kBwdStage) + sub * (512 / NV);
        int at = 0;
        int64_t pos = load_pos(p, t), pos_next = t + 1 < p.T ? load_pos(p, t + 1) : 0;
        Angles angles = load_angles<D, SPLIT>(p, pos, l, lane);
        Turn u;
        Eight w;
        bool new_token = true, new_kind = true;
        kind = part >= a.q_parts;
#pragma unroll 1
        for (int unit = begin; unit < end; ++unit) {
            if (new_token) {
                u = turn_of<D, SPLIT>(p, angles, pos, lane);
                if (unit > begin) pos_next = t + 1 < p.T ? load_pos(p, t + 1) : 0;
            }
            if (new_kind) w = load_weight<D, SPLIT>(kind ? p.wk : p.wq, l);
            const HeadsOut& out = kind ? a.dk : a.dq;
            const int h0 = (kind ? part - a.q_parts : part) * HR, mine = (kind ? a.k : a.q).heads - h0;
            uint16_t* dst = out.p + t * out.ts + (h0 + sub) * out.hs;
            const int64_t dst_step = NV * out.hs;
            // the next unit
            int t_next = t, part_next = part + 1;
            if (part_next == a.parts.d) {
                part_next = 0;
                ++t_next;
            }
            if (unit + 1 < end && t_next != t) angles = load_angles<D, SPLIT>(p, pos_next, l, lane);
            __syncwarp();
            issue();
            asm volatile("cp.async.wait_group %0;" ::"n"(kBwdStages - 1) : "memory");
            __syncwarp();
            const uint8_t* from = stage + at * kBwdStage;
            at = at == kBwdStages - 1 ? 0 : at + 1;
            // A whole unit: the sums of squares of all its vectors first, so that their reductions overlap.
            auto take = [&](auto whole) {
                constexpr bool WHOLE = decltype(whole)::value;
                auto vector_at = [&](int i) { return reinterpret_cast<const uint16_t*>(from + i * 512); };
                float ss[kBwdUnroll];
                if constexpr (WHOLE) {
#pragma unroll
                    for (int i = 0; i < kBwdUnroll; ++i) {
                        const Eight x = unpack(load_bf16<D, SPLIT>(vector_at(kBwdUnroll + i), l));
                        ss[i] = dot(x, x);
                    }
#pragma unroll
                    for (int o = NL / 2; o > 0; o >>= 1)
#pragma unroll
                        for (int i = 0; i < kBwdUnroll; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
                }
#pragma unroll
                for (int i = 0; i < kBwdUnroll; ++i) {
                    if (!WHOLE && i * NV >= mine) break;     // the same for the whole warp
                    const uint4 gv = load_bf16<D, SPLIT>(vector_at(i), l),
                                xv = load_bf16<D, SPLIT>(vector_at(kBwdUnroll + i), l);
                    const Eight dy = unpack(gv), dp = partner<SPLIT>(gv, dy, u, p.interleaved), x = unpack(xv);
                    if constexpr (!WHOLE) ss[i] = group_sum<NL>(dot(x, x));
                    // lanes without a head hold zeros, of which eps 0 makes an infinite r: they add 0 g to dw
                    const bool live = WHOLE || sub + i * NV < mine;
                    const float r = live ? inverse_root(fmaf(ss[i], 1.0f / D, p.eps)) : 0.0f;
                    const uint64_t rr = pair_of(r, r);
                    Eight wg, xh, y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t g = fma2(dy.v[e], u.c.v[e], mul2(dp.v[e], u.s.v[e] ^ kSigns));
                        wg.v[e] = mul2(w.v[e], g);
                        xh.v[e] = mul2(x.v[e], rr);
                        dw.v[e] = fma2(g, xh.v[e], dw.v[e]);
                    }
                    const float m = group_sum<NL>(dot(wg, xh)) * (-1.0f / D);
                    const uint64_t mm = pair_of(m, m);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y.v[e] = mul2(rr, fma2(xh.v[e], mm, wg.v[e]));
                    if (live) store_bf16<D, SPLIT>(dst, l, pack(y));
                    dst += dst_step;
                }
            };
            if (mine >= HR)
                take(std::true_type());
            else
                take(std::false_type());
            const int kind_next = part_next >= a.q_parts;
            new_token = t_next != t;
            new_kind = kind_next != kind;
            if (new_kind) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t other = dw.v[e];
                    dw.v[e] = dw_other.v[e];
                    dw_other.v[e] = other;
                }
            }
            if (new_token) pos = pos_next;
            t = t_next;
            part = part_next;
            kind = kind_next;
        }
    }
    __syncthreads();
    // the block's sums: over the warp's NV vectors, then over the warps
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        float f[8];
        spread(k == kind ? dw : dw_other, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int o = NL; o < 32; o <<= 1) f[e] += __shfl_xor_sync(0xffffffffu, f[e], o);
            if (sub == 0)
                sums[(warp * 2 + k) * D + (e < 4 ? first<D, SPLIT>(l) + e : second<D, SPLIT>(l) + e - 4)] = f[e];
        }
    }
    __syncthreads();
    if (threadIdx.x < 2 * D) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) v += sums[k * 2 * D + threadIdx.x];
        a.part[(int64_t)blockIdx.x * 2 * D + threadIdx.x] = v;
    }
    __syncthreads();
    bool last = false;
    if (threadIdx.x == 0) last = arrive(a.done) == (int)gridDim.x - 1;
    if (!__syncthreads_or(last)) return;
    // a thread adds four columns of every ROWS-th block's sums, many loads in flight
    constexpr int COLS = 2 * D / 4, ROWS = kBwdThreads / COLS;
    const int col = threadIdx.x % COLS, row = threadIdx.x / COLS;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int FLIGHT = (152 + ROWS - 1) / ROWS;
#pragma unroll 1
    for (int b = row; b < (int)gridDim.x; b += FLIGHT * ROWS) {
        float4 x[FLIGHT];
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (b + i * ROWS < (int)gridDim.x)
                x[i] = __ldcg(reinterpret_cast<const float4*>(a.part + (int64_t)(b + i * ROWS) * 2 * D) + col);
        }
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) v = make_float4(v.x + x[i].x, v.y + x[i].y, v.z + x[i].z, v.w + x[i].w);
    }
    float4* flat = reinterpret_cast<float4*>(sums);
    flat[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < 2 * D) {
        const float* s = sums + threadIdx.x;
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) x += s[i * 2 * D];
        (threadIdx.x < D ? a.dwq : a.dwk - D)[threadIdx.x] = x;
    }
    if (threadIdx.x == 0) *a.done = 0;
}

}  // namespace

cudaError_t launch_qk_norm_rope(int D, const HeadsIn& q, const HeadsIn& k, const RopeParams& p, const HeadsOut& qo,
                                const HeadsOut& ko, cudaStream_t st) {
    ForwardArgs a = {};
    a.q = q;
    a.k = k;
    a.qo = qo;
    a.ko = ko;
    a.rope = p;
    a.T = p.T;
    return launch_forward_d<kRope>(D, a, st);
}

cudaError_t launch_qk_norm_rope_kv4(int D, const HeadsIn& q, const HeadsIn& k, const HeadsIn& v, const RopeParams& p,
                                    const HeadsOut& qo, const Kv4Cache& c, const int64_t* slots, cudaStream_t st) {
    ForwardArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.qo = qo;
    a.rope = p;
    a.c = c;
    a.slots = slots;
    a.T = p.T;
    return launch_forward_d<kRopeCache>(D, a, st);
}

cudaError_t launch_kv4_append(int D, const HeadsIn& k, const HeadsIn& v, int64_t T, const Kv4Cache& c,
                              const int64_t* slots, int* err, cudaStream_t st) {
    ForwardArgs a = {};
    a.k = k;
    a.v = v;
    a.rope.err = err;
    a.c = c;
    a.slots = slots;
    a.T = T;
    return launch_forward_d<kAppend>(D, a, st);
}

cudaError_t launch_kv4_gather(int D, const Kv4Cache& c, const int64_t* slots, int64_t T, uint16_t* k, uint16_t* v,
                              int* err, cudaStream_t st) {
    const bool groups = T >= kGatherGroupTokens;
    const int nv = 256 / D;
    const int64_t warps = groups ? (T + 15) / 16 * c.heads : T * ((c.heads + nv - 1) / nv);
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX / (kThreads / 32)) return cudaErrorInvalidValue;
    auto kernel = D == 64 ? (groups ? gather_groups_kernel<64> : gather_kernel<64>)
                          : (groups ? gather_groups_kernel<128> : gather_kernel<128>);
    return launch_chained(kernel, (unsigned)blocks, kThreads, 0, st, c, slots, T,
                          fast_div(groups ? c.heads : (c.heads + nv - 1) / nv), k, v, err);
}

int qk_norm_rope_bwd_blocks(int sms) { return sms; }

cudaError_t launch_qk_norm_rope_bwd(int D, const HeadsIn& dqo, const HeadsIn& dko, const HeadsIn& q, const HeadsIn& k,
                                    const RopeParams& p, const HeadsOut& dq, const HeadsOut& dk, float* dwq,
                                    float* dwk, float* part, int* done, int sms, cudaStream_t st) {
    const int hr = kBwdUnroll * (256 / D), nw = kBwdThreads / 32;
    const int q_parts = (q.heads + hr - 1) / hr, k_parts = (k.heads + hr - 1) / hr;
    const int64_t units = p.T * (q_parts + k_parts);
    if (units > INT32_MAX / 2) return cudaErrorInvalidValue;
    const int64_t want = (units + nw - 1) / nw, cap = qk_norm_rope_bwd_blocks(sms);
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    const int warps = (int)grid * nw;
    const BackwardArgs a = {dqo,  dko,  q,   k,  p, dq, dk, dwq, dwk, part, done, fast_div(q_parts + k_parts), q_parts,
                            (int)(units / warps), (int)(units % warps)};
    const bool split = p.rot == D && !p.interleaved;
    auto kernel = D == 64 ? (split ? backward_kernel<64, true> : backward_kernel<64, false>)
                          : (split ? backward_kernel<128, true> : backward_kernel<128, false>);
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), kBwdSmem);
    if (e != cudaSuccess) return e;
    return launch_chained(kernel, grid, kBwdThreads, kBwdSmem, st, a);
}

}  // namespace r9q
