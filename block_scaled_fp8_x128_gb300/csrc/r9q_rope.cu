// RMS norm of query and key heads with the position rotation in the same pass,
// its gradient, and the forms that write the paged 4-bit cache.
//
// A head vector x[D] with weight w: y = w x r, r = (mean(x^2) + eps)^-1/2; then
// each pair (a, b) of the first `rot` elements turns by its position's angle to
// (a cos - b sin, b cos + a sin).  Both are linear in x once r is known, so with
// x' the pair's other element
//   out = r (x (w c) + x' (w' s')),   s' = -sin for a, +sin for b,
// and w c, w' s' depend on the token and the element only: a warp forms them
// once and uses them for all its heads of the token.  x' comes from the lane
// that holds it, one shuffle of the packed bf16 input (adjacent pairs: from the
// same register).
//
// HBM bound: each input and output once.  A head vector takes D/8 lanes of 16
// bytes; a warp takes kUnroll x (32 / (D/8)) heads of one token with all loads in
// flight before the first is used.  Neighbouring warps of a block share a token, so
// the rows of the cos and sin tables come from L1 after the first.
#include "r9q_kv4.cuh"

namespace r9q {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

template <int D>
constexpr int heads_per_warp() { return kUnroll * (256 / D); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// A lane's part of the rotation: the lane that holds its pairs' other elements
// and its eight cos and signed sin (-sin for the first element of a pair).
struct Turn {
    int src;
    float c[8], s[8];
};
template <int D>
__device__ __forceinline__ Turn load_turn(const RopeParams& p, int64_t t, int lane) {
    const int l = lane & (D / 8 - 1), d0 = 8 * l, half = p.rot / 2;
    Turn u;
    u.src = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) u.c[i] = 1.0f, u.s[i] = 0.0f;
    if (p.rot == 0) return u;
    const int64_t pos = p.pos[t];
    if (pos < 0 || pos >= p.npos) {
        if (lane == 0) record_error(p.err, kErrArg);
#pragma unroll
        for (int i = 0; i < 8; ++i) u.c[i] = u.s[i] = __int_as_float(0x7FC00000);
        return u;
    }
    if (d0 >= p.rot) return u;
    const float* cs = p.cos + pos * half;
    const float* sn = p.sin + pos * half;
    if (p.interleaved) {
        const float4 a = *reinterpret_cast<const float4*>(cs + d0 / 2), b = *reinterpret_cast<const float4*>(sn + d0 / 2);
        const float c4[4] = {a.x, a.y, a.z, a.w}, s4[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u.c[i] = c4[i / 2];
            u.s[i] = i & 1 ? s4[i / 2] : -s4[i / 2];
        }
    } else {
        const bool second = d0 >= half;
        const int at = second ? d0 - half : d0;
        u.src = second ? lane - half / 8 : lane + half / 8;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 a = *reinterpret_cast<const float4*>(cs + at + 4 * k);
            const float4 b = *reinterpret_cast<const float4*>(sn + at + 4 * k);
            const float c4[4] = {a.x, a.y, a.z, a.w}, s4[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u.c[4 * k + i] = c4[i];
                u.s[4 * k + i] = second ? s4[i] : -s4[i];
            }
        }
    }
    return u;
}

// The other elements of the lane's pairs, as packed bf16.
__device__ __forceinline__ uint4 partner(const uint4& v, const Turn& u, int interleaved) {
    if (interleaved)
        return make_uint4(__byte_perm(v.x, 0, 0x1032), __byte_perm(v.y, 0, 0x1032), __byte_perm(v.z, 0, 0x1032),
                          __byte_perm(v.w, 0, 0x1032));
    return make_uint4(__shfl_sync(0xffffffffu, v.x, u.src), __shfl_sync(0xffffffffu, v.y, u.src),
                      __shfl_sync(0xffffffffu, v.z, u.src), __shfl_sync(0xffffffffu, v.w, u.src));
}
// w c and w' s' for the lane's elements, in place of c and s.
template <int D>
__device__ __forceinline__ void fold_weight(Turn& u, const float* w, int lane, int interleaved) {
    const int d0 = 8 * (lane & (D / 8 - 1)), e0 = 8 * (u.src & (D / 8 - 1));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u.c[i] *= w[d0 + i];
        u.s[i] *= interleaved ? w[d0 + (i ^ 1)] : w[e0 + i];
    }
}

// Sum of the squares of a head vector in a fixed order, one rounding a step: 32
// partial sums of every 32nd square, in their order, then a binary tree over
// neighbouring partial sums.  Lanes that are D/32 lanes' worth of elements apart
// hold a partial sum's terms; they exchange them so that each forms 32 / NL of
// the partial sums.
template <int NL>
__device__ __forceinline__ float sum_squares_in_order(const float (&x)[8], int l) {
    float q[8], s;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(x[i], x[i]);
    if constexpr (NL == 8) {                              // lanes l, l ^ 4: four partial sums each, two terms
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
// once, and the sum of squares has a fixed order.  An evaluation of the formula
// step by step in fp32 gives the same codes.
template <int NL>
__device__ __forceinline__ void norm_rope_in_order(float (&y)[8], const float (&w)[8], const Turn& u, int lane,
                                                   const RopeParams& p) {
    const float mean = __fmul_rn(sum_squares_in_order<NL>(y, lane & (NL - 1)), 1.0f / (8 * NL));
    const float r = rsqrtf(__fadd_rn(mean, p.eps));
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(__fmul_rn(y[e], r), w[e]);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = p.interleaved ? y[e ^ 1] : __shfl_sync(0xffffffffu, y[e], u.src);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __fadd_rn(__fmul_rn(y[e], u.c[e]), __fmul_rn(z[e], u.s[e]));
}

enum Pass { kRope, kRopeCache, kAppend };

struct ForwardArgs {
    HeadsIn q, k, v;
    HeadsOut qo, ko;
    RopeParams rope;
    Kv4Cache c;
    const int64_t* slots;
    int64_t T;
    int nq, nk, nv;          // warps a token's query, key and value heads take
};

// Where a token goes: its page and place, or page -1 for padding and for a slot
// outside the cache (an error).
struct Place {
    int64_t page;
    int at;
};
__device__ __forceinline__ Place find_slot(const Kv4Cache& c, int64_t slot, int lane, int* err) {
    Place r = {-1, 0};
    if (slot >= 0) {
        const int64_t page = slot / c.page;
        if (page < c.pages) {
            r.page = page;
            r.at = (int)(slot - page * c.page);
        } else if (lane == 0) {
            record_error(err, kErrArg);
        }
    }
    return r;
}

template <int D, int PASS>
__global__ void __launch_bounds__(kThreads) forward_kernel(const ForwardArgs a) {
    constexpr int NL = D / 8, NV = 32 / NL, HPW = heads_per_warp<D>();
    const int lane = threadIdx.x & 31, l = lane & (NL - 1), sub = lane / NL;
    const int parts = a.nq + a.nk + a.nv;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = unit / parts;
    if (t >= a.T) return;
    int part = (int)(unit - t * parts);
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
    const int h0 = part * HPW + sub;
    uint4 x[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int h = h0 + i * NV;
        x[i] = h < in.heads ? *reinterpret_cast<const uint4*>(in.p + t * in.ts + h * in.hs + 8 * l)
                            : make_uint4(0u, 0u, 0u, 0u);
    }
    Place place = {-1, 0};
    if (PASS != kRope && kind > 0) place = find_slot(a.c, a.slots[t], lane, a.rope.err);
    const bool turned = PASS != kAppend && kind < 2;
    const bool in_order = PASS == kRopeCache && kind == 1;
    Turn u;
    float w[8];
    if (turned) {
        u = load_turn<D>(a.rope, t, lane);
        if (in_order) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = a.rope.wk[8 * l + e];
        } else {
            fold_weight<D>(u, kind == 0 ? a.rope.wq : a.rope.wk, lane, a.rope.interleaved);
        }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int h = h0 + i * NV;
        if (part * HPW + i * NV >= in.heads) break;      // the same for the whole warp
        float y[8];
        unpack8(x[i], y);
        if (in_order) {
            norm_rope_in_order<NL>(y, w, u, lane, a.rope);
        } else if (turned) {
            float xp[8], ss = 0.0f;
            unpack8(partner(x[i], u, a.rope.interleaved), xp);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
            const float r = rsqrtf(group_sum<NL>(ss) * (1.0f / D) + a.rope.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = r * fmaf(y[e], u.c[e], xp[e] * u.s[e]);
        }
        if (PASS == kRope || (PASS == kRopeCache && kind == 0)) {
            const HeadsOut& out = kind == 0 ? a.qo : a.ko;
            if (h < in.heads) *reinterpret_cast<uint4*>(out.p + t * out.ts + h * out.hs + 8 * l) = pack8(y);
        } else {
            uint32_t pair;
            const uint32_t codes = kv4_quantise<NL>(y, pair);
            const bool live = h < in.heads && place.page >= 0;
            const int64_t head = place.page * a.c.heads + h;
            if (kind == 1) {
                if (live) {
                    kv4_store_k(a.c.k + head * kv4_head_bytes(a.c.page, D) + (int64_t)place.at * (D / 2), l, codes);
                    if (l == 0) a.c.kp[head * a.c.page + place.at] = pair;
                }
            } else {
                kv4_store_v(live ? a.c.v + head * kv4_head_bytes(a.c.page, D) + (int64_t)(place.at >> 4) * (8 * D)
                                 : nullptr,
                            place.at & 15, l, codes);
                if (live && l == 0) a.c.vp[head * a.c.page + place.at] = pair;
            }
        }
    }
}

template <int D, int PASS>
cudaError_t launch_forward(ForwardArgs a, cudaStream_t st) {
    constexpr int HPW = heads_per_warp<D>();
    a.nq = PASS == kAppend ? 0 : (a.q.heads + HPW - 1) / HPW;
    a.nk = (a.k.heads + HPW - 1) / HPW;
    a.nv = PASS == kRope ? 0 : (a.v.heads + HPW - 1) / HPW;
    const int64_t warps = a.T * (a.nq + a.nk + a.nv);
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    forward_kernel<D, PASS><<<(unsigned)blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int PASS>
cudaError_t launch_forward_d(int D, const ForwardArgs& a, cudaStream_t st) {
    return D == 64 ? launch_forward<64, PASS>(a, st) : launch_forward<128, PASS>(a, st);
}

// ------------------------------------------------------------- read-back --

// bf16(lowest + step * code) of the tokens at `slots`, zeros for padding.
template <int D>
__global__ void __launch_bounds__(kThreads) gather_kernel(const Kv4Cache c, const int64_t* slots, int64_t T,
                                                          uint16_t* k, uint16_t* v, int* err) {
    constexpr int NL = D / 8, NV = 32 / NL;
    const int lane = threadIdx.x & 31, l = lane & (NL - 1), sub = lane / NL;
    const int parts = (c.heads + NV - 1) / NV;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = unit / parts;
    if (t >= T) return;
    const int h = (int)(unit - t * parts) * NV + sub;
    const Place place = find_slot(c, slots[t], lane, err);
    const bool live = place.page >= 0 && h < c.heads;
    const int64_t head = place.page * c.heads + h;
    uint32_t codes[2] = {0, 0}, pair[2] = {0, 0};
    if (live) {
        codes[0] = kv4_load_k(c.k + head * kv4_head_bytes(c.page, D) + (int64_t)place.at * (D / 2), l);
        pair[0] = c.kp[head * c.page + place.at];
        pair[1] = c.vp[head * c.page + place.at];
    }
    codes[1] = kv4_load_v(live ? c.v + head * kv4_head_bytes(c.page, D) + (int64_t)(place.at >> 4) * (8 * D) : nullptr,
                          place.at & 15, l);
    if (h >= c.heads) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = fmaf(bf16_lo(pair[s]), (float)((codes[s] >> (4 * i)) & 15u), bf16_hi(pair[s]));
        *reinterpret_cast<uint4*>((s == 0 ? k : v) + (t * c.heads + h) * D + 8 * l) = pack8(y);
    }
}

// -------------------------------------------------------------- gradient --

// With g = R^T dy (the turn by the opposite angle) and xh = x r:
//   dw = sum over tokens and heads of g xh,
//   dx = r (w g - xh mean(w g xh)) = r w g - x r^3 sum(w g x) / D.
// r is computed again from x: that reads nothing that dx does not need.  Blocks
// of 16 warps walk the (token, part) units in a fixed order, each lane summing
// its elements' dw in 32 bits; a block's sum goes to `part`, and the block that
// finishes last adds the blocks' sums in their order, so dw does not depend on
// timing.
constexpr int kBwdThreads = 512;
constexpr int kBwdUnroll = 2;

template <int D>
__global__ void __launch_bounds__(kBwdThreads) backward_kernel(const HeadsIn dqo, const HeadsIn dko, const HeadsIn q,
                                                               const HeadsIn k, const RopeParams p, const HeadsOut dq,
                                                               const HeadsOut dk, float* dwq, float* dwk, float* part,
                                                               int* done) {
    constexpr int NL = D / 8, NV = 32 / NL, HPW = kBwdUnroll * NV, NW = kBwdThreads / 32;
    const int lane = threadIdx.x & 31, l = lane & (NL - 1), sub = lane / NL, warp = threadIdx.x >> 5;
    const int nq = (q.heads + HPW - 1) / HPW, nk = (k.heads + HPW - 1) / HPW, parts = nq + nk;
    float dw[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.0f;
    const int64_t units = p.T * parts, stride = (int64_t)gridDim.x * NW;
    for (int64_t unit = (int64_t)blockIdx.x * NW + warp; unit < units; unit += stride) {
        const int64_t t = unit / parts;
        int pt = (int)(unit - t * parts);
        const bool key = pt >= nq;
        if (key) pt -= nq;
        const HeadsIn& gin = key ? dko : dqo;
        const HeadsIn& xin = key ? k : q;
        const HeadsOut& out = key ? dk : dq;
        const int h0 = pt * HPW + sub;
        uint4 gv[kBwdUnroll], xv[kBwdUnroll];
#pragma unroll
        for (int i = 0; i < kBwdUnroll; ++i) {
            const int h = h0 + i * NV;
            gv[i] = xv[i] = make_uint4(0u, 0u, 0u, 0u);
            if (h < xin.heads) {
                gv[i] = *reinterpret_cast<const uint4*>(gin.p + t * gin.ts + h * gin.hs + 8 * l);
                xv[i] = *reinterpret_cast<const uint4*>(xin.p + t * xin.ts + h * xin.hs + 8 * l);
            }
        }
        const Turn u = load_turn<D>(p, t, lane);
        const float* wp = (key ? p.wk : p.wq) + 8 * l;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = wp[e];
#pragma unroll
        for (int i = 0; i < kBwdUnroll; ++i) {
            const int h = h0 + i * NV;
            float g[8], gp[8], x[8], ss = 0.0f, sg = 0.0f;
            unpack8(gv[i], g);
            unpack8(partner(gv[i], u, p.interleaved), gp);
            unpack8(xv[i], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] = fmaf(g[e], u.c[e], -gp[e] * u.s[e]);
                ss = fmaf(x[e], x[e], ss);
                sg = fmaf(w[e] * g[e], x[e], sg);
            }
            ss = group_sum<NL>(ss);
            sg = group_sum<NL>(sg);
            const float r = rsqrtf(ss * (1.0f / D) + p.eps);
            const float m = r * r * r * sg * (1.0f / D);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gx = g[e] * (x[e] * r);
                if (key) dw[1][e] += gx;
                else dw[0][e] += gx;
                y[e] = fmaf(r * w[e], g[e], -x[e] * m);
            }
            if (h < xin.heads) *reinterpret_cast<uint4*>(out.p + t * out.ts + h * out.hs + 8 * l) = pack8(y);
        }
    }
    // the block's sum: over the warp's NV vectors, then over the warps
    __shared__ float sums[NW][2 * D];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = dw[s][e];
#pragma unroll
            for (int o = NL; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (sub == 0) sums[warp][s * D + 8 * l + e] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kBwdThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w2 = 0; w2 < NW; ++w2) v += sums[w2][i];
        part[(int64_t)blockIdx.x * 2 * D + i] = v;
    }
    __threadfence();
    __syncthreads();
    __shared__ int last;
    if (threadIdx.x == 0) last = atomicAdd(done, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    constexpr int ROWS = kBwdThreads / (2 * D);          // threads that share a column
    const int col = threadIdx.x % (2 * D), row = threadIdx.x / (2 * D);
    float v = 0.0f;
    for (int b = row; b < (int)gridDim.x; b += ROWS) v += __ldcg(part + (int64_t)b * 2 * D + col);
    float* flat = &sums[0][0];
    __syncthreads();
    flat[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < 2 * D) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) v += flat[i * 2 * D + col];
        if (col < D) dwq[col] = v;
        else dwk[col - D] = v;
    }
    if (threadIdx.x == 0) *done = 0;
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
    const int nv = 256 / D;
    const int64_t warps = T * ((c.heads + nv - 1) / nv), blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (D == 64) gather_kernel<64><<<(unsigned)blocks, kThreads, 0, st>>>(c, slots, T, k, v, err);
    else gather_kernel<128><<<(unsigned)blocks, kThreads, 0, st>>>(c, slots, T, k, v, err);
    return cudaGetLastError();
}

int qk_norm_rope_bwd_blocks(int sms) { return 2 * sms; }

cudaError_t launch_qk_norm_rope_bwd(int D, const HeadsIn& dqo, const HeadsIn& dko, const HeadsIn& q, const HeadsIn& k,
                                    const RopeParams& p, const HeadsOut& dq, const HeadsOut& dk, float* dwq,
                                    float* dwk, float* part, int* done, int sms, cudaStream_t st) {
    const int hpw = kBwdUnroll * (256 / D), nw = kBwdThreads / 32;
    const int64_t units = p.T * ((q.heads + hpw - 1) / hpw + (k.heads + hpw - 1) / hpw);
    const int64_t want = (units + nw - 1) / nw, cap = qk_norm_rope_bwd_blocks(sms);
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    if (D == 64)
        backward_kernel<64><<<grid, kBwdThreads, 0, st>>>(dqo, dko, q, k, p, dq, dk, dwq, dwk, part, done);
    else
        backward_kernel<128><<<grid, kBwdThreads, 0, st>>>(dqo, dko, q, k, p, dq, dk, dwq, dwk, part, done);
    return cudaGetLastError();
}

}  // namespace r9q
