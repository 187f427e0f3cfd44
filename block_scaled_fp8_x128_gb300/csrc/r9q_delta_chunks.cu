// The gated delta rule over many tokens a sequence, in chunks of 64 (formulas: r9q_delta.cuh): prompts,
// trees of drafted tokens, long accepted paths.
//
// A CTA walks one value head of a sequence.  Everything is transposed, so that row v of all
// products is value element v and belongs to one thread: with S [D values][D keys] as the
// accumulator in tensor memory, for each chunk of keys K, queries Q [64][D]
//   W = S K^T, Y = S Q^T         [D values][64 tokens]
//   x_i = beta_i (v_i - A(i, 0) W_i),  u_i = x_i - sum_{j<i} L_ij u_j   (each thread its row, in fp32)
//   O = A(., 0) Y + U P^T,  S <- A(n, 0) S + (A(n, .) U) K
// with L_ij = beta_i A(i, j) (k_i.k_j), P_ij = A(i, j) (q_i.k_j) from one product [K; Q] K^T.
// Keys and queries are the bf16 inputs themselves (exact operands); their lengths go into L, P and
// the scalars.  What is fp32 (S, u) is an operand in bf16 parts, cut off, not rounded: three parts
// hold all 24 bits and keep fp32's range, so that nothing needs a scale and a
// token's values, however large, do not touch those of earlier tokens.  Three parts for what
// goes into S and u, two (2^-16) where only outputs, which are rounded to bf16, follow.
//
// Warps 0-3: the rows.  Warps 4-7: the tokens; they copy K, Q, V (a chunk ahead), and form L and P
// of the next chunk while the rows work on this one.  Warp 8 issues the products.  In a tree the sums
// go over ancestors, and its one chunk leaves the state alone.
//
// A value that is not finite would reach earlier tokens (or other branches) through the zeros of P,
// so u is an operand with zeros in its place, and the outputs that it belongs to are NaN.
#include <cfloat>

#include "r9q_delta.cuh"

namespace r9q {

namespace {

constexpr int kChunk = 64;
constexpr int kRowThreads = 128, kTokenThreads = 128, kThreads = kRowThreads + kTokenThreads + 32;
constexpr int kLStride = 68;                 // floats between rows of L: eight rows' 16-byte pieces lie in different banks

// Scalars of a chunk's tokens.
struct Scalars {
    float r_k[kChunk], r_q[kChunk];          // 1 / length; r_q times the scale
    float beta[kChunk], fade[kChunk], left[kChunk];          // fade A(i, 0), left A(n, i)
    float hi[kChunk], lo[kChunk];            // sums of the decays' logarithms to base 2
    uint64_t above[kChunk];
    int parents[kChunk];
    NodeKind kind[kChunk];
};

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = 64 * 128;                   // 64 rows of 128 bytes, swizzled
    static constexpr int kKq = kHalves * 2 * kTile;          // of each 64 elements: K's rows, then Q's
    static constexpr int kInput = kKq + kChunk * D * 2;      // and V [64][D]
    static constexpr int kL = kChunk * kLStride * 4;
    static constexpr int kP = 2 * kTile;                     // its two parts
    static constexpr int kPairs = (kL + kP + (int)sizeof(Scalars) + 1023) / 1024 * 1024;
    static constexpr int kBytes = 2 * kInput + 2 * kPairs;
    // tensor memory, columns
    static constexpr int kS = 0, kParts = D, kW = kParts + 3 * D / 2, kY = kW + 64, kG = kY + 64;
    static constexpr int kU = kParts, kUleft = kParts + 64;  // u's two parts and (A(n, .) u)'s three, after S's
    static_assert(kG + 64 <= 512 && kUleft + 96 <= kW + (D == 64 ? 64 : 0), "tensor memory");
};

struct Barriers {
    uint64_t input_full[2], input_free[2], gram_full, gram_read, pairs_full[2], pairs_free[2], s_ready, w_full, y_full,
        u_ready, s_full, o_full, o_read;
    uint32_t tmem;
    int failed;                              // a wait gave up
};

// Two fp32 values to bf16 parts, cut off; the rest stays.
__device__ __forceinline__ uint32_t take_part(float& a, float& b) {
    uint32_t r;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    a -= bf16_lo(r);
    b -= bf16_hi(r);
    return r;
}

__device__ __forceinline__ void umma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// A from tensor memory.
__device__ __forceinline__ void umma_bf16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// bf16 operands, fp32 accumulator, M = 128; B with its K or its N contiguous.
constexpr uint32_t idesc_bf16(int N, bool n_contiguous) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((n_contiguous ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
// A descriptor as umma_sdesc_sw128's, of an operand whose N is contiguous: 64 elements a row, rows are
// K, 8 rows every 1024 bytes; the next 64 elements `apart` bytes on.
__device__ __forceinline__ uint64_t sdesc_n_contiguous(uint32_t saddr, uint32_t apart) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(apart >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&d)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::"r"(d[0]),
        "r"(d[1]), "r"(d[2]), "r"(d[3]), "r"(d[4]), "r"(d[5]), "r"(d[6]), "r"(d[7]), "r"(d[8]), "r"(d[9]), "r"(d[10]),
        "r"(d[11]), "r"(d[12]), "r"(d[13]), "r"(d[14]), "r"(d[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void token_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Bounded; after one that gave up all others do at once.
struct Waits {
    volatile int* failed;
    int* err;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
        if (*failed) return;
        if (!mbar_wait(bar, parity)) {
            *failed = 1;
            record_error(err, kErrTimeout);
        }
    }
};

template <int D, DeltaMode MODE>
__global__ void __launch_bounds__(kThreads, 1) delta_chunks_kernel(const DeltaParams p) {
    using Y = Layout<D>;
    constexpr bool TREE = MODE == kDeltaTree, HAS_Q = MODE != kDeltaCommit;
    constexpr int KS = D / 16;               // steps of a product over the keys' elements
    extern __shared__ uint8_t raw[];
    begin_chained();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / p.Hv, h = blockIdx.x - b * p.Hv, hk = h / p.ratio;
    int n;
    int64_t row0;
    delta_tokens(p, b, n, row0);
    const int32_t* path = p.path + (int64_t)b * p.P;
    if constexpr (MODE == kDeltaCommit) {
        uint64_t ends = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = i * 32 + lane, node = at < p.P ? path[at] : -1;
            ends |= (uint64_t)__ballot_sync(0xffffffffu, node < 0 || node >= p.Lq) << (32 * i);
            if (node >= p.Lq) record_error(p.err, kErrArg);
        }
        n = ends ? __ffsll((long long)ends) - 1 : p.P;
    }
    const int slot = delta_slot<!TREE>(p, b);
    if (slot < 0) {
        if constexpr (HAS_Q)
            for (int64_t x = tid; x < (int64_t)n * D; x += kThreads)
                p.o[((row0 + x / D) * p.Hv + h) * D + x % D] = slot == -1 ? 0 : 0x7FC0;
        return;
    }
    float* state = p.state + ((int64_t)slot * p.Hv + h) * D * D;
    if (n == 0) {
        if (p.from_zero)
            for (int x = tid; x < D * D; x += kThreads) state[x] = 0.0f;
        return;
    }
    const int chunks = (n + kChunk - 1) / kChunk;
    uint8_t* smem = raw + (1024u - smem_u32(raw) % 1024u) % 1024u;
    Barriers& bars = *reinterpret_cast<Barriers*>(smem + Y::kBytes);
    auto input = [&](int c) { return smem + (c & 1) * Y::kInput; };
    auto l_of = [&](int c) { return reinterpret_cast<float*>(smem + 2 * Y::kInput + (c & 1) * Y::kPairs + Y::kP); };
    auto p_of = [&](int c) { return smem + 2 * Y::kInput + (c & 1) * Y::kPairs; };
    auto scalars_of = [&](int c) {
        return reinterpret_cast<Scalars*>(smem + 2 * Y::kInput + (c & 1) * Y::kPairs + Y::kP + Y::kL);
    };
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.input_full[i], kTokenThreads);
            mbar_init(&bars.input_free[i], 1);
            mbar_init(&bars.pairs_full[i], kTokenThreads);
            mbar_init(&bars.pairs_free[i], kRowThreads);
        }
        mbar_init(&bars.gram_full, 1);
        mbar_init(&bars.gram_read, kTokenThreads);
        mbar_init(&bars.s_ready, kRowThreads);
        mbar_init(&bars.w_full, 1);
        mbar_init(&bars.y_full, 1);
        mbar_init(&bars.u_ready, kRowThreads);
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.o_full, 1);
        mbar_init(&bars.o_read, kRowThreads);
        bars.failed = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&bars.tmem, 512);
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    const uint32_t tmem = bars.tmem;
    const Waits wait = {&bars.failed, p.err};

    if (warp < 4) {
        // ---------------------------------------------------------------- rows --
        const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);
        const bool live = tid < D;           // (D = 64: the other half of the lanes is zeros)
        float* row = state + (int64_t)tid * D;
#pragma unroll 1
        for (int e = 0; e < D; e += 16) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = live && !p.from_zero ? reinterpret_cast<const uint4*>(row + e)[i] : make_uint4(0, 0, 0, 0);
                x[4 * i] = v.x;
                x[4 * i + 1] = v.y;
                x[4 * i + 2] = v.z;
                x[4 * i + 3] = v.w;
            }
            tmem_st16(mine + Y::kS + e, x);
        }
        tmem_wait_st();
        uint64_t lost = 0;                   // tokens whose u is not finite
        uint64_t before = 0;                 // that of the chunk whose outputs are due
        auto outputs = [&](int c) {
            const Scalars& sc = *scalars_of(c);
            wait(&bars.o_full, c & 1);
            umma_fence_after();
#pragma unroll 1
            for (int t0 = 0; t0 < kChunk; t0 += 16) {
                float y[16], z[16];
                tmem_ld(mine + Y::kY + t0, y);
                tmem_ld(mine + Y::kG + t0, z);
                tmem_wait_ld(y);
                tmem_wait_ld(z);
                if (t0 == kChunk - 16) {
                    umma_fence_before();
                    mbar_arrive(&bars.o_read);
                }
                if (!live) continue;
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    const int i = t0 + t, token = c * kChunk + i;
                    if (token >= n) break;
                    float o = sc.r_q[i] * fmaf(sc.fade[i], y[t], z[t]);
                    uint32_t out = pack_bf16x2(o, 0.0f);
                    if (before && (TREE ? (before & sc.above[i]) != 0 : (before & (~0ull >> (63 - i))) != 0)) out = 0x7FC0u;
                    if (TREE && sc.kind[i] != kNode) out = sc.kind[i] == kNoNode ? 0u : 0x7FC0u;
                    p.o[((row0 + token) * p.Hv + h) * D + tid] = (uint16_t)out;
                }
            }
        };
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            wait(&bars.pairs_full[c & 1], (c >> 1) & 1);
            const Scalars& sc = *scalars_of(c);
            const float* L = l_of(c);
            if (c > 0) {
                wait(&bars.s_full, (c - 1) & 1);
                if (HAS_Q) wait(&bars.o_full, (c - 1) & 1);  // (u's parts, which it reads, make room for S's)
                umma_fence_after();
            }
            // S into its parts, and what is left of it at the chunk's end
            const float left = sc.fade[kChunk - 1];
#pragma unroll 1
            for (int e = 0; e < D; e += 32) {
                float s[32];
                tmem_ld(mine + Y::kS + e, s);
                tmem_wait_ld(s);
                if constexpr (!TREE) {
                    uint32_t x[16];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(left * s[half * 16 + i]);
                        tmem_st16(mine + Y::kS + e + half * 16, x);
                    }
                }
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    uint32_t x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = take_part(s[2 * i], s[2 * i + 1]);
                    tmem_st16(mine + Y::kParts + part * (D / 2) + e / 2, x);
                }
            }
            tmem_wait_st();
            umma_fence_before();
            mbar_arrive(&bars.s_ready);
            if (HAS_Q && c > 0) {
                outputs(c - 1);
                mbar_arrive(&bars.pairs_free[(c - 1) & 1]);
            } else if (c > 0) {
                mbar_arrive(&bars.pairs_free[(c - 1) & 1]);
            }

            // ---- x, then u ----
            wait(&bars.w_full, c & 1);
            umma_fence_after();
            uint64_t u[kChunk / 2];
            const uint16_t* v = reinterpret_cast<const uint16_t*>(input(c) + Y::kKq) + (live ? tid : 0);
#pragma unroll
            for (int t0 = 0; t0 < kChunk; t0 += 32) {
                float w[32];
                tmem_ld(mine + Y::kW + t0, w);
                tmem_wait_ld(w);
#pragma unroll
                for (int t = 0; t < 32; t += 2) {
                    float x[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = t0 + t + i;
                        const float val = live ? bf16_lo(v[j * D]) : 0.0f;
                        x[i] = sc.beta[j] * fmaf(-sc.fade[j] * sc.r_k[j], w[t + i], val);
                    }
                    u[(t0 + t) / 2] = pair_of(x[0], x[1]);
                }
            }
            lost = 0;
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                uint64_t s0 = 0, s1 = 0;
#pragma unroll
                for (int j = 0; j < i; j += 4) {             // (L is zero from the diagonal on)
                    const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(L + i * kLStride + j);
                    s0 = fma2(l.x, u[j / 2], s0);
                    if (j + 2 < i) s1 = fma2(l.y, u[j / 2 + 1], s1);
                }
                const float2 a = parts_of(s0), d = parts_of(s1), old = parts_of(u[i / 2]);
                float x = (i & 1 ? old.y : old.x) - ((a.x + a.y) + (d.x + d.y));
                if constexpr (TREE) {        // another branch is not to get it through a zero of L
                    if (!(fabsf(x) <= FLT_MAX) || (lost & sc.above[i])) {
                        lost |= 1ull << i;
                        x = 0.0f;
                    }
                }
                u[i / 2] = i & 1 ? pair_of(old.x, x) : pair_of(x, old.y);
            }
            if constexpr (!TREE) {
                uint64_t any = 0;
#pragma unroll
                for (int i = 0; i < kChunk / 2; ++i) any = fma2(u[i], 0ull, any);
                const float2 a = parts_of(any);
                if (!(a.x == 0.0f && a.y == 0.0f)) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        const float2 x = parts_of(u[i / 2]);
                        if (!(fabsf(i & 1 ? x.y : x.x) <= FLT_MAX)) lost |= 1ull << i;
                    }
                }
            }
            before = lost;
            // ---- u as an operand, in place of S's parts ----
            if constexpr (HAS_Q) {
                wait(&bars.y_full, c & 1);
                umma_fence_after();
#pragma unroll
                for (int t0 = 0; t0 < kChunk; t0 += 32) {
                    float x[32];
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        const float2 f = parts_of(u[t0 / 2 + t]);
                        x[2 * t] = f.x;
                        x[2 * t + 1] = f.y;
                    }
                    if (lost) {
#pragma unroll
                        for (int t = 0; t < 32; ++t)
                            if (lost >> (t0 + t) & 1) x[t] = 0.0f;
                    }
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        uint32_t y[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = take_part(x[2 * i], x[2 * i + 1]);
                        tmem_st16(mine + Y::kU + part * 32 + t0 / 2, y);
                    }
                }
            }
            if constexpr (!TREE) {
#pragma unroll
                for (int t0 = 0; t0 < kChunk; t0 += 32) {
                    float x[32];
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        const float2 f = parts_of(u[t0 / 2 + t]);
                        x[2 * t] = f.x * (sc.left[t0 + 2 * t] * sc.r_k[t0 + 2 * t]);
                        x[2 * t + 1] = f.y * (sc.left[t0 + 2 * t + 1] * sc.r_k[t0 + 2 * t + 1]);
                    }
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        uint32_t y[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = take_part(x[2 * i], x[2 * i + 1]);
                        tmem_st16(mine + Y::kUleft + part * 32 + t0 / 2, y);
                    }
                }
            }
            tmem_wait_st();
            umma_fence_before();
            mbar_arrive(&bars.u_ready);
        }
        if constexpr (!TREE) {
            wait(&bars.s_full, (chunks - 1) & 1);
            umma_fence_after();
#pragma unroll 1
            for (int e = 0; e < D; e += 32) {
                float s[32];
                tmem_ld(mine + Y::kS + e, s);
                tmem_wait_ld(s);
                if (live)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<float4*>(row + e)[i] = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
            }
        }
        if constexpr (HAS_Q) outputs(chunks - 1);
    } else if (warp < 8) {
        // -------------------------------------------------------------- tokens --
        const int t = tid - kRowThreads;     // row of [K; Q]
        const int i = t & 63;
        const bool key = t < 64;
        const uint32_t mine = tmem + ((uint32_t)((warp - 4) * 32) << 16);
        auto place = [&](int at) { return MODE == kDeltaCommit ? (int64_t)path[at] : (p.cu ? row0 : 0) + at; };
        auto load = [&](int c) {
            const uint32_t base = smem_u32(input(c));
#pragma unroll 4
            for (int x = t; x < 3 * kChunk * (D / 8); x += kTokenThreads) {
                const int which = x / (kChunk * (D / 8)), y = x % (kChunk * (D / 8)), r = y / (D / 8), piece = y % (D / 8);
                if (!HAS_Q && which == 1) continue;          // (a commit's Q: rows that nothing uses)
                const int at = c * kChunk + r;
                const int64_t token = at < n ? place(at) : 0;
                const uint16_t* src = which == 0   ? p.k + b * p.k_bs + token * p.k_ts + hk * p.k_hs
                                      : which == 1 ? p.q + b * p.q_bs + token * p.q_ts + hk * p.q_hs
                                                   : p.v + b * p.v_bs + token * p.v_ts + h * p.v_hs;
                const uint32_t dst = which == 2 ? Y::kKq + r * (D * 2) + piece * 16
                                                : (piece >> 3) * (2 * Y::kTile) + which * Y::kTile + r * 128 +
                                                      (((piece & 7) ^ (r & 7)) << 4);
                copy16(base + dst, at < n ? src + piece * 8 : p.k, at < n);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto loaded = [&](int c) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            fence_proxy_async_smem();
            mbar_arrive(&bars.input_full[c & 1]);
        };
        // L, P and the scalars of chunk c
        auto pairs = [&](int c) {
            Scalars& sc = *scalars_of(c);
            if (c >= 2) wait(&bars.pairs_free[c & 1], ((c - 2) >> 1) & 1);
            const int at = c * kChunk + i;
            float g = 0.0f;
            if (at < n) {
                const int64_t x = ((MODE == kDeltaCommit ? row0 : p.cu ? 0 : row0) + place(at)) * p.Hv + h;
                g = p.g[x];
                if (key) sc.beta[i] = p.beta[x];
            } else if (key) {
                sc.beta[i] = 0.0f;
            }
            g = g < -200.0f ? -200.0f : g;   // (exp is 0 there; infinities have no differences)
            if constexpr (TREE) {
                if (key) {
                    sc.hi[i] = g;
                    sc.parents[i] = at < n ? p.parents[(int64_t)b * p.Lq + at] : -2;
                }
                token_barrier();
                if (key) {
                    int depth;
                    const NodeKind kind = find_node(sc.parents, i, kMostNodes, sc.above[i], depth);
                    if (kind == kBadNode) record_error(p.err, kErrArg);
                    if (kind != kNode) sc.above[i] = 0;
                    sc.kind[i] = kind;
                    double sum = 0.0;
                    for (uint64_t m = sc.above[i]; m; m &= m - 1) sum += (double)sc.hi[__ffsll((long long)m) - 1];
                    sum *= 1.4426950408889634;
                    token_barrier();
                    sc.hi[i] = (float)sum;
                    sc.lo[i] = (float)(sum - (double)sc.hi[i]);
                    sc.fade[i] = ex2(sc.hi[i]);
                } else {
                    token_barrier();
                }
            } else if (warp == 4) {          // two tokens a lane
                const int a = c * kChunk + 2 * lane;
                double x[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float gy = a + y < n ? p.g[((MODE == kDeltaCommit ? row0 : p.cu ? 0 : row0) + place(a + y)) * p.Hv + h] : 0.0f;
                    x[y] = (double)(gy < -200.0f ? -200.0f : gy) * 1.4426950408889634;
                }
                double sum = x[0] + x[1];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                const double end = __shfl_sync(0xffffffffu, sum, 31), first = sum - x[1];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const double z = y ? sum : first;
                    const int at2 = 2 * lane + y;
                    sc.hi[at2] = (float)z;
                    sc.lo[at2] = (float)(z - (double)(float)z);
                    sc.fade[at2] = ex2((float)z);
                    sc.left[at2] = ex2((float)(end - z));
                }
            }
            // the row's length
            float sum = 0.0f;
            if (key || HAS_Q) {
                wait(&bars.input_full[c & 1], (c >> 1) & 1);
                const uint8_t* rows = input(c) + (key ? 0 : Y::kTile) + i * 128;
#pragma unroll
                for (int x = 0; x < D / 8; ++x) {
                    const uint4 q = *reinterpret_cast<const uint4*>(rows + (x >> 3) * (2 * Y::kTile) + (((x & 7) ^ (i & 7)) << 4));
                    const Eight e = unpack(q);
                    sum += dot(e, e);
                }
            }
            const float r = rsqrtf(sum + p.eps);
            if (key)
                sc.r_k[i] = at < n ? r : 0.0f;
            else
                sc.r_q[i] = r * p.scale;
            token_barrier();
            wait(&bars.gram_full, c & 1);
            umma_fence_after();
            const float hi = sc.hi[i], lo = sc.lo[i], own = key ? sc.beta[i] * sc.r_k[i] : 1.0f;
            const uint64_t above = TREE ? sc.above[i] : ~0ull >> (63 - i);
            float* L = l_of(c) + i * kLStride;
            uint8_t* P = p_of(c) + i * 128;
#pragma unroll 1
            for (int j0 = 0; j0 < kChunk; j0 += 16) {
                float x[16];
                tmem_ld(mine + Y::kG + j0, x);
                tmem_wait_ld(x);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int jj = j0 + j;
                    const bool seen = (above >> jj & 1) && !(key && jj == i);
                    const float a = ex2((hi - sc.hi[jj]) + (lo - sc.lo[jj]));
                    x[j] = seen ? own * a * (sc.r_k[jj] * x[j]) : 0.0f;
                }
                if (key) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4*>(L + j0 + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                } else if constexpr (HAS_Q) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint4 w;
                            w.x = take_part(x[8 * half], x[8 * half + 1]);
                            w.y = take_part(x[8 * half + 2], x[8 * half + 3]);
                            w.z = take_part(x[8 * half + 4], x[8 * half + 5]);
                            w.w = take_part(x[8 * half + 6], x[8 * half + 7]);
                            *reinterpret_cast<uint4*>(P + part * Y::kTile + (((j0 / 8 + half) ^ (i & 7)) << 4)) = w;
                        }
                }
            }
            umma_fence_before();
            mbar_arrive(&bars.gram_read);
            fence_proxy_async_smem();
            mbar_arrive(&bars.pairs_full[c & 1]);
        };
        load(0);
        loaded(0);
        if (chunks > 1) {
            load(1);
            loaded(1);
        }
        pairs(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            if (c + 1 < chunks) pairs(c + 1);
            if (c + 2 < chunks) {
                wait(&bars.input_free[c & 1], (c >> 1) & 1);
                load(c + 2);
                loaded(c + 2);
            }
        }
    } else if (lane == 0) {
        // ------------------------------------------------------------ products --
        constexpr uint32_t kById = idesc_bf16(64, false), kUpdate = idesc_bf16(D, true);
        auto gram = [&](int c) {
            wait(&bars.input_full[c & 1], (c >> 1) & 1);
            umma_fence_after();
            const uint32_t kq = smem_u32(input(c));
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint64_t d = umma_sdesc_sw128(kq + (k >> 2) * (2 * Y::kTile) + (k & 3) * 32);
                umma_bf16(tmem + Y::kG, d, d, kById, k > 0);
            }
            umma_commit(&bars.gram_full);
        };
        gram(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint32_t kq = smem_u32(input(c)), pp = smem_u32(p_of(c));
            wait(&bars.s_ready, c & 1);
            umma_fence_after();
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    umma_bf16_tmem(tmem + Y::kW, tmem + Y::kParts + part * (D / 2) + k * 8,
                                   umma_sdesc_sw128(kq + (k >> 2) * (2 * Y::kTile) + (k & 3) * 32), kById, part + k > 0);
            umma_commit(&bars.w_full);
            if constexpr (HAS_Q) {
                if (c > 0) {
                    wait(&bars.o_read, (c - 1) & 1);
                    umma_fence_after();
                }
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        umma_bf16_tmem(tmem + Y::kY, tmem + Y::kParts + part * (D / 2) + k * 8,
                                       umma_sdesc_sw128(kq + (k >> 2) * (2 * Y::kTile) + Y::kTile + (k & 3) * 32), kById,
                                       part + k > 0);
                umma_commit(&bars.y_full);
            }
            wait(&bars.gram_read, c & 1);    // (of this chunk's: its rows are done before u is)
            umma_fence_after();
            if (c + 1 < chunks) gram(c + 1);
            wait(&bars.u_ready, c & 1);
            umma_fence_after();
            if constexpr (!TREE) {
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int k = 0; k < kChunk / 16; ++k)
                        umma_bf16_tmem(tmem + Y::kS, tmem + Y::kUleft + part * 32 + k * 8,
                                       sdesc_n_contiguous(kq + k * 2048, 2 * Y::kTile), kUpdate, true);
                umma_commit(&bars.s_full);
            }
            if constexpr (HAS_Q) {
                if (c + 1 < chunks) {
                    wait(&bars.gram_read, (c + 1) & 1);
                    umma_fence_after();
                }
                wait(&bars.pairs_full[c & 1], (c >> 1) & 1);
#pragma unroll
                for (int m = 0; m < 3; ++m)                  // parts (0, 0), (0, 1), (1, 0)
#pragma unroll
                    for (int k = 0; k < kChunk / 16; ++k)
                        umma_bf16_tmem(tmem + Y::kG, tmem + Y::kU + (m == 2 ? 32 : 0) + k * 8,
                                       umma_sdesc_sw128(pp + (m == 1 ? Y::kTile : 0) + k * 32), kById, m + k > 0);
                umma_commit(&bars.o_full);
            }
            umma_commit(&bars.input_free[c & 1]);
        }
        // all products are done, whatever else gave up
        if (!mbar_wait(&bars.input_free[(chunks - 1) & 1], ((chunks - 1) >> 1) & 1)) record_error(p.err, kErrTimeout);
    }
    __syncwarp();
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D, DeltaMode MODE>
cudaError_t launch(const DeltaParams& p, cudaStream_t st) {
    constexpr size_t smem = Layout<D>::kBytes + sizeof(Barriers) + 1024;
    const void* kernel = reinterpret_cast<const void*>(delta_chunks_kernel<D, MODE>);
    cudaError_t e = ensure_dynamic_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_chained(delta_chunks_kernel<D, MODE>, (unsigned)p.B * p.Hv, kThreads, smem, st, p);
}

}  // namespace

cudaError_t launch_delta_chunks(int D, DeltaMode mode, const DeltaParams& p, cudaStream_t st) {
    if (mode == kDeltaChain) return D == 64 ? launch<64, kDeltaChain>(p, st) : launch<128, kDeltaChain>(p, st);
    if (mode == kDeltaTree) return D == 64 ? launch<64, kDeltaTree>(p, st) : launch<128, kDeltaTree>(p, st);
    return D == 64 ? launch<64, kDeltaCommit>(p, st) : launch<128, kDeltaCommit>(p, st);
}

}  // namespace r9q
