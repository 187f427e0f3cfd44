// The gated delta rule over many tokens a sequence, in chunks of 64 (formulas: r9q_delta.cuh): prompts,
// trees of drafted tokens, long accepted paths.
//
// A CTA walks one value head of a sequence.  Everything is transposed, so that row v of all
// products is value element v and belongs to one thread: with S [D values][D keys] as the
// accumulator in tensor memory, for each chunk of keys K, queries Q [64][D]
//   W = S K^T, Y = S Q^T         [D values][64 tokens]
//   X_i = beta_i (v_i - A(i, 0) W_i),  U = X T^T,  T = (1 + L)^-1
//   O = A(., 0) Y + U P^T,  S <- A(n, 0) S + (A(n, .) U) K
// with L_ij = beta_i A(i, j) (k_i.k_j), P_ij = A(i, j) (q_i.k_j) from one product [K; Q] K^T.
// Keys and queries are the bf16 inputs themselves (exact operands); their lengths go into L, P and
// the scalars.  What is fp32 (S, X, T, u) is an operand in bf16 parts, cut off, not rounded: three parts
// hold all 24 bits and keep fp32's range, so that nothing needs a scale and a
// token's values, however large, do not touch those of earlier tokens.  Three parts for what
// goes into S and u, two (2^-16) where only outputs, which are rounded to bf16, follow.
//
// Warps 0-7, the rows: S, X and u into parts, the chain that bounds a sequence's time, half the columns each;
// they take the last chunk's outputs while W is formed and write them during U's products.  Warps 8-11, the
// tokens: L and P of the next chunk.  Warps 12-15 turn
// L into T, in fp32 by blocks of 16, 32 and 64 (as a substitution a row's thread would need all of L
// in its registers: 8300 cycles of shared memory's 128 bytes each for four warps).  Warp 16 issues the
// products, 17 and 18 copy K and Q two chunks ahead and V one.  In a tree the sums go over ancestors, and its one chunk
// leaves the state alone.
//
// What bounds it: the chain of one chunk to the next, and the code.  A chunk takes about 9,700 cycles: the update of S 900,
// its parts 1450, W 1300, X 1000, U 1450, u 2000, the rest between them.  The parts run different code at once; at 185 KB
// in all it was fetched anew every chunk over a path that the SMs of a group share, and SMs beside busy ones took 1.4 times as
// long.  So loops are rolled where nothing waits for them, and a wait is a few instructions: 91 KB, 801 -> 641 us for
// 8192 tokens and 32 heads of 128 (one sequence, 32 SMs; now 630), 425 -> 328 for 16 of 64 to 2000 (now 325, 1.5 TB/s).
//
// A value that is not finite would reach earlier tokens (or other branches) through the zeros of T and P.
// So L's rows, X and u are zero in its place, and the outputs that it belongs to are NaN, as is the state's row.
#include <cfloat>

#include "r9q_delta.cuh"

namespace r9q {

namespace {

constexpr int kChunk = 64;
constexpr int kGroup = 128;                  // threads of the tokens, and of T; twice that the rows
constexpr int kLoaders = 64;
constexpr int kThreads = 4 * kGroup + 32 + kLoaders;      // (at most 20 warps have 96 registers)
constexpr int kLStride = 68;                 // floats between rows of L: eight rows' 16-byte pieces lie in different banks
constexpr int kMStride = 36;
constexpr int kSorted = 256;                 // sequences that are put in order

// Scalars of a chunk's tokens.
struct alignas(16) Scalars {
    ulonglong2 x[kChunk / 2];                // X = x v + y W, pairs of two tokens
    float fade[kChunk], o[kChunk];           // o = o (fade Y + U P^T)
    float last[kChunk];                      // A(n, i) / |k_i|
    float4 decay[kChunk];                    // two parts of the sum of the decays' logarithms (to base 2); 1 / |k|
    uint64_t above[kChunk];                  // (of a tree)
    uint32_t lost[2][kGroup];                // tokens without a finite X or u, by half and row
    int parents[kChunk];
    NodeKind kind[kChunk];
    uint32_t bad[2];                         // tokens whose row of L is not finite
    float end;                               // A(n, 0)
};

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = 64 * 128;                   // 64 rows of 128 bytes, swizzled
    static constexpr int kKq = kHalves * 2 * kTile;          // of each 64 elements: K's rows, then Q's
    static constexpr int kV = 3 * kKq;                       // three chunks' of those; V [64][D]
    static constexpr int kP = kV + kChunk * D * 2;           // twice P's two parts
    static constexpr int kT = kP + 4 * kTile;                // T's three
    static constexpr int kL = kT + 3 * kTile;                // L, twice
    static constexpr int kM = kL + 2 * kChunk * kLStride * 4;
    static constexpr int kScalars = kM + 32 * kMStride * 4;
    static constexpr int kBars = kScalars + 4 * (int)sizeof(Scalars);
    static_assert(kL % 16 == 0 && kM % 16 == 0 && kScalars % 16 == 0 && sizeof(Scalars) % 16 == 0 && kBars % 16 == 0,
                  "16-byte loads");
    // tensor memory, columns.  S's parts are 64 columns apart.  X's third part takes a place that W alone reads (of S's
    // third), U, in two sums, those of S's first and second.  W is replaced by two parts of X and they by two of u: of
    // tokens 32 i on in the columns 32 i and 32 i + 16 on; U P^T adds to A(., 0) Y.  (A product takes 40 cycles,
    // 70 with N = 128: so U's sums are one; W is not held up by Y.)
    static constexpr int kS = 0, kParts = 128, kW = kParts + 192, kY = kW + 64, kG = kY + 64;
    // (A(n, .) u's first two parts then lie where S's third was, its third as those.)
    static constexpr int kX2 = kParts + 128, kU = kParts, kUleft = kParts + 128;
    static_assert(kG + 64 == 512, "tensor memory");
};

struct Barriers {
    uint64_t input_full[3], k_free[3], v_full, gram_full, gram_read, pairs_full[2], l_free[2], o_full[2], t_full, s_ready,
        w_full, y_free, y_full, x_ready, u_full, u_ready, s_full;
    uint32_t tmem;
    int failed;                              // a wait gave up
};

// Two fp32 values to bf16, cut off; the rest stays.  (The rest as fused multiply-adds of the bf16 values themselves: taking
// them apart with masks instead keeps the logic pipe, at half rate, busier than any other.)
__device__ __forceinline__ uint32_t take_part(uint64_t& x) {
    uint32_t r;
    float2 f = parts_of(x);
    asm("{\n\t.reg .b16 l, h, k;\n\tcvt.rz.bf16x2.f32 %0, %2, %1;\n\tmov.b32 {l, h}, %0;\n\tmov.b16 k, 0xBF80;\n\t"
        "fma.rn.f32.bf16 %1, l, k, %1;\n\tfma.rn.f32.bf16 %2, h, k, %2;\n\t}"                 // (0xBF80: -1)
        : "=&r"(r), "+f"(f.x), "+f"(f.y));
    x = pair_of(f.x, f.y);
    return r;
}
// The last part: nothing stays.
__device__ __forceinline__ uint32_t last_part(uint64_t x) {
    uint32_t r;
    const float2 f = parts_of(x);
    asm("cvt.rz.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(f.x), "f"(f.y));
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
// 16 or 8 columns of this thread's lane.
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&d)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::"r"(d[0]),
        "r"(d[1]), "r"(d[2]), "r"(d[3]), "r"(d[4]), "r"(d[5]), "r"(d[6]), "r"(d[7]), "r"(d[8]), "r"(d[9]), "r"(d[10]),
        "r"(d[11]), "r"(d[12]), "r"(d[13]), "r"(d[14]), "r"(d[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&d)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(d[0]), "r"(d[1]), "r"(d[2]),
                 "r"(d[3]), "r"(d[4]), "r"(d[5]), "r"(d[6]), "r"(d[7]), "r"(taddr)
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
// Of one group's threads.
template <int ID>
__device__ __forceinline__ void group_barrier() {
    asm volatile("bar.sync %0, 128;" ::"n"(ID) : "memory");
}
// The next part of 32 values, two a column; LAST: nothing stays.
template <bool LAST = false, int N>
__device__ __forceinline__ void take_parts(uint32_t (&y)[N], uint64_t (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = LAST ? last_part(x[i]) : take_part(x[i]);
}
template <bool LAST = false, int N>
__device__ __forceinline__ void store_part(uint32_t taddr, uint64_t (&x)[N]) {
    uint32_t y[N];
    take_parts<LAST>(y, x);
    tmem_st(taddr, y);
}
// 32 columns of this thread's lane.
__device__ __forceinline__ void load_pairs(uint32_t taddr, uint64_t (&x)[16]) {
    float f[32];
    tmem_ld(taddr, f);
    tmem_wait_ld(f);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = pair_of(f[2 * i], f[2 * i + 1]);
}
// Which of 2 N values are not finite, a bit each; those become zero.
template <int N>
__device__ __forceinline__ uint32_t not_finite(uint64_t (&x)[N]) {
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) sum = fma2(x[i], 0ull, sum);
    uint32_t m = 0;
    const float2 any = parts_of(sum);
    if (any.x + any.y != 0.0f) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float2 f = parts_of(x[i]);
            if (!(fabsf(f.x) <= FLT_MAX)) {
                m |= 1u << (2 * i);
                f.x = 0.0f;
            }
            if (!(fabsf(f.y) <= FLT_MAX)) {
                m |= 2u << (2 * i);
                f.y = 0.0f;
            }
            x[i] = pair_of(f.x, f.y);
        }
    }
    __syncwarp();                            // (a store to tensor memory, by the whole warp, follows)
    return m;
}

// Bounded; after one that gave up all others do at once.  (As little code as can be, for there are many: the error is recorded
// at the end.)
struct Waits {
    volatile int* failed;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
#pragma unroll 1
        for (uint32_t i = 0; i < kSpinLimit; ++i) {
            if (mbar_try_wait(bar, parity)) return;
            if (*failed) return;
        }
        *failed = 1;
    }
};

template <int D, DeltaMode MODE>
__global__ void __launch_bounds__(kThreads, 1) delta_chunks_kernel(const DeltaParams p) {
    using Y = Layout<D>;
    constexpr bool TREE = MODE == kDeltaTree, HAS_Q = MODE != kDeltaCommit;
    extern __shared__ uint8_t raw[];
    begin_chained();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = tid & (kGroup - 1);
    const int rank = blockIdx.x / p.Hv, h = blockIdx.x - rank * p.Hv, hk = h / p.ratio;
    // The longest sequences first, so that no long one begins when the others end (32 heads of 128; 12 of 64 to 4000 tokens:
    // 545 us in every order, as given 671 with the longest last and 541 with it first; 40 of 64 to 1000: 542, 573
    // and 535); the order of many is not worth finding.
    int b = rank;
    if (p.cu && p.B <= kSorted) {
        int* lens = reinterpret_cast<int*>(raw);
        for (int x = tid; x < p.B; x += kThreads) lens[x] = p.cu[x + 1] - p.cu[x];
        __syncthreads();
        for (int x = tid; x < p.B; x += kThreads) {
            int before = 0;
            for (int y = 0; y < p.B; ++y) before += lens[y] > lens[x] || (lens[y] == lens[x] && y < x);
            if (before == rank) lens[kSorted] = x;
        }
        __syncthreads();
        b = lens[kSorted];
        __syncthreads();
    }
    int n;
    int64_t row0;
    delta_tokens(p, b, n, row0);
    const int32_t* path = p.path + (int64_t)b * p.P;
    if constexpr (MODE == kDeltaCommit) n = path_length(p, b);
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
    Barriers& bars = *reinterpret_cast<Barriers*>(smem + Y::kBars);
    auto input = [&](int c) { return smem + c % 3 * Y::kKq; };
    auto third = [](int c) { return (uint32_t)(c / 3) & 1; };        // the phase of what there are three of
    auto p_of = [&](int c) { return smem + Y::kP + (c & 1) * 2 * Y::kTile; };
    auto l_of = [&](int c) { return reinterpret_cast<float*>(smem + Y::kL) + (c & 1) * (kChunk * kLStride); };
    uint8_t* const parts_of_t = smem + Y::kT;
    auto scalars_of = [&](int c) { return reinterpret_cast<Scalars*>(smem + Y::kScalars) + (c & 3); };
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bars.input_full[i], kLoaders);
            mbar_init(&bars.k_free[i], 1);
        }
        mbar_init(&bars.v_full, kLoaders);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.pairs_full[i], kGroup);
            mbar_init(&bars.l_free[i], kGroup);
            mbar_init(&bars.o_full[i], 1);
        }
        mbar_init(&bars.gram_full, 1);
        mbar_init(&bars.gram_read, kGroup);
        mbar_init(&bars.t_full, kGroup);
        mbar_init(&bars.s_ready, 2 * kGroup);
        mbar_init(&bars.w_full, 1);
        mbar_init(&bars.y_free, 2 * kGroup);
        mbar_init(&bars.y_full, 1);
        mbar_init(&bars.x_ready, 2 * kGroup);
        mbar_init(&bars.u_full, 1);
        mbar_init(&bars.u_ready, 2 * kGroup);
        mbar_init(&bars.s_full, 1);
        bars.failed = 0;
        fence_mbar_init();
    }
    if (warp == 16) tmem_alloc(&bars.tmem, 512);
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    const uint32_t tmem = bars.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const Waits wait = {&bars.failed};

    if (warp < 8) {
        // ---------------------------------------------------------------- rows --
        const bool live = t < D;             // (D = 64: the other half of the lanes is zeros)
        const int half = warp >> 2, e0 = half * (D / 2), t0 = half * 32;         // the thread's columns and tokens
        float* row = state + (int64_t)t * D;
#pragma unroll 1
        for (int e = e0; e < e0 + D / 2; e += 16) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = live && !p.from_zero ? reinterpret_cast<const uint4*>(row + e)[i] : make_uint4(0, 0, 0, 0);
                x[4 * i] = v.x;
                x[4 * i + 1] = v.y;
                x[4 * i + 2] = v.z;
                x[4 * i + 3] = v.w;
            }
            tmem_st(mine + Y::kS + e, x);
        }
        tmem_wait_st();
        uint32_t out[16];                    // of chunk c, two tokens each, as bf16
        auto take_outputs = [&](int c) {
            const Scalars& sc = *scalars_of(c);
            wait(&bars.o_full[c & 1], (c >> 1) & 1);
            umma_fence_after();
            float y[32];
            tmem_ld(mine + Y::kY + t0, y);
            tmem_wait_ld(y);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&sc.o[t0 + i]);
                out[i / 2] = pack_bf16x2(f.x * y[i], f.y * y[i + 1]);
                out[i / 2 + 1] = pack_bf16x2(f.z * y[i + 2], f.w * y[i + 3]);
            }
        };
        auto mark_outputs = [&](int c) {
            const Scalars& sc = *scalars_of(c);
            uint64_t lost = (uint64_t)sc.lost[1][t] << 32 | sc.lost[0][t] | *reinterpret_cast<const uint64_t*>(sc.bad);
            if (lost) {                      // NaN, and what comes from it
                if constexpr (TREE) {
#pragma unroll 1
                    for (int i = 0; i < kChunk; ++i)
                        if (sc.above[i] & lost) lost |= 1ull << i;
                } else {
                    lost = ~0ull << (__ffsll((long long)lost) - 1);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (lost >> (t0 + i) & 1) out[i / 2] = i & 1 ? (out[i / 2] & 0xFFFFu) | 0x7FC00000u : (out[i / 2] & 0xFFFF0000u) | 0x7FC0u;
            }
            __syncwarp();                    // (as there, of Y)
            if constexpr (TREE) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const NodeKind kind = sc.kind[t0 + i];
                    const uint32_t bits = kind == kNoNode ? 0u : 0x7FC07FC0u, m = i & 1 ? 0xFFFF0000u : 0xFFFFu;
                    if (kind != kNode) out[i / 2] = (out[i / 2] & ~m) | (bits & m);
                }
            }
        };
        // (A warp writes 64 bytes of a token.)
        const int64_t o_stride = (int64_t)p.Hv * D;
        uint16_t* const o_first = HAS_Q ? p.o + ((row0 + t0) * p.Hv + h) * D + t : nullptr;
        auto write_outputs = [&](int c) {
            uint16_t* o = o_first + c * kChunk * o_stride;
            const int most = live ? min(n - c * kChunk - t0, 32) : 0;
            if (most == 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    *o = (uint16_t)(out[i / 2] >> (16 * (i & 1)));
                    o += o_stride;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (i < most) *o = (uint16_t)(out[i / 2] >> (16 * (i & 1)));
                    o += o_stride;
                }
            }
        };
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            wait(&bars.pairs_full[c & 1], (c >> 1) & 1);
            Scalars& sc = *scalars_of(c);
            if (c > 0) {
                wait(&bars.s_full, (c - 1) & 1);
                umma_fence_after();
            }
            // S into its parts, and what is left of it at the chunk's end
            const float left = sc.end;
            const uint64_t left2 = pair_of(left, left);
#pragma unroll 1
            for (int e = e0; e < e0 + D / 2; e += 32) {
                uint64_t s[16];
                load_pairs(mine + Y::kS + e, s);
                if constexpr (!TREE) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t x[16];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 f = parts_of(mul2(left2, s[i * 8 + j]));
                            x[2 * j] = __float_as_uint(f.x);
                            x[2 * j + 1] = __float_as_uint(f.y);
                        }
                        tmem_st(mine + Y::kS + e + i * 16, x);
                    }
                }
                uint32_t first[16];
                take_parts(first, s);
                store_part(mine + Y::kParts + 64 + e / 2, s);
                store_part<true>(mine + Y::kParts + 128 + e / 2, s);
                tmem_st(mine + Y::kParts + e / 2, first);
            }
            tmem_wait_st();
            umma_fence_before();
            mbar_arrive(&bars.s_ready);
            if constexpr (HAS_Q) {
                if (c > 0) take_outputs(c - 1);
                umma_fence_before();
                mbar_arrive(&bars.y_free);
            }

            // ---- X ----
            const uint16_t* v = reinterpret_cast<const uint16_t*>(smem + Y::kV) + t0 * D + (live ? t : 0);
            uint32_t own[16];
            wait(&bars.v_full, c & 1);
#pragma unroll
            for (int i = 0; i < 16; ++i) own[i] = (uint32_t)v[2 * i * D] | (uint32_t)v[(2 * i + 1) * D] << 16;
            uint64_t x[16];
            wait(&bars.w_full, c & 1);
            umma_fence_after();
            load_pairs(mine + Y::kW + t0, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const ulonglong2 f = sc.x[t0 / 2 + i];
                x[i] = fma2(f.y, x[i], mul2(f.x, pair_of(bf16_lo(own[i]), bf16_hi(own[i]))));
            }
            uint32_t lost = not_finite(x);
            store_part(mine + Y::kW + t0, x);
            store_part(mine + Y::kW + t0 + 16, x);
            store_part<true>(mine + Y::kX2 + t0 / 2, x);
            tmem_wait_st();
            umma_fence_before();
            mbar_arrive(&bars.x_ready);

            // ---- the last chunk's outputs, and Y as it goes into these ----
            if constexpr (HAS_Q) {
                if (c > 0) {
                    mark_outputs(c - 1);
                    write_outputs(c - 1);
                }
                wait(&bars.y_full, c & 1);
                umma_fence_after();
                load_pairs(mine + Y::kY + t0, x);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t y[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = parts_of(mul2(*reinterpret_cast<const uint64_t*>(&sc.fade[t0 + 16 * i + 2 * j]), x[i * 8 + j]));
                        y[2 * j] = __float_as_uint(f.x);
                        y[2 * j + 1] = __float_as_uint(f.y);
                    }
                    tmem_st(mine + Y::kY + t0 + i * 16, y);
                }
            }

            // ---- u, as an operand: with A(n, .) for the state, as it is for the outputs ----
            wait(&bars.u_full, c & 1);
            umma_fence_after();
#pragma unroll 1
            for (int t1 = t0; t1 < t0 + 32; t1 += 16) {
                uint64_t u[8];
                {
                    float y[16], z[16];
                    tmem_ld(mine + Y::kU + t1, y);
                    tmem_ld(mine + Y::kU + 64 + t1, z);
                    tmem_wait_ld(y);
                    tmem_wait_ld(z);
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[j] = add2(pair_of(y[2 * j], y[2 * j + 1]), pair_of(z[2 * j], z[2 * j + 1]));
                }
                lost |= not_finite(u) << (t1 - t0);
                if constexpr (!TREE) {
                    uint64_t y[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&sc.last[t1 + 2 * i]);
                        y[i] = mul2(f.x, u[i]);
                        y[i + 1] = mul2(f.y, u[i + 1]);
                    }
                    if (t1 > t0 && (lost | sc.bad[0] | sc.bad[1])) y[0] = pair_of(__int_as_float(0x7FC00000), 0.0f);     // into the state
                    __syncwarp();
                    store_part(mine + Y::kUleft + t1 / 2, y);
                    store_part(mine + Y::kUleft + 32 + t1 / 2, y);
                    store_part<true>(mine + Y::kU + t0 + (t1 - t0) / 2, y);
                }
                if constexpr (HAS_Q) {
                    store_part(mine + Y::kW + t0 + (t1 - t0) / 2, u);
                    store_part<true>(mine + Y::kW + t0 + 16 + (t1 - t0) / 2, u);
                }
            }
            sc.lost[half][t] = lost;
            tmem_wait_st();
            umma_fence_before();
            mbar_arrive(&bars.u_ready);
        }
        if constexpr (!TREE) {
            wait(&bars.s_full, (chunks - 1) & 1);
            umma_fence_after();
#pragma unroll 1
            for (int e = e0; e < e0 + D / 2; e += 32) {
                float s[32];
                tmem_ld(mine + Y::kS + e, s);
                tmem_wait_ld(s);
                if (live)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<float4*>(row + e)[i] = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
            }
        }
        if constexpr (HAS_Q) {
            take_outputs(chunks - 1);
            mark_outputs(chunks - 1);
            write_outputs(chunks - 1);
        }
    } else if (warp < 12) {
        // -------------------------------------------------------------- tokens --
        const int i = t & 63;                // row of K or of Q
        const bool key = t < 64;
        auto rate_of = [&](int at) {
            return ((MODE == kDeltaCommit ? row0 + path[at] : row0 + at)) * p.Hv + h;
        };
        float g_next = 0.0f, beta_next = 0.0f;
        auto load_rates = [&](int c) {       // ahead of their use
            const int at = c * kChunk + i;
            g_next = at < n ? p.g[rate_of(at)] : 0.0f;
            beta_next = key && at < n ? p.beta[rate_of(at)] : 0.0f;
        };
        // L, P and the scalars of chunk c
        auto pairs = [&](int c) {
            Scalars& sc = *scalars_of(c);
            const int at = c * kChunk + i;
            // Sums of the decays' logarithms to base 2 in units of 2^-40, so that differences are exact.  (exp(-200) is 0, and
            // infinities have no differences; a NaN goes into the rate, and from there to all that follows.)
            const float beta = g_next == g_next ? beta_next : g_next;
            const long long g = __float2ll_rn(fminf(fmaxf(g_next, -200.0f), 200.0f) * (1.4426950408889634f * 0x1p40f));
            if (c + 1 < chunks) load_rates(c + 1);
            // the row's length
            wait(&bars.input_full[c % 3], third(c));
            float square = 0.0f;
            if (key || HAS_Q) {
                const uint8_t* row = input(c) + t * 128;     // (K's rows, then Q's)
#pragma unroll 4
                for (int x = 0; x < D / 8; ++x) {
                    const uint4 q = *reinterpret_cast<const uint4*>(row + (x >> 3) * (2 * Y::kTile) + (((x & 7) ^ (t & 7)) << 4));
                    const Eight e = unpack(q);
                    square += dot(e, e);
                }
            }
            const float r = at < n ? rsqrtf(square + p.eps) : 0.0f;
            uint64_t above = ~0ull >> (63 - i);
            long long sum = 0, end = 0;
            if constexpr (TREE) {
                long long* rates = reinterpret_cast<long long*>(sc.decay);
                if (key) {
                    rates[i] = g;
                    sc.parents[i] = at < n ? p.parents[(int64_t)b * p.Lq + at] : -2;
                }
                group_barrier<1>();
                int depth;
                const NodeKind kind = find_node(sc.parents, i, kMostNodes, above, depth);
                if (kind == kBadNode && key) record_error(p.err, kErrArg);
                if (kind != kNode) above = 0;
                sc.kind[i] = kind;
                sc.above[i] = above;
                for (uint64_t m = above; m; m &= m - 1) sum += rates[__ffsll((long long)m) - 1];
                group_barrier<1>();
            } else {                         // a scan over the 64 tokens, whole in each pair of warps
                sum = g;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                long long* halves = reinterpret_cast<long long*>(sc.parents);        // (a tree's)
                if (lane == 31) halves[warp & 3] = sum;
                group_barrier<1>();
                end = halves[0] + halves[1];
                if (i >= 32) sum += halves[0];
            }
            // (the sum is under 2^55: its upper word is exact as a float)
            const float hi = (float)(int)(sum >> 32) * 0x1p-8f, lo = (float)(uint32_t)sum * 0x1p-40f, fade = ex2(hi + lo);
            if (key) {
                sc.decay[i] = make_float4(hi, lo, r, 0.0f);
                float* x = reinterpret_cast<float*>(&sc.x[i / 2]) + (i & 1);
                x[0] = beta;
                x[2] = -(beta * fade * r);
                if (!TREE) sc.last[i] = ex2((float)(end - sum) * 0x1p-40f) * r;
            } else {
                sc.fade[i] = fade;
                sc.o[i] = r * p.scale;
            }
            if (t == 0) {
                sc.end = ex2((float)end * 0x1p-40f);
                sc.bad[0] = sc.bad[1] = 0;
            }
            group_barrier<1>();
            if (c >= 2) {
                wait(&bars.l_free[c & 1], ((c - 2) >> 1) & 1);
                wait(&bars.o_full[c & 1], ((c - 2) >> 1) & 1);      // (P; and what used the scalars of chunk c - 3 and before)
            }
            wait(&bars.gram_full, c & 1);
            umma_fence_after();
            const float own = key ? beta * r : 1.0f;
            if (key) above &= ~(1ull << i);
            float* Li = l_of(c) + i * kLStride;
            uint8_t* P = p_of(c) + i * 128;
            uint64_t zeros = 0;              // NaN where a value of the row is not finite
            const int first = (warp & 1) * 32;               // the warp's rows are first .. first + 31
#pragma unroll 1
            for (int j0 = 0; j0 < kChunk; j0 += 16) {
                float x[16];
                if (!TREE && j0 >= first + 32) {             // nothing of it is seen
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = 0.0f;
                } else {
                    tmem_ld(mine + Y::kG + j0, x);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float4 d = sc.decay[j0 + j];
                        x[j] = (own * ex2((hi - d.x) + (lo - d.y))) * (d.z * x[j]);
                    }
                    if (TREE || j0 >= first) {
                        const uint32_t seen = (uint32_t)(above >> j0);
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = seen >> j & 1 ? x[j] : 0.0f;
                    }
                }
                if (key) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        *reinterpret_cast<float4*>(Li + j0 + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                        zeros = fma2(pair_of(x[j], x[j + 1]), 0ull, fma2(pair_of(x[j + 2], x[j + 3]), 0ull, zeros));
                    }
                } else if constexpr (HAS_Q) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint64_t y[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] = pair_of(x[8 * half + 2 * j], x[8 * half + 2 * j + 1]);
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            uint4 w;
                            w.x = part == 1 ? last_part(y[0]) : take_part(y[0]);
                            w.y = part == 1 ? last_part(y[1]) : take_part(y[1]);
                            w.z = part == 1 ? last_part(y[2]) : take_part(y[2]);
                            w.w = part == 1 ? last_part(y[3]) : take_part(y[3]);
                            *reinterpret_cast<uint4*>(P + part * Y::kTile + (((j0 / 8 + half) ^ (i & 7)) << 4)) = w;
                        }
                    }
                }
            }
            const float2 zero = parts_of(zeros);
            if (key && zero.x + zero.y != 0.0f) {
                atomicOr(&sc.bad[i >> 5], 1u << (i & 31));
                for (int j = 0; j < kChunk; j += 4) *reinterpret_cast<float4*>(Li + j) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            umma_fence_before();
            mbar_arrive(&bars.gram_read);
            fence_proxy_async_smem();
            mbar_arrive(&bars.pairs_full[c & 1]);
        };
        load_rates(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) pairs(c);
    } else if (warp < 16) {
        // ------------------------------------------------------------ L into T --
        float* const M = reinterpret_cast<float*>(smem + Y::kM);
        auto pairs4 = [](const float* at) { return *reinterpret_cast<const ulonglong2*>(at); };
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            wait(&bars.pairs_full[c & 1], (c >> 1) & 1);
            float* const L = l_of(c);
            auto l4 = [&](int r, int col) { return *reinterpret_cast<const float4*>(L + r * kLStride + col); };
            // blocks of 16 on the diagonal, a column a thread
            if (t < 64) {
                const int at = t & 48, col = t & 15;
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float s = i == col ? 1.0f : 0.0f;
#pragma unroll
                    for (int j = 0; j < i; j += 4) {
                        const float4 l = l4(at + i, at + j);
                        s = fmaf(-l.x, x[j], s);
                        if (j + 1 < i) s = fmaf(-l.y, x[j + 1], s);
                        if (j + 2 < i) s = fmaf(-l.z, x[j + 2], s);
                        if (j + 3 < i) s = fmaf(-l.w, x[j + 3], s);
                    }
                    x[i] = s;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) L[(at + i) * kLStride + at + col] = x[i];
            }
            group_barrier<2>();
            // of 32: the lower left is -T22 (L21 T11)
            {
                const int at = (t >> 6) * 32, r = (t & 63) >> 2, col = (t & 3) * 4;
                float* m = M + (t >> 6) * (16 * kMStride);
#pragma unroll
                for (int pass = 0; pass < 2; ++pass) {
                    uint64_t s[2] = {};
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 l = l4(at + 16 + r, at + pass * 16 + k);
                        const float w[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const ulonglong2 y = pass == 0 ? pairs4(L + (at + k + x) * kLStride + at + col)
                                                           : pairs4(m + (k + x) * kMStride + col);
                            const uint64_t f = pass == 0 ? pair_of(w[x], w[x]) : pair_of(-w[x], -w[x]);
                            s[0] = fma2(f, y.x, s[0]);
                            s[1] = fma2(f, y.y, s[1]);
                        }
                    }
                    float* out = pass == 0 ? m + r * kMStride + col : L + (at + 16 + r) * kLStride + at + col;
                    *reinterpret_cast<ulonglong2*>(out) = make_ulonglong2(s[0], s[1]);
                    group_barrier<2>();
                }
            }
            // of 64, two rows and four columns a thread
            {
                const int r = (t >> 3) * 2, col = (t & 7) * 4;
#pragma unroll
                for (int pass = 0; pass < 2; ++pass) {
                    const int most = pass == 0 ? 32 : (warp & 3) * 8 + 8;    // (T22's rows end at the diagonal)
                    uint64_t s[2][2] = {};
#pragma unroll 2
                    for (int k = 0; k < most; k += 4) {
                        const float4 l0 = l4(32 + r, pass * 32 + k), l1 = l4(33 + r, pass * 32 + k);
                        const float w[2][4] = {{l0.x, l0.y, l0.z, l0.w}, {l1.x, l1.y, l1.z, l1.w}};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const ulonglong2 y = pass == 0 ? pairs4(L + (k + x) * kLStride + col) : pairs4(M + (k + x) * kMStride + col);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint64_t f = pass == 0 ? pair_of(w[i][x], w[i][x]) : pair_of(-w[i][x], -w[i][x]);
                                s[i][0] = fma2(f, y.x, s[i][0]);
                                s[i][1] = fma2(f, y.y, s[i][1]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float* out = pass == 0 ? M + (r + i) * kMStride + col : L + (32 + r + i) * kLStride + col;
                        *reinterpret_cast<ulonglong2*>(out) = make_ulonglong2(s[i][0], s[i][1]);
                    }
                    group_barrier<2>();
                }
            }
            // its parts, half a row a thread
            if (c > 0) wait(&bars.u_full, (c - 1) & 1);      // (the last chunk's are used)
            {
                const int r = t >> 1, half = t & 1;
                uint8_t* T = parts_of_t + r * 128;
#pragma unroll 1
                for (int x = 0; x < 4; ++x) {
                    const float4 a = l4(r, half * 32 + x * 8), d = l4(r, half * 32 + x * 8 + 4);
                    uint64_t y[4] = {pair_of(a.x, a.y), pair_of(a.z, a.w), pair_of(d.x, d.y), pair_of(d.z, d.w)};
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        uint4 w;
                        w.x = part == 2 ? last_part(y[0]) : take_part(y[0]);
                        w.y = part == 2 ? last_part(y[1]) : take_part(y[1]);
                        w.z = part == 2 ? last_part(y[2]) : take_part(y[2]);
                        w.w = part == 2 ? last_part(y[3]) : take_part(y[3]);
                        *reinterpret_cast<uint4*>(T + part * Y::kTile + (((half * 4 + x) ^ (r & 7)) << 4)) = w;
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bars.t_full);
            mbar_arrive(&bars.l_free[c & 1]);
        }
    } else if (warp > 16) {
        // --------------------------------------------------------------- loads --
        const int x0 = tid - (4 * kGroup + 32);
        // A thread copies the same 16 bytes of every 64 / (D/8)-th token.
        constexpr int PIECES = D / 8, STEP = kLoaders / PIECES;
        const int piece = x0 % PIECES, r0 = x0 / PIECES;
        enum { kKeys, kQueries, kValues };
        auto load = [&](int what, int c) {
            const bool values = what == kValues;
            uint32_t dst = values ? smem_u32(smem + Y::kV) + r0 * (D * 2) + piece * 16
                                  : smem_u32(input(c)) + (piece >> 3) * (2 * Y::kTile) + what * Y::kTile + r0 * 128;
            const uint16_t* src = (what == kKeys ? p.k + b * p.k_bs + hk * p.k_hs
                                   : values      ? p.v + b * p.v_bs + h * p.v_hs
                                                 : p.q + b * p.q_bs + hk * p.q_hs) + piece * 8;
            const int64_t stride = what == kKeys ? p.k_ts : values ? p.v_ts : p.q_ts;
            int at = c * kChunk + r0;
            if (MODE != kDeltaCommit) src += ((p.cu ? row0 : 0) + at) * stride;
#pragma unroll 4
            for (int x = 0; x < kChunk / STEP; ++x) {
                const uint16_t* from = src;
                if (MODE == kDeltaCommit && at < n) from += path[at] * stride;
                copy16(dst + (values ? 0 : ((piece & 7) ^ (at & 7)) << 4), at < n ? from : p.k, at < n);     // (zeros behind the last)
                dst += STEP * (values ? D * 2 : 128);
                src += MODE == kDeltaCommit ? 0 : STEP * stride;
                at += STEP;
            }
        };
#pragma unroll 1
        for (int c = -2; c < chunks; ++c) {
            if (c >= 0) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                mbar_arrive(&bars.v_full);
            }
            if (c + 2 < chunks) {            // where chunk c - 1 was
                if (c > 0) wait(&bars.k_free[(c - 1) % 3], third(c - 1));
#pragma unroll 1
                for (int what = kKeys; what <= (HAS_Q ? kQueries : kKeys); ++what) load(what, c + 2);
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                mbar_arrive(&bars.input_full[(c + 2) % 3]);
            }
            if (c + 1 < chunks && c >= -1) {
                if (c >= 0) wait(&bars.x_ready, c & 1);
                load(kValues, c + 1);
            }
        }
    } else if (elect_one()) {
        // ------------------------------------------------------------ products --
        constexpr uint32_t kById = idesc_bf16(64, false), kUpdate = idesc_bf16(D, true);
        // D[tmem] = A B^T with A the keys' and queries' rows or parts of S, B [64][D]
        auto gram = [&](int c) {
            wait(&bars.input_full[c % 3], third(c));
            if (c > 0) wait(&bars.gram_read, (c - 1) & 1);
            umma_fence_after();
            const uint32_t kq = smem_u32(input(c));
#pragma unroll 1
            for (int half = 0; half < Y::kHalves; ++half)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t d = umma_sdesc_sw128(kq + half * (2 * Y::kTile) + k * 32);
                    umma_bf16(tmem + Y::kG, d, d, kById, half + k > 0);
                }
            umma_commit(&bars.gram_full);
        };
        auto by_keys = [&](uint32_t d, uint32_t b_tile, int parts) {
#pragma unroll 1
            for (int i = 0; i < parts * Y::kHalves; ++i) {
                const int part = i / Y::kHalves, half = i % Y::kHalves;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_bf16_tmem(d, tmem + Y::kParts + part * 64 + half * 32 + k * 8,
                                   umma_sdesc_sw128(b_tile + half * (2 * Y::kTile) + k * 32), kById, i + k > 0);
            }
        };
        // D[tmem] (+)= A[tmem] B^T with B [N][64]; A's tokens from 32 on `apart` columns after the others
        auto by_tokens = [&](uint32_t d, uint32_t a, int apart, uint32_t b_tile, uint32_t idesc, bool first) {
#pragma unroll
            for (int k = 0; k < kChunk / 16; ++k)
                umma_bf16_tmem(d, a + (k >> 1) * apart + (k & 1) * 8, umma_sdesc_sw128(b_tile + k * 32), idesc, !first || k > 0);
        };
#pragma unroll 1
        for (int c = 0; c < min(chunks, 2); ++c) gram(c);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint32_t kq = smem_u32(input(c)), pp = smem_u32(p_of(c)), tt = smem_u32(parts_of_t);
            wait(&bars.s_ready, c & 1);
            umma_fence_after();
            // W, with three parts of S, then Y, with two
#pragma unroll 1
            for (int y = 0; y < (HAS_Q ? 2 : 1); ++y) {
                if (y) {
                    umma_commit(&bars.w_full);
                    wait(&bars.y_free, c & 1);
                    umma_fence_after();
                }
                by_keys(tmem + (y ? Y::kY : Y::kW), kq + y * Y::kTile, 3 - y);
            }
            umma_commit(HAS_Q ? &bars.y_full : &bars.w_full);
            wait(&bars.x_ready, c & 1);
            wait(&bars.t_full, c & 1);
            umma_fence_after();
            // parts (X, T): (0, 0) and (0, 1), (1, 0) and (1, 1), (0, 2), (2, 0)
#pragma unroll 1
            for (int i = 0; i < 4; ++i)
                by_tokens(tmem + Y::kU, tmem + (i == 3 ? Y::kX2 : i == 1 ? Y::kW + 16 : Y::kW), i == 3 ? 16 : 32,
                          tt + (i == 2 ? 2 * Y::kTile : 0), i < 2 ? idesc_bf16(128, false) : kById, i == 0);
            umma_commit(&bars.u_full);
            if (c + 2 < chunks) gram(c + 2);
            wait(&bars.u_ready, c & 1);
            umma_fence_after();
            if constexpr (!TREE) {
#pragma unroll 1
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int k = 0; k < kChunk / 16; ++k)
                        umma_bf16_tmem(tmem + Y::kS,
                                       tmem + (part < 2 ? Y::kUleft + part * 32 + k * 8 : Y::kU + (k >> 1) * 32 + (k & 1) * 8),
                                       sdesc_n_contiguous(kq + k * 2048, 2 * Y::kTile), kUpdate, true);
                umma_commit(&bars.s_full);
            }
            umma_commit(&bars.k_free[c % 3]);
            if constexpr (HAS_Q) {
                wait(&bars.pairs_full[c & 1], (c >> 1) & 1);
                // parts (u, P): (0, 0), (0, 1), (1, 0)
#pragma unroll 1
                for (int i = 0; i < 3; ++i)
                    by_tokens(tmem + Y::kY, tmem + Y::kW + (i == 2 ? 16 : 0), 32, pp + (i == 1 ? Y::kTile : 0), kById, false);
            }
            umma_commit(&bars.o_full[c & 1]);
        }
        // all products are done, whatever else gave up
        if (!mbar_wait(&bars.o_full[(chunks - 1) & 1], ((chunks - 1) >> 1) & 1)) bars.failed = 1;
    }
    __syncwarp();
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    if (warp == 16) tmem_dealloc(tmem, 512);
    if (tid == 0 && bars.failed) record_error(p.err, kErrTimeout);
}

template <int D, DeltaMode MODE>
cudaError_t launch(const DeltaParams& p, cudaStream_t st) {
    constexpr size_t smem = Layout<D>::kBars + sizeof(Barriers) + 1024;
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
