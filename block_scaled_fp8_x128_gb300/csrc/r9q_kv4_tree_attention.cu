// Attention of a tree of drafted tokens over the paged 4-bit cache, for many rows of a key-value head
// (nodes times the query heads that share it); few rows take the kernel of r9q_kv4_attention.cu, whose
// formulas and references these are.
//
// With more than a few rows the products are what costs, and they go to tcgen05: a tile of 128
// rows, a thread each, against tiles of 128 keys.  A CTA has two such streams, which take
// turns on the tensor cores: two row tiles over the same keys, or with up to 128 rows one row tile
// over the even and the odd tiles of keys.
//   S = Q Ck^T     Q in fp16, brought to [2^13, 2^14) by a power of two per row; codes in the low bits of an fp16, the
//                  subnormal c 2^-24, exactly (of two nibbles one weighs 16 times the other; so do Q's elements, inversely)
//   score = fr (sk S + lk sum(q))
//   O += P V'      P the weights in fp16, in S's place in tensor memory; V' = (c - 8) sv 2^(11 - E), fp16, E the exponent of
//                  the largest step (or 2^-10 of a lowest value) so far
// and what V' leaves out, mid = lv + 8 sv, is summed in fp32 with the weights before their rounding, so that what fp16 loses counts
// with the distance of codes from 8, however far from zero the values are.  (With mid and its weights in fp16 6 % less time,
// but an error of 2^-12 of a value's size; with mid as bf16, and what that leaves in V', 2 % more.)  Sums of (c - 8), which are near zero,
// do not drift as those of codes would.  V' holds steps down to 2^-25 of the largest in full.  References move as there: a
// row's weights are taken against top - 8 + E of its own, which moves only when a chunk of 32 weights passes 2^15, and takes
// what is summed and P with it.
// Tiles in which some row does not see some key (the tree's own, those at a window's edge or at the sequence's end) keep an
// exponent for every key, and a row takes the same steps whatever the other rows of its warp need, so that its result depends on
// nothing that it does not see; V' of a key without a finite pair is zero there and everywhere, and rows that see it are NaN.
//
// What bounds it: the softmax's chain of loads, exponentials and stores, with two warps a scheduler (256 rows x 128 heads
// of 8200 keys, D = 128: 228 us, 603 TFLOP/s; half of the issue slots, tensor cores busy for 29 %; streams that take turns
// at it took 3 % more, two threads a row 30 %, for their registers spill), and 25 us of beginning and end.
//
// Warps 0-3 and 4-7: the streams; the first of each issues its products.  Warps 8-11 read the codes of a tile ahead into
// registers, and write K and V' of the one at hand to shared memory.  Work is cut as in r9q_kv4_attention.cuh; an item that several
// CTAs share is joined by a second kernel, a warp a row.
#include <algorithm>

#include "r9q_delta.cuh"
#include "r9q_kv4_attention.cuh"

namespace r9q {

namespace {

constexpr int kTile = 128;                   // keys, and rows
constexpr int kStreamThreads = 128, kConvertThreads = 128;
constexpr int kThreads = 2 * kStreamThreads + kConvertThreads;
constexpr int kTileGroups = kTile / 16;
constexpr int kRing = 4;                     // tiles whose scalars are kept
struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};
constexpr float kNear = 4194304.0f;          // 2^22
constexpr float kMost = 32768.0f;            // a sum of 32 weights over this moves the reference

// Of a tile's keys.
struct alignas(16) KeyScalars {
    uint32_t k[kTile];                       // the pair, as in the cache
    float mid[kTile];                        // (lv + 8 sv) 2^-exponent
    float exponent[kTile];                   // biased; all the same where every row sees every key
    uint16_t v[kTile];                       // steps as fp16, 2^(11 - exponent) times
    uint32_t bad[4];                         // keys without a finite value pair
    uint32_t have;                           // groups that were read
    float one_exponent;
};
struct alignas(16) TreeNodes {
    uint64_t mask[kMostNodes];
    int first[kMostNodes], instead[kMostNodes], parents[kMostNodes];
};
struct Bars {
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], o_full[2];
    uint32_t tmem;
    int failed;
};
template <int D>
struct Shape {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalf = kTile * 128;                // 128 rows of 128 bytes, swizzled
    static constexpr int kQ = kHalves * kHalf;               // one row tile
    static constexpr int kV = 2 * D * 128;                   // [2 halves of the keys][D] of 64 keys
    static constexpr int kAtK = 2 * kQ, kAtV = kAtK + 2 * kQ, kAtScalars = kAtV + 2 * kV;
    static constexpr int kAtNodes = kAtScalars + kRing * (int)sizeof(KeyScalars);
    static constexpr int kAtMeet = kAtNodes + (int)sizeof(TreeNodes);        // references and sums of one stream for the other
    static constexpr int kAtBars = kAtMeet + 2 * kTile * 4;
    static_assert(sizeof(KeyScalars) % 16 == 0 && kAtNodes % 16 == 0 && kAtBars % 16 == 0, "16-byte loads");
    static constexpr size_t kBytes = kAtBars + sizeof(Bars) + 1024;
    static constexpr int kS = 0, kO = 256;                   // tensor memory: S (and P) of both streams, O of both
};

__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_f16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// fp16 operands with K contiguous, fp32 accumulator, M = 128.
constexpr uint32_t idesc_f16(int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24); }

__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&d)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::"r"(d[0]),
        "r"(d[1]), "r"(d[2]), "r"(d[3]), "r"(d[4]), "r"(d[5]), "r"(d[6]), "r"(d[7]), "r"(d[8]), "r"(d[9]), "r"(d[10]),
        "r"(d[11]), "r"(d[12]), "r"(d[13]), "r"(d[14]), "r"(d[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int ID, int N>
__device__ __forceinline__ void part_barrier() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory");
}

// Bounded; after one that gave up all others do at once.
struct Waits {
    volatile int* failed;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
#pragma unroll 1
        for (uint32_t i = 0; i < kSpinLimit; ++i) {
            if (mbar_try_wait(bar, parity & 1)) return;
            if (*failed) return;
        }
        *failed = 1;                         // (recorded at the end)
    }
};

// Bits [lo, hi) of 32.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    lo = min(max(lo, 0), 32);
    hi = min(max(hi, 0), 32);
    const uint32_t below_hi = hi == 32 ? 0xFFFFFFFFu : (1u << hi) - 1u, below_lo = lo == 32 ? 0xFFFFFFFFu : (1u << lo) - 1u;
    return below_hi & ~below_lo;
}

// The groups of a part, as tiles, and what is known of a tile without looking at its keys.
struct Tiles {
    int g_begin, g_end, len, all_lo, base;
    __device__ __forceinline__ int count() const { return (g_end - g_begin + kTileGroups - 1) / kTileGroups; }
    __device__ __forceinline__ int first_key(int j) const { return (g_begin + j * kTileGroups) * 16; }
    // some row does not see some of its keys before the tree
    __device__ __forceinline__ bool edge(int j) const { return first_key(j) < all_lo; }
    // every row sees all of its keys (if all its pages are there)
    __device__ __forceinline__ bool plain(int j) const {
        return first_key(j) >= all_lo && first_key(j) + kTile <= base && g_begin + (j + 1) * kTileGroups <= g_end;
    }
};
__device__ __forceinline__ Tiles tiles_of(const Kv4AttnParams& p, const Walk& walk, const Part& it) {
    const int base = walk.sp.len - p.Lq;
    return {it.g_begin, it.g_end, walk.sp.len, p.window > 0 ? base + p.Lq - p.window : 0, base};
}

constexpr int kItemCost = 24;                // groups of a CTA that take as long as beginning and ending an item
constexpr int kMinGroups = 2 * kTileGroups;  // a tile for each stream

// D: elements of a head.  DUAL: two row tiles over the same keys.
template <int D, bool DUAL>
__global__ void __launch_bounds__(kThreads, 1) tree_attention_kernel(const Kv4AttnParams p, int2* items) {
    using Z = Shape<D>;
    constexpr int ROWS = DUAL ? 2 * kTile : kTile;
    extern __shared__ uint8_t raw[];
    begin_chained();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = tid & 127;
    uint8_t* smem = raw + (1024u - smem_u32(raw) % 1024u) % 1024u;
    Bars& bars = *reinterpret_cast<Bars*>(smem + Z::kAtBars);
    auto scalars_of = [&](int tile) { return reinterpret_cast<KeyScalars*>(smem + Z::kAtScalars) + (tile & (kRing - 1)); };
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.k_full[i], kConvertThreads);
            mbar_init(&bars.k_free[i], DUAL ? 2 : 1);
            mbar_init(&bars.v_full[i], kConvertThreads);
            mbar_init(&bars.v_free[i], DUAL ? 2 : 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.o_full[i], 1);
        }
        bars.failed = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&bars.tmem, 512);
    Walk walk;
    const bool any = walk.start(p, kMinGroups, kItemCost);
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    const uint32_t tmem = bars.tmem;
    const Waits wait = {&bars.failed};
    const int rows = p.Lq * p.G;
    // Steps of a stream: every tile, or every second one.
    auto steps_of = [](int tiles, int stream) { return DUAL ? tiles : (tiles + 1 - stream) >> 1; };
    auto tile_of = [](int step, int stream) { return DUAL ? step : 2 * step + stream; };
    Part it;

    if (warp < 8) {
        // ------------------------------------------------------------- streams --
        const int stream = warp >> 2, half = DUAL ? stream : 0;
        const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t at_s = mine + Z::kS + stream * 128, at_o = mine + Z::kO + stream * 128;
        TreeNodes& nodes = *reinterpret_cast<TreeNodes*>(smem + Z::kAtNodes);
        int done = 0, tile0 = 0;             // steps and tiles of earlier parts
        while (any && walk.next(p, it)) {
            const Tiles tiles = tiles_of(p, walk, it);
            const int n = tiles.count(), steps = steps_of(n, stream);
            const int row = it.chunk * ROWS + half * kTile + t;              // of the item's rows
            const bool live = row < rows, warp_live = row - lane < rows;
            const int node = live ? row / p.group : 0, head = it.hk * p.G + (live ? row - node * p.G : 0);
            // ---- the tree ----
            if (tid < p.Lq) nodes.parents[tid] = p.parents[(int64_t)it.b * p.Lq + tid];
            part_barrier<1, 2 * kStreamThreads>();
            if (tid < p.Lq) {
                uint64_t mask;
                int depth;
                const NodeKind kind = find_node(nodes.parents, tid, p.window > 0 ? p.window : kMostNodes, mask, depth);
                const bool none = tiles.len == 0;            // an unused place of the batch: whatever its parents are
                if (kind == kBadNode && !none) record_error(p.err, kErrArg);
                nodes.mask[tid] = mask;
                nodes.first[tid] = p.window > 0 && kind == kNode ? tiles.base + depth - p.window + 1 : 0;
                nodes.instead[tid] = kind == kNode ? kAsItIs : kind == kNoNode || none ? kNothing : kNan;
            }
            // ---- the row's query ----
            float fr = 0.0f, qs = 0.0f;
            {
                uint32_t x[D / 2];
                const uint4* src = reinterpret_cast<const uint4*>(p.q + it.b * p.q_bs + node * p.q_ts + head * p.q_hs);
                uint32_t big = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = live ? src[i] : make_uint4(0, 0, 0, 0);
                    x[4 * i] = v.x;
                    x[4 * i + 1] = v.y;
                    x[4 * i + 2] = v.z;
                    x[4 * i + 3] = v.w;
                }
#pragma unroll
                for (int i = 0; i < D / 2; ++i) {
                    big = __vmaxu2(big, x[i] & 0x7FFF7FFFu);
                    qs += bf16_lo(x[i]) + bf16_hi(x[i]);
                }
                big = max(big >> 16, big & 0xFFFFu);
                const int e = (int)(big >> 7), up = e == 0 ? 0 : min(13 - (e - 127), 100);
                const float f = __uint_as_float((uint32_t)(127 + up) << 23), f16 = f * 0.0625f;
                fr = fminf(p.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23) * 0x1p24f, 3e38f);
                qs *= f * 0x1p-24f;
                if (DUAL || stream == 0) {
                    uint8_t* dst = smem + half * Z::kQ + t * 128;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {        // (the order in which a word of codes gives its elements)
                        const uint32_t* q = x + 4 * i;
                        uint4 w;
                        w.x = pack_f16x2(bf16_lo(q[0]) * f, bf16_lo(q[2]) * f);
                        w.y = pack_f16x2(bf16_hi(q[0]) * f16, bf16_hi(q[2]) * f16);
                        w.z = pack_f16x2(bf16_lo(q[1]) * f, bf16_lo(q[3]) * f);
                        w.w = pack_f16x2(bf16_hi(q[1]) * f16, bf16_hi(q[3]) * f16);
                        *reinterpret_cast<uint4*>(dst + (i >> 3) * Z::kHalf + (((i & 7) ^ (t & 7)) << 4)) = w;
                    }
                }
            }
            fence_proxy_async_smem();
            part_barrier<1, 2 * kStreamThreads>();           // (Q and the nodes are there)
            // ---- the products, by the stream's first warp ----
            auto issue_scores = [&](int i) {
                const int tile = tile0 + tile_of(i, stream), buf = tile & 1;
                wait(&bars.k_full[buf], tile >> 1);
                umma_fence_after();
                const uint32_t q = smem_u32(smem) + half * Z::kQ, k = smem_u32(smem) + Z::kAtK + buf * Z::kQ;
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x)
                        umma_f16(tmem + Z::kS + stream * 128, umma_sdesc_sw128(q + (x >> 2) * Z::kHalf + (x & 3) * 32),
                                 umma_sdesc_sw128(k + (x >> 2) * Z::kHalf + (x & 3) * 32), idesc_f16(kTile), x > 0);
                    umma_commit(&bars.s_full[stream]);
                    umma_commit(&bars.k_free[buf]);
                }
                __syncwarp();
            };
            auto issue_values = [&](int i) {
                const int tile = tile0 + tile_of(i, stream), buf = tile & 1;
                wait(&bars.v_full[buf], tile >> 1);
                umma_fence_after();
                const uint32_t v = smem_u32(smem) + Z::kAtV + buf * Z::kV;
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < kTile / 16; ++x)
                        umma_f16_tmem(tmem + Z::kO + stream * 128, tmem + Z::kS + stream * 128 + x * 8,
                                      umma_sdesc_sw128(v + (x >> 2) * (D * 128) + (x & 3) * 32), idesc_f16(D), i > 0 || x > 0);
                    umma_commit(&bars.o_full[stream]);
                    umma_commit(&bars.v_free[buf]);
                }
                __syncwarp();
            };
            const bool issues = (warp & 3) == 0;
            if (issues && steps > 0) issue_scores(0);
            const uint64_t node_mask = nodes.mask[node];
            const int first = nodes.first[node];

            // l: the sum of 2^(score - ref + 8), ref = rint(top fr), an integer, so that one fused multiply-add makes the
            // exponent (for scores under 2^22; larger ones take the difference from top first, and ref = top fr).
            // O and ml: those weights times 2^(e - e_row), e a key's exponent.
            float top = 0.0f, ref = 0.0f, l = 0.0f, ml = 0.0f;
            int e_row = 1;
            bool seen_any = false, lost = false;
            const uint64_t fr2 = pair_of(fr, fr), qs2 = pair_of(qs, qs);
#pragma unroll 1
            for (int i = 0; i < steps; ++i) {
                const int j = tile_of(i, stream), tile = tile0 + j;
                wait(&bars.s_full[stream], done + i);
                umma_fence_after();
                const KeyScalars& ks = *scalars_of(tile);
                const bool plain = tiles.plain(j) && ks.have == 0xFFu;
                if (warp_live) {
                    // which of the keys the row sees
                    uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
                    if (!plain) {
                        const int key0 = tiles.first_key(j), off = tiles.base - key0;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int s = 32 * w - off;
                            const uint32_t tree = s >= 64 || s <= -32 ? 0u : s >= 0 ? (uint32_t)(node_mask >> s) : (uint32_t)(node_mask << -s);
                            const uint32_t here = (ks.have >> (2 * w) & 1u ? 0xFFFFu : 0u) | (ks.have >> (2 * w + 1) & 1u ? 0xFFFF0000u : 0u);
                            seen[w] = (bits_between(first - key0 - 32 * w, off - 32 * w) | tree) & here &
                                      bits_between(0, tiles.len - key0 - 32 * w);
                        }
                    }
                    lost = lost || ((seen[0] & ks.bad[0]) | (seen[1] & ks.bad[1]) | (seen[2] & ks.bad[2]) | (seen[3] & ks.bad[3])) != 0;
                    // Scores of 32 keys, over fr, from their products.
                    auto scores = [&](int c, const float (&a)[32], uint64_t (&s)[16]) {
#pragma unroll
                        for (int x = 0; x < 16; x += 2) {
                            const uint4 k = *reinterpret_cast<const uint4*>(&ks.k[c * 32 + 2 * x]);
                            s[x] = fma2(pair_of(bf16_lo(k.x), bf16_lo(k.y)), pair_of(a[2 * x], a[2 * x + 1]),
                                        mul2(pair_of(bf16_hi(k.x), bf16_hi(k.y)), qs2));
                            s[x + 1] = fma2(pair_of(bf16_lo(k.z), bf16_lo(k.w)), pair_of(a[2 * x + 2], a[2 * x + 3]),
                                            mul2(pair_of(bf16_hi(k.z), bf16_hi(k.w)), qs2));
                        }
                    };
                    // The row's reference to `to` and its exponent to `to_e`; `c`: chunks of P that are written.
                    float sum = 0.0f, msum = 0.0f;           // of the tile
                    auto move = [&](float to, int to_e, int c) {
                        const bool near = fabsf(to * fr) < kNear || fabsf(ref) < kNear;
                        const float to_ref = fabsf(to * fr) < kNear ? rintf(to * fr) : to * fr;
                        const float alpha = seen_any ? ex2(near ? ref - to_ref : (top - to) * fr) : 0.0f;
                        const float alpha_w = alpha * ex2((float)(e_row - to_e));
                        top = to;
                        ref = to_ref;
                        e_row = to_e;
                        l *= alpha;
                        sum *= alpha;
                        ml *= alpha_w;
                        msum *= alpha_w;
                        if (i > 0) {                         // O, once the last tile's product is in it
                            wait(&bars.o_full[stream], done + i - 1);
                            umma_fence_after();
#pragma unroll 1
                            for (int x = 0; x < D; x += 16) {
                                float o[16];
                                uint32_t y[16];
                                tmem_ld(at_o + x, o);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int z = 0; z < 16; ++z) y[z] = __float_as_uint(o[z] * alpha_w);
                                tmem_store16(at_o + x, y);
                            }
                        }
#pragma unroll 1
                        for (int x = 0; x < c; ++x) {
                            const uint32_t both = pack_f16x2(alpha_w, alpha_w);
                            float w[16];
                            uint32_t y[16];
                            tmem_ld(at_s + x * 16, w);
                            tmem_wait_ld(w);
#pragma unroll
                            for (int z = 0; z < 16; ++z) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[z]) : "r"(__float_as_uint(w[z])), "r"(both));
                            tmem_store16(at_s + x * 16, y);
                        }
                        tmem_stored();
                    };
                    if (!plain || __any_sync(0xffffffffu, !seen_any)) {       // the largest score and exponent of what the row sees
                        float best = kNegInf, most = plain ? ks.one_exponent : 0.0f;
                        bool none = false;                   // a score that is not a number
                        float a[32];
                        tmem_ld(at_s, a);
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint64_t s[16];
                            tmem_wait_ld(a);
                            scores(c, a, s);
                            if (c < 3) tmem_ld(at_s + (c + 1) * 32, a);
                            const uint32_t m = c == 0 ? seen[0] : c == 1 ? seen[1] : c == 2 ? seen[2] : seen[3];
#pragma unroll
                            for (int x = 0; x < 32; x += 2) {
                                float2 f = parts_of(s[x / 2]);
                                if (!(m >> x & 1)) f.x = kNegInf;
                                if (!(m >> x & 2)) f.y = kNegInf;
                                none = none || f.x != f.x || f.y != f.y;
                                best = max3(best, f.x, f.y);
                            }
                            if (!plain)
#pragma unroll
                                for (int x = 0; x < 32; x += 4) {
                                    const float4 ex = *reinterpret_cast<const float4*>(&ks.exponent[c * 32 + x]);
                                    most = max3(most, m >> x & 1 ? ex.x : 0.0f, m >> x & 2 ? ex.y : 0.0f);
                                    most = max3(most, m >> x & 4 ? ex.z : 0.0f, m >> x & 8 ? ex.w : 0.0f);
                                }
                        }
                        const int e = (int)most;
                        // (a score that is not a number makes the row's sums that, whatever the reference)
                        const bool any = best > kNegInf || none;
                        // (a plain tile brings here rows that have seen something too, for others' sake)
                        const bool up = any && (!seen_any || (!plain && (best - top) * fr > (float)kSlack));
                        const int to_e = any ? max(e_row, e) : e_row;
                        if (__any_sync(0xffffffffu, up || to_e > e_row)) move(up ? (none ? 0.0f : best) : top, to_e, 0);
                        seen_any = seen_any || any;
                    } else if (__any_sync(0xffffffffu, (int)ks.one_exponent > e_row)) {
                        move(top, max(e_row, (int)ks.one_exponent), 0);
                    }
                    // Weights of 32 keys against the reference: as P's columns, and their sums.
                    auto weigh = [&](int c, const float (&a)[32], uint32_t (&out)[16], float& chunk_sum, float& chunk_mid, auto tag) {
                        constexpr bool FAST = decltype(tag)::value;
                        uint64_t s[16];
                        scores(c, a, s);
                        const uint32_t m = c == 0 ? seen[0] : c == 1 ? seen[1] : c == 2 ? seen[2] : seen[3];
                        const bool near = fabsf(ref) < kNear;
                        const uint64_t top2 = pair_of(-top, -top), shift2 = pair_of((float)kHeadroom - ref, (float)kHeadroom - ref);
                        uint64_t total = 0;
                        float mid0 = 0.0f, mid1 = 0.0f;
                        float4 mid;
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            if (x % 2 == 0) mid = *reinterpret_cast<const float4*>(&ks.mid[c * 32 + 2 * x]);
                            uint64_t at = fma2(s[x], fr2, shift2);
                            if constexpr (!FAST)
                                if (!near) at = fma2(add2(s[x], top2), fr2, pair_of((float)kHeadroom, (float)kHeadroom));
                            const float2 f = parts_of(at);
                            float p0 = ex2(f.x), p1 = ex2(f.y), w0, w1;
                            if constexpr (FAST) {
                                w0 = p0;
                                w1 = p1;
                            } else {                         // (unseen keys may have any pair)
                                const float2 ex = *reinterpret_cast<const float2*>(&ks.exponent[c * 32 + 2 * x]);
                                p0 = m >> (2 * x) & 1 ? p0 : 0.0f;
                                p1 = m >> (2 * x + 1) & 1 ? p1 : 0.0f;
                                w0 = p0 * ex2(fminf(ex.x - (float)e_row, 0.0f));
                                w1 = p1 * ex2(fminf(ex.y - (float)e_row, 0.0f));
                            }
                            total = add2(total, pair_of(p0, p1));
                            out[x] = pack_f16x2(w0, w1);
                            mid0 = fmaf(w0, x % 2 == 0 ? mid.x : mid.z, mid0);
                            mid1 = fmaf(w1, x % 2 == 0 ? mid.y : mid.w, mid1);
                        }
                        const float2 both = parts_of(total);
                        chunk_sum = both.x + both.y;
                        chunk_mid = mid0 + mid1;
                    };
                    // A row that sees all, with the same exponent as its own: a fused multiply-add and nothing else stand between a
                    // score and its weight, and the reference moves where 32 weights pass their bound.  A warp of such rows
                    // takes the short way; in any other they come to the same, bit for bit (a row's result is its own).
                    const bool short_row = plain && e_row == (int)ks.one_exponent && fabsf(ref) < kNear;
                    const bool fast = __all_sync(0xffffffffu, short_row);
                    float a[32], z[32];
                    uint32_t y[16], u[16];
                    auto weigh_tile = [&](auto tag) {        // 64 keys at a time, from S's first columns in a
#pragma unroll 1
                        for (int c = 0; c < 4; c += 2) {
                            float sum0, mid0, sum1, mid1;
                            tmem_ld(at_s + (c + 1) * 32, z);
                            tmem_wait_ld(a);
                            tmem_wait_ld(z);
                            weigh(c, a, y, sum0, mid0, tag);
                            weigh(c + 1, z, u, sum1, mid1, tag);
                            const bool over = short_row && fmaxf(sum0, sum1) > kMost;
                            if (__any_sync(0xffffffffu, over)) {             // (P of these is not written yet, and S is there)
                                float best = kNegInf;
#pragma unroll 1
                                for (int k = c; k < c + 2; ++k) {
                                    uint64_t s[16];
                                    tmem_ld(at_s + k * 32, a);
                                    tmem_wait_ld(a);
                                    scores(k, a, s);
#pragma unroll
                                    for (int x = 0; x < 16; ++x) {
                                        const float2 f = parts_of(s[x]);
                                        best = max3(best, f.x, f.y);
                                    }
                                }
                                move(over ? fmaxf(top, best) : top, e_row, c);
                                tmem_ld(at_s + c * 32, a);
                                tmem_wait_ld(a);
                                weigh(c, a, y, sum0, mid0, No());
                                tmem_ld(at_s + c * 32 + 32, a);
                                tmem_wait_ld(a);
                                weigh(c + 1, a, u, sum1, mid1, No());
                            }
                            if (c == 0) tmem_ld(at_s + 64, a);
                            sum += sum0 + sum1;
                            msum += mid0 + mid1;
                            tmem_store16(at_s + c * 16, y);
                            tmem_store16(at_s + c * 16 + 16, u);
                        }
                    };
                    tmem_ld(at_s, a);
                    if (fast) {
                        weigh_tile(Yes());
                    } else {
                        // (the reference holds for all: what the row sees was looked through; or it has another exponent, or scores
                        // too large for the short way, and it is looked through here)
                        if (plain) {
                            float best = kNegInf;
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                uint64_t s[16];
                                if (c > 0) tmem_ld(at_s + c * 32, a);
                                tmem_wait_ld(a);
                                scores(c, a, s);
#pragma unroll
                                for (int x = 0; x < 16; ++x) {
                                    const float2 f = parts_of(s[x]);
                                    best = max3(best, f.x, f.y);
                                }
                            }
                            const bool up = !short_row && (best - top) * fr > (float)kSlack;
                            if (__any_sync(0xffffffffu, up)) move(up ? best : top, e_row, 0);
                            tmem_ld(at_s, a);
                        }
                        weigh_tile(No());
                    }
                    l += sum;
                    ml += msum;
                    tmem_stored();
                }
                umma_fence_before();
                if (stream == 0)
                    part_barrier<3, kStreamThreads>();
                else
                    part_barrier<4, kStreamThreads>();
                if (issues) {
                    issue_values(i);
                    if (i + 1 < steps) {
                        wait(&bars.o_full[stream], done + i);                // (P is read: S takes its place)
                        issue_scores(i + 1);
                    }
                }
            }
            // ---- the end of the part ----
            if (steps > 0) {
                wait(&bars.o_full[stream], done + steps - 1);
                umma_fence_after();
            }
            if (lost) l = __int_as_float(0x7FC00000);
            // As partials are: both sums in units of 2^-e for one e, under which they are finite.
            const int e_out = max(e_row, kMinExponent);
            const float to_out = ex2((float)(e_row - e_out));
            l *= ex2((float)(127 - e_out));
            ml *= to_out;
            float m = seen_any ? ref + (float)(e_out - kHeadroom - 127) : kNegInf;
            float scale_o = steps > 0 && seen_any ? 0x1p-11f * to_out : 0.0f;
            float total_m = m, total_l = l;
            float* meet_m = reinterpret_cast<float*>(smem + Z::kAtMeet);
            float* meet_l = meet_m + kTile;
            float* meet_o = reinterpret_cast<float*>(smem);                  // [D / 4][128 rows] of four, over Q and K
            float own_k = 1.0f, other_k = 0.0f;
            if constexpr (!DUAL) {           // the other stream's sums, by way of shared memory
                part_barrier<1, 2 * kStreamThreads>();       // (no product reads Q any more)
                if (stream == 1) {
                    meet_m[t] = m;
                    meet_l[t] = l;
#pragma unroll 1
                    for (int x = 0; x < D; x += 16) {
                        float o[16];
                        tmem_ld(at_o + x, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int z = 0; z < 16; z += 4)
                            reinterpret_cast<float4*>(meet_o)[(x + z) / 4 * kTile + t] =
                                seen_any ? make_float4(fmaf(o[z], scale_o, ml), fmaf(o[z + 1], scale_o, ml), fmaf(o[z + 2], scale_o, ml), fmaf(o[z + 3], scale_o, ml))
                                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
                }
                part_barrier<1, 2 * kStreamThreads>();
                if (stream == 0) {
                    const float om = meet_m[t], ol = meet_l[t];
                    total_m = fmaxf(m, om);
                    const float base = total_m > kNegInf ? total_m : 0.0f;
                    own_k = ex2(m - base);
                    other_k = ex2(om - base);
                    total_l = l * own_k + ol * other_k;
                }
            }
            if (warp_live && (DUAL || stream == 0)) {
                const Instead instead = (Instead)nodes.instead[node];
                float* part = p.part + ((size_t)blockIdx.x * 2 + (it.begins ? 1 : 0)) * ((size_t)ROWS * (D + 2));
                const int r = half * kTile + t;
                const int64_t out = ((int64_t)it.b * p.Lq + node) * (p.c.heads * p.G) + head;
                const float inv = total_l != 0.0f ? 1.0f / total_l : 0.0f;
#pragma unroll 1
                for (int x = 0; x < D; x += 16) {
                    float o[16];
                    tmem_ld(at_o + x, o);    // (by the whole warp)
                    tmem_wait_ld(o);
#pragma unroll
                    for (int z = 0; z < 16; ++z) o[z] = steps > 0 && seen_any ? own_k * fmaf(o[z], scale_o, ml) : 0.0f;
                    if constexpr (!DUAL) {
#pragma unroll
                        for (int z = 0; z < 16; z += 4) {
                            const float4 v = reinterpret_cast<const float4*>(meet_o)[(x + z) / 4 * kTile + t];
                            o[z] = fmaf(other_k, v.x, o[z]);
                            o[z + 1] = fmaf(other_k, v.y, o[z + 1]);
                            o[z + 2] = fmaf(other_k, v.z, o[z + 2]);
                            o[z + 3] = fmaf(other_k, v.w, o[z + 3]);
                        }
                    }
                    if (live && it.whole) {
                        uint32_t w[8];
#pragma unroll
                        for (int z = 0; z < 8; ++z) {
                            w[z] = pack_bf16x2(o[2 * z] * inv, o[2 * z + 1] * inv);
                            if (instead != kAsItIs) w[z] = instead == kNothing ? 0u : 0x7FC07FC0u;
                        }
                        uint4* dst = reinterpret_cast<uint4*>(p.o + out * D + x);
                        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    } else if (live) {
#pragma unroll
                        for (int z = 0; z < 16; z += 4)
                            reinterpret_cast<float4*>(part)[(x + z) / 4 * ROWS + r] = make_float4(o[z], o[z + 1], o[z + 2], o[z + 3]);
                    }
                    __syncwarp();            // (the next load is by the whole warp again)
                }
                if (live && it.whole && p.lse)
                    p.lse[out] = instead == kNothing ? kNegInf : instead == kNan ? __int_as_float(0x7FC00000) : log_sum_exp(total_m, total_l);
                if (live && !it.whole) {
                    part[(size_t)ROWS * D + r] = total_m;
                    part[(size_t)ROWS * D + ROWS + r] = total_l;
                }
            }
            if (tid == 0 && it.begins) {     // for the kernel that joins: the CTAs that have the item
                int c0 = 0, c1 = 0;
                if (!it.whole) walk.sharers(c0, c1);
                items[(int64_t)it.b * walk.items_per_seq + walk.item] = make_int2(c0, c1);
            }
            umma_fence_before();
            part_barrier<1, 2 * kStreamThreads>();           // (the nodes, Q and what met are free)
            done += steps;
            tile0 += n;
            if (walk.parted) break;
        }
    } else {
        // --------------------------------------------------------------- codes --
        int tile0 = 0;
        while (any && walk.next(p, it)) {
            const Tiles tiles = tiles_of(p, walk, it);
            const int n = tiles.count(), gmax = min(it.g_end, (tiles.len + 15) >> 4);
            const int32_t* table = p.table + (int64_t)it.b * p.max_pages;
            // Thread t: key t; and of the values the eight rows r = t % 8 of half a head or all (D = 64: of two groups).
            constexpr int VG = kConvertThreads / (8 * (D / 64));             // groups at a time
            const int vr = t & 7, vc = D == 128 ? (t >> 3) & 1 : 0, vg = t / (8 * (D / 64));
            static_assert(VG == kTileGroups || VG == 2 * kTileGroups, "groups of a tile");
            auto group_at = [&](int j, int g) {
                const int at = it.g_begin + j * kTileGroups + g;
                return g < kTileGroups && at < gmax ? find_group(p, table, at, it.hk) : kNoGroup;
            };
            uint32_t k_at = group_at(0, t >> 4), v_at = group_at(0, vg), k_next = kNoGroup, v_next = kNoGroup;
            uint4 kq[D / 32], vq[4];
            uint32_t kp = 0, vp = 0;
            auto load = [&]() {              // the codes at k_at and v_at
                if (k_at != kNoGroup) {
                    const uint4* src = reinterpret_cast<const uint4*>(p.c.k + ((uint64_t)k_at + (t & 15)) * (D / 2));
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) kq[i] = src[i];
                    kp = p.c.kp[(uint64_t)k_at + (t & 15)];
                    vp = p.c.vp[(uint64_t)k_at + (t & 15)];
                }
                if (v_at != kNoGroup) {
                    const uint4* src = reinterpret_cast<const uint4*>(p.c.v + (uint64_t)v_at * (D / 2) + vc * 512 + vr * 64);
#pragma unroll
                    for (int i = 0; i < 4; ++i) vq[i] = src[i];
                }
            };
#pragma unroll
            for (int i = 0; i < D / 32; ++i) kq[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) vq[i] = make_uint4(0, 0, 0, 0);
            int e_part = 1;                  // the largest exponent of a key that all rows see
            load();
            if (n > 1) {
                k_next = group_at(1, t >> 4);
                v_next = group_at(1, vg);
            }
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const int tile = tile0 + j, buf = tile & 1;
                KeyScalars& ks = *scalars_of(tile);
                uint8_t* K = smem + Z::kAtK + buf * Z::kQ;
                uint8_t* V = smem + Z::kAtV + buf * Z::kV;
                if (tile >= 2) wait(&bars.k_free[buf], (tile - 2) >> 1);
                // ---- the key's pairs ----
                const bool here = k_at != kNoGroup && tiles.first_key(j) + t < tiles.len;
                const uint32_t kpair = here ? kp : 0u, vpair = here ? vp : 0u;
                const int xs = (int)(vpair >> 7) & 255, xl = (int)(vpair >> 23) & 255;
                const bool bad = xs == 255 || xl == 255;
                int e = bad ? 1 : min(max(max(xs, xl - kLowestBits), 1), 253);
                const uint32_t got = __ballot_sync(0xffffffffu, k_at != kNoGroup), not_good = __ballot_sync(0xffffffffu, bad);
                if (lane == 0) {
                    ks.bad[warp & 3] = not_good;
                    uint8_t* have = reinterpret_cast<uint8_t*>(ks.exponent);         // (for a moment)
                    have[warp & 3] = (uint8_t)((got & 1u) | (got >> 16 & 1u) << 1);
                }
                // (what every row sees has one exponent, the largest so far)
                const bool all_see = !tiles.edge(j) && tiles.first_key(j) + t < tiles.base;
                int most = all_see && here ? e : 1;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                if (lane == 0) reinterpret_cast<int*>(ks.mid)[warp & 3] = most;      // (likewise)
                part_barrier<2, kConvertThreads>();
                const uint32_t four = *reinterpret_cast<const uint32_t*>(ks.exponent);
                const int4 all = *reinterpret_cast<const int4*>(ks.mid);
                part_barrier<2, kConvertThreads>();
                const uint32_t have = (four & 3u) | (four >> 6 & 12u) | (four >> 12 & 48u) | (four >> 18 & 192u);
                e_part = max(e_part, max(max(all.x, all.y), max(all.z, all.w)));
                if (all_see) e = e_part;
                ks.k[t] = kpair;
                const float sv = bad ? 0.0f : bf16_lo(vpair), lv = bad ? 0.0f : bf16_hi(vpair);
                const float down = __uint_as_float((uint32_t)(254 - e) << 23);
                ks.mid[t] = fmaf(8.0f, sv * down, lv * down);
                ks.exponent[t] = (float)e;
                // 2^(11 + 127 - e) in two factors, so that neither is out of range
                ks.v[t] = (uint16_t)pack_f16x2(sv * down * 2048.0f, 0.0f);
                if (t == 0) {
                    ks.have = have;
                    ks.one_exponent = (float)e_part;
                }
                // ---- keys: a word's four masks are 16 bytes of the row ----
                uint8_t* dst = K + t * 128;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t q[4] = {kq[i].x, kq[i].y, kq[i].z, kq[i].w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int word = 4 * i + x;
                        const uint32_t w = q[x], y = w >> 8;
                        *reinterpret_cast<uint4*>(dst + (word >> 3) * Z::kHalf + (((word & 7) ^ (t & 7)) << 4)) =
                            make_uint4(w & 0x000F000Fu, w & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars.k_full[buf]);
                // ---- values ----
                if (tile >= 2) wait(&bars.v_free[buf], (tile - 2) >> 1);
                part_barrier<2, kConvertThreads>();          // (the steps of all keys)
                if (vg < kTileGroups) {
                    const uint4 s0 = *reinterpret_cast<const uint4*>(&ks.v[vg * 16]), s1 = *reinterpret_cast<const uint4*>(&ks.v[vg * 16 + 8]);
                    const uint32_t lo[4] = {s0.x, s0.y, s0.z, s0.w}, hi[4] = {s1.x, s1.y, s1.z, s1.w};
                    auto value = [](uint32_t codes, uint32_t magic, uint32_t middle, uint32_t step) {
                        uint32_t r;
                        asm("{\n\t.reg .b32 x;\n\tsub.rn.f16x2 x, %1, %2;\n\tmul.rn.f16x2 %0, x, %3;\n\t}" : "=r"(r) : "r"(codes | magic), "r"(middle), "r"(step));
                        return r;
                    };
                    uint8_t* row = V + (vg >> 2) * (D * 128) + (vc * 64 + vr) * 128;
                    const int at0 = ((vg & 3) * 2) ^ vr, at1 = ((vg & 3) * 2 + 1) ^ vr;
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        uint32_t a[4], c[4], x[4], y[4];     // of tokens 2j, 2j + 1 and 8 on; element r and r + 8
#pragma unroll
                        for (int jj = 0; jj < 4; ++jj) {
                            const uint32_t w = m == 0 ? vq[jj].x : m == 1 ? vq[jj].y : m == 2 ? vq[jj].z : vq[jj].w, h = w >> 8;
                            // 1024 + code (steps of one), 64 + code (steps of 1/16)
                            a[jj] = value(w & 0x000F000Fu, 0x64006400u, 0x64086408u, lo[jj]);
                            c[jj] = value(h & 0x000F000Fu, 0x64006400u, 0x64086408u, hi[jj]);
                            x[jj] = value(w & 0x00F000F0u, 0x54005400u, 0x54805480u, lo[jj]);
                            y[jj] = value(h & 0x00F000F0u, 0x54005400u, 0x54805480u, hi[jj]);
                        }
                        uint8_t* d0 = row + m * (16 * 128);
                        *reinterpret_cast<uint4*>(d0 + (at0 << 4)) = make_uint4(a[0], a[1], a[2], a[3]);
                        *reinterpret_cast<uint4*>(d0 + (at1 << 4)) = make_uint4(c[0], c[1], c[2], c[3]);
                        *reinterpret_cast<uint4*>(d0 + 8 * 128 + (at0 << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
                        *reinterpret_cast<uint4*>(d0 + 8 * 128 + (at1 << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars.v_full[buf]);
                // the next tile's codes are on their way meanwhile
                k_at = k_next;
                v_at = v_next;
                if (j + 1 < n) load();
                k_next = j + 2 < n ? group_at(j + 2, t >> 4) : kNoGroup;
                v_next = j + 2 < n ? group_at(j + 2, vg) : kNoGroup;
            }
            tile0 += n;
            if (walk.parted) break;
        }
    }
    __syncwarp();
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
    if (tid == 0 && bars.failed) record_error(p.err, kErrTimeout);
}

// Items that several CTAs share.  A partial is [D / 4][ROWS] of four elements, then the rows' references and sums; a thread
// joins four elements of a row, a warp those of 32 rows.
constexpr int kJoinRows = 32, kJoinPieces = 8;
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinRows * kJoinPieces) join_kernel(const Kv4AttnParams p, const int2* items, int row_blocks) {
    begin_chained();
    constexpr int PIECES = D / 4 / kJoinPieces;              // blocks that share a row
    const int x = blockIdx.x / PIECES, item = x / row_blocks;
    const int r = (x - item * row_blocks) * kJoinRows + (threadIdx.x & 31);
    const int piece = (blockIdx.x - x * PIECES) * kJoinPieces + (threadIdx.x >> 5);
    const int2 by = items[item];
    if (by.x == by.y || r >= ROWS) return;
    const int chunks = p.chunks.d, per_seq = p.c.heads * chunks, b = item / per_seq, rest = item - b * per_seq;
    const int hk = rest / chunks, chunk = rest - hk * chunks, row = chunk * ROWS + r;
    if (row >= p.Lq * p.G) return;
    const int node = row / p.G, head = hk * p.G + (row - node * p.G);
    // the node, as the other kernel found it
    const int32_t* parents = p.parents + (int64_t)b * p.Lq;
    Instead instead = kAsItIs;
    if (parents[node] == -2) {
        instead = kNothing;
    } else {
        for (int t = node; t >= 0;) {
            const int up = parents[t];
            if (up != -1 && (up < 0 || up >= t)) {
                instead = kNan;
                break;
            }
            t = up;
        }
    }
    auto slot = [&](int c) { return p.part + ((size_t)c * 2 + (c == by.x ? 1 : 0)) * ((size_t)ROWS * (D + 2)); };
    float top = kNegInf;
#pragma unroll 4
    for (int c = by.x; c <= by.y; ++c) top = fmaxf(top, slot(c)[(size_t)ROWS * D + r]);
    const float base = top > kNegInf ? top : 0.0f;
    float sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int c = by.x; c <= by.y; ++c) {
        const float* s = slot(c);
        const float k = ex2(s[(size_t)ROWS * D + r] - base);
        const float4 v = reinterpret_cast<const float4*>(s)[piece * ROWS + r];
        sum = fmaf(k, s[(size_t)ROWS * D + ROWS + r], sum);
        o = make_float4(fmaf(k, v.x, o.x), fmaf(k, v.y, o.y), fmaf(k, v.z, o.z), fmaf(k, v.w, o.w));
    }
    const int64_t out = ((int64_t)b * p.Lq + node) * (p.c.heads * p.G) + head;
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    uint2 w = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (instead != kAsItIs) w.x = w.y = instead == kNothing ? 0u : 0x7FC07FC0u;
    *reinterpret_cast<uint2*>(p.o + out * D + piece * 4) = w;
    if (p.lse && piece == 0)
        p.lse[out] = instead == kNothing ? kNegInf : instead == kNan ? __int_as_float(0x7FC00000) : log_sum_exp(top, sum);
}

template <int D, bool DUAL>
cudaError_t launch(Kv4AttnParams p, int2* items, int sms, cudaStream_t st) {
    constexpr int ROWS = DUAL ? 2 * kTile : kTile;
    const void* kernel = reinterpret_cast<const void*>(tree_attention_kernel<D, DUAL>);
    cudaError_t e = ensure_dynamic_smem(kernel, Shape<D>::kBytes);
    if (e != cudaSuccess) return e;
    p.chunks = fast_div((p.Lq * p.G + ROWS - 1) / ROWS);
    p.group = fast_div(p.G);
    p.page_groups = fast_div(p.c.page / 16);
    e = launch_chained(tree_attention_kernel<D, DUAL>, used_sms(sms), kThreads, Shape<D>::kBytes, st, p, items);
    if (e != cudaSuccess) return e;
    const int row_blocks = (std::min(ROWS, p.Lq * p.G) + kJoinRows - 1) / kJoinRows;
    return launch_chained(join_kernel<D, ROWS>, (unsigned)p.B * p.c.heads * p.chunks.d * row_blocks * (D / 4 / kJoinPieces),
                          kJoinRows * kJoinPieces, 0, st, p, static_cast<const int2*>(items), row_blocks);
}

}  // namespace

// This kernel takes about 25 us for a part's beginning and end (the other about 9), and a quarter to a half of the other's
// time for a row and key.  So: rows that fill at least half of a tile, and work, in 16 rows of 16 keys, worth the difference
// (us, the other / this; rows, sequences x heads, tokens; D = 128 but where said): 64 x 128 of 8200 150/152; 80 x 128 of
// 8200 180/157; 96 x 32 of 4100 45/40, x 128 124/97; 128 x 8 of 8200 34/38, x 64 of 2100 55/42, of 8200 148/92; 147 x 4 of 5000
// (D = 64) 17/34, x 32 55/49; 256 x 8 of 4100 34/36, of 65600 301/114, x 128 of 8200 533/229; 512 x 128 of 350 119/65.  By
// what the pages can hold, as the other's rules: short sequences with a table for long ones pay for its beginning and end.
bool kv4_tree_wide(const Kv4AttnParams& p) {
    const int64_t rows = (int64_t)p.Lq * p.G, groups = std::min(p.room, p.reach) / 16 + 1;
    return rows > kTreeFewRows && (int64_t)p.B * p.c.heads * groups * ((rows + 15) / 16) > 36000;
}

// Bytes: the items' CTAs, then the partials of two slots a CTA.
size_t kv4_tree_items_bytes(int64_t rows, int64_t heads) {
    return (size_t)(heads * ((rows + kTile - 1) / kTile)) * sizeof(int2) / 256 * 256 + 256;
}
size_t kv4_tree_part_floats(int D, int64_t rows, int sms) {
    return (size_t)used_sms(sms) * 2 * (rows > kTile ? 2 * kTile : kTile) * (D + 2);
}

cudaError_t launch_kv4_tree_attention(int D, const Kv4AttnParams& p, void* items, int sms, cudaStream_t st) {
    int2* at = static_cast<int2*>(items);
    const bool dual = p.Lq * p.G > kTile;
    if (D == 64) return dual ? launch<64, true>(p, at, sms, st) : launch<64, false>(p, at, sms, st);
    return dual ? launch<128, true>(p, at, sms, st) : launch<128, false>(p, at, sms, st);
}

}  // namespace r9q
