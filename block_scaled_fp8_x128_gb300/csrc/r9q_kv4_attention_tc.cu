// Attention over the paged 4-bit cache for more than 16 rows of a key-value head
// (drafted tokens, prompts), on the tensor cores' tcgen05 path.  D = 128.
//
// The arithmetic is that of r9q_kv4_attention.cu: products of bare codes, held as fp16
// subnormals, with the pairs applied to scores and weights, and weights against a
// reference that moves rarely.  There, a warp's registers hold the accumulators, which
// ends at 16 rows; here they are in tensor memory and a chunk has R = 32 or 64 rows.  A CTA of
// eight warps takes tiles of 128 keys:
//   S [128 keys x R] = Ck [128 x 128] Q^T       (M = 128, N = R, 8 steps of K = 16)
//   a thread has one key and half of the rows: scores, weights, its share of both sums,
//   O^T [128 elements x R] += Cv^T [128 x 128 keys] P^T
// with both operands of codes written to shared memory as fp16 in turn (the same 32 KB:
// K's are read before V's are written), K-major with the 128-byte swizzle.  The order of the elements
// along K is that in which the masks give them (0 4 1 5 2 6 3 7 of every eight), for
// codes and queries alike; the high nibbles' factor of 16 is taken out of the queries'
// elements 1 5 3 7, and of the rows of O at the end.
//
// What bounds it: instructions and shared memory, about 700 cycles a tile and SM for the
// codes (5 instructions for 8, and 64 KB written) and R = 32 rows (12 instructions a
// score).  Two CTAs an SM overlap one another's barriers and products.
#include "r9q_kv4_attention.cuh"

namespace r9q {

namespace {

constexpr int kD = 128;
constexpr int kTile = 128;                   // keys
constexpr int kThreads = 256;
constexpr int kRow = 80;                     // bytes that 64 bytes of codes take in a stage: no bank conflicts
constexpr int kStage = 2 * kTile * kRow + kTile * 8;       // K, V, pairs of both
constexpr int kOperand = kTile * kD * 2;

// Shared memory, from a 1024-byte boundary: the codes' operand, P, Q, two stages, then this.
template <int R>
struct Small {
    float4 row[R];           // fr, qs (score = fr (sk acc + lk qs)), top, shift (r9q_kv4_attention.cu, State)
    int hi[R], seen[R];      // last key that a row sees; whether it has seen one
    uint32_t most[R];        // of a move: the largest score, in the order of unsigned integers
    int exponent[R];
    float alpha[R];
    float l[4][R], ml[4][R];
    uint64_t s_done, o_done; // products that are complete
    uint32_t tmem;
    float sv_bound;
    int least, failed, joins;
    alignas(8) uint8_t have[2][8];           // groups of a stage that were loaded (read eight at a time)
};
template <int R>
constexpr int small_at() { return kOperand + 2 * R * kD * 2 + 2 * kStage; }
template <int R>
constexpr int smem_bytes() { return 1024 + small_at<R>() + (int)sizeof(Small<R>); }
static_assert(join_bytes(32, kThreads, kJoinRows<32>) <= small_at<32>(), "room to join");
static_assert(join_bytes(64, kThreads, kJoinRows<64>) <= small_at<64>(), "room to join");

// kind::f16 descriptor: D fp32, A and B fp16, both K-major.
constexpr uint32_t idesc_f16(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }
__device__ __forceinline__ void umma_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[128 x R] (+)= A[128 x 128] B[R x 128]^T: operands of two blocks of 64 along K.
template <int R>
__device__ __forceinline__ void product(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t accumulate) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
        umma_f16(tmem_d, umma_sdesc_sw128(a + (k >> 2) * (kTile * 128) + (k & 3) * 32),
                 umma_sdesc_sw128(b + (k >> 2) * (R * 128) + (k & 3) * 32), idesc_f16(128, R),
                 accumulate || k > 0 ? 1u : 0u);
}
template <int NC>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&d)[NC]) {
    static_assert(NC == 16, "tcgen05.st width");
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "f"(d[0]), "f"(d[1]), "f"(d[2]), "f"(d[3]), "f"(d[4]), "f"(d[5]), "f"(d[6]), "f"(d[7]), "f"(d[8]), "f"(d[9]),
        "f"(d[10]), "f"(d[11]), "f"(d[12]), "f"(d[13]), "f"(d[14]), "f"(d[15])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Element k of row `row` of a K-major operand of `rows` rows: the 16-byte chunk of 8 elements.
__device__ __forceinline__ uint32_t chunk_at(int rows, int row, int chunk) {
    return (chunk >> 3) * (rows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Floats in the order of unsigned integers; a NaN is 0, below all.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
    return v != v ? 0u : (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return u == 0 ? kNegInf : __uint_as_float((u >> 31) ? u & 0x7FFFFFFFu : ~u);
}

// A lane's share of a group of 16 tokens (the warp copies what it will convert itself): 64-byte rows kRow apart.
__device__ __forceinline__ void copy_rows(bool live, uint32_t k_dst, const uint8_t* k, uint32_t v_dst, const uint8_t* v,
                                          uint32_t pair_dst, const uint32_t* pair) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
        "@p cp.async.cg.shared.global [%1], [%2], 16;\n\t"
        "@p cp.async.cg.shared.global [%1+640], [%2+512], 16;\n\t"
        "@p cp.async.cg.shared.global [%3], [%4], 16;\n\t"
        "@p cp.async.cg.shared.global [%3+640], [%4+512], 16;\n\t"
        "@p cp.async.ca.shared.global [%5], [%6], 4;\n\t}" ::"r"((int)live),
        "r"(k_dst), "l"(k), "r"(v_dst), "l"(v), "r"(pair_dst), "l"(pair)
        : "memory");
}

template <int R>
__global__ void __launch_bounds__(kThreads, R == 32 ? 2 : 1) kv4_attention_tc_kernel(const Kv4AttnParams p) {
    begin_chained();
    constexpr int H = R / 2;                 // rows of a thread
    constexpr int kCols = 2 * R;             // TMEM: S, then O
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    const uint32_t op = smem_u32(smem), pp = op + kOperand, qq = pp + R * kD * 2, stages = qq + R * kD * 2;
    uint8_t* stage_ptr = smem + kOperand + 2 * R * kD * 2;
    Small<R>& sm = *reinterpret_cast<Small<R>*>(smem + small_at<R>());

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int key = (warp & 3) * 32 + lane;  // the thread's key of a tile, and element of the result
    const int n0 = (warp >> 2) * H;          // its first row
    const int rows = p.Lq * p.G;
    Walk walk;
    if (!walk.start(p, 2 * kTile / 16)) return;

    if (warp == 0) tmem_alloc(&sm.tmem, kCols);
    if (tid == 0) {
        mbar_init(&sm.s_done, 1);
        mbar_init(&sm.o_done, 1);
        fence_mbar_init();
        sm.failed = 0;
    }
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    const uint32_t tmem = sm.tmem, lane_at = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem, to = tmem + R;
    uint32_t s_phase = 0, o_phase = 0;
    bool failed = false;

    const uint8_t* k_lane = p.c.k + lane * 16;
    const uint8_t* v_lane = p.c.v + lane * 16;
    const uint32_t* pair_lane = (lane < 16 ? p.c.kp : p.c.vp) + (lane & 15);
    // stage: [128 K rows][128 V rows][128 K pairs][128 V pairs]; a warp's group is 16 of each
    const uint32_t k_dst = (warp * 16 + (lane >> 2)) * kRow + (lane & 3) * 16, v_dst = kTile * kRow + k_dst;
    const uint32_t pair_dst = 2 * kTile * kRow + (lane >> 4) * (kTile * 4) + (warp * 16 + (lane & 15)) * 4;

    Part it;
    while (walk.next(p, it)) {
        const Span& sp = walk.sp;
        const int chunk0 = it.chunk * R, live = min(R, rows - chunk0);
        const int tiles = (it.g_end - it.g_begin + 7) >> 3;
        const int32_t* table = p.table + (int64_t)it.b * p.max_pages;
        const int gmax = min(it.g_end, (sp.len + 15) >> 4);
        // lane x holds the token index of the warp's group of the x-th of 32 tiles
        auto groups_of = [&](int tile) {
            const int g = it.g_begin + 8 * (tile + lane) + warp;
            return g < gmax ? find_group(p, table, g, it.hk) : kNoGroup;
        };
        uint32_t groups = groups_of(0);
        auto issue = [&](int tile) {
            if (tile > 0 && (tile & 31) == 0) groups = groups_of(tile);
            const uint32_t at = __shfl_sync(0xffffffffu, groups, tile & 31), st = stages + (tile & 1) * kStage;
            const bool have = at != kNoGroup;
            if (lane == 0) sm.have[tile & 1][warp] = have;
            copy_rows(have, st + k_dst, k_lane + (uint64_t)at * (kD / 2), st + v_dst, v_lane + (uint64_t)at * (kD / 2),
                      st + pair_dst, pair_lane + at);
            cp_commit();
        };
        issue(0);

        // ---- queries: an operand, scaled by a power of two per row (r9q_kv4_attention.cu) ----
        {
            constexpr int TPR = kThreads / R, WORDS = kD / 8 / TPR;      // threads of a row; eights of a thread
            const int n = tid / TPR, part = tid % TPR, row = chunk0 + n;
            uint4 raw[WORDS];
#pragma unroll
            for (int i = 0; i < WORDS; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows) {
                const int i = row / p.group, head = it.hk * p.G + (row - i * p.G);
                const uint4* src = reinterpret_cast<const uint4*>(p.q + it.b * p.q_bs + i * p.q_ts + head * p.q_hs) +
                                   part * WORDS;
#pragma unroll
                for (int k = 0; k < WORDS; ++k) raw[k] = src[k];
            }
            float sum = 0.0f;
            uint32_t big = 0;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    big = __vmaxu2(big, w[k] & 0x7FFF7FFFu);
                    sum += bf16_lo(w[k]) + bf16_hi(w[k]);
                }
            }
            big = max(big >> 16, big & 0xFFFFu);
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) {
                big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            const int e = (int)(big >> 7), up = e == 0 ? 0 : min(13 - (e - 127), 100);
            const float f = __uint_as_float((uint32_t)(127 + up) << 23), f16 = f * 0.0625f;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                sts16(qq + chunk_at(R, n, part * WORDS + i), pack_f16x2(bf16_lo(w[0]) * f, bf16_lo(w[2]) * f),
                      pack_f16x2(bf16_hi(w[0]) * f16, bf16_hi(w[2]) * f16),
                      pack_f16x2(bf16_lo(w[1]) * f, bf16_lo(w[3]) * f),
                      pack_f16x2(bf16_hi(w[1]) * f16, bf16_hi(w[3]) * f16));
            }
            if (part == 0) {
                const float over = __uint_as_float((uint32_t)(127 - up) << 23);
                sm.row[n] = make_float4(fminf(p.scale_log2 * over * 0x1p24f, 3e38f), sum * f * 0x1p-24f, 0.0f,
                                        (float)(kHeadroom + 127 - kMinExponent));
                sm.hi[n] = sp.len - p.Lq + min(row, rows - 1) / p.group;
                sm.seen[n] = 0;
            }
            if (tid == 0) sm.sv_bound = -1.0f;               // the first tile moves the references
        }
        const int all_hi = sp.len - p.Lq + chunk0 / p.group;
        const int last_hi = sp.len - p.Lq + (min(rows, chunk0 + R) - 1) / p.group;
        const int window = p.window > 0 ? p.window : kNoWindow;

        float l[H], ml[H];
#pragma unroll
        for (int i = 0; i < H; ++i) l[i] = ml[i] = 0.0f;

        for (int tile = 0; tile < tiles; ++tile) {
            const uint8_t* stp = stage_ptr + (tile & 1) * kStage;
            cp_wait<0>();
            __syncwarp();
            if (tile > 0) {                                  // the last tile's product has read the operand and P
                if (!mbar_wait(&sm.o_done, o_phase)) sm.failed = 1;
                o_phase ^= 1;
            }
            // ---- K's codes ----
            {
                const int r0 = warp * 16 + (lane & 7), j = lane >> 3;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = r0 + 8 * h;
                    const uint4 v = *reinterpret_cast<const uint4*>(stp + row * kRow + j * 16);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x = w[i] >> 8;
                        sts16(op + chunk_at(kTile, row, 4 * j + i), w[i] & 0x000F000Fu, w[i] & 0x00F000F0u,
                              x & 0x000F000Fu, x & 0x00F000F0u);
                    }
                }
            }
            fence_proxy_async_smem();
            umma_fence_before();
            __syncthreads();
            failed = sm.failed;
            if (failed) break;
            if (tid == 0) {
                umma_fence_after();
                product<R>(ts, op, qq, 0);
                umma_commit(&sm.s_done);
            }
            if (tile + 1 < tiles) issue(tile + 1);

            // ---- the thread's key ----
            const int key0 = (it.g_begin + 8 * tile) << 4, at = key0 + key;
            const uint2 have8 = *reinterpret_cast<const uint2*>(sm.have[tile & 1]);
            const bool have = sm.have[tile & 1][key >> 4];
            const bool plain = have8.x == 0x01010101u && have8.y == 0x01010101u && key0 > last_hi - window &&
                               key0 + kTile - 1 <= all_hi;
            const uint32_t* pairs = reinterpret_cast<const uint32_t*>(stp + 2 * kTile * kRow);
            uint32_t kq = pairs[key], vq = pairs[kTile + key];
            if (!have || at >= sp.len) kq = vq = 0u;
            const float sk = bf16_lo(kq), lk = bf16_hi(kq), sv = bf16_lo(vq), lv = bf16_hi(vq);

            float v[H];
            if (!mbar_wait(&sm.s_done, s_phase)) sm.failed = 1;
            s_phase ^= 1;
            umma_fence_after();
            tmem_ld<H>(ts + lane_at + n0, v);
            tmem_wait_ld(v);

            // ---- scores over fr, and whether the references hold ----
            bool move = !plain || fmaxf(sv, fabsf(lv) * kLowestShare) > sm.sv_bound;
            float far = kNegInf;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float4 row = sm.row[n0 + i];
                float s = fmaf(sk, v[i], lk * row.y);
                if (!plain) {
                    const int hi = sm.hi[n0 + i];
                    if (!have || at > hi || at <= hi - window) s = kNegInf;
                }
                v[i] = s;
                far = fmaxf(far, (s - row.z) * row.x);
            }
            move = move || far > (float)kSlack;
            if (__syncthreads_or(move)) {
                if (tid < R) {
                    sm.most[tid] = 0;
                    sm.exponent[tid] = 0;
                    if (tid == 0) sm.least = 255;
                }
                __syncthreads();
                const int xs = (int)(vq >> 7) & 255, xl = (int)(vq >> 23) & 255;
                const int ek = xs == 255 || xl == 255 ? 0 : max(xs, xl - kLowestBits);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const uint32_t most = __reduce_max_sync(0xffffffffu, ordered(v[i]));
                    const int e = __reduce_max_sync(0xffffffffu, v[i] != kNegInf ? ek : 0);
                    if (lane == 0) {
                        atomicMax(&sm.most[n0 + i], most);
                        atomicMax(&sm.exponent[n0 + i], e);
                    }
                }
                __syncthreads();
                if (tid < R) {
                    float4 row = sm.row[tid];
                    const bool seen = sm.seen[tid];
                    const float x = fmaxf(unordered(sm.most[tid]), seen ? row.z : kNegInf);
                    const int e = max(sm.exponent[tid], kHeadroom + 127 - (int)row.w);
                    const float shift = (float)(kHeadroom + 127 - e);
                    float alpha = 0.0f;
                    if (x > kNegInf) {
                        if (seen) alpha = ex2(fmaf(row.z - x, row.x, shift - row.w));
                        sm.seen[tid] = 1;
                        row.z = x;
                    }
                    row.w = shift;
                    sm.row[tid] = row;
                    sm.alpha[tid] = alpha;
                    atomicMin(&sm.least, e);
                }
                __syncthreads();
                if (tid == 0) sm.sv_bound = __uint_as_float((uint32_t)(sm.least + 1) << 23);   // (read after the next barrier)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float alpha = sm.alpha[n0 + i];
                    l[i] *= alpha;
                    ml[i] *= alpha;
                }
                if (tile > 0) {
#pragma unroll
                    for (int c = 0; c < H; c += 16) {
                        float o[16];
                        tmem_ld<16>(to + lane_at + n0 + c, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= sm.alpha[n0 + c + i];
                        tmem_st<16>(to + lane_at + n0 + c, o);
                    }
                }
            }

            // ---- weights ----
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float4 row = sm.row[n0 + i];
                const float pr = ex2(fmaf(v[i] - row.z, row.x, row.w));
                float w = pr * sv, add = pr * lv;
                if (!plain && v[i] == kNegInf) w = add = 0.0f;              // not 0 * infinity
                l[i] += pr;
                ml[i] += add;
                const uint32_t h = pack_f16x2(w, 0.0f);
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(pp + chunk_at(R, n0 + i, key >> 3) + (key & 7) * 2),
                             "h"((uint16_t)h)
                             : "memory");
            }
            // ---- V's codes, in the place of K's ----
            {
                const int r = lane & 7, half = (lane >> 3) & 1, c = lane >> 4;
                const uint8_t* src = stp + kTile * kRow + (warp * 16 + c * 8 + r) * kRow + half * 8;
                uint2 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint2*>(src + j * 16);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int d = 64 * c + 16 * (2 * half + m) + r;
                    uint32_t x[4], y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[j] = m == 0 ? w[j].x : w[j].y;
                        y[j] = x[j] >> 8;
                    }
                    // tokens 0..7 and 8..15 of the group, elements d and d + 8
                    sts16(op + chunk_at(kD, d, 2 * warp), x[0] & 0x000F000Fu, x[1] & 0x000F000Fu, x[2] & 0x000F000Fu,
                          x[3] & 0x000F000Fu);
                    sts16(op + chunk_at(kD, d, 2 * warp + 1), y[0] & 0x000F000Fu, y[1] & 0x000F000Fu,
                          y[2] & 0x000F000Fu, y[3] & 0x000F000Fu);
                    sts16(op + chunk_at(kD, d + 8, 2 * warp), x[0] & 0x00F000F0u, x[1] & 0x00F000F0u,
                          x[2] & 0x00F000F0u, x[3] & 0x00F000F0u);
                    sts16(op + chunk_at(kD, d + 8, 2 * warp + 1), y[0] & 0x00F000F0u, y[1] & 0x00F000F0u,
                          y[2] & 0x00F000F0u, y[3] & 0x00F000F0u);
                }
            }
            fence_proxy_async_smem();
            umma_fence_before();
            __syncthreads();
            failed = sm.failed;
            if (failed) break;
            if (tid == 0) {
                umma_fence_after();
                product<R>(to, op, pp, tile > 0);
                umma_commit(&sm.o_done);
            }
        }
        cp_wait<0>();
        if (failed) break;

        // ---- the sums over the keys of a row ----
        if (!mbar_wait(&sm.o_done, o_phase)) sm.failed = 1;
        o_phase ^= 1;
        umma_fence_after();
#pragma unroll
        for (int i = 0; i < H; ++i) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
                ml[i] += __shfl_xor_sync(0xffffffffu, ml[i], o);
            }
            if (lane == 0) {
                sm.l[warp & 3][n0 + i] = l[i];
                sm.ml[warp & 3][n0 + i] = ml[i];
            }
        }
        __syncthreads();
        failed = sm.failed;
        if (failed) break;
        const float unscale = key & 8 ? 0x1p20f : 0x1p24f;
        float* part = partial_of<kD, R>(p, blockIdx.x, it.begins);
#pragma unroll
        for (int c = 0; c < H; c += 16) {
            float o[16];
            tmem_ld<16>(to + lane_at + n0 + c, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int n = n0 + c + i;
                if (n >= live) break;
                const float sum = (sm.l[0][n] + sm.l[1][n]) + (sm.l[2][n] + sm.l[3][n]);
                const float low = (sm.ml[0][n] + sm.ml[1][n]) + (sm.ml[2][n] + sm.ml[3][n]);
                const float x = fmaf(o[i], unscale, low);
                const float4 row = sm.row[n];
                const float top = sm.seen[n] ? fmaf(row.z, row.x, -row.w) : kNegInf;
                if (it.whole) {
                    const int grow = chunk0 + n, q = grow / p.group;
                    const int64_t out = ((int64_t)it.b * p.Lq + q) * (p.c.heads * p.G) + it.hk * p.G + (grow - q * p.G);
                    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
                    p.o[out * kD + key] = (uint16_t)pack_bf16x2(x * inv, 0.0f);
                    if (p.lse && key == 0) p.lse[out] = log_sum_exp(top, sum);
                } else {
                    part[n * kD + key] = x;
                    if (key == 0) {
                        part[R * kD + n] = top;
                        part[R * kD + R + n] = sum;
                    }
                }
            }
        }
        umma_fence_before();
        if (!it.whole) {
            int c0, c1;
            walk.sharers(c0, c1);
            __syncthreads();
            if (tid == 0) {
                const bool last = arrive(p.done + c0) == c1 - c0;
                if (last) p.done[c0] = 0;
                sm.joins = last;
            }
            __syncthreads();
            if (sm.joins) join_partials<kD, R, kThreads>(p, it, c0, c1, live, reinterpret_cast<float*>(smem));
        }
        if (walk.parted) break;
        __syncthreads();                     // shared memory is free for the next item
    }
    cp_wait<0>();
    if (failed) {
        if (tid == 0) record_error(p.err, kErrTimeout);
        // what was issued may still be on its way: give it as long again before its memory is let go
        (void)mbar_wait(&sm.s_done, s_phase);
        (void)mbar_wait(&sm.o_done, o_phase);
    }
    umma_fence_before();
    __syncthreads();
    if (warp == 0) {
        umma_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

template <int R>
cudaError_t launch(Kv4AttnParams p, int sms, cudaStream_t st) {
    p.chunks = fast_div((p.Lq * p.G + R - 1) / R);
    p.group = fast_div(p.G);
    p.page_groups = fast_div(p.c.page / 16);
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kv4_attention_tc_kernel<R>), smem_bytes<R>());
    if (e != cudaSuccess) return e;
    return launch_chained(kv4_attention_tc_kernel<R>, used_sms(sms) * kv4_attention_tc_ctas(R), kThreads,
                          smem_bytes<R>(), st, p);
}

}  // namespace

cudaError_t launch_kv4_attention_tc(const Kv4AttnParams& p, int sms, cudaStream_t st) {
    return launch<32>(p, sms, st);
}

}  // namespace r9q
