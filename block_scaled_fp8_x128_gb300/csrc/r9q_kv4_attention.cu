// Attention of a few new tokens per sequence over the paged 4-bit cache.
//
// Rows are the new tokens' query heads that share a key-value head (Lq x G of
// them); 8 NT rows make a chunk.  With keys k = lk + sk ck and values
// v = lv + sv cv (c the 4-bit codes, one pair per token)
//   score = scale (sk (q . ck) + lk sum(q)),   o = (sum (p sv) cv + sum p lv) / sum p,
// so both products run on the bare codes and the pairs act on scores and
// weights.  Products are transposed, tokens or elements as the 16 rows of an
// m16n8k16 fp16 product and query rows as its 8 columns:
//   S^T [16 tokens x 8 rows] += Ck [16 x D] Q^T,   O^T [D x 8 rows] += Cv^T [D x 16 tokens] P^T,
// which wastes nothing for eight rows and takes each code through the registers
// once.  A code in the low bits of an fp16 is the subnormal c 2^-24, exactly, and
// tensor cores take subnormals: fragments come out of the packed bytes with one
// mask each and one shift for every two (w & 0x000F000F, w & 0x00F000F0, the same
// of w >> 8).  The high nibbles weigh 16 times the low ones; for K that is taken
// out of the query's elements, for V (where they are rows of their own) at the end.
// The queries are scaled by a power of two per row to a largest element in
// [2^13, 2^14), where fp16 holds bf16 values exactly down to 2^-27 of it.  The
// weights P sv are rounded to fp16 (11 bits; bf16 would keep 8).  What a weight loses counts
// with the code's distance from 7.5, half of what it would from 0: with w the rounded weight
//   sum (p sv) c + sum p lv  is formed as  sum w c + sum (p (lv + 7.5 sv) - 7.5 w).
// Tensor cores cut an accumulator's low bits off, always towards zero, which in a sum of
// codes, none negative, adds up over a long sequence.  So every second group of 16 keys has
// weights of the other sign and codes 15 - c (the same mask, of the complement): the sum stays
// near zero and the cuts cancel.  131072 tokens, error before the result's rounding: 1.9e-4 of
// the result, with plain sums 8.0e-4; it costs 1.5 % of the time.  To keep them in
// its range a row's weights are taken not against its largest score alone but against
// largest score - 8 + E, E the exponent of the largest step its keys have had.  This
// reference moves only when a weight passes it by 2^6 (or a step is larger than any
// before): weights stay under 2^15, 2^-22 of the largest still has full precision, and
// most steps neither reduce a maximum over the warp nor touch the accumulators.
// Both sums use the same weights, so the power of two cancels.  Scores, maxima,
// sums and accumulators are fp32.
//
// The warps of a CTA take 32-key steps of a part in turn, each with its own reference,
// and meet in shared memory at its end.
//
// Lanes copy exactly the bytes they will use (cp.async, 16 bytes, a ring of stages in
// shared memory per warp), so a stage needs no barrier.
//
// What bounds it.  Up to 8 rows: HBM (136 bytes a token and head at D = 128) and the
// taking apart of the codes, 64 masks for 16 tokens of a head, alike: 64 sequences of up
// to 16384 tokens, 64/8 heads, take 108 us, 5.4 TB/s (the bytes alone 87).  More rows:
// latency at low occupancy, eight warps an SM of 255 registers, 44 % of the issue slots (16
// sequences of 8191 tokens with 4 new ones 82 us, 208 TFLOP/s; the products alone 29), and
// every chunk takes the codes apart again.  Small batches:
// latency, about 5.7 us from launch to the result for one short sequence, and with
// parts to join about 9.  A prompt's chunks each walk the whole sequence: the keys past a
// chunk's last row, or before its window, are masked and not left out.
// A step's score products formed before the last step's weights, and
// the queries in shared memory for a third more warps, were slower (113 and 97 us,
// against 108 and 81).  So was tcgen05 with the codes as an operand in tensor memory, for 32
// rows: 103 us against 81, since converting them and two barriers a tile of 128 keys cost
// more than the products save.
#include <algorithm>

#include "r9q_kv4_attention.cuh"

namespace r9q {

namespace {

constexpr int kStep = 32;                    // keys a warp takes at a time: two groups of 16
constexpr int kStages = 4;                   // steps in a warp's ring (three, and a CTA more an SM: 128 us against 115)

// The warps that an SM holds (registers) make CTAs of two or four, or one CTA.
enum Width { kNarrow, kMiddle, kWide };
constexpr int sm_warps(int D, int NT) { return 4 * ((D == 64 ? 4 : 3) - (NT - 1)); }
constexpr int cta_warps(int D, int NT, Width w) { return w == kWide ? sm_warps(D, NT) : w == kMiddle ? 4 : 2; }
constexpr int ctas_per_sm(int D, int NT, Width w) { return sm_warps(D, NT) / cta_warps(D, NT, w); }

// Groups of a CTA that take as long as beginning and ending an item.
constexpr int item_cost(int NT, Width w) { return NT == 1 && w == kNarrow ? 16 : 24; }
constexpr int stage_bytes(int D) { return kStep * D + kStep * 8; }
constexpr int out_stride(int D) { return D + 4; }      // floats a row of the CTA's exchange takes
// Shared memory: the rings, and in their place the warps' exchange [warps][R][out_stride] with references and sums,
// and the joining of partials.
constexpr int work_bytes(int D, int NT, Width width) {
    const int w = cta_warps(D, NT, width), R = 8 * NT;
    return largest(largest(w * kStages * stage_bytes(D), w * R * (out_stride(D) + 2) * 4), join_bytes(R, w * 32));
}
constexpr int smem_bytes(int D, int NT, Width w) { return work_bytes(D, NT, w) + 16; }   // and a flag

// Transposes an 8x8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A warp's state for NT tiles of 8 rows; a lane has columns (rows of the query)
// 2j and 2j + 1 of each.
template <int D, int NT>
struct State {
    uint32_t qf[NT][D / 16][2];              // query fragments
    float fr[NT][2], qs[NT][2];              // score = fr (sk acc + lk qs)
    int hi[NT][2];                           // the last key that the column sees
    float acc[NT][D / 16][4], l[NT][2], ml[NT][2];
    // A weight is 2^((score - top) + shift) with the largest score and the values' exponent of the last move; taken
    // as a difference first, so that it holds for scores of any size.
    float top[NT][2], shift[NT][2];          // (top over fr, 0 while the column has seen no key; shift 8 - exponent)
    float bound[NT][2], sv_bound;            // when to move: a lane's weights of a step, a step (or share of a lowest)
    uint32_t seen;                           // columns that have seen a key
};

// Takes the columns' references to the largest score and the largest values they have
// seen, this step's included, and what was summed against the old ones with them.
template <int D, int NT, bool MASKED>
__device__ __forceinline__ void move_reference(State<D, NT>& s, const float (&sc)[NT][2][4],
                                               const uint32_t (&vq)[2][2]) {
    int ek[2][2];                            // the exponent of a key's values; none for a pair that is not finite
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int xs = (int)(vq[i][h] >> 7) & 255, xl = (int)(vq[i][h] >> 23) & 255;
            ek[i][h] = xs == 255 || xl == 255 ? 0 : max(xs, xl - kLowestBits);
        }
    int es_min = 255;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t bit = 1u << (2 * nt + c);
            float x = max3(max3(sc[nt][0][c], sc[nt][0][c + 2], sc[nt][1][c]), sc[nt][1][c + 2],
                           s.seen & bit ? s.top[nt][c] : kNegInf);
            int e = kHeadroom + 127 - (int)s.shift[nt][c];     // only of keys that the column sees
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (!MASKED || sc[nt][i][2 * h + c] != kNegInf) e = max(e, ek[i][h]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                e = max(e, __shfl_xor_sync(0xffffffffu, e, o));
            }
            float alpha = 0.0f;              // nothing seen before: the sums are zero
            s.bound[nt][c] = 0.0f;           // (nothing seen now either: no weight is over 0)
            const float shift = (float)(kHeadroom + 127 - e);
            if (x > kNegInf) {
                if (s.seen & bit) alpha = ex2(fmaf(s.top[nt][c] - x, s.fr[nt][c], shift - s.shift[nt][c]));
                s.seen |= bit;
                s.top[nt][c] = x;
                s.bound[nt][c] = ex2(shift + kSlack);
            }
            s.shift[nt][c] = shift;
            es_min = min(es_min, e);
            s.l[nt][c] *= alpha;
            s.ml[nt][c] *= alpha;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
                s.acc[nt][t][c] *= alpha;
                s.acc[nt][t][c + 2] *= alpha;
            }
        }
    s.sv_bound = __uint_as_float((uint32_t)(es_min + 1) << 23);          // the next power of two
}

// One step: 32 keys in the stage `st`, of which groups `bits` were loaded.
// MASKED: some column does not see some key, or a group is missing.
template <int D, int NT, bool MASKED>
__device__ __forceinline__ void attend(State<D, NT>& s, const uint8_t* st, int key0, uint32_t bits, int len,
                                       int window, int lane) {
    constexpr int KW = D / 32;
    const int r = lane >> 2;
    // pairs of the lane's keys r + 8h of group i
    const uint4 kp = *reinterpret_cast<const uint4*>(st + kStep * D + r * 16);
    uint4 vp = *reinterpret_cast<const uint4*>(st + kStep * D + kStep * 4 + r * 16);
    uint32_t kq[2][2] = {{kp.x, kp.y}, {kp.z, kp.w}}, vq[2][2] = {{vp.x, vp.y}, {vp.z, vp.w}};
    if (MASKED) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (!((bits >> i) & 1u) || key0 + 16 * i + 8 * h + r >= len) kq[i][h] = vq[i][h] = 0u;
    }

    // ---- scores over fr ----
    float sc[NT][2][4];
    uint32_t k0[2][KW], k1[2][KW];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint8_t* kb = st + i * 16 * (D / 2) + lane * (KW * 4);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            k0[i][w] = reinterpret_cast<const uint32_t*>(kb)[w];
            k1[i][w] = reinterpret_cast<const uint32_t*>(kb + 8 * (D / 2))[w];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[nt][i][c] = 0.0f;
    }
    // (the products that add to one accumulator lie apart, so that they need not wait for one another)
#pragma unroll
    for (int w = 0; w < KW; ++w) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(sc[nt][i], k0[i][w] & 0x000F000Fu, k1[i][w] & 0x000F000Fu, k0[i][w] & 0x00F000F0u,
                              k1[i][w] & 0x00F000F0u, s.qf[nt][2 * w][0], s.qf[nt][2 * w][1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t x0 = k0[i][w] >> 8, x1 = k1[i][w] >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(sc[nt][i], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x00F000F0u,
                              s.qf[nt][2 * w + 1][0], s.qf[nt][2 * w + 1][1]);
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t pair = kq[i][c >> 1];
                float v = fmaf(bf16_lo(pair), sc[nt][i][c], bf16_hi(pair) * s.qs[nt][c & 1]);
                if (MASKED) {
                    const int key = key0 + 16 * i + 8 * (c >> 1) + r;
                    if (key > s.hi[nt][c & 1] || key <= s.hi[nt][c & 1] - window || !((bits >> i) & 1u)) v = kNegInf;
                }
                sc[nt][i][c] = v;
            }

    // ---- weights, once the reference holds ----
    // It does while no step is larger than any before, and no weight passes its bound; weights are not negative, so
    // a lane checks the sum of its four of a column, which it needs in any case.
    const float sv_max = max3(max3(bf16_lo(vq[0][0]), bf16_lo(vq[0][1]), bf16_lo(vq[1][0])), bf16_lo(vq[1][1]),
                              max3(fabsf(bf16_hi(vq[0][0])), fabsf(bf16_hi(vq[0][1])),
                                   max3(fabsf(bf16_hi(vq[1][0])), fabsf(bf16_hi(vq[1][1])), 0.0f)) * kLowestShare);
    bool move = MASKED || sv_max > s.sv_bound;
    float pr[NT][2][4], sum[NT][2];
    auto weigh = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        pr[nt][i][2 * h + c] =
                            ex2(fmaf(sc[nt][i][2 * h + c] - s.top[nt][c], s.fr[nt][c], s.shift[nt][c]));
                sum[nt][c] = (pr[nt][0][c] + pr[nt][0][c + 2]) + (pr[nt][1][c] + pr[nt][1][c + 2]);
                move = move || sum[nt][c] > s.bound[nt][c];
            }
    };
    weigh();
    if (__any_sync(0xffffffffu, move)) {
        move_reference<D, NT, MASKED>(s, sc, vq);
        weigh();
    }
    uint32_t pf[NT][2][2];
    float mid[2][2];                         // the value in the middle of the codes
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) mid[i][h] = fmaf(7.5f, bf16_lo(vq[i][h]), bf16_hi(vq[i][h]));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) s.l[nt][c] += sum[nt][c];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float sv = bf16_lo(vq[i][h]), mv = mid[i][h];
                    if (MASKED && sc[nt][i][2 * h + c] == kNegInf) sv = mv = 0.0f;      // not 0 * infinity
                    w[c] = pr[nt][i][2 * h + c] * (i ? -sv : sv);
                    s.ml[nt][c] = fmaf(pr[nt][i][2 * h + c], mv, s.ml[nt][c]);
                }
                const uint32_t both = pack_f16x2(w[0], w[1]);
                less_mid(s.ml[nt][0], s.ml[nt][1], both);
                pf[nt][i][h] = transpose_8x8(both);
            }
    }

    // ---- values: the codes of the first group, 15 less those of the second with weights of the other sign ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t flip = i ? 0xFFFFFFFFu : 0u;
        const uint8_t* vb = st + kStep * (D / 2) + i * 16 * (D / 2) + lane * 16;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(vb + c * 512);
            const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t x = q[m] ^ flip, y = (q[m] >> 8) ^ flip;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16_16816(s.acc[nt][4 * c + m], x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu,
                                  y & 0x00F000F0u, pf[nt][i][0], pf[nt][i][1]);
            }
        }
    }
}

template <int D, int NT, Width WIDTH>
__global__ void __launch_bounds__(32 * cta_warps(D, NT, WIDTH), ctas_per_sm(D, NT, WIDTH))
    kv4_attention_kernel(const Kv4AttnParams p) {
    constexpr int W = cta_warps(D, NT, WIDTH), kThreads = 32 * W;
    constexpr int KW = D / 32;               // 32-bit words of a key that a lane holds
    constexpr int MT = D / 16;               // 16-element tiles
    constexpr int R = 8 * NT;                // rows of a chunk
    constexpr int ST = kStages;
    constexpr int kMinGroups = 2 * W;        // groups a CTA takes at least: one step for each warp
    extern __shared__ __align__(16) uint8_t smem[];
    begin_chained();
    int* joins = reinterpret_cast<int*>(smem + work_bytes(D, NT, WIDTH));     // the CTA joins an item's partials

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, j = lane & 3;
    const int rows = p.Lq * p.G;
    Walk walk;
    if (!walk.start(p, kMinGroups, item_cost(NT, WIDTH))) return;
    uint8_t* ring = smem + warp * (ST * stage_bytes(D));
    const uint32_t ring_u = smem_u32(ring);
    const uint8_t* k_lane = p.c.k + lane * (KW * 4);
    const uint8_t* v_lane = p.c.v + lane * 16;
    const uint32_t* pair_lane = (lane < 16 ? p.c.kp : p.c.vp) + (lane & 15);
    const uint32_t pair_dst = kStep * D + (lane >> 4) * (kStep * 4) + ((lane & 7) * 4 + ((lane >> 3) & 1)) * 4;

    Part it;
    while (walk.next(p, it)) {
        const Span& sp = walk.sp;
        const int b = it.b, hk = it.hk, chunk = it.chunk, g_begin = it.g_begin, g_end = it.g_end;

        // ---- the warp's steps ----
        const int steps_all = (g_end - g_begin + 1) >> 1;
        const int steps = steps_all > warp ? (steps_all - warp + W - 1) / W : 0;
        const int32_t* table = p.table + (int64_t)b * p.max_pages;
        const int gmax = min(g_end, (sp.len + 15) >> 4);
        // Lane x holds the cache's token index of the x-th group of the next 16 steps, and of the 16 after them.
        auto groups_of = [&](int first_step) {
            const int g = g_begin + 2 * ((first_step + (lane >> 1)) * W + warp) + (lane & 1);
            return g < gmax ? find_group(p, table, g, hk) : kNoGroup;
        };
        uint32_t groups_now = 0, groups_next = groups_of(0);

        // ---- query fragments and this lane's two columns of every tile ----
        State<D, NT> s;
        s.sv_bound = -1.0f;                  // the first step moves the references
        s.seen = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = chunk * R + nt * 8 + r;
            uint32_t raw[D / 8];
            if (row < rows) {
                const int i = row / p.group, head = hk * p.G + (row - i * p.G);
                const uint4* src = reinterpret_cast<const uint4*>(p.q + b * p.q_bs + i * p.q_ts + head * p.q_hs +
                                                                  j * (D / 4));
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint4 v = src[x];
                    raw[4 * x] = v.x;
                    raw[4 * x + 1] = v.y;
                    raw[4 * x + 2] = v.z;
                    raw[4 * x + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int x = 0; x < D / 8; ++x) raw[x] = 0;
            }
            float sum = 0.0f;
            uint32_t big = 0;
#pragma unroll
            for (int x = 0; x < D / 8; ++x) {
                big = __vmaxu2(big, raw[x] & 0x7FFF7FFFu);
                sum += bf16_lo(raw[x]) + bf16_hi(raw[x]);
            }
            big = max(big >> 16, big & 0xFFFFu);           // the largest magnitude, as bf16 bits
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            // power of two that brings it to [2^13, 2^14); 1 for a row of zeros
            const int e = (int)(big >> 7);
            const int up = e == 0 ? 0 : min(13 - (e - 127), 100);
            const float f = __uint_as_float((uint32_t)(127 + up) << 23), f16 = f * 0.0625f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                // elements 8w .. 8w+7 of the lane's quarter; a word's bytes 0 and 2 give 0, 4 (low) and 1, 5 (high),
                // bytes 1 and 3 give 2, 6 and 3, 7
                const uint32_t* q = raw + 4 * w;
                s.qf[nt][2 * w][0] = pack_f16x2(bf16_lo(q[0]) * f, bf16_lo(q[2]) * f);
                s.qf[nt][2 * w][1] = pack_f16x2(bf16_hi(q[0]) * f16, bf16_hi(q[2]) * f16);
                s.qf[nt][2 * w + 1][0] = pack_f16x2(bf16_lo(q[1]) * f, bf16_lo(q[3]) * f);
                s.qf[nt][2 * w + 1][1] = pack_f16x2(bf16_hi(q[1]) * f16, bf16_hi(q[3]) * f16);
            }
            const float over = __uint_as_float((uint32_t)(127 - up) << 23);       // 1 / f
            const float row_fr = fminf(p.scale_log2 * over * 0x1p24f, 3e38f), row_qs = sum * f * 0x1p-24f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = 2 * j + c;
                s.fr[nt][c] = __shfl_sync(0xffffffffu, row_fr, col * 4);
                s.qs[nt][c] = __shfl_sync(0xffffffffu, row_qs, col * 4);
                const int ci = min(chunk * R + nt * 8 + col, rows - 1) / p.group;
                s.hi[nt][c] = sp.len - p.Lq + ci;
                s.top[nt][c] = s.bound[nt][c] = s.l[nt][c] = s.ml[nt][c] = 0.0f;
                s.shift[nt][c] = (float)(kHeadroom + 127 - kMinExponent);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) s.acc[nt][t][c] = 0.0f;
        }
        // keys that all rows of the chunk see
        const int i_first = chunk * R / p.group, i_last = (min(rows, chunk * R + R) - 1) / p.group;
        const int all_hi = sp.len - p.Lq + i_first, all_lo = p.window > 0 ? sp.len - p.Lq + i_last - p.window + 1 : 0;

        const int window = p.window > 0 ? p.window : kNoWindow;
        uint32_t have = 0;                   // two bits a step in flight: which of its groups were loaded
        uint32_t put = ring_u;               // stage that is loaded next
        const uint8_t* get = ring;           // stage that is used next
        for (int n = 1 - ST; n < steps; ++n) {
            if (n >= 0) {
                cp_wait<ST - 2>();
                __syncwarp();
            }
            const int ahead = n + ST - 1;
            const uint32_t bits = have >> (2 * (ST - 2)) & 3u;
            have <<= 2;
            if (ahead < steps) {
                if ((ahead & 15) == 0) {
                    groups_now = groups_next;
                    if (ahead + 16 < steps) groups_next = groups_of(ahead + 16);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t at = __shfl_sync(0xffffffffu, groups_now, 2 * (ahead & 15) + i);
                    const bool live = at != kNoGroup;
                    have |= live ? 1u << i : 0u;
                    copy_group<D>(live, put + i * 16 * (D / 2) + lane * (KW * 4), k_lane + (uint64_t)at * (D / 2),
                                  put + kStep * (D / 2) + i * 16 * (D / 2) + lane * 16, v_lane + (uint64_t)at * (D / 2),
                                  put + pair_dst + i * 8, pair_lane + at);
                }
                put = put == ring_u + (ST - 1) * stage_bytes(D) ? ring_u : put + stage_bytes(D);
            }
            cp_commit();
            if (n < 0) continue;
            const int key0 = (g_begin + 2 * (n * W + warp)) << 4;
            if (bits == 3u && key0 >= all_lo && key0 + kStep - 1 <= all_hi)
                attend<D, NT, false>(s, get, key0, bits, sp.len, window, lane);
            else
                attend<D, NT, true>(s, get, key0, bits, sp.len, window, lane);
            get = get == ring + (ST - 1) * stage_bytes(D) ? ring : get + stage_bytes(D);
        }
        cp_wait<0>();

        // ---- the warps' sums meet ----
        __syncthreads();                     // the ring is free
        float* ex_m = reinterpret_cast<float*>(smem);                  // [W][R] references
        float* ex_l = ex_m + W * R;
        float* ex_o = ex_l + W * R;                               // [W][R][out_stride]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = s.l[nt][c], ml = s.ml[nt][c];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    l += __shfl_xor_sync(0xffffffffu, l, o);
                    ml += __shfl_xor_sync(0xffffffffu, ml, o);
                }
                const int row = nt * 8 + 2 * j + c;
                if (r == 0) {
                    ex_m[warp * R + row] =
                        s.seen >> (2 * nt + c) & 1u ? fmaf(s.top[nt][c], s.fr[nt][c], -s.shift[nt][c]) : kNegInf;
                    ex_l[warp * R + row] = l;
                }
                float* o = ex_o + (warp * R + row) * out_stride(D);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    o[16 * t + r] = fmaf(s.acc[nt][t][c], 0x1p24f, ml);
                    o[16 * t + 8 + r] = fmaf(s.acc[nt][t][c + 2], 0x1p20f, ml);
                }
            }
        __syncthreads();

        const int live = min(R, rows - chunk * R);
        // a thread takes four elements of every (kThreads / (D / 4))-th row
        const int ed = (tid % (D / 4)) * 4, row0 = tid / (D / 4);
        constexpr int ROWS = kThreads / (D / 4);
        float* part = partial_of<D, R>(p, blockIdx.x, it.begins);
#pragma unroll 1
        for (int row = row0; row < live; row += ROWS) {
            float top = kNegInf, sum = 0.0f;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < W; ++w) top = fmaxf(top, ex_m[w * R + row]);
            const float base = top > kNegInf ? top : 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float k = ex2(ex_m[w * R + row] - base);
                const float4 v = *reinterpret_cast<const float4*>(ex_o + (w * R + row) * out_stride(D) + ed);
                sum = fmaf(k, ex_l[w * R + row], sum);
                x = make_float4(fmaf(k, v.x, x.x), fmaf(k, v.y, x.y), fmaf(k, v.z, x.z), fmaf(k, v.w, x.w));
            }
            if (it.whole) {
                finish_row<D>(p, it, chunk * R + row, ed, x, sum, top);
            } else {
                *reinterpret_cast<float4*>(part + row * D + ed) = x;
                if (ed == 0) {
                    part[R * D + row] = top;
                    part[R * D + R + row] = sum;
                }
            }
        }
        if (!it.whole) {
            int c0, c1;
            walk.sharers(c0, c1);
            __syncthreads();
            if (tid == 0) {
                const bool last = arrive(p.done + c0) == c1 - c0;
                if (last) p.done[c0] = 0;
                *joins = last;
            }
            __syncthreads();
            if (*joins) join_partials<D, R, kThreads>(p, it, c0, c1, live, reinterpret_cast<float*>(smem));
        }
        if (walk.parted) return;
        __syncthreads();                     // the exchange is free for the next item's ring
    }
}

// Tiles of eight rows that a chunk has.  Two take each code through the registers for twice the rows, in 1.62 times the
// time of one (1.74 at D = 64), and have fewer warps an SM, so that an item's beginning and end weigh more: 32 (40)
// groups of a CTA against 24.  Both add up, with the groups that the pages can hold, to a time for either; us, one tile /
// two, 64/8 heads of 128: 16 rows, 16 sequences of 4000 tokens 37.3/32.3, 2 of them 13.1/16.9, 64 of 300 23.6/19.2; 24
// rows 48.1/48.9 and, of 300, 25.5/29.4; 32 rows of 8191 100.0/81.1; 40 rows of 4000 71.9/66.5, of 300 35.6/41.1.  (What
// the pages can hold stands for the lengths, which only the device knows: all these have tables as wide as the longest
// sequence.  16 sequences of 300 with 16 rows in a table of 131072 tokens take two tiles, 14.7 us against 12.0.)
int row_tiles(int D, const Kv4AttnParams& p, int sms) {
    const int64_t rows = (int64_t)p.Lq * p.G, seqs = (int64_t)p.B * p.c.heads;
    if (rows <= 8) return 1;
    const float groups = (float)(std::min(p.room, p.reach) / 16 + 1);
    auto time = [&](int tiles, float group, float item) {
        const float items = (float)(seqs * ((rows + 8 * tiles - 1) / (8 * tiles)));
        return items * groups * group / (float)ctas_per_sm(D, 1, kMiddle) +
               item * std::max((float)used_sms(sms), items / (float)ctas_per_sm(D, tiles, kMiddle));
    };
    return time(1, 1.0f, 24.0f) <= time(2, D == 64 ? 1.74f : 1.62f, D == 64 ? 40.0f : 32.0f) ? 1 : 2;
}

template <int D, int NT, Width WIDTH>
cudaError_t launch(const Kv4AttnParams& p, int sms, cudaStream_t st) {
    const void* kernel = reinterpret_cast<const void*>(kv4_attention_kernel<D, NT, WIDTH>);
    cudaError_t e = ensure_dynamic_smem(kernel, smem_bytes(D, NT, WIDTH));
    if (e != cudaSuccess) return e;
    return launch_chained(kv4_attention_kernel<D, NT, WIDTH>, used_sms(sms) * ctas_per_sm(D, NT, WIDTH),
                          32 * cta_warps(D, NT, WIDTH), smem_bytes(D, NT, WIDTH), st, p);
}

template <int D, int NT>
cudaError_t launch(Kv4AttnParams p, int sms, cudaStream_t st) {
    p.chunks = fast_div((p.Lq * p.G + 8 * NT - 1) / (8 * NT));
    p.group = fast_div(p.G);
    p.page_groups = fast_div(p.c.page / 16);
    // Few long items: one CTA an SM leaves a third as many partials to join (one sequence of 131072 tokens 32.1 us
    // against 38.9, two of 16000 16.9 against 19.6).  More, or ones too short to give such a CTA's warps two steps
    // each: CTAs of four warps (64 sequences of up to 16384 tokens 110 us against 132).  More items than such CTAs:
    // of two warps, which begin and end twice as many items at a time (us, four warps / two; sequences x tokens, 32 or
    // 64/8 heads: 100 x 30 13.5/9.2, 256 x 300 31.9/26.8, 256 x 1000 51.3/45.7, 64 x 4 new of 4000 122/92, 64 x 16384
    // 107.7/106.9; with fewer items: 32 x 1000 13.7/14.6, 2 x 4000 12.3/22.6, 16 x 4 new of 8191 80.9/86.4).  Again by what
    // the pages can hold: two sequences of 300 in a table of 131072 tokens have one CTA an SM, 6.5 us (four warps, as in a
    // table of their length, 8.9), one of 77 5.8 (5.4); 8 or 64 of 1000 take the same in either table.
    const int64_t items = (int64_t)p.B * p.c.heads * p.chunks.d, ctas = used_sms(sms);
    if (8 * items <= ctas && items * (p.room / 16) >= ctas * 4 * cta_warps(D, NT, kWide))
        return launch<D, NT, kWide>(p, sms, st);
    return items > ctas * ctas_per_sm(D, NT, kMiddle) ? launch<D, NT, kNarrow>(p, sms, st)
                                                      : launch<D, NT, kMiddle>(p, sms, st);
}

}  // namespace

size_t kv4_attention_part_floats(int D, int64_t rows, int sms) {
    size_t most = 0;
    for (int tiles = 1; tiles <= (rows <= 8 ? 1 : 2); ++tiles)
        most = std::max(most, (size_t)used_sms(sms) * ctas_per_sm(D, tiles, kNarrow) * 2 * (8 * tiles) * (D + 2));
    return most;
}

cudaError_t launch_kv4_attention(int D, const Kv4AttnParams& p, int sms, cudaStream_t st) {
    const bool one = row_tiles(D, p, sms) == 1;
    if (D == 64) return one ? launch<64, 1>(p, sms, st) : launch<64, 2>(p, sms, st);
    return one ? launch<128, 1>(p, sms, st) : launch<128, 2>(p, sms, st);
}

}  // namespace r9q
