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
// weights P sv are rounded to fp16 (11 bits; bf16 would keep 8).  To keep them in
// its range a row's weights are taken not against its largest score alone but
// against m2 = largest score - 14 + E, E the exponent of the largest step its keys
// have had: they stay under 2^15, and 2^-28 of the largest still has full precision.
// Both sums use the same weights, so the power of two cancels.  Scores, maxima,
// sums and accumulators are fp32.
//
// Work is cut in groups of 16 keys.  All CTAs are resident; each takes an equal,
// contiguous range of the groups of all (sequence, kv head, row chunk) items,
// counted on the device from the lengths, so ragged batches and single long
// sequences fill the GPU alike.  The four warps of a CTA take 32-key steps of its
// range in turn, each with its own running maximum, and meet in shared memory at
// the item's end.  An item that several CTAs share leaves fp32 partials; the CTA
// that arrives last joins them in CTA order.
//
// HBM bound (136 bytes a token and head at D = 128).  Lanes copy exactly the
// bytes they will use (cp.async, 16 bytes, a ring of stages in shared memory per
// warp), so a stage needs no barrier.
#include "r9q_kv4.cuh"

namespace r9q {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;                    // keys a warp takes at a time: two groups of 16
constexpr int kStages = 4;
constexpr int kMinGroups = 8;                // groups a CTA takes at least: one step for each warp
constexpr int kMinExponent = 67;             // value steps under 2^-60 count as that (keeps the sums finite)
constexpr float kLn2 = 0.69314718055994531f;

constexpr int stage_bytes(int D) { return kStep * D + kStep * 8; }
constexpr int ring_bytes(int D) { return kWarps * kStages * stage_bytes(D); }
constexpr int out_stride(int D) { return D + 4; }      // floats a row of the CTA's exchange takes
constexpr int exchange_bytes(int D, int NT) { return kWarps * 8 * NT * (out_stride(D) + 2) * 4; }
constexpr int work_bytes(int D, int NT) {              // the rings, and after them the exchange in their place
    return ring_bytes(D) > exchange_bytes(D, NT) ? ring_bytes(D) : exchange_bytes(D, NT);
}
// What the threads of a CTA tell one another about its range.
struct Shared {
    long long scan[kWarps], first;
    int seq, last;
};
constexpr int smem_bytes(int D, int NT) { return work_bytes(D, NT) + (int)sizeof(Shared); }
constexpr int ctas_per_sm(int D, int NT) { return (D == 64 ? 4 : 3) - (NT - 1); }

template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Transposes an 8x8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A sequence's keys: [lo, len) are seen by at least one new token.
struct Span {
    int len, g0;             // tokens; first group that holds a visible key
    int groups;              // groups of an item of it, at least one (an empty one writes zeros)
};
__device__ __forceinline__ Span span_of(const Kv4AttnParams& p, int b) {
    Span s;
    const int64_t room = (int64_t)p.max_pages * p.c.page;
    int len = p.lens[b];
    if (len < 0 || len > room) {
        if (threadIdx.x == 0) record_error(p.err, kErrArg);
        len = len < 0 ? 0 : (int)room;
    }
    s.len = len;
    const int64_t lo = p.window > 0 ? (int64_t)len - p.Lq - p.window + 1 : 0;
    s.g0 = lo > 0 ? (int)(lo >> 4) : 0;
    const int n = ((len + 15) >> 4) - s.g0;
    s.groups = n > 0 ? n : 1;
    return s;
}

// What a column's weights are taken against (m2 above); 0 while it has seen no key.
__device__ __forceinline__ float reference(float m, float fr, int es) {
    return m > -__builtin_huge_valf() ? fmaf(m, fr, (float)(es - 127 - 14)) : 0.0f;
}

// The log of the sum of exponentials, from the sum of weights l and their reference m.
__device__ __forceinline__ float log_sum_exp(float m, float l) {
    return l > 0.0f || l != l ? (m + log2f(l)) * kLn2 : __int_as_float(0xFF800000);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT)) kv4_attention_kernel(const Kv4AttnParams p) {
    constexpr int KW = D / 32;               // 32-bit words of a key that a lane holds
    constexpr int MT = D / 16;               // 16-element tiles
    constexpr int R = 8 * NT;                // rows of a chunk
    constexpr float kNegInf = -__builtin_huge_valf();
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + work_bytes(D, NT));

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, j = lane & 3;
    const int rows = p.Lq * p.G, chunks = (rows + R - 1) / R;
    const int items_per_seq = p.c.heads * chunks;

    // ---- this CTA's range of groups [u0, u1) and the sequence it begins in ----
    const int per_thread = (p.B + kThreads - 1) / kThreads;
    const int b_first = tid * per_thread, b_end = min(p.B, b_first + per_thread);
    long long mine = 0;
    for (int b = b_first; b < b_end; ++b) mine += (long long)span_of(p, b).groups * items_per_seq;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sh.scan[w];
        total += sh.scan[w];
    }
    long long per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kMinGroups) per = kMinGroups;
    const long long u0 = (long long)blockIdx.x * per;
    const long long u1 = u0 + per < total ? u0 + per : total;
    if (u0 >= total) return;
    if (u0 >= before && u0 < before + mine) {
        long long at = before;
        int b = b_first;
        for (;; ++b) {
            const long long n = (long long)span_of(p, b).groups * items_per_seq;
            if (u0 < at + n) break;
            at += n;
        }
        sh.seq = b;
        sh.first = at;
    }
    __syncthreads();
    int b = sh.seq;
    long long seq_first = sh.first;           // first unit of sequence b

    uint8_t* ring = smem + warp * (kStages * stage_bytes(D));
    const uint32_t ring_u = smem_u32(ring);
    const int gpp = p.c.page >> 4;           // groups of a page

    long long u = u0;
    Span sp = span_of(p, b);
    while (u < u1) {
        while (u >= seq_first + (long long)sp.groups * items_per_seq) {
            seq_first += (long long)sp.groups * items_per_seq;
            sp = span_of(p, ++b);
        }
        const int item = (int)((u - seq_first) / sp.groups);
        const long long item_first = seq_first + (long long)item * sp.groups, item_end = item_first + sp.groups;
        const int hk = item / chunks, chunk = item - hk * chunks;
        const long long seg_end = item_end < u1 ? item_end : u1;
        const int g_begin = sp.g0 + (int)(u - item_first), g_end = sp.g0 + (int)(seg_end - item_first);
        const bool whole = u == item_first && seg_end == item_end;

        // ---- query fragments and this lane's two columns of every tile ----
        uint32_t qf[NT][MT][2];
        float fr[NT][2], qs[NT][2];          // score = fr (sk acc + lk qs)
        int hi[NT][2], lo[NT][2];            // a column's keys: [lo, hi]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = chunk * R + nt * 8 + r;
            uint32_t raw[D / 8];
            if (row < rows) {
                const int i = row / p.G, head = hk * p.G + (row - i * p.G);
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
            float amax = 0.0f, sum = 0.0f;
#pragma unroll
            for (int x = 0; x < D / 8; ++x) {
                amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(raw[x])), fabsf(bf16_hi(raw[x]))));
                sum += bf16_lo(raw[x]) + bf16_hi(raw[x]);
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            // power of two that brings amax to [2^13, 2^14); 1 for a row of zeros
            int e = (int)(__float_as_uint(amax) >> 23);
            int up = e == 0 ? 0 : 13 - (e - 127);
            up = up > 100 ? 100 : up;
            const float f = __uint_as_float((uint32_t)(127 + (up < -126 ? -126 : up)) << 23);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                // elements 8w .. 8w+7 of the lane's quarter; a word's bytes 0 and 2 give 0, 4 (low) and 1, 5 (high),
                // bytes 1 and 3 give 2, 6 and 3, 7
                const uint32_t* q = raw + 4 * w;
                const float f16 = f * 0.0625f;
                qf[nt][2 * w][0] = pack_f16x2(bf16_lo(q[0]) * f, bf16_lo(q[2]) * f);
                qf[nt][2 * w][1] = pack_f16x2(bf16_hi(q[0]) * f16, bf16_hi(q[2]) * f16);
                qf[nt][2 * w + 1][0] = pack_f16x2(bf16_lo(q[1]) * f, bf16_lo(q[3]) * f);
                qf[nt][2 * w + 1][1] = pack_f16x2(bf16_hi(q[1]) * f16, bf16_hi(q[3]) * f16);
            }
            const float row_fr = fminf(p.scale_log2 * (16777216.0f / f), 3e38f), row_qs = sum * f * (1.0f / 16777216.0f);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = 2 * j + c;
                fr[nt][c] = __shfl_sync(0xffffffffu, row_fr, col * 4);
                qs[nt][c] = __shfl_sync(0xffffffffu, row_qs, col * 4);
                const int crow = chunk * R + nt * 8 + col;
                const int ci = (crow < rows ? crow : rows - 1) / p.G;
                hi[nt][c] = sp.len - p.Lq + ci;
                lo[nt][c] = p.window > 0 ? hi[nt][c] - p.window + 1 : 0;
            }
        }
        // keys that all rows of the chunk see
        const int i_first = chunk * R / p.G, i_last = (min(rows, chunk * R + R) - 1) / p.G;
        const int all_hi = sp.len - p.Lq + i_first, all_lo = p.window > 0 ? sp.len - p.Lq + i_last - p.window + 1 : 0;

        float acc[NT][MT][4], m[NT][2], l[NT][2], ml[NT][2];
        int es[NT][2];                       // exponent field that stands for the columns' values so far
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[nt][t][c] = 0.0f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[nt][c] = kNegInf;
                l[nt][c] = ml[nt][c] = 0.0f;
                es[nt][c] = kMinExponent;
            }
        }

        // ---- the warp's steps ----
        const int steps_all = (g_end - g_begin + 1) >> 1;
        const int steps = steps_all > warp ? (steps_all - warp + kWarps - 1) / kWarps : 0;
        const int32_t* table = p.table + (int64_t)b * p.max_pages;
        // lane x holds the page of the x-th group of the next 16 steps (-1: none), and of the 16 after them
        const int gmax = min(g_end, (sp.len + 15) >> 4);
        auto page_of = [&](int first_step) {
            const int g = g_begin + 2 * ((first_step + (lane >> 1)) * kWarps + warp) + (lane & 1);
            int page = -1;
            if (g < gmax) {
                page = table[g / gpp];
                if (page < 0 || page >= p.c.pages) {
                    record_error(p.err, kErrArg);
                    page = -1;
                }
            }
            return page;
        };
        int pages_now = steps > 0 ? page_of(0) : -1, pages_next = -1;
        uint32_t have = 0;                   // two bits a step in flight: which of its groups were loaded
        auto issue = [&](int n) {
            if (n < steps) {
                if ((n & 15) == 0) {
                    if (n > 0) pages_now = pages_next;
                    pages_next = n + 16 < steps ? page_of(n + 16) : -1;
                }
                const uint32_t st = ring_u + (n % kStages) * stage_bytes(D);
                uint32_t bits = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int page = __shfl_sync(0xffffffffu, pages_now, 2 * (n & 15) + i);
                    if (page >= 0) {
                        bits |= 1u << i;
                        const int g = g_begin + 2 * (n * kWarps + warp) + i;
                        const int at = (g % gpp) * 16;
                        const int64_t head = (int64_t)page * p.c.heads + hk;
                        const int64_t base = head * kv4_head_bytes(p.c.page, D) + (int64_t)at * (D / 2);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            cp_async<KW * 4>(st + i * 16 * (D / 2) + h * 8 * (D / 2) + lane * (KW * 4),
                                             p.c.k + base + h * 8 * (D / 2) + lane * (KW * 4));
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            cp_async<16>(st + kStep * (D / 2) + i * 16 * (D / 2) + c * 512 + lane * 16,
                                         p.c.v + base + c * 512 + lane * 16);
                        const uint32_t* pair = (lane < 16 ? p.c.kp : p.c.vp) + head * p.c.page + at + (lane & 15);
                        cp_async<4>(st + kStep * D + (lane >> 4) * (kStep * 4) + i * 64 + (lane & 15) * 4, pair);
                    }
                }
                have = (have << 2) | bits;
            } else {
                have <<= 2;
            }
            cp_commit();
        };
#pragma unroll
        for (int n = 0; n < kStages - 1; ++n) issue(n);

        for (int n = 0; n < steps; ++n) {
            cp_wait<kStages - 2>();
            __syncwarp();
            const uint32_t bits = (have >> (2 * (kStages - 2))) & 3u;
            issue(n + kStages - 1);
            const uint8_t* st = ring + (n % kStages) * stage_bytes(D);
            const int key0 = (g_begin + 2 * (n * kWarps + warp)) << 4;

            // pairs of the lane's keys r + 8h of group i
            float sk[2][2], lk[2][2], sv[2][2], lv[2][2];
            const uint32_t* kp = reinterpret_cast<const uint32_t*>(st + kStep * D);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a = kp[16 * i + 8 * h + r], v = kp[kStep + 16 * i + 8 * h + r];
                    sk[i][h] = bf16_lo(a);
                    lk[i][h] = bf16_hi(a);
                    sv[i][h] = bf16_lo(v);
                    lv[i][h] = bf16_hi(v);
                }
            const bool plain = bits == 3u && key0 >= all_lo && key0 + kStep - 1 <= all_hi;
            if (!plain) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = key0 + 16 * i + 8 * h + r;
                        if (!((bits >> i) & 1u) || key >= sp.len) sk[i][h] = lk[i][h] = sv[i][h] = lv[i][h] = 0.0f;
                    }
            }
            // ---- scores ----
            float s[NT][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t k0[KW], k1[KW];
                const uint8_t* kb = st + i * 16 * (D / 2) + lane * (KW * 4);
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    k0[w] = reinterpret_cast<const uint32_t*>(kb)[w];
                    k1[w] = reinterpret_cast<const uint32_t*>(kb + 8 * (D / 2))[w];
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[nt][i][c] = 0.0f;
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    const uint32_t x0 = k0[w] >> 8, x1 = k1[w] >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16_16816(s[nt][i], k0[w] & 0x000F000Fu, k1[w] & 0x000F000Fu, k0[w] & 0x00F000F0u,
                                      k1[w] & 0x00F000F0u, qf[nt][2 * w][0], qf[nt][2 * w][1]);
                        mma_f16_16816(s[nt][i], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u,
                                      x1 & 0x00F000F0u, qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int h = c >> 1;
                        float v = fmaf(sk[i][h], s[nt][i][c], lk[i][h] * qs[nt][c & 1]);
                        if (!plain) {
                            const int key = key0 + 16 * i + 8 * h + r;
                            if (key > hi[nt][c & 1] || key < lo[nt][c & 1] || !((bits >> i) & 1u)) v = kNegInf;
                        }
                        s[nt][i][c] = v;
                    }

            // ---- running maximum, weights ----
            // The exponent of a key's values: that of its step, or of its lowest value when that is over 2^10 steps
            // (the sum of p lv is kept in the same scale); none for a pair that is not finite.
            int ek[2][2], e = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int xs = (int)(__float_as_uint(sv[i][h]) >> 23) & 255;
                    const int xl = (int)(__float_as_uint(lv[i][h]) >> 23) & 255;
                    ek[i][h] = xs == 255 || xl == 255 ? 0 : max(xs, xl - 10);
                    e = max(e, ek[i][h]);
                }
            if (plain) e = __reduce_max_sync(0xffffffffu, e);
            float alpha[NT][2];
            bool moved = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = fmaxf(fmaxf(s[nt][0][c], s[nt][0][c + 2]), fmaxf(s[nt][1][c], s[nt][1][c + 2]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                    int ec = e;
                    if (!plain) {            // only the keys that the column sees
                        ec = 0;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (s[nt][i][2 * h + c] != kNegInf) ec = max(ec, ek[i][h]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) ec = max(ec, __shfl_xor_sync(0xffffffffu, ec, o));
                    }
                    const float mn = fmaxf(m[nt][c], x);
                    const int en = max(es[nt][c], ec);
                    const bool up = mn > m[nt][c] || en > es[nt][c];
                    // nothing seen before (m = -inf): the sums are zero, and so is the factor
                    alpha[nt][c] = up ? ex2(mn > kNegInf ? fmaf(m[nt][c] - mn, fr[nt][c], (float)(es[nt][c] - en)) : 0.0f)
                                      : 1.0f;
                    moved = moved || up;
                    m[nt][c] = mn;
                    es[nt][c] = en;
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        l[nt][c] *= alpha[nt][c];
                        ml[nt][c] *= alpha[nt][c];
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            acc[nt][t][c] *= alpha[nt][c];
                            acc[nt][t][c + 2] *= alpha[nt][c];
                        }
                    }
            }
            uint32_t pf[NT][2][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float m2[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) m2[c] = reference(m[nt][c], fr[nt][c], es[nt][c]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float w[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float sc = s[nt][i][2 * h + c];
                            const float pr = ex2(fmaf(sc, fr[nt][c], -m2[c]));
                            w[c] = pr * sv[i][h];
                            float add = pr * lv[i][h];
                            if (!plain && sc == kNegInf) w[c] = add = 0.0f;     // not 0 * infinity
                            l[nt][c] += pr;
                            ml[nt][c] += add;
                        }
                        pf[nt][i][h] = transpose_8x8(pack_f16x2(w[0], w[1]));
                    }
            }

            // ---- values ----
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t* vb = st + kStep * (D / 2) + i * 16 * (D / 2) + lane * 16;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint4 q4 = *reinterpret_cast<const uint4*>(vb + c * 512);
                    const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t y = q[x] >> 8;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(acc[nt][4 * c + x], q[x] & 0x000F000Fu, q[x] & 0x00F000F0u, y & 0x000F000Fu,
                                          y & 0x00F000F0u, pf[nt][i][0], pf[nt][i][1]);
                    }
                }
            }
        }
        cp_wait<0>();

        // ---- the warps' sums meet: rows' maxima, then weighted accumulators ----
        __syncthreads();                     // the ring is free
        float* ex_m = reinterpret_cast<float*>(smem);                  // [kWarps][R]
        float* ex_l = ex_m + kWarps * R;
        float* ex_o = ex_l + kWarps * R;                               // [kWarps][R][out_stride]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], o);
                    ml[nt][c] += __shfl_xor_sync(0xffffffffu, ml[nt][c], o);
                }
                const int row = nt * 8 + 2 * j + c;
                if (r == 0) {
                    ex_m[warp * R + row] = m[nt][c] > kNegInf ? reference(m[nt][c], fr[nt][c], es[nt][c]) : kNegInf;
                    ex_l[warp * R + row] = l[nt][c];
                }
                float* o = ex_o + (warp * R + row) * out_stride(D);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    o[16 * t + r] = fmaf(acc[nt][t][c], 0x1p24f, ml[nt][c]);
                    o[16 * t + 8 + r] = fmaf(acc[nt][t][c + 2], 0x1p20f, ml[nt][c]);
                }
            }
        __syncthreads();

        const int live = min(R, rows - chunk * R);
        // a thread takes two elements of every (kThreads / (D / 2))-th row
        const int ed = (tid % (D / 2)) * 2;
        const int cta = blockIdx.x;
        const size_t slot_floats = (size_t)R * (D + 2);
        for (int row = tid / (D / 2); row < live; row += kThreads / (D / 2)) {
            float top = kNegInf, sum = 0.0f, x0 = 0.0f, x1 = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ex_m[w * R + row]);
            const float base = top > kNegInf ? top : 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float k = ex2(ex_m[w * R + row] - base);
                const float2 v = *reinterpret_cast<const float2*>(ex_o + (w * R + row) * out_stride(D) + ed);
                sum = fmaf(k, ex_l[w * R + row], sum);
                x0 = fmaf(k, v.x, x0);
                x1 = fmaf(k, v.y, x1);
            }
            if (whole) {
                const int grow = chunk * R + row, i = grow / p.G;
                const int64_t out = ((int64_t)b * p.Lq + i) * (p.c.heads * p.G) + hk * p.G + (grow - i * p.G);
                const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
                *reinterpret_cast<uint32_t*>(p.o + out * D + ed) = pack_bf16x2(x0 * inv, x1 * inv);
                if (p.lse && ed == 0) p.lse[out] = log_sum_exp(top, sum);
            } else {
                // slot 1: the item begins in this CTA; slot 0: it began in an earlier one
                float* part = p.part + ((size_t)cta * 2 + (u == item_first ? 1 : 0)) * slot_floats;
                *reinterpret_cast<float2*>(part + row * D + ed) = make_float2(x0, x1);
                if (ed == 0) {
                    part[R * D + row] = top;
                    part[R * D + R + row] = sum;
                }
            }
        }
        if (!whole) {
            const int c0 = (int)(item_first / per), c1 = (int)((item_end - 1) / per);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const bool last = atomicAdd(p.done + c0, 1) == c1 - c0;
                if (last) p.done[c0] = 0;
                sh.last = last;
            }
            __syncthreads();
            if (sh.last) {
                __threadfence();
                for (int row = tid / (D / 2); row < live; row += kThreads / (D / 2)) {
                    float top = kNegInf, sum = 0.0f, x0 = 0.0f, x1 = 0.0f;
                    for (int c = c0; c <= c1; ++c)
                        top = fmaxf(top, __ldcg(p.part + ((size_t)c * 2 + (c == c0)) * slot_floats + R * D + row));
                    const float base = top > kNegInf ? top : 0.0f;
                    for (int c = c0; c <= c1; ++c) {
                        const float* part = p.part + ((size_t)c * 2 + (c == c0)) * slot_floats;
                        const float k = ex2(__ldcg(part + R * D + row) - base);
                        const float2 v = __ldcg(reinterpret_cast<const float2*>(part + row * D + ed));
                        sum = fmaf(k, __ldcg(part + R * D + R + row), sum);
                        x0 = fmaf(k, v.x, x0);
                        x1 = fmaf(k, v.y, x1);
                    }
                    const int grow = chunk * R + row, i = grow / p.G;
                    const int64_t out = ((int64_t)b * p.Lq + i) * (p.c.heads * p.G) + hk * p.G + (grow - i * p.G);
                    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
                    *reinterpret_cast<uint32_t*>(p.o + out * D + ed) = pack_bf16x2(x0 * inv, x1 * inv);
                    if (p.lse && ed == 0) p.lse[out] = log_sum_exp(top, sum);
                }
            }
        }
        __syncthreads();                     // the exchange is free for the next item's ring
        u = seg_end;
    }
}

int row_tiles(int64_t rows) { return rows <= 8 ? 1 : 2; }

template <int D, int NT>
cudaError_t launch(const Kv4AttnParams& p, int sms, cudaStream_t st) {
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kv4_attention_kernel<D, NT>), smem_bytes(D, NT));
    if (e != cudaSuccess) return e;
    kv4_attention_kernel<D, NT><<<sms * ctas_per_sm(D, NT), kThreads, smem_bytes(D, NT), st>>>(p);
    return cudaGetLastError();
}

}  // namespace

int kv4_attention_ctas(int D, int64_t rows, int sms) { return sms * ctas_per_sm(D, row_tiles(rows)); }

size_t kv4_attention_part_floats(int D, int64_t rows, int sms) {
    return (size_t)kv4_attention_ctas(D, rows, sms) * 2 * (8 * row_tiles(rows)) * (D + 2);
}

cudaError_t launch_kv4_attention(int D, const Kv4AttnParams& p, int sms, cudaStream_t st) {
    const bool one = row_tiles((int64_t)p.Lq * p.G) == 1;
    if (D == 64) return one ? launch<64, 1>(p, sms, st) : launch<64, 2>(p, sms, st);
    return one ? launch<128, 1>(p, sms, st) : launch<128, 2>(p, sms, st);
}

}  // namespace r9q
