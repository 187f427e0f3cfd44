// The frame of the attention over the 4-bit cache (r9q_kv4_attention.cu): how the work is
// cut, the copies of a group of 16 tokens, the partial results of an item that several
// CTAs have, and how they are joined.
//
// An item is a sequence's row chunk (R query rows that share a key-value head); its work
// is counted in groups of 16 keys.  Work is cut on the device, from the lengths, so that ragged
// batches and single long sequences fill the GPU alike.  All CTAs are resident.  With
// few items each is cut into equal parts, one a CTA; with many, each CTA takes an equal,
// contiguous range of all items' groups (each item counting some more for what it costs
// to begin), its ends moved to an item's end where that is near.  An item that several
// CTAs share leaves fp32 partials; the CTA that arrives last joins them in CTA order.
#pragma once

#include "r9q_kv4.cuh"

namespace r9q {

constexpr int kMinExponent = 67;             // value steps under 2^-60 count as that (keeps the sums finite)
constexpr int kHeadroom = 8;                 // weights at the reference score are 2^8 to 2^9
constexpr int kSlack = 6;                    // powers of two they may pass it by
// A lowest value counts as a step of 2^-10 of it: the sums of p lv are kept in the weights' scale.
constexpr int kLowestBits = 10;
constexpr float kLowestShare = 1.0f / (1 << kLowestBits);
constexpr int kNoWindow = 0x7FE00000;        // over any length (Lq is at most 2^20)
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr uint32_t kNoGroup = 0xFFFFFFFFu;
constexpr int kMaxSms = 160;                 // more are left idle
inline int used_sms(int sms) { return sms < kMaxSms ? sms : kMaxSms; }
constexpr int largest(int a, int b) { return a > b ? a : b; }

// Copies a lane's share of one group of 16 tokens into a stage, if `live`: its two K rows' parts (8 rows apart), its
// V pieces, and a (step, lowest) pair.
template <int D>
__device__ __forceinline__ void copy_group(bool live, uint32_t k_dst, const uint8_t* k, uint32_t v_dst,
                                           const uint8_t* v, uint32_t pair_dst, const uint32_t* pair) {
    if constexpr (D == 128) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
            "@p cp.async.cg.shared.global [%1], [%2], 16;\n\t"
            "@p cp.async.cg.shared.global [%1+512], [%2+512], 16;\n\t"
            "@p cp.async.cg.shared.global [%3], [%4], 16;\n\t"
            "@p cp.async.cg.shared.global [%3+512], [%4+512], 16;\n\t"
            "@p cp.async.ca.shared.global [%5], [%6], 4;\n\t}" ::"r"((int)live),
            "r"(k_dst), "l"(k), "r"(v_dst), "l"(v), "r"(pair_dst), "l"(pair)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
            "@p cp.async.ca.shared.global [%1], [%2], 8;\n\t"
            "@p cp.async.ca.shared.global [%1+256], [%2+256], 8;\n\t"
            "@p cp.async.cg.shared.global [%3], [%4], 16;\n\t"
            "@p cp.async.ca.shared.global [%5], [%6], 4;\n\t}" ::"r"((int)live),
            "r"(k_dst), "l"(k), "r"(v_dst), "l"(v), "r"(pair_dst), "l"(pair)
            : "memory");
    }
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
// Takes 7.5 times the fp16 values in the halves of w from a and b, one rounding each.
__device__ __forceinline__ void less_mid(float& a, float& b, uint32_t w) {
    asm("{\n\t.reg .b16 l, h, k;\n\tmov.b32 {l, h}, %2;\n\tmov.b16 k, 0xC780;\n\tfma.rn.f32.f16 %0, l, k, %0;\n\t"
        "fma.rn.f32.f16 %1, h, k, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(w));                               // (0xC780: -7.5)
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
static __device__ __noinline__ long long div64(long long a, long long b) { return a / b; }

// A sequence's keys and the groups an item of it has.  `room`: tokens that its pages
// can hold; `reach`: the most tokens that its new ones see.
struct Span {
    int len, g0;             // tokens; first group that holds a visible key
    int groups;              // at least one (an empty sequence's items write zeros)
};
static __device__ __noinline__ Span span_of(const int32_t* at, int room, int reach, int* err) {
    Span s;
    int len = *at;
    if (len < 0 || len > room) {
        if (threadIdx.x == 0) record_error(err, kErrArg);
        len = len < 0 ? 0 : room;
    }
    s.len = len;
    s.g0 = len > reach ? (len - reach) >> 4 : 0;
    const int n = ((len + 15) >> 4) - s.g0;
    s.groups = n > 0 ? n : 1;
    return s;
}

// The warp's inclusive scan of one value a lane; `total` over all.
__device__ __forceinline__ long long warp_scan(long long v, long long& total) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    total = __shfl_sync(0xffffffffu, v, 31);
    return v;
}

// The log of the sum of exponentials, from the sum of weights l and their reference m
// (both of powers of two).
__device__ __forceinline__ float log_sum_exp(float m, float l) {
    return l > 0.0f || l != l ? (m + log2f(l)) * kLn2 : __int_as_float(0xFF800000);
}

// A part of an item.
struct Part {
    int b, hk, chunk;        // sequence, key-value head, row chunk
    int g_begin, g_end;      // groups, from the sequence's beginning
    bool whole, begins;      // all of the item; its first part
};

// What a CTA has to do.  Every warp finds it for itself, a lane for every so many sequences.
struct Walk {
    bool parted;             // one part of one item a CTA; else a range of all items' groups
    int begin_cost, b, item, items_per_seq, parts, even, counted;
    long long per, u, range_end, seq_first, first;
    Span sp;                 // of sequence b

    __device__ __forceinline__ Span span(const Kv4AttnParams& p, int at) const {
        return span_of(p.lens + at, p.room, p.reach, p.err);
    }
    // An end of a range inside an item goes to the item's end where that is within so many groups of it.
    __device__ __forceinline__ int snap(int groups) const {
        return min(min(8, (int)min(per / 4, 8ll)), (groups - 1) / 2);
    }
    __device__ __forceinline__ long long moved(long long x, long long from, int groups) const {
        const int n = groups + begin_cost, s = snap(groups);
        const long long item_at = from + div64(x - from, n) * n;
        return x - item_at <= begin_cost + s ? item_at : item_at + n - x <= s ? item_at + n : x;
    }

    // False: nothing.  min_groups: the groups that a CTA takes at least; item_cost: those that take it as long as
    // beginning and ending an item.
    __device__ __forceinline__ bool start(const Kv4AttnParams& p, int min_groups, int item_cost) {
        const int lane = threadIdx.x & 31;
        items_per_seq = p.c.heads * p.chunks.d;
        const long long items = (long long)p.B * items_per_seq, ctas = gridDim.x;
        parted = 2 * items <= ctas;
        begin_cost = parted ? 0 : item_cost;
        const int per_lane = (p.B + 31) / 32, b_first = lane * per_lane, b_end = min(p.B, b_first + per_lane);
        long long mine = 0, total;
#pragma unroll 1
        for (int at = b_first; at < b_end; ++at) mine += span(p, at).groups + begin_cost;
        mine *= items_per_seq;
        long long upto = warp_scan(mine, total);
        if (parted) {
            // The even share, if parts of that size are no more than the CTAs; else total / (ctas - items): the sum
            // of ceil(groups / per) over the items is at most total / per + items.
            const long long all = total;
            per = (all + ctas - 1) / ctas;
            for (int attempt = 1;; ++attempt) {
                if (per < min_groups) per = min_groups;
                mine = 0;                    // from here on: parts
#pragma unroll 1
                for (int at = b_first; at < b_end; ++at) mine += (span(p, at).groups + (int)per - 1) / (int)per;
                mine *= items_per_seq;
                upto = warp_scan(mine, total);
                if (total <= ctas || attempt == 2) break;
                per = (all + ctas - items - 1) / (ctas - items);
            }
        } else {
            per = div64(total + ctas - 1, ctas);
            if (per < min_groups) per = min_groups;
        }
        u = parted ? blockIdx.x : blockIdx.x * per;
        if (u >= total) return false;
        const bool here = u >= upto - mine && u < upto;  // one lane's
        b = b_first;
        seq_first = upto - mine;             // first part or group of sequence b
        if (here) {
#pragma unroll 1
            for (;; ++b) {
                const int g = span(p, b).groups;
                const long long n = (long long)(parted ? (g + (int)per - 1) / (int)per : g + begin_cost) * items_per_seq;
                if (u < seq_first + n) break;
                seq_first += n;
            }
        }
        const int owner = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        b = __shfl_sync(0xffffffffu, b, owner);
        seq_first = __shfl_sync(0xffffffffu, seq_first, owner);
        sp = span(p, b);
        // parts of `even` groups, one after another; rounding may leave the last of those counted above without any
        counted = parted ? (sp.groups + (int)per - 1) / (int)per : 0;
        even = parted ? (sp.groups + counted - 1) / counted : 0;
        parts = parted ? (sp.groups + even - 1) / even : 0;
        range_end = 0;
        if (!parted) {
            const long long end = u + per;
            u = moved(u, seq_first, sp.groups);
            if (end >= total) {
                range_end = total;
            } else {                         // it may lie in a later sequence
                long long from = seq_first;
                int be = b, g = sp.groups;
#pragma unroll 1
                while (end >= from + (long long)(g + begin_cost) * items_per_seq) {
                    from += (long long)(g + begin_cost) * items_per_seq;
                    g = span(p, ++be).groups;
                }
                range_end = moved(end, from, g);
            }
        }
        return true;
    }

    // The next part; false where there is none.
    __device__ __forceinline__ bool next(const Kv4AttnParams& p, Part& x) {
        if (parted) {
            const int at = (int)(u - seq_first);
            item = at / counted;
            const int part = at - item * counted;
            if (part >= parts) return false;
            x.g_begin = part * even;
            x.g_end = min(sp.groups, x.g_begin + even);
        } else {
            if (u >= range_end) return false;
#pragma unroll 1
            while (u >= seq_first + (long long)(sp.groups + begin_cost) * items_per_seq) {
                seq_first += (long long)(sp.groups + begin_cost) * items_per_seq;
                sp = span(p, ++b);
            }
            const int n = sp.groups + begin_cost;
            item = (int)div64(u - seq_first, n);
            first = seq_first + (long long)item * n;
            x.g_begin = max(0, (int)(u - first) - begin_cost);
            x.g_end = (int)min((long long)n, range_end - first) - begin_cost;
            u = first + begin_cost + x.g_end;
        }
        x.whole = x.g_begin == 0 && x.g_end == sp.groups;
        x.begins = x.g_begin == 0;
        x.g_begin += sp.g0;
        x.g_end += sp.g0;
        x.b = b;
        x.hk = item / p.chunks;
        x.chunk = item - x.hk * p.chunks.d;
        return true;
    }

    // The CTAs that share the item of the part that next() gave.
    __device__ __forceinline__ void sharers(int& c0, int& c1) const {
        if (parted) {
            c0 = (int)(seq_first + (long long)item * counted);
            c1 = c0 + parts - 1;
        } else {
            const int n = sp.groups + begin_cost, s = snap(sp.groups);
            c0 = (int)div64(first + begin_cost + s, per);
            c1 = (int)div64(first + n - s - 1, per);
        }
    }
};

// The token index in the cache of group g of a sequence, or kNoGroup where its page is not one (an error).
__device__ __forceinline__ uint32_t find_group(const Kv4AttnParams& p, const int32_t* table, int g, int hk) {
    const int pg = g / p.page_groups, page = table[pg];
    if (page >= 0 && page < p.c.pages)
        return ((uint32_t)page * p.c.heads + hk) * p.c.page + (g - pg * p.page_groups.d) * 16;
    record_error(p.err, kErrArg);
    return kNoGroup;
}

// What a row is to be in place of its sums.
enum Instead { kAsItIs, kNothing, kNan };
struct AsItIs {
    __device__ __forceinline__ Instead operator()(int) const { return kAsItIs; }
};

// Four elements from ed of a row: o = x / sum, and the row's log of the sum of exponentials.  `instead`: of the row's
// token.
template <int D, typename INSTEAD>
__device__ __forceinline__ void finish_row(const Kv4AttnParams& p, const Part& it, int row, int ed, float4 x,
                                           float sum, float top, const INSTEAD& instead) {
    const int i = row / p.group;
    const Instead other = instead(i);
    if (other == kNothing) {
        x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        sum = 0.0f;
    } else if (other == kNan) {
        x.x = x.y = x.z = x.w = sum = __int_as_float(0x7FC00000);
    }
    const int64_t out = ((int64_t)it.b * p.Lq + i) * (p.c.heads * p.G) + it.hk * p.G + (row - i * p.G);
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    *reinterpret_cast<uint2*>(p.o + out * D + ed) =
        make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
    if (p.lse && ed == 0) p.lse[out] = log_sum_exp(top, sum);
}

// A CTA's partial of an item, floats: [R][D] sums, [R] references, [R] sums of weights.  Slot 1 of a CTA: the item
// begins in it; slot 0: it began in an earlier one.
template <int D, int R>
constexpr size_t kSlotFloats = (size_t)R * (D + 2);
template <int D, int R>
__device__ __forceinline__ float* partial_of(const Kv4AttnParams& p, int cta, bool begins) {
    return p.part + ((size_t)cta * 2 + (begins ? 1 : 0)) * kSlotFloats<D, R>;
}

// Shared memory of join_partials.
constexpr int join_bytes(int R, int threads) { return 2 * R * 4 + threads * R * 16; }

// Joins an item's partials, all threads of the CTA that arrived last: the rows' references and sums over all partials
// first, then the weighted sum.  The warps that hold a row's elements take every ROWS-th partial each (all the rows'
// loads in flight) and meet at the end.
template <int D, int R, int THREADS, typename INSTEAD>
__device__ __forceinline__ void join_partials(const Kv4AttnParams& p, const Part& it, int c0, int c1, int live,
                                              float* smem, const INSTEAD& instead) {
    constexpr int ROWS = THREADS / (D / 4);
    const int tid = threadIdx.x, lane = tid & 31, ed = (tid % (D / 4)) * 4, row0 = tid / (D / 4), n = c1 - c0 + 1;
    float *total_m = smem, *total_l = total_m + R, *meet = total_l + R;
    auto slot = [&](int c) { return partial_of<D, R>(p, c0 + c, c == 0); };
    for (int row = tid >> 5; row < R; row += THREADS / 32) {
        float top = kNegInf, sum = 0.0f;
        auto join = [&](float m, float l) {
            const float both = fmaxf(top, m), base = both > kNegInf ? both : 0.0f;
            sum = sum * ex2(top - base) + l * ex2(m - base);
            top = both;
        };
        if (row < live)
            for (int c = lane; c < n; c += 32) join(__ldcg(slot(c) + R * D + row), __ldcg(slot(c) + R * D + R + row));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float m = __shfl_xor_sync(0xffffffffu, top, o), l = __shfl_xor_sync(0xffffffffu, sum, o);
            join(m, l);
        }
        if (lane == 0) {
            total_l[row] = sum;
            total_m[row] = top;
        }
    }
    __syncthreads();
    float4 x[R];
    float base[R];
#pragma unroll
    for (int row = 0; row < R; ++row) {
        x[row] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        base[row] = total_m[row] > kNegInf ? total_m[row] : 0.0f;
    }
#pragma unroll 2
    for (int c = row0; c < n; c += ROWS) {
        const float* src = slot(c) + ed;
#pragma unroll
        for (int row = 0; row < R; ++row)
            if (row < live) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(src + row * D));
                const float k = ex2(__ldcg(slot(c) + R * D + row) - base[row]);
                x[row] = make_float4(fmaf(k, v.x, x[row].x), fmaf(k, v.y, x[row].y), fmaf(k, v.z, x[row].z),
                                     fmaf(k, v.w, x[row].w));
            }
    }
#pragma unroll
    for (int row = 0; row < R; ++row) *reinterpret_cast<float4*>(meet + ((size_t)row0 * R + row) * D + ed) = x[row];
    __syncthreads();
    for (int row = row0; row < live; row += ROWS) {
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(meet + ((size_t)k * R + row) * D + ed);
            y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
        }
        finish_row<D>(p, it, it.chunk * R + row, ed, y, total_l[row], total_m[row], instead);
    }
}

}  // namespace r9q
