// The gated delta rule over a few tokens a sequence (formulas: r9q_delta.cuh): decode steps,
// small trees of drafted tokens, accepted paths.
//
// The state is what costs: 4 D D bytes a head in and, where it changes, out.  So a
// sequence's head is cut by rows (values), which do not meet: a warp holds 16 rows of S
// in registers, row r + 4i in the lanes 8r .. 8r + 7, each with D/8 of its elements.  Groups
// of up to 16 tokens pass over it: S k and S q of eight at a time (the eight partial sums of four
// rows and two products meet in seven shuffles, which leaves one result a lane), then the
// sums over earlier tokens, at last the update with all of the group's u at once.  What does
// not depend on the row, the products of keys and queries among themselves and the decays,
// is formed once for the CTA, a warp following a token's ancestors and adding up their decays as
// it goes.  In a tree S stays as it is.
//
// What bounds it: with one token HBM (128 sequences, 32 heads of 128: 79 us, 6.8 TB/s); with more about 1 us a token
// for the sums over earlier tokens (16 trees of 16 nodes: 41 us, 64 paths of 5: 53 us, 5.1 TB/s).  A head's CTA of 8 warps
// against one of 4 warps for half of it: the products among the tokens are formed once (53 -> 40 us).
#include "r9q_delta.cuh"

namespace r9q {

namespace {

constexpr int kGroup = 16, kAtOnce = 8;      // tokens between updates of S, and that are multiplied with it at a time
constexpr int kRows = 16;                    // of a warp
constexpr int warps_of(int D) { return D / kRows; }          // of a CTA, which has a head

template <int D>
struct Shared {
    float kn[kGroup][D], qn[kGroup][D];      // of unit length
    float solve[kGroup][kGroup], weigh[kGroup][kGroup];      // beta A (k.k), scale A (q.k), of ancestors
    float g[kGroup], beta[kGroup], fade[kGroup], left[kGroup];       // fade A(i, 0), left A(n, i)
    float u[warps_of(D)][kGroup][kRows];
    int parents[kGroup];
    uint64_t above[kGroup];                  // a node's ancestors, itself among them
    NodeKind kind[kGroup];
};

// 32/8 lanes of a quarter warp hold `N` partial sums each (N 8 or 4); lane c of 8 gets the sum of the c-th (c/2-th).
template <int N>
__device__ __forceinline__ float meet8(const float (&x)[N], int c) {
    float y[N / 2], z[N / 4];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float keep = c & 4 ? x[i + N / 2] : x[i], give = c & 4 ? x[i] : x[i + N / 2];
        y[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float keep = c & 2 ? y[i + N / 4] : y[i], give = c & 2 ? y[i] : y[i + N / 4];
        z[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    if constexpr (N == 4) return z[0] + __shfl_xor_sync(0xffffffffu, z[0], 1);
    const float keep = c & 1 ? z[N / 4 - 1] : z[0], give = c & 1 ? z[0] : z[N / 4 - 1];
    return keep + __shfl_xor_sync(0xffffffffu, give, 1);
}

// A bf16 head vector, D/32 elements a lane, as fp32 of unit length in shared memory.
template <int D>
__device__ __forceinline__ void unit_vector(const uint16_t* src, float* dst, float eps, int lane) {
    float x[D / 32];
    if constexpr (D == 128) {
        const uint2 w = reinterpret_cast<const uint2*>(src)[lane];
        x[0] = bf16_lo(w.x);
        x[1] = bf16_hi(w.x);
        x[2] = bf16_lo(w.y);
        x[3] = bf16_hi(w.y);
    } else {
        const uint32_t w = reinterpret_cast<const uint32_t*>(src)[lane];
        x[0] = bf16_lo(w);
        x[1] = bf16_hi(w);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) sum = fmaf(x[i], x[i], sum);
    const float r = rsqrtf(group_sum<32>(sum) + eps);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) dst[lane * (D / 32) + i] = x[i] * r;
}

template <int D, DeltaMode MODE>
__global__ void __launch_bounds__(32 * warps_of(D), D == 64 ? 4 : 2) delta_rows_kernel(const DeltaParams p) {
    constexpr int W = warps_of(D), M = D / 32;               // warps; 16-byte pieces of a row that a lane has
    constexpr bool TREE = MODE == kDeltaTree, HAS_Q = MODE != kDeltaCommit;
    __shared__ Shared<D> sh;
    begin_chained();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 7, r = lane >> 3;
    const int b = blockIdx.x / p.Hv, h = blockIdx.x - b * p.Hv, hk = h / p.ratio;
    const int row0 = warp * kRows;
    int n;
    int64_t row;
    delta_tokens(p, b, n, row);
    const int32_t* path = p.path + (int64_t)b * p.P;
    if constexpr (MODE == kDeltaCommit) n = path_length(p, b);
    const int first_slot = p.slots[b];       // (its rows are on their way while the slot is checked)
    float* rows = p.state + (((int64_t)(first_slot >= 0 && first_slot < p.n_states ? first_slot : 0) * p.Hv + h) * D + row0) * D;
    uint64_t s[4][2 * M];                    // pairs of rows r + 4i
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            ulonglong2 x = make_ulonglong2(0ull, 0ull);
            if (!p.from_zero) x = *reinterpret_cast<const ulonglong2*>(rows + (r + 4 * i) * D + m * 32 + c * 4);
            s[i][2 * m] = x.x;
            s[i][2 * m + 1] = x.y;
        }
    const bool second = HAS_Q && (c & 1);    // the lane gets S q of its row; else S k
    const int own = row0 + r + 4 * (c >> 1); // that row
    const int64_t at0 = p.cu ? row : 0;      // the first token in q, k and v
    int slot = -1;

#pragma unroll 1
    for (int base = 0; base < max(n, 1); base += kGroup) {
        const int cnt = min(kGroup, n - base);
        auto token = [&](int t) { return MODE == kDeltaCommit ? path[base + t] : base + t; };
        if (base > 0) __syncthreads();       // what the last group left is used
        for (int t = warp; t < cnt; t += W) {
            const int64_t at = at0 + token(t);
            unit_vector<D>(p.k + b * p.k_bs + at * p.k_ts + hk * p.k_hs, sh.kn[t], p.eps, lane);
            if constexpr (HAS_Q) unit_vector<D>(p.q + b * p.q_bs + at * p.q_ts + hk * p.q_hs, sh.qn[t], p.eps, lane);
        }
        if (tid < cnt) {
            const int64_t at = (row + token(tid)) * p.Hv + h;
            sh.g[tid] = p.g[at];
            sh.beta[tid] = p.beta[at];
            if constexpr (TREE) sh.parents[tid] = p.parents[(int64_t)b * p.Lq + tid];
        }
        if (base == 0) {
            slot = delta_slot<!TREE>(p, b);
            if (slot < 0) {                  // no state: outputs of zero, or NaN where it should have been one
                if constexpr (HAS_Q)
                    for (int64_t x = tid; x < (int64_t)n * D; x += 32 * W)
                        p.o[((row + x / D) * p.Hv + h) * D + x % D] = slot == -1 ? 0 : 0x7FC0;
                return;
            }
        }
        __syncthreads();
        // products among the tokens, a warp for each: along its ancestors, or the tokens before it
        for (int i = warp; i < cnt; i += W) {
            NodeKind kind = kNode;
            uint64_t above = 0;
            if constexpr (TREE) {
                int depth;
                kind = find_node(sh.parents, i, kMostNodes, above, depth);
                if (kind == kBadNode && lane == 0) record_error(p.err, kErrArg);
                if (kind != kNode) above = 0;
                if (lane == 0) {
                    sh.kind[i] = kind;
                    sh.above[i] = above;
                }
            }
            float k[D / 32], q[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                k[e] = sh.kn[i][e * 32 + lane];
                q[e] = HAS_Q ? sh.qn[i][e * 32 + lane] : 0.0f;
            }
            const float beta = sh.beta[i];
            float sum = 0.0f;                // of the decays after j, up to i
            if (kind == kNode)
                for (int j = i; j >= 0; j = TREE ? sh.parents[j] : j - 1) {
                    float kk = 0.0f, qk = 0.0f;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        const float x = sh.kn[j][e * 32 + lane];
                        kk = fmaf(k[e], x, kk);
                        qk = fmaf(q[e], x, qk);
                    }
                    // both sums at once: half the lanes go on with one each
                    const float give = lane & 16 ? kk : qk, keep = lane & 16 ? qk : kk;
                    float v = keep + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    const float a = expf(sum);
                    if (lane == 0) sh.solve[i][j] = j == i ? 0.0f : beta * a * v;
                    if (lane == 16) sh.weigh[i][j] = p.scale * a * v;
                    sum += sh.g[j];
                }
            if (lane == 0) sh.fade[i] = expf(sum);
            if constexpr (!TREE) {
                float after = 0.0f;
                for (int j = i + 1; j < cnt; ++j) after += sh.g[j];
                if (lane == 0) sh.left[i] = expf(after);
            }
        }
        __syncthreads();

#pragma unroll 1
        for (int t0 = 0; t0 < cnt; t0 += kAtOnce) {
            float v[kAtOnce], val[kAtOnce], u[kAtOnce];      // S k or S q, then the sums
#pragma unroll
            for (int t = 0; t < kAtOnce; ++t)
                v[t] = t0 + t < cnt ? bf16_lo(p.v[b * p.v_bs + (at0 + token(t0 + t)) * p.v_ts + h * p.v_hs + own]) : 0.0f;
#pragma unroll
            for (int t = 0; t < kAtOnce; ++t) {
                if (t0 + t >= cnt) break;
                float x[HAS_Q ? 8 : 4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint64_t wk = 0, wq = 0; // (two zeros)
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&sh.kn[t0 + t][m * 32 + c * 4]);
                        wk = fma2(s[i][2 * m], k.x, wk);
                        wk = fma2(s[i][2 * m + 1], k.y, wk);
                        if constexpr (HAS_Q) {
                            const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&sh.qn[t0 + t][m * 32 + c * 4]);
                            wq = fma2(s[i][2 * m], q.x, wq);
                            wq = fma2(s[i][2 * m + 1], q.y, wq);
                        }
                    }
                    const float2 a = parts_of(wk), d = parts_of(wq);
                    x[HAS_Q ? 2 * i : i] = a.x + a.y;
                    if constexpr (HAS_Q) x[2 * i + 1] = d.x + d.y;
                }
                val[t] = meet8(x, c);
            }
            float (*mine)[kGroup] = second ? sh.weigh : sh.solve;
            const float sign = second ? 1.0f : -1.0f;
#pragma unroll
            for (int t = 0; t < kAtOnce; ++t) {
                const int i = t0 + t;
                if (i >= cnt) break;
                float x = sh.fade[i] * val[t];
                x = second ? p.scale * x : sh.beta[i] * (v[t] - x);
                // (a node takes its ancestors alone: the others may hold anything)
                const uint64_t above = TREE ? sh.above[i] : ~0ull;
                for (int j = 0; j < t0; ++j)
                    if (!TREE || (above >> j & 1)) x = fmaf(sign * mine[i][j], sh.u[warp][j][r * 4 + (c >> 1)], x);
#pragma unroll
                for (int j = 0; j < t; ++j)
                    if (!TREE || (above >> (t0 + j) & 1)) x = fmaf(sign * mine[i][t0 + j], u[j], x);
                u[t] = HAS_Q ? __shfl_sync(0xffffffffu, x, lane & ~1) : x;
                if (second) {
                    uint32_t out = 0;
                    const NodeKind kind = TREE ? sh.kind[i] : kNode;
                    if (kind == kNode)
                        out = pack_bf16x2(fmaf(mine[i][i], u[t], x), 0.0f);
                    else if (kind == kBadNode)
                        out = 0x7FC0u;
                    p.o[((row + base + i) * p.Hv + h) * D + own] = (uint16_t)out;
                }
                if (!(c & 1)) sh.u[warp][i][r * 4 + (c >> 1)] = u[t];
            }
            __syncwarp();
        }
        if constexpr (!TREE) {
            if (cnt > 0) {
                const float a = sh.fade[cnt - 1];
                const uint64_t all = pair_of(a, a);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int m = 0; m < 2 * M; ++m) s[i][m] = mul2(s[i][m], all);
            }
#pragma unroll 4
            for (int t = 0; t < cnt; ++t) {
                const float left = sh.left[t];
                const float4 w = *reinterpret_cast<const float4*>(&sh.u[warp][t][r * 4]);
                const float x[4] = {left * w.x, left * w.y, left * w.z, left * w.w};
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&sh.kn[t][m * 32 + c * 4]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[i][2 * m] = fma2(pair_of(x[i], x[i]), k.x, s[i][2 * m]);
                        s[i][2 * m + 1] = fma2(pair_of(x[i], x[i]), k.y, s[i][2 * m + 1]);
                    }
                }
            }
        }
    }
    if constexpr (!TREE) {
        if (n == 0 && !p.from_zero) return;  // as it is
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < M; ++m)
                *reinterpret_cast<ulonglong2*>(rows + (r + 4 * i) * D + m * 32 + c * 4) =
                    make_ulonglong2(s[i][2 * m], s[i][2 * m + 1]);
    }
}

// The eight elements' pairs that a lane has of a bf16 head vector (those of its share of a state's row), and the vector's
// 1 / length.
template <int D>
__device__ __forceinline__ float lane_vector(const uint16_t* src, int c, uint64_t (&x)[D / 16], float eps) {
    uint64_t sum = 0;
#pragma unroll
    for (int m = 0; m < D / 32; ++m) {
        const uint2 w = *reinterpret_cast<const uint2*>(src + m * 32 + c * 4);
        x[2 * m] = pair_of(bf16_lo(w.x), bf16_hi(w.x));
        x[2 * m + 1] = pair_of(bf16_lo(w.y), bf16_hi(w.y));
        sum = fma2(x[2 * m], x[2 * m], sum);
        sum = fma2(x[2 * m + 1], x[2 * m + 1], sum);
    }
    const float2 f = parts_of(sum);
    return rsqrtf(group_sum<8>(f.x + f.y) + eps);
}

// One token a sequence: every warp for itself, without shared memory.
constexpr int kWarps = 4, kThreads = 32 * kWarps;
template <int D>
__global__ void __launch_bounds__(kThreads, 4) delta_one_kernel(const DeltaParams p) {
    constexpr int PARTS = D / (kWarps * kRows), M = D / 32;
    begin_chained();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 7, r = lane >> 3;
    const int part = blockIdx.x % PARTS, bh = blockIdx.x / PARTS, b = bh / p.Hv, h = bh - b * p.Hv, hk = h / p.ratio;
    const int row0 = (part * kWarps + warp) * kRows, own = row0 + r + 4 * (c >> 1);
    const int first_slot = p.slots[b];
    float* rows = p.state + (((int64_t)(first_slot >= 0 && first_slot < p.n_states ? first_slot : 0) * p.Hv + h) * D + row0) * D;
    uint64_t s[4][2 * M];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            ulonglong2 x = make_ulonglong2(0ull, 0ull);
            if (!p.from_zero) x = *reinterpret_cast<const ulonglong2*>(rows + (r + 4 * i) * D + m * 32 + c * 4);
            s[i][2 * m] = x.x;
            s[i][2 * m + 1] = x.y;
        }
    uint16_t* o = p.o + ((int64_t)b * p.Hv + h) * D + own;
    const float g = p.g[(int64_t)b * p.Hv + h], beta = p.beta[(int64_t)b * p.Hv + h];
    const float v = bf16_lo(p.v[b * p.v_bs + h * p.v_hs + own]);
    uint64_t k[2 * M], q[2 * M];
    const float rk = lane_vector<D>(p.k + b * p.k_bs + hk * p.k_hs, c, k, p.eps);
    const float rq = lane_vector<D>(p.q + b * p.q_bs + hk * p.q_hs, c, q, p.eps);
    const uint64_t rk2 = pair_of(rk, rk);
    uint64_t kq = 0;
#pragma unroll
    for (int m = 0; m < 2 * M; ++m) {
        k[m] = mul2(k[m], rk2);
        kq = fma2(k[m], q[m], kq);
    }
    const float2 both = parts_of(kq);
    const float qk = group_sum<8>(both.x + both.y), a = expf(g);
    const int slot = delta_slot<true>(p, b);
    if (slot < 0) {
        if (c & 1) *o = slot == -1 ? 0 : 0x7FC0;
        return;
    }
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t wk = 0, wq = 0;
#pragma unroll
        for (int m = 0; m < 2 * M; ++m) {
            wk = fma2(s[i][m], k[m], wk);
            wq = fma2(s[i][m], q[m], wq);
        }
        const float2 d = parts_of(wk), e = parts_of(wq);
        x[2 * i] = d.x + d.y;
        x[2 * i + 1] = e.x + e.y;
    }
    const float val = a * meet8(x, c);
    const float u = __shfl_sync(0xffffffffu, beta * (v - val), lane & ~1);
    if (c & 1) *o = (uint16_t)pack_bf16x2(p.scale * rq * fmaf(qk, u, val), 0.0f);
    const uint64_t a2 = pair_of(a, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float w = __shfl_sync(0xffffffffu, u, (lane & 24) | (2 * i));
        const uint64_t w2 = pair_of(w, w);
#pragma unroll
        for (int m = 0; m < M; ++m)
            *reinterpret_cast<ulonglong2*>(rows + (r + 4 * i) * D + m * 32 + c * 4) =
                make_ulonglong2(fma2(w2, k[2 * m], mul2(a2, s[i][2 * m])), fma2(w2, k[2 * m + 1], mul2(a2, s[i][2 * m + 1])));
    }
}

template <int D>
cudaError_t launch_one(const DeltaParams& p, cudaStream_t st) {
    return launch_chained(delta_one_kernel<D>, (unsigned)p.B * p.Hv * (D / (kWarps * kRows)), kThreads, 0, st, p);
}

template <int D, DeltaMode MODE>
cudaError_t launch_rows(const DeltaParams& p, cudaStream_t st) {
    return launch_chained(delta_rows_kernel<D, MODE>, (unsigned)p.B * p.Hv, 32 * warps_of(D), 0, st, p);
}

}  // namespace

cudaError_t launch_delta(int D, DeltaMode mode, const DeltaParams& p, cudaStream_t st) {
    // This file's kernel takes about 1 us a token beyond its loads, for all of a wave of CTAs; the one
    // in chunks 10 to 16 us for up to 64 tokens, with one CTA an SM.  Measured, us here and in chunks, of the
    // steps of n tokens: one sequence of 32 heads of 128: n = 8 9.8 and 14.7, 12 14.5 and 14.8, 16 18.0 and 14.8; 16
    // sequences: 16 47 and 56, 24 66 and 56; 64: 16 184 and 200, 24 255 and 203; 12 heads of 64, 16 sequences: 16
    // 19.7 and 20.8, 24 27 and 21.  Trees alike: one of 12 nodes 11.8 and 12.3, of 16 14.8 and 12.4, 16 of 16 41 and 49 (with the
    // states in L2 35 and 45).
    const bool waves = (int64_t)p.B * p.Hv > 152;
    bool few = p.Lq <= (waves ? kGroup : 12);
    // A path is as long as what was accepted, not as its width: of 64 sequences 32 wide 111 and 191 with a third
    // of it taken, 262 and 201 with all; 48 wide 148 and 195, 378 and 212.
    if (mode == kDeltaCommit) few = p.P <= 32;
    // One of the packed sequences may have all of their tokens.  (Of a token each they are steps.)
    if (p.cu) few = p.T <= max(p.B, 12);
    if (!few) return launch_delta_chunks(D, mode, p, st);
    if (mode == kDeltaChain && !p.cu && p.Lq == 1) return D == 64 ? launch_one<64>(p, st) : launch_one<128>(p, st);
    if (mode == kDeltaChain) return D == 64 ? launch_rows<64, kDeltaChain>(p, st) : launch_rows<128, kDeltaChain>(p, st);
    if (mode == kDeltaTree) return D == 64 ? launch_rows<64, kDeltaTree>(p, st) : launch_rows<128, kDeltaTree>(p, st);
    return D == 64 ? launch_rows<64, kDeltaCommit>(p, st) : launch_rows<128, kDeltaCommit>(p, st);
}

}  // namespace r9q
