// The gated delta rule: parameters and helpers of its kernels.
//
// A value head's memory is a matrix S [D values][D keys] in fp32; a token of unit key k and
// query q, value v, decay a = exp(g) and rate beta does
//   S <- a S + u k^T,  u = beta (v - a S k),  o = scale S q.
// Over tokens 1..n from a state S the same in sums, with A(i, j) = exp(g_j+1 + ... + g_i):
//   u_i = beta_i (v_i - A(i, 0) S k_i - sum_{j<i} A(i, j) (k_i.k_j) u_j)
//   o_i = scale (A(i, 0) S q_i + sum_{j<=i} A(i, j) (q_i.k_j) u_j)
//   S   <- A(n, 0) S + sum_j A(n, j) u_j k_j^T
// and along a tree with the sums over a node's ancestors and A along the path.  Decays are
// always taken forward (no quotient of them), so that any g <= 0 holds, -infinity too.
#pragma once

#include "r9q_kv4.cuh"

namespace r9q {

// The slot of sequence b.  One that is out of range or, where states are written, that an earlier sequence of the
// call has too is an error; the whole CTA calls this.
template <bool WRITES>
__device__ __forceinline__ int delta_slot(const DeltaParams& p, int b) {
    const int slot = p.slots[b];
    bool bad = slot >= p.n_states;
    if constexpr (WRITES) {
        bool twice = false;
        if (slot >= 0)
            for (int x = threadIdx.x; x < b; x += blockDim.x) twice = twice || p.slots[x] == slot;
        bad = __syncthreads_or(twice) || bad;
    }
    if (bad) {
        if (threadIdx.x == 0) record_error(p.err, kErrArg);
        return -2;
    }
    return slot < 0 ? -1 : slot;
}

// Where sequence b's tokens are.  Offsets that decrease or leave the tokens are an error: no tokens.
__device__ __forceinline__ void delta_tokens(const DeltaParams& p, int b, int& n, int64_t& row) {
    n = p.Lq;
    row = (int64_t)b * p.Lq;
    if (p.cu) {
        const int from = p.cu[b], to = p.cu[b + 1];
        const bool ok = from >= 0 && from <= to && to <= p.T;
        if (!ok && threadIdx.x == 0) record_error(p.err, kErrArg);
        n = ok ? to - from : 0;
        row = ok ? from : 0;
    }
}

// The nodes of sequence b's path: up to the first entry that is not one, an error where that is Lq or more.  What stands behind
// it, or in the path of a place without a sequence, is not looked at.  Whole warps call this.
__device__ __forceinline__ int path_length(const DeltaParams& p, int b) {
    const int32_t* path = p.path + (int64_t)b * p.P;
    const int lane = threadIdx.x & 31;
    uint64_t ends = 0, out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = i * 32 + lane, node = at < p.P ? path[at] : -1;
        ends |= (uint64_t)__ballot_sync(0xffffffffu, node < 0 || node >= p.Lq) << (32 * i);
        out |= (uint64_t)__ballot_sync(0xffffffffu, node >= p.Lq) << (32 * i);
    }
    if (ends == 0) return p.P;
    const int n = __ffsll((long long)ends) - 1;
    if (threadIdx.x == 0 && (out >> n & 1) && p.slots[b] >= 0) record_error(p.err, kErrArg);
    return n;
}

// A node of a tree, found by following its parents in shared memory: its ancestors and itself, a bit each; fewer
// than all of them where `most` (a window) ends before the tree does.
enum NodeKind { kNode, kNoNode, kBadNode };
__device__ __forceinline__ NodeKind find_node(const int* parents, int i, int most, uint64_t& mask, int& depth) {
    mask = 0;
    depth = 0;
    if (parents[i] == -2) return kNoNode;
    for (int t = i;; ++depth) {
        if (depth < most) mask |= 1ull << t;
        const int up = parents[t];
        if (up == -1) return kNode;
        if (up < 0 || up >= t) return kBadNode;
        t = up;
    }
}

}  // namespace r9q
