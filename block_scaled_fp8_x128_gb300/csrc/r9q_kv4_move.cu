// Tokens moved between places of the 4-bit cache: what an accepted path of drafted tokens
// leaves is made contiguous.  Codes and pairs are copied as they are, so nothing is rounded
// again.
//
// A CTA takes one head of a row of moves: all its tokens (136 bytes each at D = 128) come
// into shared memory before any is written, so that a row may move tokens over one another.
// A token's value codes are single bytes among those of 15 others (r9q_kv4.cuh), read
// and written as such.  Bound: latency, the chain slots -> codes -> shared memory -> codes.
#include "r9q_delta.cuh"

namespace r9q {

namespace {

constexpr int kThreads = 128;

// A token of a head: the first byte of its keys, of its value group, its place in it, and its pairs' index.
struct Spot {
    int64_t k, v, pair;
};
template <int D>
__device__ __forceinline__ Spot spot_of(const Kv4Cache& c, int64_t slot, int h) {
    const int64_t page = slot / c.page, head = page * c.heads + h, at = slot - page * c.page;
    return {(head * c.page + at) * (D / 2), head * kv4_head_bytes(c.page, D) + (at >> 4) * (8 * D) + kv4_v_token_byte((int)at & 15),
            head * c.page + at};
}

template <int D>
__global__ void __launch_bounds__(kThreads) move_kernel(const Kv4Cache c, const int64_t* src, const int64_t* dst, int n,
                                                        int* err) {
    constexpr int NL = D / 8;                // threads of a token: four bytes of keys and four of values each
    __shared__ int64_t from[kMostNodes], to[kMostNodes];
    __shared__ uint32_t kq[kMostNodes][NL], vq[kMostNodes][NL], pairs[kMostNodes][2];
    begin_chained();
    const int tid = threadIdx.x, row = blockIdx.x / c.heads, h = blockIdx.x - row * c.heads;
    const int l = tid % NL;
    if (tid < n) {
        int64_t a = src[(int64_t)row * n + tid], b = dst[(int64_t)row * n + tid];
        const int64_t end = c.pages * c.page;
        if (a >= end || b >= end) record_error(err, kErrArg);
        if (a < 0 || b < 0 || a >= end || b >= end) a = b = -1;
        from[tid] = a;
        to[tid] = b;
    }
    __syncthreads();
    for (int i = tid / NL; i < n; i += kThreads / NL) {
        if (from[i] < 0) continue;
        const Spot s = spot_of<D>(c, from[i], h);
        kq[i][l] = reinterpret_cast<const uint32_t*>(c.k + s.k)[l];
        uint32_t w = 0;                      // rows r = 4 (l & 1) .. + 3 of element tile l >> 1
        const uint8_t* at = c.v + s.v + (l >> 3) * 512 + ((l >> 1) & 3) * 4 + (l & 1) * 256;
#pragma unroll
        for (int x = 0; x < 4; ++x) w |= (uint32_t)at[x * 64] << (8 * x);
        vq[i][l] = w;
        if (l < 2) pairs[i][l] = (l ? c.vp : c.kp)[s.pair];
    }
    __syncthreads();
    for (int i = tid / NL; i < n; i += kThreads / NL) {
        bool live = from[i] >= 0;
        for (int x = i + 1; live && x < n; ++x) live = to[x] != to[i];       // of two at one place the later stays
        if (!live) continue;
        const Spot s = spot_of<D>(c, to[i], h);
        reinterpret_cast<uint32_t*>(c.k + s.k)[l] = kq[i][l];
        uint8_t* at = c.v + s.v + (l >> 3) * 512 + ((l >> 1) & 3) * 4 + (l & 1) * 256;
#pragma unroll
        for (int x = 0; x < 4; ++x) at[x * 64] = (uint8_t)(vq[i][l] >> (8 * x));
        if (l < 2) (l ? c.vp : c.kp)[s.pair] = pairs[i][l];
    }
}

}  // namespace

cudaError_t launch_kv4_move(int D, const Kv4Cache& c, const int64_t* src, const int64_t* dst, int64_t rows, int per_row,
                            int* err, cudaStream_t st) {
    auto kernel = D == 64 ? move_kernel<64> : move_kernel<128>;
    return launch_chained(kernel, (unsigned)(rows * c.heads), kThreads, 0, st, c, src, dst, per_row, err);
}

}  // namespace r9q
