// C ABI of the attention operators (declared in include/r9q.h): QK norm with
// rotation, its gradient, the paged 4-bit cache and the attention over it.
// Argument checks and dispatch, as in r9q_api.cu.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "r9q.h"
#include "r9q_kernels.h"

namespace r9q {
namespace {

constexpr size_t kCounterHeader = 64 * 1024;     // the workspace header that every call leaves at zero

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Half-open byte range of a tensor.
struct Extent {
    uintptr_t lo, hi;
};
Extent bytes_of(const void* p, int64_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + (p ? (uintptr_t)n : 0)};
}
bool meet(const Extent& a, const Extent& b) { return a.lo < b.hi && b.lo < a.hi; }

bool dims_ok(int64_t T, int64_t heads, int64_t D) {
    return T >= 0 && T <= INT_MAX && heads >= 1 && heads <= 4096 && (D == 64 || D == 128);
}

// Stride of a dimension of n: one that is never used counts as none.
bool stride_ok(int64_t n, int64_t s) { return n <= 1 || (s >= 0 && s <= ((int64_t)1 << 40)); }
bool stride_aligned(int64_t n, int64_t s) { return n <= 1 || s % 8 == 0; }
// A [T][heads][D] bf16 tensor with free token and head strides (elements).
int check_heads(const void* p, int64_t T, int64_t ts, int64_t heads, int64_t hs) {
    if (!p) return R9Q_ERR_NULL;
    if (!stride_ok(T, ts) || !stride_ok(heads, hs)) return R9Q_ERR_ARG;
    return aligned(p, 16) && stride_aligned(T, ts) && stride_aligned(heads, hs) ? R9Q_OK : R9Q_ERR_ALIGN;
}
// An output's vectors may not share memory with one another.
bool spread(int64_t T, int64_t heads, int64_t D, int64_t ts, int64_t hs) {
    if (T == 1) return heads == 1 || hs >= D;
    if (heads == 1) return ts >= D;
    return hs <= ts ? hs >= D && ts >= (heads - 1) * hs + D : ts >= D && hs >= (T - 1) * ts + D;
}
Extent extent(const void* p, int64_t T, int64_t heads, int64_t D, int64_t ts, int64_t hs) {
    return bytes_of(p, 2 * ((T > 1 ? (T - 1) * ts : 0) + (heads > 1 ? (heads - 1) * hs : 0) + D));
}

int check_rope(const float* wq, const float* wk, const float* cos, const float* sin, const int64_t* pos, int64_t D,
               int64_t rot, int64_t npos, float eps, int flags) {
    if (flags & ~R9Q_ROPE_INTERLEAVED) return R9Q_ERR_ARG;
    if (!wq || !wk || (rot > 0 && (!cos || !sin || !pos))) return R9Q_ERR_NULL;
    if (rot < 0 || rot > D || rot % 16 || (rot > 0 && npos < 1)) return R9Q_ERR_DIM;
    if (!(eps >= 0.0f) || std::isinf(eps)) return R9Q_ERR_ARG;
    if (!aligned(wq, 4) || !aligned(wk, 4) || !aligned(cos, 16) || !aligned(sin, 16) || !aligned(pos, 8))
        return R9Q_ERR_ALIGN;
    return R9Q_OK;
}
// An output over what the rotation reads.
bool rope_meets(const float* wq, const float* wk, const float* cos, const float* sin, const int64_t* pos, int64_t T,
                int64_t D, int64_t rot, int64_t npos, const Extent& x) {
    if (meet(bytes_of(wq, D * 4), x) || meet(bytes_of(wk, D * 4), x)) return true;
    const int64_t table = std::min(npos, (int64_t)1 << 40) * rot * 2;          // (rot / 2 floats a row)
    return rot > 0 && (meet(bytes_of(cos, table), x) || meet(bytes_of(sin, table), x) || meet(bytes_of(pos, T * 8), x));
}
RopeParams rope_params(const float* wq, const float* wk, const float* cos, const float* sin, const int64_t* pos,
                       int64_t T, int64_t rot, int64_t npos, float eps, int flags, int* err) {
    RopeParams p = {};
    p.wq = wq;
    p.wk = wk;
    p.cos = cos;
    p.sin = sin;
    p.pos = pos;
    p.T = T;
    p.npos = npos;
    p.rot = (int)rot;
    p.eps = eps;
    p.interleaved = flags & R9Q_ROPE_INTERLEAVED ? 1 : 0;
    p.err = err;
    return p;
}

int check_cache(const void* k, const void* kp, const void* v, const void* vp, int64_t pages, int64_t heads,
                int64_t page) {
    if (!k || !kp || !v || !vp) return R9Q_ERR_NULL;
    if (pages < 1 || pages > INT_MAX || page < 16 || page % 16 || page > 65536) return R9Q_ERR_DIM;
    if (pages * page > ((int64_t)1 << 32) / heads) return R9Q_ERR_DIM;      // (the kernels count vectors in 32 bits)
    return aligned(k, 16) && aligned(v, 16) && aligned(kp, 4) && aligned(vp, 4) ? R9Q_OK : R9Q_ERR_ALIGN;
}
Kv4Cache cache_of(const void* k, const void* kp, const void* v, const void* vp, int64_t pages, int64_t heads,
                  int64_t page) {
    Kv4Cache c = {};
    c.k = static_cast<uint8_t*>(const_cast<void*>(k));
    c.kp = static_cast<uint32_t*>(const_cast<void*>(kp));
    c.v = static_cast<uint8_t*>(const_cast<void*>(v));
    c.vp = static_cast<uint32_t*>(const_cast<void*>(vp));
    c.pages = pages;
    c.heads = (int)heads;
    c.page = (int)page;
    return c;
}
// The four buffers apart from one another, and from [x, x + n) of the others.
bool cache_meets(const Kv4Cache& c, int64_t D, const Extent& x) {
    const int64_t vectors = c.pages * c.heads * c.page;
    return meet(bytes_of(c.k, vectors * (D / 2)), x) || meet(bytes_of(c.v, vectors * (D / 2)), x) ||
           meet(bytes_of(c.kp, vectors * 4), x) || meet(bytes_of(c.vp, vectors * 4), x);
}
bool cache_meets_rope(const Kv4Cache& c, int64_t D, const float* wq, const float* wk, const float* cos, const float* sin,
                      const int64_t* pos, int64_t T, int64_t rot, int64_t npos) {
    const int64_t vectors = c.pages * c.heads * c.page;
    for (const Extent& x : {bytes_of(c.k, vectors * (D / 2)), bytes_of(c.v, vectors * (D / 2)), bytes_of(c.kp, vectors * 4),
                            bytes_of(c.vp, vectors * 4)})
        if (rope_meets(wq, wk, cos, sin, pos, T, D, rot, npos, x)) return true;
    return false;
}
bool cache_overlaps_itself(const Kv4Cache& c, int64_t D) {
    const int64_t vectors = c.pages * c.heads * c.page;
    const Extent e[4] = {bytes_of(c.k, vectors * (D / 2)), bytes_of(c.v, vectors * (D / 2)), bytes_of(c.kp, vectors * 4),
                         bytes_of(c.vp, vectors * 4)};
    for (int i = 0; i < 4; ++i)
        for (int k = 0; k < i; ++k)
            if (meet(e[i], e[k])) return true;
    return false;
}

HeadsIn heads_in(const void* p, int64_t ts, int64_t hs, int64_t heads) {
    return {static_cast<const uint16_t*>(p), ts, hs, (int)heads};
}
HeadsOut heads_out(void* p, int64_t ts, int64_t hs) { return {static_cast<uint16_t*>(p), ts, hs}; }

int status(cudaError_t e) {
    if (e == cudaSuccess) return R9Q_OK;
    (void)cudaGetLastError();                    // no pending error is left for the caller
    return R9Q_ERR_LAUNCH;
}

// The device's SM count; a GB300's where a workspace is asked for without one.
int sms_or_default() {
    int* err = nullptr;
    int sms = 0;
    return device_error_word_and_sms(&err, &sms) == R9Q_OK ? sms : 152;
}

}  // namespace

size_t decode_workspace(int op, int64_t M, int64_t N, int* rc) {
    *rc = R9Q_OK;
    if (N != 64 && N != 128) {
        *rc = R9Q_ERR_DIM;
        return 0;
    }
    if (op == R9Q_OP_QK_NORM_ROPE_BWD)
        return kCounterHeader + (size_t)qk_norm_rope_bwd_blocks(sms_or_default()) * 2 * (size_t)N * 4;
    if (M < 1) {
        *rc = R9Q_ERR_DIM;
        return 0;
    }
    return kCounterHeader + kv4_attention_part_floats((int)N, M, sms_or_default()) * 4;
}

}  // namespace r9q

using namespace r9q;

extern "C" {

int r9q_qk_norm_rope(const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts, int64_t k_hs,
                     const float* wq, const float* wk, const float* cos, const float* sin, const int64_t* pos,
                     void* q_out, int64_t qo_ts, int64_t qo_hs, void* k_out, int64_t ko_ts, int64_t ko_hs, int64_t T,
                     int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t npos, float eps, int flags,
                     void* stream) {
    if (!dims_ok(T, Hq, D) || !dims_ok(T, Hk, D)) return R9Q_ERR_DIM;
    if (T == 0) return R9Q_OK;
    int rc = check_rope(wq, wk, cos, sin, pos, D, rot, npos, eps, flags);
    if (!rc) rc = check_heads(q, T, q_ts, Hq, q_hs);
    if (!rc) rc = check_heads(k, T, k_ts, Hk, k_hs);
    if (!rc) rc = check_heads(q_out, T, qo_ts, Hq, qo_hs);
    if (!rc) rc = check_heads(k_out, T, ko_ts, Hk, ko_hs);
    if (rc) return rc;
    if (!spread(T, Hq, D, qo_ts, qo_hs) || !spread(T, Hk, D, ko_ts, ko_hs)) return R9Q_ERR_ARG;
    const Extent in[2] = {extent(q, T, Hq, D, q_ts, q_hs), extent(k, T, Hk, D, k_ts, k_hs)};
    const Extent out[2] = {extent(q_out, T, Hq, D, qo_ts, qo_hs), extent(k_out, T, Hk, D, ko_ts, ko_hs)};
    for (const Extent& o : out) {
        if (rope_meets(wq, wk, cos, sin, pos, T, D, rot, npos, o)) return R9Q_ERR_ARG;
        for (const Extent& i : in)
            if (meet(i, o)) return R9Q_ERR_ARG;
    }
    int *err = nullptr, sms = 0;
    rc = device_error_word_and_sms(&err, &sms);
    if (rc) return rc;
    return status(launch_qk_norm_rope((int)D, heads_in(q, q_ts, q_hs, Hq), heads_in(k, k_ts, k_hs, Hk),
                                      rope_params(wq, wk, cos, sin, pos, T, rot, npos, eps, flags, err),
                                      heads_out(q_out, qo_ts, qo_hs), heads_out(k_out, ko_ts, ko_hs),
                                      static_cast<cudaStream_t>(stream)));
}

int r9q_qk_norm_rope_bwd(const void* dq_out, int64_t dqo_ts, int64_t dqo_hs, const void* dk_out, int64_t dko_ts,
                         int64_t dko_hs, const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts,
                         int64_t k_hs, const float* wq, const float* wk, const float* cos, const float* sin,
                         const int64_t* pos, void* dq, int64_t dq_ts, int64_t dq_hs, void* dk, int64_t dk_ts,
                         int64_t dk_hs, float* dwq, float* dwk, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                         int64_t rot, int64_t npos, float eps, int flags, void* workspace, size_t workspace_bytes,
                         void* stream) {
    if (!dims_ok(T, Hq, D) || !dims_ok(T, Hk, D)) return R9Q_ERR_DIM;
    if (!dwq || !dwk) return R9Q_ERR_NULL;
    if (!aligned(dwq, 4) || !aligned(dwk, 4)) return R9Q_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int *err = nullptr, sms = 0;
    if (T == 0) {                                             // no token: the weights' gradients are zero
        const int rc = device_error_word_and_sms(&err, &sms);
        if (rc) return rc;
        if (cudaMemsetAsync(dwq, 0, D * 4, st) != cudaSuccess || cudaMemsetAsync(dwk, 0, D * 4, st) != cudaSuccess)
            return R9Q_ERR_LAUNCH;
        return R9Q_OK;
    }
    int rc = check_rope(wq, wk, cos, sin, pos, D, rot, npos, eps, flags);
    if (!rc) rc = check_heads(dq_out, T, dqo_ts, Hq, dqo_hs);
    if (!rc) rc = check_heads(dk_out, T, dko_ts, Hk, dko_hs);
    if (!rc) rc = check_heads(q, T, q_ts, Hq, q_hs);
    if (!rc) rc = check_heads(k, T, k_ts, Hk, k_hs);
    if (!rc) rc = check_heads(dq, T, dq_ts, Hq, dq_hs);
    if (!rc) rc = check_heads(dk, T, dk_ts, Hk, dk_hs);
    if (rc) return rc;
    if (!spread(T, Hq, D, dq_ts, dq_hs) || !spread(T, Hk, D, dk_ts, dk_hs)) return R9Q_ERR_ARG;
    const Extent in[4] = {extent(dq_out, T, Hq, D, dqo_ts, dqo_hs), extent(dk_out, T, Hk, D, dko_ts, dko_hs),
                          extent(q, T, Hq, D, q_ts, q_hs), extent(k, T, Hk, D, k_ts, k_hs)};
    const Extent out[4] = {extent(dq, T, Hq, D, dq_ts, dq_hs), extent(dk, T, Hk, D, dk_ts, dk_hs),
                           bytes_of(dwq, D * 4), bytes_of(dwk, D * 4)};
    for (const Extent& o : out) {
        if (rope_meets(wq, wk, cos, sin, pos, T, D, rot, npos, o)) return R9Q_ERR_ARG;
        for (const Extent& i : in)
            if (meet(i, o)) return R9Q_ERR_ARG;
    }
    if (meet(out[2], out[3]) || meet(out[0], out[2]) || meet(out[0], out[3]) || meet(out[1], out[2]) ||
        meet(out[1], out[3]))
        return R9Q_ERR_ARG;
    rc = device_error_word_and_sms(&err, &sms);
    if (rc) return rc;
    const size_t need = decode_workspace(R9Q_OP_QK_NORM_ROPE_BWD, 1, D, &rc);
    if (!workspace || workspace_bytes < need) return R9Q_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return R9Q_ERR_ALIGN;
    const Extent ws = bytes_of(workspace, (int64_t)need);
    if (rope_meets(wq, wk, cos, sin, pos, T, D, rot, npos, ws)) return R9Q_ERR_ARG;
    for (const Extent& i : in)
        if (meet(i, ws)) return R9Q_ERR_ARG;
    for (const Extent& o : out)
        if (meet(o, ws)) return R9Q_ERR_ARG;
    return status(launch_qk_norm_rope_bwd(
        (int)D, heads_in(dq_out, dqo_ts, dqo_hs, Hq), heads_in(dk_out, dko_ts, dko_hs, Hk), heads_in(q, q_ts, q_hs, Hq),
        heads_in(k, k_ts, k_hs, Hk), rope_params(wq, wk, cos, sin, pos, T, rot, npos, eps, flags, err),
        heads_out(dq, dq_ts, dq_hs), heads_out(dk, dk_ts, dk_hs), dwq, dwk,
        reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterHeader), static_cast<int*>(workspace), sms,
        st));
}

int r9q_qk_norm_rope_kv4(const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts, int64_t k_hs,
                         const void* v, int64_t v_ts, int64_t v_hs, const float* wq, const float* wk,
                         const float* cos, const float* sin, const int64_t* pos, void* q_out, int64_t qo_ts,
                         int64_t qo_hs, uint8_t* kc, void* kp, uint8_t* vc, void* vp, const int64_t* slots, int64_t T,
                         int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t npos, int64_t pages, int64_t page,
                         float eps, int flags, void* stream) {
    if (!dims_ok(T, Hq, D) || !dims_ok(T, Hk, D)) return R9Q_ERR_DIM;
    if (T == 0) return R9Q_OK;
    int rc = check_rope(wq, wk, cos, sin, pos, D, rot, npos, eps, flags);
    if (!rc) rc = check_heads(q, T, q_ts, Hq, q_hs);
    if (!rc) rc = check_heads(k, T, k_ts, Hk, k_hs);
    if (!rc) rc = check_heads(v, T, v_ts, Hk, v_hs);
    if (!rc) rc = check_heads(q_out, T, qo_ts, Hq, qo_hs);
    if (!rc) rc = check_cache(kc, kp, vc, vp, pages, Hk, page);
    if (!rc && !slots) rc = R9Q_ERR_NULL;
    if (!rc && !aligned(slots, 8)) rc = R9Q_ERR_ALIGN;
    if (rc) return rc;
    if (!spread(T, Hq, D, qo_ts, qo_hs)) return R9Q_ERR_ARG;
    const Kv4Cache c = cache_of(kc, kp, vc, vp, pages, Hk, page);
    const Extent in[3] = {extent(q, T, Hq, D, q_ts, q_hs), extent(k, T, Hk, D, k_ts, k_hs),
                          extent(v, T, Hk, D, v_ts, v_hs)};
    const Extent out = extent(q_out, T, Hq, D, qo_ts, qo_hs);
    for (const Extent& i : in)
        if (meet(i, out) || cache_meets(c, D, i)) return R9Q_ERR_ARG;
    if (cache_meets(c, D, out) || cache_overlaps_itself(c, D)) return R9Q_ERR_ARG;
    const Extent at = bytes_of(slots, T * 8);
    if (meet(at, out) || cache_meets(c, D, at) || rope_meets(wq, wk, cos, sin, pos, T, D, rot, npos, out) ||
        cache_meets_rope(c, D, wq, wk, cos, sin, pos, T, rot, npos))
        return R9Q_ERR_ARG;
    int *err = nullptr, sms = 0;
    rc = device_error_word_and_sms(&err, &sms);
    if (rc) return rc;
    return status(launch_qk_norm_rope_kv4((int)D, heads_in(q, q_ts, q_hs, Hq), heads_in(k, k_ts, k_hs, Hk),
                                          heads_in(v, v_ts, v_hs, Hk),
                                          rope_params(wq, wk, cos, sin, pos, T, rot, npos, eps, flags, err),
                                          heads_out(q_out, qo_ts, qo_hs), c, slots, static_cast<cudaStream_t>(stream)));
}

int r9q_kv4_append(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, uint8_t* kc,
                   void* kp, uint8_t* vc, void* vp, const int64_t* slots, int64_t T, int64_t Hk, int64_t D,
                   int64_t pages, int64_t page, void* stream) {
    if (!dims_ok(T, Hk, D)) return R9Q_ERR_DIM;
    if (T == 0) return R9Q_OK;
    int rc = check_heads(k, T, k_ts, Hk, k_hs);
    if (!rc) rc = check_heads(v, T, v_ts, Hk, v_hs);
    if (!rc) rc = check_cache(kc, kp, vc, vp, pages, Hk, page);
    if (!rc && !slots) rc = R9Q_ERR_NULL;
    if (!rc && !aligned(slots, 8)) rc = R9Q_ERR_ALIGN;
    if (rc) return rc;
    const Kv4Cache c = cache_of(kc, kp, vc, vp, pages, Hk, page);
    if (cache_meets(c, D, extent(k, T, Hk, D, k_ts, k_hs)) || cache_meets(c, D, extent(v, T, Hk, D, v_ts, v_hs)) ||
        cache_meets(c, D, bytes_of(slots, T * 8)) || cache_overlaps_itself(c, D))
        return R9Q_ERR_ARG;
    int *err = nullptr, sms = 0;
    rc = device_error_word_and_sms(&err, &sms);
    if (rc) return rc;
    return status(launch_kv4_append((int)D, heads_in(k, k_ts, k_hs, Hk), heads_in(v, v_ts, v_hs, Hk), T, c, slots, err,
                                    static_cast<cudaStream_t>(stream)));
}

int r9q_kv4_gather(const uint8_t* kc, const void* kp, const uint8_t* vc, const void* vp, const int64_t* slots,
                   int64_t T, int64_t Hk, int64_t D, int64_t pages, int64_t page, void* k, void* v, void* stream) {
    if (!dims_ok(T, Hk, D)) return R9Q_ERR_DIM;
    if (T == 0) return R9Q_OK;
    int rc = check_cache(kc, kp, vc, vp, pages, Hk, page);
    if (!rc && (!slots || !k || !v)) rc = R9Q_ERR_NULL;
    if (!rc && (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16))) rc = R9Q_ERR_ALIGN;
    if (rc) return rc;
    const Kv4Cache c = cache_of(kc, kp, vc, vp, pages, Hk, page);
    const Extent ke = bytes_of(k, 2 * T * Hk * D), ve = bytes_of(v, 2 * T * Hk * D);
    const Extent at = bytes_of(slots, T * 8);
    if (meet(ke, ve) || meet(ke, at) || meet(ve, at) || cache_meets(c, D, ke) || cache_meets(c, D, ve)) return R9Q_ERR_ARG;
    int *err = nullptr, sms = 0;
    rc = device_error_word_and_sms(&err, &sms);
    if (rc) return rc;
    return status(launch_kv4_gather((int)D, c, slots, T, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), err,
                                    static_cast<cudaStream_t>(stream)));
}

int r9q_kv4_attention(const void* q, int64_t q_bs, int64_t q_ts, int64_t q_hs, const uint8_t* kc, const void* kp,
                      const uint8_t* vc, const void* vp, const int32_t* block_table, const int32_t* seq_lens, void* o,
                      float* lse, int64_t B, int64_t Lq, int64_t Hq, int64_t Hk, int64_t D, int64_t pages,
                      int64_t page, int64_t max_pages, int64_t window, float scale, void* workspace,
                      size_t workspace_bytes, void* stream) {
    if (!dims_ok(Lq, Hq, D) || !dims_ok(Lq, Hk, D) || B < 0 || Hq % Hk) return R9Q_ERR_DIM;
    if (B > INT_MAX / 64 || Lq > (1 << 20) || B * Lq > INT_MAX || max_pages < 0 || max_pages > INT_MAX || window < 0)
        return R9Q_ERR_DIM;
    const int64_t rows = Lq * (Hq / Hk);
    if (rows > (1 << 24) || Hk * rows > ((int64_t)1 << 30)) return R9Q_ERR_DIM;
    if (B == 0 || Lq == 0) return R9Q_OK;
    int rc = check_heads(q, Lq, q_ts, Hq, q_hs);
    if (!rc && !stride_ok(B, q_bs)) rc = R9Q_ERR_ARG;
    if (!rc && !stride_aligned(B, q_bs)) rc = R9Q_ERR_ALIGN;
    if (!rc) rc = check_cache(kc, kp, vc, vp, pages, Hk, page);
    if (rc) return rc;
    if (!seq_lens || !o || (max_pages > 0 && !block_table)) return R9Q_ERR_NULL;
    if (!aligned(o, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4)) return R9Q_ERR_ALIGN;
    if (!(scale > 0.0f) || std::isinf(scale) || max_pages * page > 0x7FE00000) return R9Q_ERR_ARG;
    const size_t need = decode_workspace(R9Q_OP_KV4_ATTENTION, rows, D, &rc);
    if (!workspace || workspace_bytes < need) return R9Q_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return R9Q_ERR_ALIGN;
    const Kv4Cache c = cache_of(kc, kp, vc, vp, pages, Hk, page);
    const Extent qe = bytes_of(q, (B > 1 ? 2 * (B - 1) * q_bs : 0) +
                                      (int64_t)(extent(q, Lq, Hq, D, q_ts, q_hs).hi - reinterpret_cast<uintptr_t>(q)));
    const Extent tables[2] = {bytes_of(block_table, B * max_pages * 4), bytes_of(seq_lens, B * 4)};
    const Extent out[3] = {bytes_of(o, 2 * B * Lq * Hq * D), bytes_of(lse, 4 * B * Lq * Hq),
                           bytes_of(workspace, (int64_t)need)};
    for (int i = 0; i < 3; ++i) {
        if (out[i].lo == 0) continue;                         // no lse
        if (meet(out[i], qe) || meet(out[i], tables[0]) || meet(out[i], tables[1]) || cache_meets(c, D, out[i]))
            return R9Q_ERR_ARG;
        for (int n = 0; n < i; ++n)
            if (meet(out[i], out[n])) return R9Q_ERR_ARG;
    }
    int *err = nullptr, sms = 0;
    rc = device_error_word_and_sms(&err, &sms);
    if (rc) return rc;
    Kv4AttnParams p = {};
    p.q = static_cast<const uint16_t*>(q);
    p.q_bs = q_bs;
    p.q_ts = q_ts;
    p.q_hs = q_hs;
    p.c = c;
    p.table = block_table;
    p.lens = seq_lens;
    p.o = static_cast<uint16_t*>(o);
    p.lse = lse;
    p.done = static_cast<int*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterHeader);
    p.err = err;
    p.B = (int)B;
    p.Lq = (int)Lq;
    p.G = (int)(Hq / Hk);
    p.max_pages = (int)max_pages;
    // a window longer than any sequence is none
    p.window = window > max_pages * page ? 0 : (int)window;
    p.room = (int)(max_pages * page);
    p.reach = p.window > 0 ? (int)(p.window > INT_MAX - Lq ? INT_MAX : p.window + Lq - 1) : INT_MAX;
    p.scale_log2 = scale * 1.4426950408889634f;
    return status(launch_kv4_attention((int)D, p, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
