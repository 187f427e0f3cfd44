"""QK norm with rotation and its gradient, the paged 4-bit cache and the
attention over it, against their definitions in 64 bits.

Bounds, from the arithmetic (u = 2^-8 the unit roundoff of bf16: eight significant bits):
  * norm + rotation: one rounding to bf16 of an fp32 value whose own error is a
    few roundings of the head's elements: u |y| + 2^-20 max|y of the head|;
  * gradient: the same for dx; dw is an fp32 sum: 2^-20 sum |terms|;
  * 4-bit codes and pairs of bf16 inputs: every step is an IEEE fp32 operation,
    so they are equal bit for bit;
  * attention: scores carry fp32 errors of at most 2^-18 sum |q k| scale (the
    sums of 128 products, taken apart as q.c and q.1), which move every weight by
    that factor; weights are rounded to fp16 (2^-11) and multiply codes, up to the
    vector's range; the result is rounded to bf16:
    u |o| + 2^-11 sum p range + 2^-17 S sum p |v|, S = max(1, largest sum |q k| scale);
    lse: 2^-17 S.
"""
import numpy as np
import pytest
import torch

import _attention_ref as ref
from _helpers import dev

U = 2.0 ** -8


@pytest.fixture(scope="module")
def r9q():
    import __graft_entry__
    __graft_entry__.build()
    import block_scaled_fp8_x128_gb300 as lib
    return lib


def rand(shape, seed, scale=1.0):
    """bf16 normals (a CPU tensor)."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def np64(t):
    return t.detach().cpu().double().numpy()


def tables(npos, rot):
    a = np.arange(npos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def on(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev())


def rope_inputs(T, Hq, Hk, D, rot, seed, npos=5000):
    """Slices of one [T][Hq + 2 Hk][D] buffer, weights, tables and positions."""
    qkv = rand((T, Hq + 2 * Hk, D), seed, 1.5).to(dev())
    g = np.random.default_rng(seed)
    wq, wk = (g.normal(1, 0.3, D).astype(np.float32) for _ in range(2))
    pos = g.integers(0, npos, T)
    cos, sin = tables(npos, rot) if rot else (None, None)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], wq, wk, cos, sin, pos


def rope_args(wq, wk, cos, sin, pos):
    return (on(wq), on(wk)) + ((None,) * 3 if cos is None else (on(cos), on(sin), on(pos)))


def rope_bound(y):
    return U * np.abs(y) * 1.01 + 2.0 ** -20 * np.abs(y).max(-1, keepdims=True)


# (T, Hq, Hk, D, rot, interleaved)
ROPE = [(1, 1, 1, 128, 128, False), (1, 32, 8, 128, 128, False), (3, 9, 5, 128, 64, True), (17, 5, 1, 64, 64, False),
        (33, 14, 2, 64, 32, True), (5, 8, 8, 64, 16, False), (7, 40, 8, 128, 0, False), (130, 32, 32, 128, 96, False),
        (257, 17, 3, 128, 128, True), (4, 3, 3, 64, 48, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", ROPE)
def test_norm_rope(r9q, T, Hq, Hk, D, rot, inter):
    q, k, _, wq, wk, cos, sin, pos = rope_inputs(T, Hq, Hk, D, rot, 1)
    qo, ko = r9q.r9q_qk_norm_rope(q, k, *rope_args(wq, wk, cos, sin, pos), eps=1e-5, interleaved=inter)
    c, s = (None, None) if cos is None else (cos[pos], sin[pos])
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        e = ref.norm_rope(np64(x), w, c, s, 1e-5, inter)
        assert (np.abs(np64(y) - e) <= rope_bound(e)).all()
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
def test_norm_rope_layouts(r9q):
    """Head-major inputs and outputs inside one buffer, on another stream: the same values as contiguous ones."""
    T, Hq, Hk, D = 19, 6, 2, 128
    q, k, _, wq, wk, cos, sin, pos = rope_inputs(T, Hq, Hk, D, D, 2)
    args = rope_args(wq, wk, cos, sin, pos)
    a = r9q.r9q_qk_norm_rope(q, k, *args)
    qh = q.transpose(0, 1).contiguous().transpose(0, 1)
    buf = torch.full((T, Hq + Hk + 1, D), 7.0, dtype=torch.bfloat16, device=dev())
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    r9q.r9q_qk_norm_rope(qh, k, *args, q_out=buf[:, :Hq], k_out=buf[:, Hq:Hq + Hk], stream=st)
    st.synchronize()
    assert torch.equal(buf[:, :Hq], a[0]) and torch.equal(buf[:, Hq:Hq + Hk], a[1])
    assert bool((buf[:, -1] == 7).all())


@pytest.mark.gpu
def test_norm_rope_zero_vectors_and_bad_positions(r9q):
    T, D = 6, 128
    q, k, _, wq, wk, cos, sin, pos = rope_inputs(T, 4, 4, D, D, 3, npos=100)
    q[2] = 0
    pos[4], pos[5] = 100, -1
    qo, ko = r9q.r9q_qk_norm_rope(q, k, *rope_args(wq, wk, cos, sin, pos))
    assert r9q.r9q_last_device_error() == -8
    assert r9q.r9q_last_device_error() == 0
    assert bool((qo[2] == 0).all()) and bool(torch.isfinite(qo[:4]).all()) and bool(torch.isfinite(ko[:4]).all())
    assert bool(torch.isnan(qo[4:]).all()) and bool(torch.isnan(ko[4:]).all())


GRAD = ROPE + [(2500, 8, 2, 128, 128, False), (6001, 3, 1, 64, 64, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", GRAD)
def test_norm_rope_grad(r9q, T, Hq, Hk, D, rot, inter):
    q, k, _, wq, wk, cos, sin, pos = rope_inputs(T, Hq, Hk, D, rot, 4)
    dq, dk = rand((T, Hq, D), 5).to(dev()), rand((T, Hk, D), 6).to(dev())
    args = (dq, dk, q, k) + rope_args(wq, wk, cos, sin, pos)
    out = r9q.r9q_qk_norm_rope_bwd(*args, eps=1e-5, interleaved=inter)
    again = r9q.r9q_qk_norm_rope_bwd(*args, eps=1e-5, interleaved=inter)
    c, s = (None, None) if cos is None else (cos[pos], sin[pos])
    for x, w, dy, dx, dw in ((q, wq, dq, out[0], out[2]), (k, wk, dk, out[1], out[3])):
        ex, ew, mass = ref.norm_rope_grad(np64(dy), np64(x), w, c, s, 1e-5, inter)
        # dx = r (w g) - (x r) (...): its error goes with the larger of the two
        big = np.abs(ex).max(-1, keepdims=True) + np.abs(np64(dy)).max(-1, keepdims=True)
        assert (np.abs(np64(dx) - ex) <= U * np.abs(ex) * 1.01 + 2.0 ** -19 * big).all()
        assert (np.abs(np64(dw) - ew) <= 2.0 ** -20 * mass).all()
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.gpu
def test_norm_rope_grad_of_no_tokens(r9q):
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device=dev())
    w = torch.ones(128, device=dev())
    dq, dk, dwq, dwk = r9q.r9q_qk_norm_rope_bwd(e, e, e, e, w, w)
    assert dq.shape == (0, 4, 128) and bool((dwq == 0).all()) and bool((dwk == 0).all())


def test_reference_gradient_against_differences():
    """The gradient's formula against central differences of the forward, in 64 bits."""
    g = np.random.default_rng(0)
    T, H, D, rot = 2, 2, 64, 32
    cos, sin = tables(9, rot)
    cos, sin = cos[[3, 8]], sin[[3, 8]]
    x, dy, w = g.normal(size=(T, H, D)), g.normal(size=(T, H, D)), g.normal(1, 0.3, D)
    for inter in (False, True):
        def loss(x, w):
            return (ref.norm_rope(x, w, cos, sin, 1e-5, inter) * dy).sum()
        dx, dw, _ = ref.norm_rope_grad(dy, x, w, cos, sin, 1e-5, inter)
        h = 1e-5
        for i in ((0, 0, 0), (0, 1, 17), (1, 0, 31), (1, 1, 63)):
            d = np.zeros_like(x)
            d[i] = h
            assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[i]) < 1e-7
        for i in (0, 5, 31, 40):
            d = np.zeros_like(w)
            d[i] = h
            assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[i]) < 1e-7


@pytest.mark.gpu
def test_gradient_against_differences_of_the_forward(r9q):
    """The two kernels against one another: along a random direction d, the forward's change equals <dx, d>.
    With steps of 1/16 of unit inputs the outputs move by far more than their rounding; the central difference
    of the rounded outputs is off by at most the roundings (random, 2^-8 each) and the third-order term."""
    T, Hq, Hk, D = 64, 8, 2, 128
    q, k, _, wq, wk, cos, sin, pos = rope_inputs(T, Hq, Hk, D, D, 8)
    args = rope_args(wq, wk, cos, sin, pos)
    dq, dk = rand((T, Hq, D), 9).to(dev()), rand((T, Hk, D), 10).to(dev())
    gq, gk, _, _ = r9q.r9q_qk_norm_rope_bwd(dq, dk, q, k, *args)
    for x, dy, g, which in ((q, dq, gq, 0), (k, dk, gk, 1)):
        step = (x.float() + torch.where(g.float() > 0, 1 / 16, -1 / 16)).to(torch.bfloat16)
        back = (x.float() - torch.where(g.float() > 0, 1 / 16, -1 / 16)).to(torch.bfloat16)
        a = r9q.r9q_qk_norm_rope(*((step, k) if which == 0 else (q, step)), *args)[which]
        b = r9q.r9q_qk_norm_rope(*((back, k) if which == 0 else (q, back)), *args)[which]
        change = ((a.double() - b.double()) * dy.double()).sum().item()
        slope = (g.double() * (step.double() - back.double())).sum().item()
        assert abs(change - slope) < 0.02 * abs(slope)


# ------------------------------------------------------------------ cache --

def codes_of(cache):
    kc, vc = ref.cache_codes(cache.k.cpu().numpy(), cache.v.cpu().numpy(), cache.k.shape[2], 2 * cache.k.shape[3])
    return kc, vc, np64(cache.kp), np64(cache.vp)


# (T, heads, D, page, pages)
CACHE = [(1, 1, 128, 16, 1), (40, 3, 128, 16, 3), (61, 2, 64, 48, 2), (33, 8, 64, 16, 9), (100, 5, 128, 32, 4),
         (16, 1, 128, 64, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,D,page,pages", CACHE)
@pytest.mark.parametrize("shuffled", [False, True])
def test_append_and_gather(r9q, T, H, D, page, pages, shuffled):
    """Codes and pairs bit for bit, at scattered and at consecutive places; other places stay as they were."""
    g = np.random.default_rng(T)
    kv = rand((T, 2 * H, D), 11, 2.0)
    kv[0, 0] = 3.0                                    # constant: step 0
    kv[T // 2, H, :] = 0.0
    if T > 8:
        kv[5, H - 1, 7] = float("inf")
        kv[6, H, 0] = float("nan")
        kv[7, :, 1] = 3.0e38                          # near the end of the range
        kv[7, :, 2:] = 1.0e38
    kv = kv.to(dev())
    slots = g.permutation(pages * page)[:T] if shuffled else np.arange(T) + (pages * page - T) // 2
    if T > 3:
        slots[2] = -5                                 # padding
    cache = r9q.r9q_kv4_cache(pages, H, page, D)
    for t in cache:
        t.view(torch.uint8).fill_(0x5A)
    k, v = kv[:, :H], kv[:, H:]
    r9q.r9q_kv4_append(k, v, cache, on(slots))
    kc, vc, kp, vp = codes_of(cache)
    written = np.zeros((pages, page), bool)
    for x, codes, pair in ((k, kc, kp), (v, vc, vp)):
        ec, es, el = ref.quantise32(np64(x).astype(np.float32))
        for t in range(T):
            if slots[t] < 0:
                continue
            p, at = slots[t] // page, slots[t] % page
            written[p, at] = True
            for h in range(H):
                vec = np64(x[t, h])
                if np.isfinite(vec).all():
                    assert (codes[p, h, at] == ec[t, h]).all()
                    assert pair[p, h, at, 0] == es[t, h, 0] and pair[p, h, at, 1] == el[t, h, 0]
                else:
                    assert np.isnan(pair[p, h, at]).all()
    for codes in (kc, vc):
        assert set(np.unique(codes.transpose(0, 2, 1, 3)[~written])) <= {5, 10}
    gk, gv = r9q.r9q_kv4_gather(cache, on(slots))
    for x, codes, pair in ((gk, kc, kp), (gv, vc, vp)):
        x = np64(x)
        for t in range(T):
            if slots[t] < 0:
                assert (x[t] == 0).all()
                continue
            p, at = slots[t] // page, slots[t] % page
            e = pair[p, :, at, 1:] + pair[p, :, at, :1] * codes[p, :, at]
            assert np.array_equal(np.isnan(x[t]), np.isnan(e))
            ok = np.abs(x[t] - e) <= U * np.abs(e) * 1.01
            assert (ok | np.isnan(e)).all()
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
def test_bad_slots_write_nothing(r9q):
    cache = r9q.r9q_kv4_cache(2, 2, 16, 128)
    before = [t.clone() for t in cache]
    k = rand((3, 2, 128), 1).to(dev())
    slots = on(np.array([32, -1, 1 << 40]))
    r9q.r9q_kv4_append(k, k, cache, slots)
    assert r9q.r9q_last_device_error() == -8
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    gk, gv = r9q.r9q_kv4_gather(cache, slots)
    assert r9q.r9q_last_device_error() == -8
    assert bool((gk == 0).all()) and bool((gv == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", ROPE)
def test_norm_rope_into_cache(r9q, T, Hq, Hk, D, rot, inter):
    """q as from r9q_qk_norm_rope, v as from r9q_kv4_append, both bit for bit; k quantised from its fp32 value:
    codes as from the 64-bit value, except within 2^-10 of a tie (an fp32 error of 2^-20 of the largest element is
    under 2^-15 of a step; a pair may be off by a rounding)."""
    page = 16 * (1 + T % 3)
    q, k, v, wq, wk, cos, sin, pos = rope_inputs(T, Hq, Hk, D, rot, 21)
    args = rope_args(wq, wk, cos, sin, pos)
    pages = T // page + 2
    slots = np.random.default_rng(T).permutation(pages * page)[:T]
    a, b = r9q.r9q_kv4_cache(pages, Hk, page, D), r9q.r9q_kv4_cache(pages, Hk, page, D)
    qo = r9q.r9q_qk_norm_rope_kv4(q, k, v, *args, a, on(slots), interleaved=inter)
    assert torch.equal(qo, r9q.r9q_qk_norm_rope(q, k, *args, interleaved=inter)[0])
    r9q.r9q_kv4_append(k, v, b, on(slots))
    assert torch.equal(a.v, b.v) and torch.equal(a.vp, b.vp)
    c, s = (None, None) if cos is None else (cos[pos], sin[pos])
    e = ref.norm_rope(np64(k), wk, c, s, 1e-6, inter)
    kc, _, kp, _ = codes_of(a)
    codes, pair = kc[slots // page, :, slots % page], kp[slots // page, :, slots % page]
    step, low = pair[..., :1], pair[..., 1:]
    _, es, el = ref.quantise32(e.astype(np.float32))
    assert (np.abs(step - es) <= 2.0 ** -7 * es).all() and (np.abs(low - el) <= 2.0 ** -7 * np.abs(el)).all()
    x = np.clip((e - low) / step, 0, 15)
    near = np.abs(x - np.floor(x) - 0.5) < 2.0 ** -10
    assert (near | (codes == np.rint(x))).all()
    assert near.mean() < 0.05 or near.size < 2000


# -------------------------------------------------------------- attention --

def make_cache(r9q, lens, Hk, D, page, seed, extra=2, garbage=True, v_scale=1.0):
    """A cache that holds sequences of these lengths on shuffled pages.  Places that hold no token are NaN."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    order = np.random.default_rng(seed).permutation(pages)
    cache = r9q.r9q_kv4_cache(pages, Hk, page, D)
    if garbage:
        for t in (cache.kp, cache.vp):
            t.fill_(float("nan"))
        for t in (cache.k, cache.v):
            t.fill_(0xFF)
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at, slots = 0, []
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        t = np.arange(n)
        slots.append(table[b, t // page].astype(np.int64) * page + t % page)
    slots = np.concatenate(slots) if sum(lens) else np.zeros(0, np.int64)
    k = rand((len(slots), Hk, D), seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    v = (torch.randn((len(slots), Hk, D), generator=g) * v_scale *
         torch.exp(torch.randn((len(slots), Hk, 1), generator=g))).to(torch.bfloat16)
    if len(slots):
        r9q.r9q_kv4_append(k.to(dev()), v.to(dev()), cache, on(slots))
    return cache, table, slots


def check_attention(r9q, cache, table, lens, q, o, lse, window=0, scale=None, skip=()):
    page, D = cache.k.shape[2], 2 * cache.k.shape[3]
    kc, vc, kp, vp = codes_of(cache)
    scale = D ** -0.5 if scale is None else scale
    q, o, lse = np64(q), np64(o), np64(lse)
    for b, n in enumerate(lens):
        t = np.arange(n)
        p, at = table[b, t // page], t % page
        k = kp[p, :, at, 1:] + kp[p, :, at, :1] * kc[p, :, at]
        v = vp[p, :, at, 1:] + vp[p, :, at, :1] * vc[p, :, at]
        eo, el, wide, mass, top = ref.attention(q[b], k, v, 15 * vp[p, :, at, 0], scale, window)
        S = np.maximum(1, top)
        empty = np.isneginf(el)
        assert np.array_equal(empty, np.isneginf(lse[b])), b
        d = np.abs(np.where(empty, 0, lse[b]) - np.where(empty, 0, el))
        assert (d <= 2.0 ** -17 * S).all(), (b, d.max())
        bound = U * np.abs(eo) * 1.01 + 2.0 ** -11 * wide[..., None] + 2.0 ** -17 * S[..., None] * mass
        assert (np.abs(o[b] - eo) <= bound).all(), (b, (np.abs(o[b] - eo) - bound).max())
        assert (o[b][empty] == 0).all()


# (lens, Lq, Hq, Hk, D, page, window)
ATTENTION = [
    ([1], 1, 1, 1, 128, 16, 0), ([0], 1, 4, 1, 128, 16, 0), ([5, 0, 16, 17, 15, 33], 1, 8, 2, 128, 16, 0),
    ([77], 1, 32, 32, 128, 16, 0), ([129, 64, 1000], 1, 32, 8, 128, 64, 0), ([511, 3], 1, 14, 2, 64, 48, 0),
    ([2, 700, 0, 31], 4, 8, 2, 128, 32, 0),                  # drafts, more of them than tokens
    ([300, 40], 5, 12, 4, 64, 16, 0), ([260], 1, 16, 1, 128, 80, 0), ([200, 90], 3, 40, 2, 128, 16, 0),
    ([1000, 10, 0, 127], 1, 7, 1, 64, 16, 100), ([333, 64], 3, 8, 8, 128, 32, 1), ([333, 64], 3, 8, 8, 128, 32, 5),
    ([600], 17, 4, 2, 128, 64, 40), ([90], 90, 4, 2, 128, 16, 0), ([4000], 1, 8, 8, 128, 128, 3999),
    ([20000], 1, 8, 1, 128, 64, 0), ([9000, 100], 1, 16, 2, 64, 16, 0), ([5000], 2, 64, 8, 128, 256, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Lq,Hq,Hk,D,page,window", ATTENTION)
def test_attention(r9q, lens, Lq, Hq, Hk, D, page, window):
    cache, table, _ = make_cache(r9q, lens, Hk, D, page, 31)
    if window:                                            # pages that no new token sees any more are given back
        for b, n in enumerate(lens):
            table[b, :max(0, n - Lq - window + 1) // page] = -1
    q = rand((len(lens), Lq, Hq, D), 33).to(dev())
    args = (q, cache, on(table), on(np.array(lens, np.int32)))
    o, lse = r9q.r9q_kv4_attention(*args, window=window, return_lse=True)
    assert r9q.r9q_last_device_error() == 0
    check_attention(r9q, cache, table, lens, q, o, lse, window)
    again = r9q.r9q_kv4_attention(*args, window=window, return_lse=True)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert torch.equal(o, r9q.r9q_kv4_attention(*args, window=window))


@pytest.mark.gpu
def test_attention_many_sequences(r9q):
    lens = [int(n) for n in np.random.default_rng(3).integers(0, 90, 300)]
    cache, table, _ = make_cache(r9q, lens, 2, 128, 16, 41)
    q = rand((300, 1, 8, 128), 42).to(dev())
    o, lse = r9q.r9q_kv4_attention(q, cache, on(table), on(np.array(lens, np.int32)), return_lse=True)
    check_attention(r9q, cache, table, lens, q, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale,v_scale,scale", [(1e-30, 1e-25, None), (1e4, 1e20, 1e-5), (30.0, 1e-3, None),
                                                   (1.0, 0.0, 2.0)])
def test_attention_magnitudes(r9q, q_scale, v_scale, scale):
    """Queries and values far from 1, and a cache of zero values."""
    lens = [300, 17]
    cache, table, _ = make_cache(r9q, lens, 2, 128, 16, 51, v_scale=v_scale)
    q = rand((2, 2, 8, 128), 52, q_scale).to(dev())
    o, lse = r9q.r9q_kv4_attention(q, cache, on(table), on(np.array(lens, np.int32)), scale=scale, return_lse=True)
    check_attention(r9q, cache, table, lens, q, o, lse, scale=scale)


@pytest.mark.gpu
def test_attention_strided_queries_on_a_stream_and_in_a_graph(r9q):
    lens = [120, 999, 45]
    cache, table, _ = make_cache(r9q, lens, 2, 128, 32, 61)
    buf = rand((3, 2, 12, 128), 62).to(dev())
    q = buf[:, :, :8]
    t, n = on(table), on(np.array(lens, np.int32))
    ws = torch.zeros(r9q.r9q_workspace_bytes(r9q.R9Q_OP_KV4_ATTENTION, 8, 128, 0), dtype=torch.uint8, device=dev())
    o = r9q.r9q_kv4_attention(q.contiguous(), cache, t, n)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    other = torch.empty_like(o)
    r9q.r9q_kv4_attention(q, cache, t, n, out=other, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(o, other)
    g = torch.cuda.CUDAGraph()
    other.zero_()
    with torch.cuda.graph(g):
        r9q.r9q_kv4_attention(q, cache, t, n, out=other, workspace=ws)
    for _ in range(3):
        other.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, other)
    n.copy_(on(np.array([0, 500, 45], np.int32)))         # the lengths are read when it runs
    g.replay()
    torch.cuda.synchronize()
    assert bool((other[0] == 0).all()) and torch.equal(other[2], o[2])


@pytest.mark.gpu
def test_what_is_masked_does_not_reach_the_result(r9q):
    """Three new tokens; the last one's key and value hold huge numbers, infinities or NaN: the first two tokens'
    results are what they are without it, bit for bit, and the last one's are not finite where that follows."""
    n, Lq, Hq, Hk, D, page = 100, 3, 4, 2, 128, 16
    cache, table, slots = make_cache(r9q, [n], Hk, D, page, 71)
    q = rand((1, Lq, Hq, D), 72).to(dev())
    args = (q, cache, on(table), on(np.array([n], np.int32)))
    base = r9q.r9q_kv4_attention(*args, return_lse=True)
    last = on(slots[-1:])
    for x in (-3.3895313892515355e38, 1e30, float("inf"), float("nan")):
        k = rand((1, Hk, D), 73).to(dev())
        v = k.clone()
        k[0, 0, 3], v[0, 0, 5] = x, x
        r9q.r9q_kv4_append(k, v, cache, last)
        o, lse = r9q.r9q_kv4_attention(*args, return_lse=True)
        assert torch.equal(o[:, :2], base[0][:, :2]) and torch.equal(lse[:, :2], base[1][:, :2]), x
        assert bool(torch.isfinite(o[:, 2, 2:]).all())      # the other key-value head
        if x != x or x == float("inf"):
            assert bool(torch.isnan(o[:, 2, :2]).all())


@pytest.mark.gpu
def test_attention_of_bad_tables(r9q):
    """A page out of range, and a length that the table has no room for: an error in the device word, nothing out of
    bounds, the other sequences' results as ever."""
    lens = [40, 40]
    cache, table, _ = make_cache(r9q, lens, 2, 64, 16, 81)
    q = rand((2, 1, 4, 64), 82).to(dev())
    good = r9q.r9q_kv4_attention(q, cache, on(table), on(np.array(lens, np.int32)))
    bad = table.copy()
    bad[0, 1] = 1 << 30
    o = r9q.r9q_kv4_attention(q, cache, on(bad), on(np.array(lens, np.int32)))
    assert r9q.r9q_last_device_error() == -8
    assert torch.equal(o[1], good[1]) and bool(torch.isfinite(o[0]).all())
    r9q.r9q_kv4_attention(q, cache, on(table), on(np.array([1 << 30, 40], np.int32)))
    assert r9q.r9q_last_device_error() == -8
    o = r9q.r9q_kv4_attention(q, cache, on(table), on(np.array([-3, 40], np.int32)))
    assert r9q.r9q_last_device_error() == -8
    assert bool((o[0] == 0).all()) and torch.equal(o[1], good[1])


# --------------------------------------------------------------- refusals --

def test_refusals():
    """Argument checks, on the host and before any CUDA call (the pointers are not addresses)."""
    import ctypes
    import __graft_entry__
    __graft_entry__._builder().build()
    import block_scaled_fp8_x128_gb300 as r9q
    lib, M = r9q._lib, 1 << 24
    DIM, NULL, ALIGN, ARG, WS = -2, -1, -3, -8, -4

    def rope(q=M, ts=512, hs=128, cos=7 * M, qo=3 * M, T=4, Hq=4, D=128, rot=128, npos=9, eps=1e-6, flags=0, w=5 * M):
        return lib.r9q_qk_norm_rope(q, ts, hs, 2 * M, 512, 128, w, 6 * M, cos, 8 * M, 9 * M, qo, 512, 128, 4 * M, 512,
                                    128, T, Hq, 2, D, rot, npos, eps, flags, None)
    assert rope(D=96) == DIM and rope(Hq=0) == DIM and rope(T=-1) == DIM and rope(rot=24) == DIM
    assert rope(rot=144) == DIM and rope(npos=0) == DIM
    assert rope(q=None) == NULL and rope(cos=None) == NULL and rope(w=None) == NULL
    assert rope(q=M + 8) == ALIGN and rope(ts=516) == ALIGN and rope(hs=132) == ALIGN and rope(cos=7 * M + 4) == ALIGN
    assert rope(flags=2) == ARG and rope(eps=-1.0) == ARG and rope(eps=float("nan")) == ARG
    assert rope(qo=M) == ARG and rope(ts=-512) == ARG
    assert rope(T=0) == 0
    # an output whose vectors lie over one another
    assert lib.r9q_qk_norm_rope(M, 512, 128, 2 * M, 512, 128, 5 * M, 6 * M, 7 * M, 8 * M, 9 * M, 3 * M, 128, 128, 4 * M,
                                512, 128, 4, 4, 2, 128, 128, 9, 1e-6, 0, None) == ARG

    def cache(slots=9 * M, pages=4, page=16, kc=5 * M, T=4, D=128, k=M):
        return lib.r9q_kv4_append(k, 256, 128, 2 * M, 256, 128, kc, 6 * M, 7 * M, 8 * M, slots, T, 2, D, pages, page,
                                  None)
    assert cache(page=24) == DIM and cache(page=0) == DIM and cache(pages=0) == DIM and cache(D=32) == DIM
    assert cache(slots=None) == NULL and cache(kc=None) == NULL and cache(kc=5 * M + 8) == ALIGN
    assert cache(slots=9 * M + 4) == ALIGN and cache(k=5 * M) == ARG and cache(kc=7 * M) == ARG and cache(T=0) == 0

    def gather(k=M, v=2 * M):
        return lib.r9q_kv4_gather(5 * M, 6 * M, 7 * M, 8 * M, 9 * M, 4, 2, 128, 4, 16, k, v, None)
    assert gather(k=None) == NULL and gather(v=M) == ARG and gather(k=5 * M) == ARG and gather(v=2 * M + 2) == ALIGN

    def attn(q=M, o=2 * M, B=2, Lq=1, Hq=4, Hk=2, D=128, page=16, max_pages=3, window=0, scale=0.1, ws=10 * M,
             wsb=1 << 26, lens=9 * M, table=4 * M):
        return lib.r9q_kv4_attention(q, 512, 512, 128, 5 * M, 6 * M, 7 * M, 8 * M, table, lens, o, None, B, Lq, Hq, Hk, D,
                                     4, page, max_pages, window, scale, ws, wsb, None)
    assert attn(Hq=5) == DIM and attn(D=256) == DIM and attn(page=8) == DIM and attn(window=-1) == DIM
    assert attn(B=-1) == DIM and attn(Hk=0) == DIM
    assert attn(q=None) == NULL and attn(lens=None) == NULL and attn(table=None) == NULL and attn(o=None) == NULL
    assert attn(scale=0.0) == ARG and attn(scale=-1.0) == ARG and attn(scale=float("nan")) == ARG
    assert attn(ws=None) == WS and attn(wsb=1000) == WS and attn(ws=10 * M + 16) == ALIGN
    assert attn(o=M) == ARG and attn(o=10 * M) == ARG and attn(q=M + 2) == ALIGN
    assert attn(B=0) == 0 and attn(Lq=0) == 0
    n = ctypes.c_size_t(0)
    assert lib.r9q_workspace_bytes(r9q.R9Q_OP_KV4_ATTENTION, 8, 256, 0, 0, 0, ctypes.byref(n)) == DIM
    assert lib.r9q_workspace_bytes(r9q.R9Q_OP_KV4_ATTENTION, 0, 128, 0, 0, 0, ctypes.byref(n)) == DIM
    assert lib.r9q_workspace_bytes(r9q.R9Q_OP_QK_NORM_ROPE_BWD, 1, 128, 0, 0, 0, ctypes.byref(n)) == 0 and n.value > 65536
    with pytest.raises(ValueError):
        r9q.r9q_qk_norm_rope(*(torch.zeros((2, 2, 128), dtype=torch.bfloat16),) * 2, *(torch.ones(128),) * 2)
    with pytest.raises(ValueError):
        r9q.r9q_kv4_cache(2, 2, 20, 128, device="cpu")


# ------------------------------------------------- many tokens at a time --

def prompt_slots(T, page, pages, how, seed):
    """Places of T tokens: page after page from the start of one, from its fourth token, or anywhere; padding in it."""
    order = np.random.default_rng(seed).permutation(pages)
    t = np.arange(T) + (3 if how == "late" else 0)
    slots = order[t // page] * page + t % page
    if how == "anywhere":
        slots = np.random.default_rng(seed).permutation(pages * page)[:T]
    if how != "aligned":
        slots[[7, T // 2]] = -1
    return slots


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,D,page", [(512, 2, 128, 16), (777, 3, 128, 48), (1000, 1, 64, 16), (515, 5, 64, 64)])
@pytest.mark.parametrize("how", ["aligned", "late", "anywhere"])
def test_append_and_gather_of_a_prompt(r9q, T, H, D, page, how):
    """As test_append_and_gather, at sizes where whole groups of 16 tokens are put together."""
    pages = T // page + 2
    slots = prompt_slots(T, page, pages, how, T)
    kv = rand((T, 2 * H, D), 91, 2.0).to(dev())
    kv[3, 0] = 1.0
    k, v = kv[:, :H], kv[:, H:]
    cache = r9q.r9q_kv4_cache(pages, H, page, D)
    for t in cache:
        t.view(torch.uint8).fill_(0x5A)
    r9q.r9q_kv4_append(k, v, cache, on(slots))
    kc, vc, kp, vp = codes_of(cache)
    kept = slots >= 0
    p, at = slots[kept] // page, slots[kept] % page
    written = np.zeros((pages, page), bool)
    written[p, at] = True
    gk, gv = r9q.r9q_kv4_gather(cache, on(slots))
    for x, codes, pair, got in ((k, kc, kp, gk), (v, vc, vp, gv)):
        ec, es, el = ref.quantise32(np64(x).astype(np.float32)[kept])
        assert np.array_equal(codes[p, :, at], ec)
        assert np.array_equal(pair[p, :, at], np.concatenate([es, el], -1).astype(np.float64))
        assert set(np.unique(codes.transpose(0, 2, 1, 3)[~written])) <= {5, 10}
        e = el + es * ec
        got = np64(got)
        assert (np.abs(got[kept] - e) <= U * np.abs(e) * 1.01).all() and (got[~kept] == 0).all()
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", [(520, 4, 2, 128, 128, False), (700, 3, 1, 64, 64, False),
                                                (513, 2, 2, 128, 64, True), (600, 5, 1, 64, 32, False)])
def test_norm_rope_of_a_prompt_into_cache(r9q, T, Hq, Hk, D, rot, inter):
    """The same cache, bit for bit, as from the tokens a few at a time (which the tests above hold to 64 bits)."""
    page, pages = 16, T // 16 + 2
    q, k, v, wq, wk, cos, sin, pos = rope_inputs(T, Hq, Hk, D, rot, 95)
    args = rope_args(wq, wk, cos, sin, pos)
    slots = on(prompt_slots(T, page, pages, "late" if T % 2 else "aligned", T))
    a, b = r9q.r9q_kv4_cache(pages, Hk, page, D), r9q.r9q_kv4_cache(pages, Hk, page, D)
    qo = r9q.r9q_qk_norm_rope_kv4(q, k, v, *args, a, slots, interleaved=inter)
    for i in range(0, T, 100):
        s = slice(i, min(T, i + 100))
        part = r9q.r9q_qk_norm_rope_kv4(q[s], k[s], v[s], *args[:4], args[4][s].contiguous(), b, slots[s].contiguous(),
                                        interleaved=inter)
        assert torch.equal(part, qo[s])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,D", [(4, 1, 128), (16, 1, 128), (7, 1, 64), (12, 1, 64)])
def test_attention_of_one_long_sequence(r9q, Hq, Hk, D):
    """Long enough for one CTA an SM (and its partials from every one of them)."""
    lens, page = [150000], 256
    cache, table, _ = make_cache(r9q, lens, Hk, D, page, 97, garbage=False)
    q = rand((1, 1, Hq, D), 98).to(dev())
    o, lse = r9q.r9q_kv4_attention(q, cache, on(table), on(np.array(lens, np.int32)), return_lse=True)
    check_attention(r9q, cache, table, lens, q, o, lse)
    n = on(np.array([1234], np.int32))
    o, lse = r9q.r9q_kv4_attention(q, cache, on(table), n, return_lse=True)
    check_attention(r9q, cache, table, [1234], q, o, lse)


@pytest.mark.gpu
def test_attention_of_thousands_of_sequences(r9q):
    """More sequences than threads of a CTA, most of them short or empty."""
    lens = [int(n) for n in np.random.default_rng(4).integers(0, 20, 2500)]
    lens[77], lens[2499] = 700, 300
    cache, table, _ = make_cache(r9q, lens, 1, 64, 16, 101)
    q = rand((2500, 1, 2, 64), 102).to(dev())
    o, lse = r9q.r9q_kv4_attention(q, cache, on(table), on(np.array(lens, np.int32)), return_lse=True)
    check_attention(r9q, cache, table, lens, q, o, lse)


# ------------------------------------- variants that sizes of these orders take --

@pytest.mark.gpu
@pytest.mark.parametrize("T,H,D,page", [(1024, 2, 128, 16), (1777, 3, 128, 48), (8192, 1, 64, 16), (8205, 2, 128, 64)])
@pytest.mark.parametrize("how", ["aligned", "late", "anywhere"])
def test_append_and_gather_of_a_long_prompt(r9q, T, H, D, page, how):
    """At sizes where writes, and for the longest read-backs too, take a group of the cache at a time."""
    test_append_and_gather_of_a_prompt(r9q, T, H, D, page, how)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", [(1040, 4, 2, 128, 128, False), (1301, 3, 1, 64, 64, False),
                                                (1025, 2, 2, 128, 64, True), (1200, 5, 1, 64, 32, False)])
def test_norm_rope_of_a_long_prompt_into_cache(r9q, T, Hq, Hk, D, rot, inter):
    test_norm_rope_of_a_prompt_into_cache(r9q, T, Hq, Hk, D, rot, inter)


def room_for(table, page, tokens):
    """The table with places for so many tokens a sequence: what it could hold decides how the work is laid out."""
    return np.pad(table, ((0, 0), (0, tokens // page - table.shape[1])), constant_values=-1)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Lq,Hq,Hk,D,page,window", [
    ([1], 1, 9, 1, 128, 16, 0), ([260], 1, 16, 1, 128, 80, 0), ([2, 700, 0, 31], 4, 8, 2, 128, 32, 0),
    ([300, 40], 5, 12, 4, 64, 16, 0), ([0, 33, 1000], 2, 14, 2, 64, 48, 100), ([200, 90], 5, 16, 2, 128, 16, 0),
    ([600], 17, 4, 2, 128, 64, 40), ([90], 90, 4, 2, 128, 16, 0), ([61], 40, 1, 1, 64, 16, 3),
])
@pytest.mark.parametrize("copies", [1, 20])
def test_attention_of_many_rows(r9q, lens, Lq, Hq, Hk, D, page, window, copies):
    """More than eight rows of a key-value head, in two tiles (a batch with room for long sequences), in few items and in
    many; and the same numbers, to rounding, in one."""
    lens = lens * copies
    cache, table, _ = make_cache(r9q, lens, Hk, D, page, 111)
    q = rand((len(lens), Lq, Hq, D), 112).to(dev())
    n = on(np.array(lens, np.int32))
    for t in (room_for(table, page, 1 << 20), table):
        o, lse = r9q.r9q_kv4_attention(q, cache, on(t), n, window=window, return_lse=True)
        assert r9q.r9q_last_device_error() == 0
        check_attention(r9q, cache, table, lens, q, o, lse, window)


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale,v_scale,scale", [(1e-30, 1e-25, None), (1e4, 1e20, 1e-5), (30.0, 1e-3, None),
                                                   (1.0, 0.0, 2.0)])
def test_attention_magnitudes_of_many_rows(r9q, q_scale, v_scale, scale):
    lens = [300, 17]
    cache, table, _ = make_cache(r9q, lens, 2, 128, 16, 121, v_scale=v_scale)
    q = rand((2, 4, 8, 128), 122, q_scale).to(dev())
    o, lse = r9q.r9q_kv4_attention(q, cache, on(room_for(table, 16, 1 << 20)), on(np.array(lens, np.int32)), scale=scale,
                                   return_lse=True)
    check_attention(r9q, cache, table, lens, q, o, lse, scale=scale)


@pytest.mark.gpu
def test_what_is_masked_does_not_reach_the_result_of_many_rows(r9q):
    n, Lq, Hq, Hk, D, page = 100, 3, 8, 2, 128, 16
    cache, table, slots = make_cache(r9q, [n], Hk, D, page, 131)
    q = rand((1, Lq, Hq, D), 132).to(dev())
    args = (q, cache, on(room_for(table, page, 1 << 20)), on(np.array([n], np.int32)))
    base = r9q.r9q_kv4_attention(*args, return_lse=True)
    last = on(slots[-1:])
    for x in (-3.3895313892515355e38, 1e30, float("inf"), float("nan")):
        k = rand((1, Hk, D), 133).to(dev())
        v = k.clone()
        k[0, 0, 3], v[0, 0, 5] = x, x
        r9q.r9q_kv4_append(k, v, cache, last)
        o, lse = r9q.r9q_kv4_attention(*args, return_lse=True)
        assert torch.equal(o[:, :2], base[0][:, :2]) and torch.equal(lse[:, :2], base[1][:, :2]), x
        assert bool(torch.isfinite(o[:, 2, 4:]).all())
        if x != x or x == float("inf"):
            assert bool(torch.isnan(o[:, 2, :4]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", [(1500, 19, 3, 128, 64, False), (1100, 40, 9, 64, 64, True),
                                                (3333, 1, 9, 128, 128, False), (2000, 7, 7, 64, 0, False)])
def test_norm_rope_grad_of_long_batches(r9q, T, Hq, Hk, D, rot, inter):
    """Several units a warp, which cross tokens and go from query to key heads and back, and last ones of odd sizes."""
    test_norm_rope_grad(r9q, T, Hq, Hk, D, rot, inter)


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (64, 32, False), (128, 128, True)])
def test_norm_rope_grad_layouts_and_bad_positions(r9q, D, rot, inter):
    T, Hq, Hk = 2100, 6, 2
    q, k, _, wq, wk, cos, sin, pos = rope_inputs(T, Hq, Hk, D, rot, 141, npos=500)
    dq, dk = rand((T, Hq, D), 142).to(dev()), rand((T, Hk, D), 143).to(dev())
    args = rope_args(wq, wk, cos, sin, pos)
    want = r9q.r9q_qk_norm_rope_bwd(dq, dk, q, k, *args, interleaved=inter)
    # slices of one buffer, for what is read and for what is written, on another stream
    x = torch.cat([q, k, dq, dk], 1)
    out = torch.full((T, Hq + Hk + 1, D), 7.0, dtype=torch.bfloat16, device=dev())
    dwq, dwk = torch.empty(D, device=dev()), torch.empty(D, device=dev())
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    r9q.r9q_qk_norm_rope_bwd(x[:, Hq + Hk:2 * Hq + Hk], x[:, 2 * Hq + Hk:], x[:, :Hq], x[:, Hq:Hq + Hk], *args,
                             interleaved=inter, dq=out[:, :Hq], dk=out[:, Hq:Hq + Hk], dwq=dwq, dwk=dwk, stream=st)
    st.synchronize()
    got = (out[:, :Hq], out[:, Hq:Hq + Hk], dwq, dwk)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and bool((out[:, -1] == 7).all())
    bad = args[4].clone()
    bad[0], bad[1234], bad[-1] = 500, -1, 1 << 40
    got = r9q.r9q_qk_norm_rope_bwd(dq, dk, q, k, *args[:4], bad, interleaved=inter)
    assert r9q.r9q_last_device_error() == -8
    kept = torch.ones(T, dtype=torch.bool, device=dev())
    kept[[0, 1234, -1]] = False
    for a, b in zip(want[:2], got[:2]):
        assert torch.equal(a[kept], b[kept]) and bool(torch.isnan(b[~kept]).all())
