"""The attention block at the ends of what its calls accept, against 64 bits: eps of zero, inputs far from one,
other streams and devices, workspaces of captured graphs, the codes of keys to the last bit."""
import numpy as np
import pytest
import torch

import _attention_ref as ref
from _helpers import dev
from test_attention_block import U, np64, on, r9q, rand, rope_args, tables  # noqa: F401  (r9q: the fixture)


# (T, Hq, Hk, D, rot, interleaved): head counts that leave lanes of a warp without a head, and some that do not
HEADS = [(5, 14, 2, 64, 32, True), (777, 14, 2, 64, 64, False), (9, 5, 1, 64, 0, False), (3, 8, 8, 64, 64, False),
         (5, 3, 1, 128, 128, False), (1100, 7, 5, 128, 64, True), (4, 1, 1, 128, 96, False), (6, 8, 4, 128, 128, False)]


def grad_case(T, Hq, Hk, D, rot, scale, seed):
    """Queries, keys, their outputs' gradients, weights, and the angles of T positions."""
    x = [rand((T, h, D), seed + i, scale).to(dev()) for i, h in enumerate((Hq, Hk))]
    dy = [rand((T, h, D), seed + 2 + i).to(dev()) for i, h in enumerate((Hq, Hk))]
    g = np.random.default_rng(seed)
    w = [g.normal(1, 0.3, D).astype(np.float32) for _ in range(2)]
    pos = g.integers(0, 5000, T)
    cos, sin = tables(5000, rot) if rot else (None, None)
    return x, dy, w, cos, sin, pos


def check_grad(r9q, T, Hq, Hk, D, rot, inter, scale, eps, seed):
    """Bounds: dx = r (w g - xh mean(w g xh)), xh = x r, in fp32 and then one rounding to bf16.  g is two products, the
    mean D of them, r and xh carry a few roundings each: 2^-19 of the terms' largest sums.  dw: 2^-20 sum |terms|."""
    x, dy, w, cos, sin, pos = grad_case(T, Hq, Hk, D, rot, scale, seed)
    out = r9q.r9q_qk_norm_rope_bwd(*dy, *x, *rope_args(*w, cos, sin, pos), eps=eps, interleaved=inter)
    c, s = (None, None) if cos is None else (cos[pos].astype(np.float64), sin[pos].astype(np.float64))
    for i in range(2):
        xi, gi, wi = np64(x[i]), np64(dy[i]), w[i].astype(np.float64)
        ex, ew, mass = ref.norm_rope_grad(gi, xi, w[i], c, s, eps, inter)
        terms = np.abs(gi)
        if c is not None:
            own = ref.rotate(gi, c, 0 * s, inter)
            terms = np.abs(own) + np.abs(ref.rotate(gi, c, -s, inter) - own)
        r = 1 / np.sqrt((xi * xi).mean(-1, keepdims=True) + eps)
        t = terms * np.abs(wi)
        big = r * (t.max(-1, keepdims=True) +
                   np.abs(xi * r).max(-1, keepdims=True) * (t * np.abs(xi * r)).mean(-1, keepdims=True))
        assert (np.abs(np64(out[i]) - ex) <= U * np.abs(ex) * 1.01 + 2.0 ** -19 * big).all()
        assert (np.abs(np64(out[2 + i]) - ew) <= 2.0 ** -20 * mass).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", HEADS)
def test_gradient_with_eps_of_zero(r9q, T, Hq, Hk, D, rot, inter):  # noqa: F811
    """Lanes that have no head add nothing to the weights' gradients, though 1 / sqrt(0) is infinite."""
    check_grad(r9q, T, Hq, Hk, D, rot, inter, 1.0, 0.0, 201)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", HEADS)
@pytest.mark.parametrize("scale,eps", [(1e-14, 0.0), (1e-12, 0.0), (1e-6, 1e-6), (1e10, 1e-6), (1e14, 1e-6), (1e15, 0.0),
                                       (1e17, 1e-6)])
def test_gradient_of_inputs_far_from_one(r9q, T, Hq, Hk, D, rot, inter, scale, eps):  # noqa: F811
    check_grad(r9q, T, Hq, Hk, D, rot, inter, scale, eps, 211)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", HEADS)
@pytest.mark.parametrize("scale,eps", [(1.0, 0.0), (1e-14, 0.0), (1e-6, 1e-6), (1e10, 1e-6), (1e17, 1e-6)])
def test_norm_of_inputs_far_from_one(r9q, T, Hq, Hk, D, rot, inter, scale, eps):  # noqa: F811
    """u |y| + 2^-20 of the head's largest element, as for inputs near one."""
    x, _, w, cos, sin, pos = grad_case(T, Hq, Hk, D, rot, scale, 221)
    out = r9q.r9q_qk_norm_rope(*x, *rope_args(*w, cos, sin, pos), eps=eps, interleaved=inter)
    c, s = (None, None) if cos is None else (cos[pos], sin[pos])
    for xi, wi, y in zip(x, w, out):
        e = ref.norm_rope(np64(xi), wi, c, s, eps, inter)
        assert (np.abs(np64(y) - e) <= U * np.abs(e) * 1.01 + 2.0 ** -20 * np.abs(e).max(-1, keepdims=True)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [1e-6, 1e-30])
def test_gradient_of_zero_vectors(r9q, eps):  # noqa: F811
    """dx = w dy / sqrt(eps), however large 1 / sqrt(eps) is, and nothing for dw."""
    T, H, D = 3, 5, 128
    x, dy = torch.zeros((T, H, D), dtype=torch.bfloat16, device=dev()), rand((T, H, D), 231).to(dev())
    w = on(np.random.default_rng(231).normal(1, 0.3, D).astype(np.float32))
    dq, _, dwq, _ = r9q.r9q_qk_norm_rope_bwd(dy, dy, x, x, w, w, eps=eps)
    e = np64(dy) * np64(w) / np.sqrt(float(np.float32(eps)))
    assert (np.abs(np64(dq) - e) <= (U * 1.01 + 2.0 ** -20) * np.abs(e)).all() and bool((dwq == 0).all())


# ---------------------------------------------------------------- autograd --

@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", HEADS)
def test_autograd(r9q, T, Hq, Hk, D, rot, inter):  # noqa: F811
    """backward() of a call gives what r9q_qk_norm_rope_bwd gives (which the tests above hold to 64 bits): of slices of
    one tensor, with gradients of any layout, and from one output alone."""
    x, dy, w, cos, sin, pos = grad_case(T, Hq, Hk, D, rot, 1.5, 301)
    x, dy = [t + 0 for t in x], [t + 0 for t in dy]
    qk = torch.cat(x, 1).requires_grad_()
    wq, wk, *angles = rope_args(*w, cos, sin, pos)
    wq.requires_grad_(), wk.requires_grad_()
    q, k = qk[:, :Hq], qk[:, Hq:]
    plain = r9q.r9q_qk_norm_rope(*x, wq.detach(), wk.detach(), *angles, eps=1e-5, interleaved=inter)
    out = r9q.r9q_qk_norm_rope(q, k, wq, wk, *angles, eps=1e-5, interleaved=inter)
    assert all(torch.equal(a, b) and a.requires_grad and not b.requires_grad for a, b in zip(out, plain))
    for far in (dy, [d.transpose(1, 2).contiguous().transpose(1, 2) for d in dy]):
        got = torch.autograd.grad(out, (qk, wq, wk), far, retain_graph=True)
        want = r9q.r9q_qk_norm_rope_bwd(*dy, *x, wq, wk, *angles, eps=1e-5, interleaved=inter)
        assert torch.equal(got[0], torch.cat(want[:2], 1)) and torch.equal(got[1], want[2]) and torch.equal(got[2], want[3])
    got = torch.autograd.grad(out[0].float().sum(), (qk, wq, wk))          # (a gradient of stride 0, none for the keys)
    ones, none = torch.ones_like(x[0]), torch.zeros_like(x[1])
    want = r9q.r9q_qk_norm_rope_bwd(ones, none, *x, wq, wk, *angles, eps=1e-5, interleaved=inter)
    assert torch.equal(got[0], torch.cat(want[:2], 1)) and torch.equal(got[1], want[2]) and bool((got[2] == 0).all())
    with torch.no_grad():
        assert not r9q.r9q_qk_norm_rope(q, k, wq, wk, *angles, eps=1e-5, interleaved=inter)[0].requires_grad


@pytest.mark.gpu
def test_autograd_trains_and_refuses_a_second_derivative(r9q):  # noqa: F811
    """Steps down the gradient of ((norm(x) - t)^2).sum() lower it, on a stream of their own; what is not recorded says so."""
    T, H, D = 40, 3, 64
    with torch.cuda.stream(torch.cuda.Stream()):
        x, t = rand((T, H, D), 311).to(dev()), rand((T, H, D), 312, 0.5).to(dev())
        w = torch.ones(D, device=dev(), requires_grad=True)
        losses = []
        for _ in range(5):
            q, k = r9q.r9q_qk_norm_rope(x, x, w, w)
            loss = ((q.float() - t.float()) ** 2).mean() + ((k.float() - t.float()) ** 2).mean()
            g, = torch.autograd.grad(loss, w)
            losses.append(loss.item())
            w = (w - 5 * g).detach().requires_grad_()
        assert all(b < a for a, b in zip(losses, losses[1:]))
        y = r9q.r9q_qk_norm_rope(x, x, w, w)[0]
        g, = torch.autograd.grad(y.float().square().sum(), w, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()
        buf = torch.empty_like(x)
        assert not r9q.r9q_qk_norm_rope(x, x, w, w, q_out=buf)[0].requires_grad


# --------------------------------------------------- the keys' codes, exactly --

def key_in_order(x, w, c, s, eps, inter):
    """x fp32 [T][H][D], c and s fp32 [T][rot/2] or None: norm and rotation in fp32 with the roundings that include/r9q.h
    fixes.  Only the root is the GPU's (torch.rsqrt, which is rsqrtf)."""
    f32 = np.float32
    q = x * x
    sums = q[..., :32]
    for i in range(32, q.shape[-1], 32):
        sums = sums + q[..., i:i + 32]
    while sums.shape[-1] > 1:
        sums = sums[..., 0::2] + sums[..., 1::2]
    t = sums * f32(1 / x.shape[-1]) + f32(eps)
    r = torch.rsqrt(on(t)).cpu().numpy()
    y = (x * r) * w
    assert y.dtype == np.float32
    if c is None:
        return y
    c, s, half = c[:, None], s[:, None], c.shape[-1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
    z = y.copy()
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    assert z.dtype == np.float32
    return z


def check_codes(r9q, k, w, cos, sin, pos, inter):  # noqa: F811
    """Codes and pairs of keys k, written few or many at a time, against key_in_order."""
    T, Hk, D = k.shape
    cache, slots = r9q.r9q_kv4_cache(-(-T // 16), Hk, 16, D), torch.arange(T, device=dev())
    r9q.r9q_qk_norm_rope_kv4(k, k, k, *rope_args(w, w, cos, sin, pos), cache, slots, eps=1e-6, interleaved=inter)
    c, s = (None, None) if cos is None else (cos[pos], sin[pos])
    codes, step, low = ref.quantise32(key_in_order(k.float().cpu().numpy(), w, c, s, 1e-6, inter))
    at = np.arange(T)
    kb = cache.k.cpu().numpy()[at // 16, :, at % 16]
    assert np.array_equal(kb & 15, codes[..., 0::2]) and np.array_equal(kb >> 4, codes[..., 1::2])
    pair = cache.kp.float().cpu().numpy()[at // 16, :, at % 16]
    assert np.array_equal(pair, np.concatenate([step, low], -1))


@pytest.mark.gpu
@pytest.mark.parametrize("Hk,D,rot,inter", [(3, 128, 128, False), (2, 128, 128, True), (2, 128, 64, False),
                                           (1, 128, 0, False), (3, 64, 64, False), (5, 64, 64, True), (1, 64, 32, False),
                                           (2, 64, 48, True)])
@pytest.mark.parametrize("T", [40, 1025])
def test_codes_of_keys_are_those_of_the_stated_roundings(r9q, Hk, D, rot, inter, T):  # noqa: F811
    """Every code and pair, ties included, from few tokens and from a prompt: on the stated order of the sum of squares,
    single roundings and no fused product."""
    (_, k), _, (_, w), cos, sin, pos = grad_case(T, 1, Hk, D, rot, 1.5, 321)
    k[3] = 0
    check_codes(r9q, k, w, cos, sin, pos, inter)


def near_one(T, H, D, rot, seed):
    """Keys of elements of many sizes, which their weights and angles make nearly equal, so that a step of the codes is
    some thousand units of fp32 and not a million: another order of the sum or a fused product moves several of the codes."""
    g = np.random.default_rng(seed)
    size = np.exp2(g.uniform(-6, 6, D)).astype(np.float32)
    k = torch.from_numpy((size * (1 + g.integers(0, 3, (T, H, D)) / 128)).astype(np.float32)).to(torch.bfloat16).to(dev())
    w = ((1 + g.normal(0, 2.0 ** -8, D)) / size).astype(np.float32)
    cos = (1 - np.abs(g.normal(0, 2.0 ** -9, (500, rot // 2)))).astype(np.float32)
    sin = g.normal(0, 2.0 ** -8, (500, rot // 2)).astype(np.float32)
    return k, w, cos, sin, g.integers(0, 500, T)


@pytest.mark.gpu
@pytest.mark.parametrize("Hk,D,rot,inter", [(8, 128, 128, False), (8, 64, 64, False), (8, 128, 128, True), (8, 64, 32, False),
                                           (8, 128, 64, True)])
@pytest.mark.parametrize("T", [900, 1500])
def test_codes_of_keys_near_one_are_those_of_the_stated_roundings(r9q, Hk, D, rot, inter, T):  # noqa: F811
    check_codes(r9q, *near_one(T, Hk, D, rot, 331), inter)


# ------------------------------------------------------------- long sequences --

@pytest.mark.gpu
@pytest.mark.parametrize("Hq,D,batch", [(1, 128, 2000), (2, 64, 2000), (12, 128, 1000), (16, 64, 1000)])
def test_sums_over_long_sequences_do_not_drift(r9q, Hq, D, batch):  # noqa: F811
    """Queries of zero: every weight is the same power of two, exact in any format, and the result the mean of 100,000
    values, a three-hundredth of one.  So many sequences that a warp has half of one (3125 groups of 16 keys).  Partial
    sums of both signs are of the order of sqrt(n) terms, and err by 2^-23 of that each, in all 2^-23 sqrt(3125) = 2^-17 of
    a term: of the values' range.  (Sums of one sign, cut off, would drift by n / 2 units: 2^-14.)"""
    n, page = 100_000, 256
    per = -(-n // page)
    cache = r9q.r9q_kv4_cache(per, 1, page, D)
    v = rand((n, 1, D), 341).to(dev())
    slots = torch.arange(n, device=dev())
    r9q.r9q_kv4_append(v, v, cache, slots)
    q = torch.zeros((batch, 1, Hq, D), dtype=torch.bfloat16, device=dev())
    table = torch.arange(per, dtype=torch.int32, device=dev()).expand(batch, per).contiguous()    # (all the same pages)
    o, lse = r9q.r9q_kv4_attention(q, cache, table, torch.full((batch,), n, dtype=torch.int32, device=dev()), return_lse=True)
    codes, pair = cache.v.cpu().numpy(), cache.vp.double().cpu().numpy()
    _, vc = ref.cache_codes(cache.k.cpu().numpy(), codes, page, D)
    e = (pair[:, 0, :, 1:] + pair[:, 0, :, :1] * vc[:, 0]).reshape(-1, D)[:n].mean(0)
    spread = 15 * pair[:, 0, :, 0].reshape(-1)[:n].mean()
    assert (np.abs(np64(o) - e) <= U * np.abs(e) * 1.01 + 2.0 ** -17 * spread).all()
    assert (np.abs(np64(lse) - np.log(n)) <= 2.0 ** -17).all()


# ----------------------------------------------------- streams and devices --

def attention_inputs(r9q, Hq=4, Hk=2, D=128, n=40, seed=241):  # noqa: F811
    """One sequence in a cache: (q, cache, table, lengths)."""
    cache = r9q.r9q_kv4_cache(-(-n // 16), Hk, 16, D)
    kv = rand((n, 2 * Hk, D), seed).to(dev())
    r9q.r9q_kv4_append(kv[:, :Hk], kv[:, Hk:], cache, torch.arange(n, device=dev()))
    return (rand((1, 1, Hq, D), seed + 1).to(dev()), cache, torch.arange(-(-n // 16), dtype=torch.int32, device=dev())[None],
            torch.tensor([n], dtype=torch.int32, device=dev()))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rope", "grad", "write", "gather", "attention"])
def test_outputs_belong_to_the_stream_of_the_call(r9q, name):  # noqa: F811
    """The current stream still has work on a block that it has let go; outputs of a call on another stream are not
    made of that block."""
    T, H, D = 2048, 8, 128
    x, w = rand((T, H, D), 251).to(dev()), torch.ones(D, device=dev())
    q, cache, table, lens = attention_inputs(r9q)
    qs, many = q.expand(4096, 1, 4, D), (table.expand(4096, -1).contiguous(), lens.expand(4096).contiguous())
    big, slots = r9q.r9q_kv4_cache(T // 16, H, 16, D), torch.arange(T, device=dev())
    calls = {"rope": lambda **k: r9q.r9q_qk_norm_rope(x, x, w, w, **k),
             "grad": lambda **k: r9q.r9q_qk_norm_rope_bwd(x, x, x, x, w, w, **k),
             "write": lambda **k: r9q.r9q_qk_norm_rope_kv4(x, x, x, w, w, None, None, None, big, slots, **k),
             "gather": lambda **k: r9q.r9q_kv4_gather(big, slots, **k),
             "attention": lambda **k: r9q.r9q_kv4_attention(qs, cache, *many, return_lse=True, **k)}
    r9q.r9q_kv4_append(x, x, big, slots)
    st = torch.cuda.Stream()
    want = calls[name]()
    with torch.cuda.stream(st):
        calls[name]()                                         # (workspaces, and blocks that the stream can have again)
    torch.cuda.synchronize()
    want = want if isinstance(want, tuple) else (want,)
    first = want[0]
    room = first.untyped_storage().nbytes()
    block = torch.empty(room, dtype=torch.uint8, device=dev())
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    block.fill_(7)
    del block
    got = calls[name](stream=st)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
def test_calls_run_on_the_device_of_their_tensors(r9q, monkeypatch):  # noqa: F811
    """With another device current (as the binding sees it), a call makes the tensors' own current; a stream of another
    device is refused."""
    x, w = rand((3, 2, 64), 261).to(dev()), torch.ones(64, device=dev())
    q, cache, table, lens = attention_inputs(r9q)
    want, o = r9q.r9q_qk_norm_rope(x, x, w, w), r9q.r9q_kv4_attention(q, cache, table, lens)
    entered, now = [], [1]

    class Device(torch.cuda.device):
        def __enter__(self):
            entered.append(self.idx)
            now.append(self.idx)
            return super().__enter__()

        def __exit__(self, *error):
            now.pop()
            return super().__exit__(*error)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(r9q, "_current_device", lambda: now[-1])
    got = r9q.r9q_qk_norm_rope(x, x, w, w)
    assert entered == [0] and all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(o, r9q.r9q_kv4_attention(q, cache, table, lens)) and entered == [0, 0] and now == [1]

    class Other:
        device = torch.device("cuda", 1)
        cuda_stream = 12345
    with pytest.raises(ValueError):
        r9q.r9q_qk_norm_rope(x, x, w, w, stream=Other())


@pytest.mark.gpu
def test_out_of_memory_is_torch_s(r9q):  # noqa: F811
    """Outputs that do not fit (of a small share of the memory that the process may have): the error that torch raises."""
    cache, slots = r9q.r9q_kv4_cache(4, 8, 16, 128), torch.zeros(2_000_000, dtype=torch.int64, device=dev())
    torch.cuda.set_per_process_memory_fraction(0.01)
    try:
        with pytest.raises(torch.cuda.OutOfMemoryError):
            r9q.r9q_kv4_gather(cache, slots)                  # 8 GB
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    k, v = r9q.r9q_kv4_gather(cache, slots[:16])
    assert k.shape == (16, 8, 128) and r9q.r9q_last_device_error() == 0


# --------------------------------------------- workspaces of captured graphs --

def sequences(r9q, count, n, Hq, Hk, D, Lq, seed):  # noqa: F811
    """`count` sequences of n tokens, long enough that several CTAs share each: (q, cache, table, lengths)."""
    page = 64
    per = -(-n // page)
    cache = r9q.r9q_kv4_cache(count * per, Hk, page, D)
    kv = rand((count * per * page, 2 * Hk, D), seed).to(dev())
    r9q.r9q_kv4_append(kv[:, :Hk], kv[:, Hk:], cache, torch.arange(len(kv), device=dev()))
    return (rand((count, Lq, Hq, D), seed + 1).to(dev()), cache,
            torch.arange(count * per, dtype=torch.int32, device=dev()).view(count, per),
            torch.full((count,), n, dtype=torch.int32, device=dev()))


def captured(f, stream=None):
    """The graph of f() and its outputs."""
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = f()
    return g, out


def occupy():
    """Memory of the stream that is current, full of ones, in blocks of the sizes that workspaces have."""
    return [torch.full((2 ** k,), -1, dtype=torch.int8, device=dev()) for k in range(16, 26) for _ in range(4)]


@pytest.mark.gpu
def test_a_graph_keeps_its_workspace(r9q):  # noqa: F811
    """A decode step is captured; then, on the stream it was captured on, a call that needs a larger workspace, an error
    that lets the workspaces go, and other tensors.  Replays are what they were."""
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        few = sequences(r9q, 2, 3000, 8, 2, 128, 1, 271)
        many = sequences(r9q, 2, 3000, 8, 2, 128, 4, 272)
        want = r9q.r9q_kv4_attention(*few)
        x, w = rand((700, 9, 128), 273).to(dev()), torch.ones(128, device=dev())
        dwant = r9q.r9q_qk_norm_rope_bwd(x, x, x, x, w, w)
        st.synchronize()
        g, out = captured(lambda: (r9q.r9q_kv4_attention(*few), *r9q.r9q_qk_norm_rope_bwd(x, x, x, x, w, w)), st)
        r9q.r9q_kv4_attention(*many)
        bad = few[2].clone()
        bad[0, 0] = 1 << 20
        r9q.r9q_kv4_attention(few[0], few[1], bad, few[3])
        assert r9q.r9q_last_device_error() == -8
        kept = occupy()
        for _ in range(3):
            for t in out:
                t.zero_()
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip((want, *dwant), out))
        assert all(bool((t == -1).all()) for t in kept)
        assert torch.equal(r9q.r9q_kv4_attention(*few), want)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_graphs_of_one_stream_stand_alone(r9q):  # noqa: F811
    """Nothing has run on the stream before it is captured, twice; the second graph is replayed first, the first one is
    let go, and two graphs run at the same time on two streams."""
    cases = [sequences(r9q, 1 + i, 5000 + 900 * i, 8, 2, 128, 1, 281 + i) for i in range(3)]
    want = [r9q.r9q_kv4_attention(*c) for c in cases]
    gemm = (rand((64, 1024), 291).to(dev()), *r9q.r9q_quant_weight_block128(rand((4096, 1024), 292).float().to(dev())))
    y = r9q.r9q_gemm_fp8_block_qa(*gemm)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graphs = [captured(lambda c=c: (r9q.r9q_kv4_attention(*c), r9q.r9q_gemm_fp8_block_qa(*gemm)), st) for c in cases]
    for i in (1, 0, 2, 1):
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[i][1][0], want[i]) and torch.equal(graphs[i][1][1], y)
    graphs[0] = None
    kept = occupy()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in (1, 2):
            graphs[i][1][0].zero_()
        torch.cuda.synchronize()
        for i, s in zip((1, 2), streams):
            with torch.cuda.stream(s):
                for _ in range(5):
                    graphs[i][0].replay()
        torch.cuda.synchronize()
        for i in (1, 2):
            assert torch.equal(graphs[i][1][0], want[i]) and torch.equal(graphs[i][1][1], y)
    assert all(bool((t == -1).all()) for t in kept)


@pytest.mark.gpu
def test_capture_ids(r9q):  # noqa: F811
    st, seen = torch.cuda.Stream(), []
    torch.ones(1, device=dev())
    with torch.cuda.stream(st):
        assert r9q.r9q_stream_capture_id() == 0
        for _ in range(2):
            captured(lambda: (seen.append(r9q.r9q_stream_capture_id()), seen.append(r9q.r9q_stream_capture_id(st)),
                              torch.ones(1, device=dev())), st)
        assert r9q.r9q_stream_capture_id() == 0
    assert seen[0] == seen[1] != 0 and seen[2] == seen[3] != 0 and seen[0] != seen[2]


def test_capture_id_refusal(r9q):  # noqa: F811
    assert r9q._lib.r9q_stream_capture_id(None, None) == -1


# ----------------------------------------------------------------- refusals --

def test_outputs_over_weights_tables_positions_and_slots_are_refused(r9q):  # noqa: F811
    """On the host, before any CUDA call (the pointers are not addresses)."""
    lib, M, ARG = r9q._lib, 1 << 24, -8
    at = {"wq": 11 * M, "wk": 12 * M, "cos": 13 * M, "sin": 14 * M, "pos": 15 * M, "slots": 16 * M}

    def rope(**over):
        p = {"q_out": 3 * M, "k_out": 4 * M, **over}
        return lib.r9q_qk_norm_rope(M, 512, 128, 2 * M, 512, 128, at["wq"], at["wk"], at["cos"], at["sin"], at["pos"],
                                    p["q_out"], 512, 128, p["k_out"], 512, 128, 4, 4, 2, 128, 128, 9, 1e-6, 0, None)

    def grad(**over):
        p = {"dq": 5 * M, "dk": 6 * M, "dwq": 7 * M, "dwk": 8 * M, "ws": 20 * M, **over}
        return lib.r9q_qk_norm_rope_bwd(M, 512, 128, 2 * M, 512, 128, 3 * M, 512, 128, 4 * M, 512, 128, at["wq"], at["wk"],
                                        at["cos"], at["sin"], at["pos"], p["dq"], 512, 128, p["dk"], 512, 128, p["dwq"],
                                        p["dwk"], 4, 4, 2, 128, 128, 9, 1e-6, 0, p["ws"], 1 << 22, None)

    def write(**over):
        p = {"q_out": 4 * M, "kc": 5 * M, "kp": 6 * M, "vc": 7 * M, "vp": 8 * M, **over}
        return lib.r9q_qk_norm_rope_kv4(M, 512, 128, 2 * M, 256, 128, 3 * M, 256, 128, at["wq"], at["wk"], at["cos"],
                                        at["sin"], at["pos"], p["q_out"], 512, 128, p["kc"], p["kp"], p["vc"], p["vp"],
                                        at["slots"], 4, 4, 2, 128, 128, 9, 4, 16, 1e-6, 0, None)
    for name in ("wq", "wk", "cos", "sin", "pos"):
        assert all(rope(**{o: at[name]}) == ARG for o in ("q_out", "k_out")), name
        assert all(write(**{o: at[name]}) == ARG for o in ("q_out", "kc", "kp", "vc", "vp")), name
        assert all(grad(**{o: at[name]}) == ARG for o in ("dq", "dk", "dwq", "dwk")), name
    assert all(write(**{o: at["slots"]}) == ARG for o in ("q_out", "kc", "kp", "vc", "vp"))
    append = (M, 256, 128, 2 * M, 256, 128)
    for i in range(4):
        c = [5 * M, 6 * M, 7 * M, 8 * M]
        c[i] = at["slots"]
        assert lib.r9q_kv4_append(*append, *c, at["slots"], 4, 2, 128, 4, 16, None) == ARG
    for k, v in ((at["slots"], 2 * M), (M, at["slots"])):
        assert lib.r9q_kv4_gather(5 * M, 6 * M, 7 * M, 8 * M, at["slots"], 4, 2, 128, 4, 16, k, v, None) == ARG
