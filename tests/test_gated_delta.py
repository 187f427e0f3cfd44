"""The gated delta rule (packed prompts, steps, trees of drafted tokens, accepted paths) against
its definition in 64 bits; the bounds are derived in _delta_ref.py."""
import numpy as np
import pytest
import torch

import _delta_ref as ref
from _helpers import dev
from test_attention_block import np64, on, rand, r9q  # noqa: F401


def rates(shape, seed, low=0.02, high=8.0):
    """g and beta: heads from hardly forgetting to forgetting at once."""
    r = np.random.default_rng(seed)
    g = -np.exp(r.uniform(np.log(low), np.log(high), shape[-1:])) * np.log1p(np.exp(r.normal(-2, 1, shape)))
    return g.astype(np.float32), (1 / (1 + np.exp(-r.normal(0, 1, shape)))).astype(np.float32)


def some_state(n, Hv, D, seed, scale=0.3):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((n, Hv, D, D), generator=g) * scale


def inputs(shape, Hk, Hv, D, seed):
    """q, k, v as slices of one buffer [..., 2 Hk + Hv, D], g and beta."""
    x = (rand((*shape, 2 * Hk + Hv, D), seed, 1.3) + 0.2).to(dev())
    g, beta = rates((*shape, Hv), seed + 1)
    return x[..., :Hk, :], x[..., Hk:2 * Hk, :], x[..., 2 * Hk:, :], g, beta


def check_state(got, want, bound):
    d = np.abs(np64(got) - want)
    assert (d <= bound[..., None]).all(), (d / np.maximum(bound[..., None], 1e-300)).max()


# (lens, Hk, Hv, D)
PROMPTS = [([1], 1, 1, 128), ([0], 1, 2, 128), ([7, 1, 0, 64, 65], 2, 4, 128), ([63, 128, 2], 1, 3, 64),
           ([200], 4, 4, 64), ([129, 30, 5], 1, 2, 128), ([31, 17, 16, 15, 33], 2, 2, 64), ([400, 191], 1, 1, 128),
           ([8, 9, 10, 11], 3, 6, 128), ([1] * 40, 1, 2, 128), ([0] * 20 + [36] + [0] * 24, 1, 2, 128),
           ([7, 0, 5], 2, 4, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hk,Hv,D", PROMPTS)
@pytest.mark.parametrize("from_zero", [False, True])
def test_prompts(r9q, lens, Hk, Hv, D, from_zero):  # noqa: F811
    """Rows before the first sequence and behind the last stay as they are, and so do the states of others."""
    first, after, B = 3, 5, len(lens)
    T = first + sum(lens) + after
    q, k, v, g, beta = inputs((T,), Hk, Hv, D, 401)
    cu = np.cumsum([first, *lens]).astype(np.int32)
    state = some_state(B + 2, Hv, D, 403)
    slots = np.random.default_rng(404).permutation(B + 2)[:B].astype(np.int32)
    s = state.to(dev())
    out = torch.full((T, Hv, D), 7.0, dtype=torch.bfloat16, device=dev())
    args = (q, k, v, on(g), on(beta))
    o = r9q.r9q_gated_delta(*args, s, on(slots), on(cu), from_zero=from_zero, out=out)
    assert o is out and r9q.r9q_last_device_error() == 0
    again = state.to(dev())
    o2 = r9q.r9q_gated_delta(*args, again, on(slots), on(cu), from_zero=from_zero)
    assert torch.equal(again, s) and torch.equal(o2[first:T - after], o[first:T - after])
    assert bool((o[:first] == 7).all()) and bool((o[T - after:] == 7).all())
    q, k, v, o = (np64(x) for x in (q, k, v, o))
    for b, n in enumerate(lens):
        at = slice(cu[b], cu[b + 1])
        S = np64(state[slots[b]]) * (not from_zero)
        S, E, e, w = ref.chain(S, q[at], k[at], v[at], g[at], beta[at], D ** -0.5)
        check_state(s[int(slots[b])], S, E)
        assert (np.abs(o[at] - e) <= w).all()
    for x in set(range(B + 2)) - set(slots.tolist()):
        assert torch.equal(s[x].cpu(), state[x])


@pytest.mark.gpu
@pytest.mark.parametrize("B,Lq,Hk,Hv,D", [(1, 1, 1, 1, 128), (5, 1, 2, 4, 64), (3, 2, 1, 3, 128), (2, 5, 4, 4, 64),
                                          (2, 9, 1, 2, 128), (1, 20, 2, 2, 64), (3, 70, 1, 1, 128)])
def test_steps(r9q, B, Lq, Hk, Hv, D):  # noqa: F811
    q, k, v, g, beta = inputs((B, Lq), Hk, Hv, D, 411)
    state = some_state(B + 1, Hv, D, 413)
    slots = np.random.default_rng(414).permutation(B + 1)[:B].astype(np.int32)
    s = state.to(dev())
    o = r9q.r9q_gated_delta_step(q, k, v, on(g), on(beta), s, on(slots), scale=0.3, eps=1e-3)
    assert r9q.r9q_last_device_error() == 0 and o.shape == (B, Lq, Hv, D)
    q, k, v = (np64(x) for x in (q, k, v))
    for b in range(B):
        S, E, e, w = ref.chain(np64(state[slots[b]]), q[b], k[b], v[b], g[b], beta[b], 0.3, 1e-3)
        check_state(s[int(slots[b])], S, E)
        assert (np.abs(np64(o[b]) - e) <= w).all()


def random_parents(B, n, seed):
    r = np.random.default_rng(seed)
    p = np.stack([np.maximum(np.floor(np.arange(1, n + 1) * r.random(n) ** 0.5).astype(np.int64) - 1, -1) for _ in range(B)])
    return np.minimum(p, np.arange(n) - 1).astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,Hk,Hv,D", [(1, 1, 1, 1, 128), (4, 3, 1, 2, 64), (3, 8, 2, 2, 128), (2, 9, 1, 3, 128),
                                         (2, 17, 2, 4, 64), (3, 33, 1, 1, 128), (2, 64, 1, 2, 128), (1, 64, 2, 2, 64)])
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
def test_trees(r9q, B, n, Hk, Hv, D, kind):  # noqa: F811
    q, k, v, g, beta = inputs((B, n), Hk, Hv, D, 421)
    parents = {"random": random_parents(B, n, 422), "chain": np.tile(np.arange(n) - 1, (B, 1)),
               "star": np.full((B, n), -1)}[kind].astype(np.int32)
    if n > 2:                                                 # places without a node, whatever they hold
        parents[0, n - 2:] = -2
        x = v.clone()
        x[0, n - 2:] = float("nan")
        v = x
        g[0, n - 2:], beta[0, n - 1] = np.nan, np.inf
    state = some_state(B, Hv, D, 423)
    s = state.to(dev())
    slots = np.arange(B)[::-1].astype(np.int32)
    o = r9q.r9q_gated_delta_tree(q, k, v, on(g), on(beta), s, on(slots), on(parents))
    assert r9q.r9q_last_device_error() == 0 and torch.equal(s.cpu(), state)
    q, k, v = (np64(x) for x in (q, k, v))
    for b in range(B):
        e, w = ref.tree(np64(state[slots[b]]), q[b], k[b], v[b], g[b], beta[b], parents[b], D ** -0.5)
        assert (np.abs(np64(o[b]) - e) <= w).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,P,Hk,Hv,D", [(5, 3, 2, 4, 128), (8, 1, 1, 1, 64), (20, 13, 1, 2, 128), (64, 64, 1, 1, 128),
                                         (64, 40, 1, 2, 64), (3, 5, 1, 1, 64), (40, 32, 2, 4, 128), (50, 31, 1, 2, 64)])
def test_commits(r9q, n, P, Hk, Hv, D):  # noqa: F811
    """Paths of any nodes in any order, none, ending early, and a padded place of the batch."""
    B = 4
    _, k, v, g, beta = inputs((B, n), Hk, Hv, D, 431)
    r = np.random.default_rng(432)
    path = r.integers(0, n, (B, P)).astype(np.int32)
    path[1, 0] = -1
    path[2, P // 2:] = -1
    state = some_state(B + 1, Hv, D, 433)
    slots = np.array([4, 1, 0, -1], np.int32)
    s = state.to(dev())
    r9q.r9q_gated_delta_commit(k, v, on(g), on(beta), s, on(slots), on(path))
    assert r9q.r9q_last_device_error() == 0
    k, v = np64(k), np64(v)
    assert torch.equal(s[1:4].cpu(), state[1:4])
    for b in (0, 2):
        way = [int(x) for x in path[b]]
        way = way[:way.index(-1)] if -1 in way else way
        S, E, _, _ = ref.chain(np64(state[slots[b]]), k[b, way], k[b, way], v[b, way], g[b, way], beta[b, way], 1.0)
        check_state(s[int(slots[b])], S, E)


# ------------------------------------------------------------ hard values --

HARD = ["no decay", "forgets", "forgets all", "strong then weak", "one key", "opposite keys", "rate 0", "rate 2", "no keys",
        "large values", "small values", "large state", "mixed rows", "large keys", "small keys"]


def hard(kind, n, Hk, Hv, D, seed):
    """q, k, v (CPU), g, beta, state for one sequence of n tokens."""
    x = rand((n, 2 * Hk + Hv, D), seed, 1.3)
    q, k, v = x[:, :Hk].clone(), x[:, Hk:2 * Hk].clone(), x[:, 2 * Hk:].clone()
    g, beta = rates((n, Hv), seed + 1)
    state = some_state(1, Hv, D, seed + 2)
    if kind == "no decay":
        g[:] = 0
    if kind == "forgets":
        g[::3] = -np.inf
    if kind == "forgets all":
        g[:] = -1e30
    if kind == "strong then weak":
        g[:] = -1e-3
        g[::5] = -90
        g[2::7] = -3e4
    if kind == "one key":
        k[:] = k[:1]
        g[:], beta[:] = -1e-4, 1
    if kind == "opposite keys":
        k[:] = k[:1]
        k[1::2] *= -1
        g[:], beta[:] = 0, 0.9
    if kind == "rate 0":
        beta[:] = 0
    if kind == "rate 2":
        beta[:] = 2
        g[:] = -0.01
    if kind == "no keys":
        k[::2], q[1::4] = 0, 0
    if kind == "large values":
        v *= 1e30
    if kind == "small values":
        v *= 1e-30
        state *= 1e-30
    if kind == "large state":
        state *= 1e25
    if kind == "mixed rows":
        v *= torch.exp2(torch.linspace(-60, 60, D)).to(torch.bfloat16)
        state *= torch.exp2(torch.linspace(-60, 60, D))[:, None]
    if kind == "large keys":
        k *= 1e17
        q[:, :, ::2] *= 1e17
    if kind == "small keys":                                  # mean squares near eps
        k *= 1e-4
        q *= 1e-5
    return q, k, v, g, beta, state


@pytest.mark.gpu
@pytest.mark.parametrize("kind", HARD)
@pytest.mark.parametrize("n,D", [(5, 128), (150, 128), (70, 64)])
def test_hard_values(r9q, kind, n, D):  # noqa: F811
    """In a packed sequence, and in a tree that is a chain."""
    Hk, Hv = 1, 2
    q, k, v, g, beta, state = hard(kind, n, Hk, Hv, D, 441)
    args = [x.to(dev()) for x in (q, k, v)] + [on(g), on(beta)]
    s, slots = state.to(dev()), on(np.zeros(1, np.int32))
    o = r9q.r9q_gated_delta(*args, s, slots, on(np.array([0, n], np.int32)))
    S, E, e, w = ref.chain(np64(state[0]), *(np64(x) for x in (q, k, v)), g, beta, D ** -0.5)
    assert r9q.r9q_last_device_error() == 0
    check_state(s[0], S, E)
    assert (np.abs(np64(o) - e) <= w).all(), (np.abs(np64(o) - e) - w).max()
    m = min(n, 64)
    o = r9q.r9q_gated_delta_tree(*(x[None, :m].contiguous() for x in args), state.to(dev()), slots,
                                 on(np.arange(-1, m - 1, dtype=np.int32)[None]))
    assert (np.abs(np64(o[0]) - e[:m]) <= w[:m]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.3e38])
def test_what_is_not_finite_stays_in_its_branch_and_head(r9q, bad):  # noqa: F811
    """A node's value, key, rate or decay that is not finite reaches that node and what comes from it, of its heads,
    and nothing else; in packed sequences the tokens from there on."""
    n, Hk, Hv, D = 12, 2, 4, 128
    q, k, v, g, beta = inputs((1, n), Hk, Hv, D, 451)
    parents = np.array([[-1, 0, 0, 1, 2, 2, -1, 6, 4, 3, 7, 10]], np.int32)
    below = [2, 4, 5, 8]                                      # node 2 and what comes from it
    s, slots = some_state(1, Hv, D, 453).to(dev()), on(np.zeros(1, np.int32))
    base = r9q.r9q_gated_delta_tree(q, k, v, on(g), on(beta), s, slots, on(parents))
    cu = on(np.array([0, n], np.int32))
    s1 = s.clone()
    packed = r9q.r9q_gated_delta(q[0], k[0], v[0], on(g[0]), on(beta[0]), s1, slots, cu)
    for what in range(4):
        kk, vv, gg, bb = k.clone(), v.clone(), on(g), on(beta)
        heads = [0] if what != 1 else [0, 1]
        if what == 0:
            vv[0, 2, 0, 3] = bad
        if what == 1:
            kk[0, 2, 0, 3] = bad
        if what == 2:
            gg[0, 2, 0] = bad
        if what == 3:
            bb[0, 2, 0] = bad
        o = r9q.r9q_gated_delta_tree(q, kk, vv, gg, bb, s, slots, on(parents))
        keep = torch.ones((n, Hv), dtype=torch.bool)
        keep[np.ix_(below, heads)] = False
        keep = keep.to(dev())
        assert torch.equal(o[0][keep], base[0][keep])
        s2 = s.clone()
        o = r9q.r9q_gated_delta(q[0], kk[0], vv[0], gg[0], bb[0], s2, slots, cu)
        keep = torch.ones((n, Hv), dtype=torch.bool)
        keep[2:, heads] = False
        assert torch.equal(o[keep.to(dev())], packed[keep.to(dev())])
        assert torch.equal(s2[0, len(heads):], s1[0, len(heads):])
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n,at,D", [(12, 2, 128), (40, 0, 128), (40, 39, 64), (64, 29, 64), (64, 35, 128), (64, 63, 128),
                                    (150, 3, 64), (150, 45, 128), (150, 64, 128), (150, 95, 64), (150, 149, 128)])
def test_what_is_not_finite_shows_and_stays(r9q, bad, n, at, D):  # noqa: F811
    """A value, key, rate, decay or query that is not finite, in either half of a chunk, in the first, a middle or the last one:
    what comes from it is not finite, and the rest stays, bit for bit."""
    Hk, Hv, m = 2, 4, min(n, 64)                              # m: nodes of a tree
    q, k, v, g, beta = inputs((n,), Hk, Hv, D, 521)
    g, beta = on(g), on(beta)
    parents = random_parents(1, m, 522)
    below = [at] if at < m else []
    for i in range(at + 1, m):
        if parents[0, i] in below:
            below.append(i)
    s, slots, cu = some_state(1, Hv, D, 523).to(dev()), on(np.zeros(1, np.int32)), on(np.array([0, n], np.int32))

    def both(*x):
        state = s.clone()
        packed = r9q.r9q_gated_delta(*x, state, slots, cu)
        return packed, state, r9q.r9q_gated_delta_tree(*(t[None, :m].contiguous() for t in x), s, slots, on(parents))[0]
    want = both(q, k, v, g, beta)
    for what in range(5):
        x = [t.clone() for t in (v, k, g, beta, q)]
        heads, rows, after, branch = [0], slice(None), list(range(at, n)), below
        if what == 0:
            x[0][at, 0, 3], rows = bad, slice(3, 4)           # (one value's row)
        elif what in (1, 4):
            x[what][at, 0, 3], heads = bad, [0, 1]
        else:
            x[what][at, 0] = bad
        if what == 4:                                         # (nothing comes from a query but its output)
            after, branch = [at], [at] if at < m else []
        got = both(x[4], x[1], x[0], x[2], x[3])
        if not (what == 2 and bad == -float("inf")):          # (which forgets the state)
            assert not torch.isfinite(got[0][after][:, heads, rows]).any(), what
            assert not torch.isfinite(got[2][branch][:, heads, rows]).any(), what
            assert what == 4 or not torch.isfinite(got[1][0, heads][:, rows]).any(), what
        for o, old, touched, tokens in ((got[0], want[0], after, n), (got[2], want[2], branch, m)):
            keep = torch.ones((tokens, Hv), dtype=torch.bool)
            keep[np.ix_(touched, heads)] = False
            keep = keep.to(dev())
            assert torch.equal(o[keep], old[keep]), what
        spared = slice(None) if what == 4 else slice(len(heads), None)
        assert torch.equal(got[1][0, spared], want[1][0, spared]), what
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [3.3e38, -1e30])
@pytest.mark.parametrize("n,at,D", [(14, 2, 128), (40, 0, 64), (64, 29, 128), (64, 50, 64), (150, 64, 128), (150, 100, 64)])
def test_a_large_value_stays_in_its_branch_row_and_head(r9q, bad, n, at, D):  # noqa: F811
    """However large: earlier tokens, other branches and the state's other rows stay, bit for bit."""
    Hk, Hv, m = 2, 4, min(n, 64)
    q, k, v, g, beta = inputs((n,), Hk, Hv, D, 571)
    g, beta = on(g), on(beta)
    parents = random_parents(1, m, 572)
    below = [at] if at < m else []
    for i in range(at + 1, m):
        if parents[0, i] in below:
            below.append(i)
    s, slots, cu = some_state(1, Hv, D, 573).to(dev()), on(np.zeros(1, np.int32)), on(np.array([0, n], np.int32))
    got = []
    for x in (v, v.clone()):
        if got:
            x[at, 1, 9] = bad
        state = s.clone()
        packed = r9q.r9q_gated_delta(q, k, x, g, beta, state, slots, cu)
        nodes = r9q.r9q_gated_delta_tree(*(t[None, :m].contiguous() for t in (q, k, x, g, beta)), s, slots, on(parents))[0]
        got.append((packed, nodes, state[0]))
    for old, new, touched in ((got[0][0], got[1][0], range(at, n)), (got[0][1], got[1][1], below)):
        same = torch.ones_like(old, dtype=torch.bool)
        same[list(touched), 1, 9] = False
        assert torch.equal(old[same], new[same])
        assert at >= m or not torch.equal(old, new)
    same = torch.ones((Hv, D), dtype=torch.bool)
    same[1, 9] = False
    same = same.to(dev())
    assert torch.equal(got[0][2][same], got[1][2][same]) and not torch.equal(got[0][2][1, 9], got[1][2][1, 9])
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,D", [(17, 128), (40, 64), (64, 128)])
def test_bad_parents_of_larger_trees(r9q, n, D):  # noqa: F811
    """A parent that is not one, in either half of a chunk: its node and what comes from it are NaN, the rest stays."""
    q, k, v, g, beta = inputs((2, n), 1, 2, D, 531)
    parents = random_parents(2, n, 532)
    args, s, slots = (q, k, v, on(g), on(beta)), some_state(2, 2, D, 533).to(dev()), on(np.arange(2, dtype=np.int32))
    base = r9q.r9q_gated_delta_tree(*args, s, slots, on(parents))
    assert r9q.r9q_last_device_error() == 0
    for at in (0, 3, n - 2):
        for x in (at, at + 1, -3, 1 << 30, -2147483648):
            p = parents.copy()
            p[1, at] = x
            lost = [at]
            for i in range(at + 1, n):
                if p[1, i] in lost:
                    lost.append(i)
            keep = [i for i in range(n) if i not in lost]
            o = r9q.r9q_gated_delta_tree(*args, s, slots, on(p))
            assert r9q.r9q_last_device_error() == -8
            assert torch.equal(o[0], base[0]) and torch.equal(o[1, keep], base[1, keep])
            assert bool(torch.isnan(o[1, lost]).all())


# ----------------------------------------------- places, layouts, streams --

@pytest.mark.gpu
@pytest.mark.parametrize("Lq", [1, 70])
def test_slots(r9q, Lq):  # noqa: F811
    """Padding gives zeros; a slot out of range or one that an earlier sequence has gives NaN and an error; none of them
    changes a state."""
    Hk, Hv, D = 1, 2, 128
    q, k, v, g, beta = inputs((6, Lq), Hk, Hv, D, 461)
    state = some_state(4, Hv, D, 463)
    a, b = state.to(dev()), state.to(dev())
    args = (q, k, v, on(g), on(beta))
    good = r9q.r9q_gated_delta_step(*args, a, on(np.array([2, -1, 0, -7, 1, -1], np.int32)))
    assert r9q.r9q_last_device_error() == 0
    assert bool((good[[1, 3, 5]] == 0).all()) and torch.equal(a[3].cpu(), state[3])
    o = r9q.r9q_gated_delta_step(*args, b, on(np.array([2, 4, 0, 2, 1, 1 << 30], np.int32)))
    assert r9q.r9q_last_device_error() == -8
    assert torch.equal(o[[0, 2, 4]], good[[0, 2, 4]]) and bool(torch.isnan(o[[1, 3, 5]]).all()) and torch.equal(a, b)
    # trees write no states: two may have the same one
    n = min(Lq, 64)
    tree = [x[:, :n].contiguous() for x in args]
    parents = on(np.tile(np.arange(-1, n - 1, dtype=np.int32), (6, 1)))
    o = r9q.r9q_gated_delta_tree(*tree, a, on(np.array([0, 0, -1, 4, 0, 0], np.int32)), parents)
    assert r9q.r9q_last_device_error() == -8
    assert bool(torch.isfinite(o[[0, 1, 4, 5]]).all()) and bool((o[2] == 0).all()) and bool(torch.isnan(o[3]).all())


@pytest.mark.gpu
def test_bad_offsets_parents_and_paths(r9q):  # noqa: F811
    Hk, Hv, D, T = 1, 2, 64, 30
    q, k, v, g, beta = inputs((T,), Hk, Hv, D, 471)
    state = some_state(3, Hv, D, 473)
    args, slots = (q, k, v, on(g), on(beta)), on(np.arange(3, dtype=np.int32))
    for cu in ([0, 10, 5, 20], [0, 10, 20, 31], [-1, 10, 20, 30]):
        s = state.to(dev())
        out = torch.full((T, Hv, D), 7.0, dtype=torch.bfloat16, device=dev())
        r9q.r9q_gated_delta(*args, s, slots, on(np.array(cu, np.int32)), out=out)
        assert r9q.r9q_last_device_error() == -8
        for b in range(3):
            ok = 0 <= cu[b] <= cu[b + 1] <= T
            assert torch.equal(s[b].cpu(), state[b]) != ok
            if ok:
                assert bool((out[cu[b]:cu[b + 1]] != 7).any())
    tree = [x[None, :8].contiguous() for x in args]
    base = r9q.r9q_gated_delta_tree(*tree, state.to(dev()), slots[:1], on(np.array([[-1, 0, 1, 0, 3, 3, 5, -1]], np.int32)))
    for parents, lost in (([-1, 0, 1, 3, 3, 3, 5, -1], [3, 4, 5, 6]), ([-1, 0, 1, 0, -3, 3, 5, -1], [4]),
                          ([-1, 0, 1, 0, 3, 1 << 30, 5, -1], [5, 6]), ([-1, 0, 1, -2, 3, 3, 5, -1], [4, 5, 6])):
        o = r9q.r9q_gated_delta_tree(*tree, state.to(dev()), slots[:1], on(np.array([parents], np.int32)))
        assert r9q.r9q_last_device_error() == -8
        keep = [i for i in range(8) if i not in lost and parents[i] != -2]
        assert torch.equal(o[0, keep], base[0, keep]) and bool(torch.isnan(o[0, lost]).all())
        assert all(bool((o[0, i] == 0).all()) for i in range(8) if parents[i] == -2)
    a, b = state.to(dev()), state.to(dev())
    r9q.r9q_gated_delta_commit(*tree[1:], a, slots[:1], on(np.array([[0, 3, 8, 5]], np.int32)))
    assert r9q.r9q_last_device_error() == -8
    r9q.r9q_gated_delta_commit(*tree[1:], b, slots[:1], on(np.array([[0, 3, -1, 5]], np.int32)))
    assert r9q.r9q_last_device_error() == 0 and torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [6, 32, 33, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_what_stands_behind_a_path(r9q, P, D):  # noqa: F811
    """Entries behind a path's end, and the path of a place without a sequence, are not looked at; a node out of range before
    that is an error and ends the path."""
    n, Hk, Hv = 40, 1, 2
    _, k, v, g, beta = inputs((4, n), Hk, Hv, D, 541)
    state = some_state(4, Hv, D, 543)
    args, slots = (k, v, on(g), on(beta)), on(np.array([2, -1, 0, 1], np.int32))

    def after(rest):
        path = np.full((4, P), rest, np.int64)
        path[0, :3] = 0, 3, -1
        path[2, :5] = 1, 2, 4, 7, -9
        path[3, 0] = -1
        s = state.to(dev())
        r9q.r9q_gated_delta_commit(*args, s, slots, on(path.astype(np.int32)))
        return s
    want = after(-1)
    assert r9q.r9q_last_device_error() == 0
    for rest in (n, 999, 2147483647, 5, -2147483648):
        assert torch.equal(after(rest), want) and r9q.r9q_last_device_error() == 0, rest
    for at in (0, 4, P - 1):
        s, path = state.to(dev()), np.tile(np.arange(P) % n, (4, 1)).astype(np.int32)
        path[3, at] = n
        short = path.copy()
        short[3, at] = -1
        r9q.r9q_gated_delta_commit(*args, s, slots, on(path))
        assert r9q.r9q_last_device_error() == -8
        t = state.to(dev())
        r9q.r9q_gated_delta_commit(*args, t, slots, on(short))
        assert r9q.r9q_last_device_error() == 0 and torch.equal(s, t)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 100])
def test_layouts_a_stream_and_a_graph(r9q, n):  # noqa: F811
    """Head-major and broadcast inputs, another stream, and a captured call replayed: the same values."""
    B, Hk, Hv, D = 2, 2, 4, 128
    q, k, v, g, beta = inputs((B, n), Hk, Hv, D, 481)
    k = k[:, :, :1].expand(B, n, Hk, D)                       # one key for all heads
    g, beta, slots = on(g), on(beta), on(np.array([1, 0], np.int32))
    start = some_state(2, Hv, D, 483).to(dev())
    s = start.clone()
    want = r9q.r9q_gated_delta_step(q.contiguous(), k.contiguous(), v.contiguous(), g, beta, s, slots)
    heads_first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, v)]
    t = start.clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o = r9q.r9q_gated_delta_step(heads_first[0], k, heads_first[1], g, beta, t, slots, stream=st)
    st.synchronize()
    assert torch.equal(o, want) and torch.equal(s, t)
    cu = on(np.array([0, n, 2 * n], np.int32))
    t = start.clone()
    o = r9q.r9q_gated_delta(*(x.flatten(0, 1) for x in (q, k, v, g, beta)), t, slots, cu)
    # (few tokens a sequence take another kernel as steps than packed: each is within its bound of the definition)
    kk = np64(k)
    for b in range(B):
        S, E, e, w = ref.chain(np64(start[int(slots[b])]), np64(q[b]), kk[b], np64(v[b]), np64(g[b]), np64(beta[b]), D ** -0.5)
        check_state(t[int(slots[b])], S, E)
        assert (np.abs(np64(o.view_as(want)[b]) - e) <= w).all()
    assert n < 10 or (torch.equal(o.view_as(want), want) and torch.equal(s, t))
    graph = torch.cuda.CUDAGraph()
    t = start.clone()
    with torch.cuda.graph(graph):
        o = r9q.r9q_gated_delta_step(q, k, v, g, beta, t, slots)
    for _ in range(2):
        t.copy_(start)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(s, t)
    assert not o.requires_grad


@pytest.mark.gpu
def test_states_beyond_32_bits(r9q):  # noqa: F811
    """The last of states that take 4.6 GB, and of inputs whose heads lie 2^32 elements apart."""
    n, D = 70_000, 128
    state = torch.zeros((n, 1, D, D), device=dev())
    q, k, v, g, beta = inputs((1, 2), 1, 1, D, 491)
    slots = on(np.array([n - 1], np.int32))
    o = r9q.r9q_gated_delta_step(q, k, v, on(g), on(beta), state, slots)
    S, E, e, w = ref.chain(np.zeros((1, D, D)), *(np64(x[0]) for x in (q, k, v)), g[0], beta[0], D ** -0.5)
    check_state(state[n - 1], S, E)
    assert (np.abs(np64(o[0]) - e) <= w).all() and bool((state[:2] == 0).all()) and not state[n - 2].any()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 70])
def test_inputs_beyond_32_bits(r9q, n):  # noqa: F811
    """Heads, tokens and sequences of the inputs 2^32 elements and more apart: as of ordinary inputs, bit for bit."""
    B, Hk, Hv, D = 2, 2, 4, 64
    q, k, v, g, beta = inputs((B, n), Hk, Hv, D, 561)
    g, beta, slots = on(g), on(beta), on(np.arange(B, dtype=np.int32))
    start = some_state(B, Hv, D, 563).to(dev())
    far = torch.empty((1 << 32) + (1 << 27), dtype=torch.bfloat16, device=dev())
    m = min(n, 64)
    parents = on(random_parents(B, m, 564))
    path = on(np.tile(np.arange(m), (B, 1)).astype(np.int32))
    cu = on(np.array([0, n], np.int32))

    def run(q, k, v):
        """All four calls, and one of the first sequence packed: outputs and states."""
        s, t, u = start.clone(), start.clone(), start.clone()
        few = [x[:, :m] for x in (q, k, v)] + [x[:, :m].contiguous() for x in (g, beta)]
        return [r9q.r9q_gated_delta_step(q, k, v, g, beta, s, slots), s, r9q.r9q_gated_delta_tree(*few, start, slots, parents),
                r9q.r9q_gated_delta_commit(*few[1:], t, slots, path), t,
                r9q.r9q_gated_delta(q[0], k[0], v[0], g[0], beta[0], u, slots[:1], cu), u]
    want = run(q, k, v)
    # strides of sequences, tokens and heads; what is 2^32 apart comes last in memory
    last = 1 << 32
    for strides in ((1 << 18, 1 << 11, last // (Hk - 1)), (last, 1 << 11, 1 << 8), (1 << 25, -(-last // (n - 1)) + 7 & ~7, 1 << 8)):
        def spread(x, offset):
            hs = strides[2] // (3 if strides[2] > 1 << 20 and x.shape[2] > Hk else 1) // 8 * 8        # (four heads in the same room)
            y = far.as_strided(x.shape, (strides[0], strides[1], hs, 1), offset)
            y.copy_(x)
            assert torch.equal(y, x)
            return y
        apart = [spread(x, 64 * (i if i < 2 else 8)) for i, x in enumerate((q, k, v))]
        assert max(sum((d - 1) * st for d, st in zip(x.shape, x.stride())) for x in apart) >= 1 << 32
        for x, y in zip((q, k, v), apart):                    # (one did not write over another)
            assert torch.equal(x, y)
        for a, b in zip(run(*apart), want):
            assert (a is None and b is None) or torch.equal(a, b)
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
def test_a_long_sequence_in_parts(r9q):  # noqa: F811
    """Three thousand tokens at once, in parts of any size, and the last ones as steps: within the bounds of one another
    and of the definition."""
    n, Hk, Hv, D = 3000, 1, 2, 128
    q, k, v, g, beta = inputs((n,), Hk, Hv, D, 501)
    slots = on(np.zeros(1, np.int32))
    S, E, e, w = ref.chain(np.zeros((Hv, D, D)), *(np64(x) for x in (q, k, v)), g, beta, D ** -0.5)
    g, beta = on(g), on(beta)
    a = torch.full((1, Hv, D, D), 9.0, device=dev())
    o = r9q.r9q_gated_delta(q, k, v, g, beta, a, slots, on(np.array([0, n], np.int32)), from_zero=True)
    check_state(a[0], S, E)
    assert (np.abs(np64(o) - e) <= w).all()
    a.zero_()
    at = 0
    for m in (1000, 1, 63, 64, 65, 900, 128, 700, 70, 1, 8):
        cu = on(np.array([0, m], np.int32))
        x = [t[at:at + m] for t in (q, k, v, g, beta)]
        if m > 8:
            got = r9q.r9q_gated_delta(*x, a, slots, cu)
        else:
            got = r9q.r9q_gated_delta_step(*(t[None] for t in x), a, slots)[0]
        assert (np.abs(np64(got) - e[at:at + m]) <= w[at:at + m]).all()
        at += m
    assert at == n
    check_state(a[0], S, E)


# --------------------------------------------------------------- refusals --

def test_refusals():
    """Argument checks, on the host and before any CUDA call (the pointers are not addresses)."""
    import __graft_entry__
    __graft_entry__._builder().build()
    import block_scaled_fp8_x128_gb300 as lib
    c, M = lib._lib, 1 << 30
    DIM, NULL, ALIGN, ARG = -2, -1, -3, -8

    def prompt(q=M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, cu=6 * M, slots=7 * M, state=8 * M, o=9 * M, T=10, B=2, Hk=2,
               Hv=4, D=128, n=3, scale=0.1, eps=1e-6, flags=0, ts=1024):
        return c.r9q_gated_delta(q, ts, 128, k, 1024, 128, v, 1024, 128, g, beta, cu, slots, state, o, T, B, Hk, Hv, D, n,
                                 scale, eps, flags, None)
    assert prompt(D=96) == DIM and prompt(Hv=3) == DIM and prompt(Hk=0) == DIM and prompt(T=-1) == DIM
    assert prompt(n=0) == DIM and prompt(B=-1) == DIM
    for name in ("q", "k", "v", "g", "beta", "cu", "slots", "state", "o"):
        assert prompt(**{name: None}) == NULL, name
    assert prompt(q=M + 2) == ALIGN and prompt(ts=1028) == ALIGN and prompt(state=8 * M + 4) == ALIGN
    assert prompt(o=9 * M + 2) == ALIGN and prompt(cu=6 * M + 2) == ALIGN
    assert prompt(o=M) == ARG and prompt(state=3 * M) == ARG and prompt(o=8 * M) == ARG and prompt(state=4 * M) == ARG
    assert prompt(scale=0.0) == ARG and prompt(scale=float("nan")) == ARG and prompt(eps=-1.0) == ARG
    assert prompt(flags=2) == ARG and prompt(ts=-1024) == ARG and prompt(B=0) == 0

    def step(q=M, B=2, Lq=3, bs=4096, o=9 * M, state=8 * M):
        return c.r9q_gated_delta_step(q, bs, 1024, 128, 2 * M, bs, 1024, 128, 3 * M, bs, 1024, 128, 4 * M, 5 * M, 7 * M,
                                      state, o, B, Lq, 2, 4, 128, 3, 0.1, 1e-6, 0, None)
    assert step(B=-1) == DIM and step(Lq=-1) == DIM and step(q=None) == NULL and step(bs=4100) == ALIGN
    assert step(o=2 * M + 4096) == ARG and step(state=7 * M) == ARG and step(B=0) == 0 and step(Lq=0) == 0

    def tree(parents=6 * M, Lq=3, o=9 * M, state=8 * M):
        return c.r9q_gated_delta_tree(M, 4096, 1024, 128, 2 * M, 4096, 1024, 128, 3 * M, 4096, 1024, 128, 4 * M, 5 * M,
                                      parents, 7 * M, state, o, 2, Lq, 2, 4, 128, 3, 0.1, 1e-6, None)
    assert tree(Lq=65) == DIM and tree(parents=None) == NULL and tree(parents=6 * M + 1) == ALIGN and tree(o=6 * M) == ARG
    assert tree(o=8 * M) == ARG and tree(Lq=0) == 0

    def commit(path=6 * M, P=3, Lq=4, state=8 * M, eps=1e-6):
        return c.r9q_gated_delta_commit(2 * M, 4096, 1024, 128, 3 * M, 4096, 1024, 128, 4 * M, 5 * M, path, 7 * M, state,
                                        2, Lq, P, 2, 4, 128, 3, eps, None)
    assert commit(P=65) == DIM and commit(Lq=65) == DIM and commit(path=None) == NULL and commit(path=6 * M + 2) == ALIGN
    assert commit(state=6 * M) == ARG and commit(eps=float("inf")) == ARG and commit(P=0) == 0 and commit(state=None) == NULL

    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    f, i = torch.zeros((2, 2)), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):                           # not on a GPU
        lib.r9q_gated_delta(x, x, x, f, f, torch.zeros((1, 2, 128, 128)), i, torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("T,B,taken", [(1 << 20, 2047, True), (1 << 20, 2048, True), (524288, 4096, True), (40, 1 << 28, True),
                                       ((1 << 31) - 1, 1, True), (1 << 31, 1, False), (10, 1 << 29, False)])
def test_how_many_packed_tokens_and_sequences(T, B, taken):
    """T counts the tokens of all sequences: no product of the two is limited.  (A refusal that comes later, of eps, ends the
    call on the host.)"""
    import __graft_entry__
    __graft_entry__._builder().build()
    import block_scaled_fp8_x128_gb300 as lib
    M = 1 << 30
    r = lib._lib.r9q_gated_delta(M, 128, 128, 2 * M, 128, 128, 3 * M, 128, 128, 4 * M, 5 * M, 6 * M, 7 * M, 8 * M, 9 * M, T, B,
                                 1, 1, 128, 3, 0.1, -1.0, 0, None)
    assert r == (-8 if taken else -2)


@pytest.mark.gpu
def test_thousands_of_packed_sequences(r9q):  # noqa: F811
    """4100 of up to 256 tokens, 524,800 in all."""
    B, Hk, Hv, D = 4100, 1, 1, 64
    lens = np.arange(B) * 101 % 256
    lens[:524_800 - lens.sum()] += 1
    assert lens.sum() == 524_800 and B * 524_800 > 1 << 31
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    q, k, v, g, beta = inputs((cu[-1],), Hk, Hv, D, 551)
    slots = np.random.default_rng(552).permutation(B).astype(np.int32)
    s = torch.zeros((B, Hv, D, D), device=dev())
    o = r9q.r9q_gated_delta(q, k, v, on(g), on(beta), s, on(slots), on(cu))
    assert r9q.r9q_last_device_error() == 0 and bool(torch.isfinite(o).all())
    for b in (0, 1, 255, 256, 2049, B - 1):
        at = slice(cu[b], cu[b + 1])
        S, E, e, w = ref.chain(np.zeros((Hv, D, D)), *(np64(x[at]) for x in (q, k, v)), g[at], beta[at], D ** -0.5)
        check_state(s[int(slots[b])], S, E)
        assert (np.abs(np64(o[at]) - e) <= w).all()


@pytest.mark.gpu
def test_tensors_of_other_types_and_shapes(r9q):  # noqa: F811
    q, k, v, g, beta = inputs((6,), 1, 2, 64, 511)
    g, beta, s = on(g), on(beta), some_state(2, 2, 64, 513).to(dev())
    slots, cu = on(np.zeros(1, np.int32)), on(np.array([0, 6], np.int32))
    for args in ((q, k, v, g, beta, s.double(), slots, cu), (q, k, v, g, beta, s, slots.long(), cu),
                 (q.float(), k, v, g, beta, s, slots, cu), (q, k, v, g.double(), beta, s, slots, cu)):
        with pytest.raises(TypeError):
            r9q.r9q_gated_delta(*args)
    for args in ((q, k, v, g, beta, s[:, :1].contiguous(), slots, cu), (q, k, v, g, beta, s, slots, cu[:1].contiguous()),
                 (q[:5], k, v, g, beta, s, slots, cu), (q, k, v, g[:5], beta, s, slots, cu),
                 (q, k, v, g, beta, s.transpose(2, 3), slots, cu), (q, k, v, g, beta, s.cpu(), slots, cu)):
        with pytest.raises(ValueError):
            r9q.r9q_gated_delta(*args)
