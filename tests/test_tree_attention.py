"""Attention of a tree of drafted tokens over the 4-bit cache, and moves of tokens within it.  The
bounds are those of the attention of newest tokens (test_attention_block.py), with the keys that a node sees."""
import numpy as np
import pytest
import torch

import _attention_ref as ref
from _helpers import dev
from test_attention_block import U, codes_of, make_cache, np64, on, r9q, rand  # noqa: F401
from test_gated_delta import random_parents


def way_to(parents, i):
    """The nodes from the tree's beginning to i, or None where one of them is not a node."""
    way = []
    while i != -1:
        up = parents[i]
        if up < -1 or up >= i:
            return None
        way.append(i)
        i = up
    return way[::-1]


def widened(table, page, heads, rows):
    """The table with room for sequences so long that, with more than 64 rows, the call takes the kernel for many (which
    one does, is decided by what the pages can hold)."""
    tokens = 16 * (36000 // (len(table) * heads * -(-rows // 16)) + 2)
    return np.concatenate((table, np.full((len(table), max(0, -(-tokens // page) - table.shape[1])), -1, np.int32)), 1)


def check(r9q, cache, table, lens, parents, q, o, lse, window=0, scale=None):  # noqa: F811
    """Each node as the one newest token of the keys that it sees."""
    page, D = cache.k.shape[2], 2 * cache.k.shape[3]
    kc, vc, kp, vp = codes_of(cache)
    scale = D ** -0.5 if scale is None else scale
    q, o, lse = np64(q), np64(o), np64(lse)
    n = q.shape[1]
    for b, length in enumerate(lens):
        t = np.arange(length)
        p, at = table[b, t // page], t % page
        k = kp[p, :, at, 1:] + kp[p, :, at, :1] * kc[p, :, at]
        v = vp[p, :, at, 1:] + vp[p, :, at, :1] * vc[p, :, at]
        for i in range(n):
            way = way_to(parents[b], i)
            if parents[b, i] == -2 or length == 0:
                assert (o[b, i] == 0).all() and np.isneginf(lse[b, i]).all()
                continue
            if way is None:
                assert np.isnan(o[b, i]).all() and np.isnan(lse[b, i]).all()
                continue
            keys = list(range(max(0, length - n))) + [length - n + x for x in way]
            if window:                                        # (positions: a path's tokens follow one another)
                keys = keys[-window:]
            keys = [x for x in keys if x >= 0]
            if not keys:
                assert (o[b, i] == 0).all() and np.isneginf(lse[b, i]).all()
                continue
            eo, el, wide, mass, top = ref.attention(q[b, i:i + 1], k[keys], v[keys], 15 * vp[p, :, at, 0][keys], scale, 0)
            S = np.maximum(1, top)
            assert (np.abs(lse[b, i] - el[0]) <= 2.0 ** -17 * S[0]).all()
            bound = U * np.abs(eo) * 1.01 + 2.0 ** -11 * wide[..., None] + 2.0 ** -17 * S[..., None] * mass
            assert (np.abs(o[b, i] - eo[0]) <= bound[0]).all(), (b, i, (np.abs(o[b, i] - eo[0]) - bound[0]).max())


# (tokens of each sequence, the tree's among them; nodes, Hq, Hk, D, page, window)
TREES = [([1], 1, 1, 1, 128, 16, 0), ([9, 0, 24, 70], 8, 8, 2, 128, 16, 0), ([77], 8, 32, 32, 128, 16, 0),
         ([300, 16, 17], 16, 14, 2, 64, 48, 0), ([64, 1000], 64, 4, 1, 128, 64, 0), ([200, 90], 33, 8, 2, 64, 16, 0),
         ([3, 40], 7, 4, 4, 128, 32, 0),                      # fewer tokens than nodes
         ([500, 60], 21, 7, 1, 64, 16, 10), ([333, 64], 20, 16, 2, 128, 32, 1), ([700], 12, 8, 2, 128, 16, 300),
         ([2000], 30, 40, 8, 128, 128, 0), ([4096, 129, 128, 127], 48, 8, 1, 128, 64, 0), ([5000], 64, 64, 8, 64, 256, 0),
         ([260, 31], 63, 12, 4, 128, 80, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,n,Hq,Hk,D,page,window", TREES)
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("wide", [False, True])
def test_trees(r9q, lens, n, Hq, Hk, D, page, window, kind, wide):  # noqa: F811
    B = len(lens)
    cache, table, _ = make_cache(r9q, lens, Hk, D, page, 601)
    if wide:
        if n * Hq // Hk <= 64 or window and window < 50:      # (never many; a short window never makes enough to do)
            return
        table = widened(table, page, Hk, n * Hq // Hk)
    parents = {"random": random_parents(B, n, 602), "chain": np.tile(np.arange(n) - 1, (B, 1)),
               "star": np.full((B, n), -1)}[kind].astype(np.int32)
    if n > 6:
        parents[-1, n - 3:] = -2
    if window:                                                # pages that no node sees any more are given back
        for b, length in enumerate(lens):
            table[b, :max(0, length - n - window + 1) // page] = -1
    q = rand((B, n, Hq, D), 603).to(dev())
    args = (q, cache, on(table), on(np.array(lens, np.int32)), on(parents))
    o, lse = r9q.r9q_kv4_tree_attention(*args, window=window, return_lse=True)
    assert r9q.r9q_last_device_error() == 0
    check(r9q, cache, table, lens, parents, q, o, lse, window)
    again = r9q.r9q_kv4_tree_attention(*args, window=window, return_lse=True)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert torch.equal(o, r9q.r9q_kv4_tree_attention(*args, window=window))


@pytest.mark.gpu
@pytest.mark.parametrize("B,length,n,Hq,Hk,D", [(70, 90, 5, 8, 2, 128), (300, 40, 16, 4, 1, 64), (40, 300, 33, 8, 2, 128),
                                                (320, 200, 17, 8, 1, 64), (90, 700, 20, 32, 4, 128), (170, 500, 64, 2, 1, 128)])
def test_many_trees(r9q, B, length, n, Hq, Hk, D):  # noqa: F811
    """More of them than CTAs of the kernel at a time."""
    lens = [1 + (i * 37) % length for i in range(B)]
    cache, table, _ = make_cache(r9q, lens, Hk, D, 16, 611)
    parents = random_parents(B, n, 612)
    parents[::3, n - 1] = -2
    q = rand((B, n, Hq, D), 613).to(dev())
    o, lse = r9q.r9q_kv4_tree_attention(q, cache, on(table), on(np.array(lens, np.int32)), on(parents), return_lse=True)
    assert r9q.r9q_last_device_error() == 0
    check(r9q, cache, table, lens, parents, q, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale,v_scale,scale", [(1e-30, 1e-25, None), (1e4, 1e20, 1e-5), (30.0, 1e-3, None),
                                                   (1e3, 1.0, 1.0), (0.0, 1.0, None)])
@pytest.mark.parametrize("n,Hq,D,wide", [(9, 2, 128, False), (40, 8, 128, False), (40, 8, 128, True), (40, 8, 64, True),
                                          (12, 8, 128, True)])
def test_magnitudes(r9q, q_scale, v_scale, scale, n, Hq, D, wide):  # noqa: F811
    lens = [150, 700]
    cache, table, _ = make_cache(r9q, lens, 1, D, 32, 621, v_scale=v_scale)
    table = widened(table, 32, 1, n * Hq) if wide else table
    parents = random_parents(2, n, 622)
    q = rand((2, n, Hq, D), 623, q_scale).to(dev())
    o, lse = r9q.r9q_kv4_tree_attention(q, cache, on(table), on(np.array(lens, np.int32)), on(parents), scale=scale,
                                        return_lse=True)
    check(r9q, cache, table, lens, parents, q, o, lse, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq,D,wide", [(10, 2, 128, False), (40, 8, 128, False), (40, 8, 128, True), (33, 16, 64, True),
                                          (10, 8, 128, True)])
def test_what_a_node_does_not_see(r9q, n, Hq, D, wide):  # noqa: F811
    """A node's key and value of huge numbers, infinities or NaN reach that node and what comes from it alone: the others'
    results stay, bit for bit."""
    length, Hk = 200, 2
    cache, table, slots = make_cache(r9q, [length], Hk, D, 16, 631)
    table = widened(table, 16, Hk, n * Hq) if wide else table
    parents = random_parents(1, n, 632)
    parents[0, 4] = 1
    q = rand((1, n, Hq * Hk, D), 633).to(dev())
    args = (q, cache, on(table), on(np.array([length], np.int32)), on(parents))
    base = r9q.r9q_kv4_tree_attention(*args, return_lse=True)
    below = [i for i in range(n) if 4 in way_to(parents[0], i)]
    keep = [i for i in range(n) if i not in below]
    at = on(slots[length - n + 4:length - n + 5])
    for x in (-3.3895313892515355e38, 1e30, float("inf"), float("nan")):
        k = rand((1, Hk, D), 634).to(dev())
        v = k.clone()
        k[0, 0, 3], v[0, 0, 5] = x, x
        r9q.r9q_kv4_append(k, v, cache, at)
        o, lse = r9q.r9q_kv4_tree_attention(*args, return_lse=True)
        assert torch.equal(o[:, keep], base[0][:, keep]) and torch.equal(lse[:, keep], base[1][:, keep]), x
        assert bool(torch.isfinite(o[:, below, Hq:]).all())   # the other key-value head
        if x != x or x == float("inf"):
            assert bool(torch.isnan(o[:, below, :Hq]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq,wide", [(9, 2, False), (40, 8, False), (40, 8, True), (10, 8, True)])
def test_bad_parents_and_tables(r9q, n, Hq, wide):  # noqa: F811
    """Parents that are none, and those of an unused place of the batch; a page and a length out of range."""
    lens = [100, 60, 0]
    cache, table, _ = make_cache(r9q, lens, 1, 128, 16, 641)
    table = widened(table, 16, 1, n * Hq) if wide else table
    q = rand((3, n, Hq, 128), 642).to(dev())
    parents = random_parents(3, n, 643)
    parents[2] = 1 << 20                                      # not looked at
    t, lengths = on(table), on(np.array(lens, np.int32))
    good = r9q.r9q_kv4_tree_attention(q, cache, t, lengths, on(parents), return_lse=True)
    assert r9q.r9q_last_device_error() == 0 and bool((good[0][2] == 0).all())
    for at, x in ((0, 0), (3, 3), (5, -3), (6, 1 << 30), (2, -2147483648)):
        p = parents.copy()
        p[0, at] = x
        o, lse = r9q.r9q_kv4_tree_attention(q, cache, t, lengths, on(p), return_lse=True)
        assert r9q.r9q_last_device_error() == -8
        lost = [way_to(p[0], i) is None for i in range(n)]
        for i in range(n):
            if lost[i]:
                assert bool(torch.isnan(o[0, i]).all()) and bool(torch.isnan(lse[0, i]).all())
            else:
                assert torch.equal(o[0, i], good[0][0, i])
        assert lost[at] and torch.equal(o[1:], good[0][1:])
    bad = table.copy()
    bad[0, 1] = 1 << 30
    o = r9q.r9q_kv4_tree_attention(q, cache, on(bad), lengths, on(parents))
    assert r9q.r9q_last_device_error() == -8 and torch.equal(o[1], good[0][1]) and bool(torch.isfinite(o[0]).all())
    for x in (1 << 30, -3):
        o = r9q.r9q_kv4_tree_attention(q, cache, t, on(np.array([x, 60, 0], np.int32)), on(parents))
        assert r9q.r9q_last_device_error() == -8 and torch.equal(o[1], good[0][1])


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq,wide", [(9, 2, False), (40, 8, False), (40, 8, True), (12, 8, True)])
def test_layouts_a_stream_and_graphs(r9q, n, Hq, wide):  # noqa: F811
    """Strided queries, another stream with a workspace of one's own, and two graphs replayed on two streams."""
    lens = [3000, 999, 450]
    cache, table, _ = make_cache(r9q, lens, 2, 128, 32, 651)
    table = widened(table, 32, 2, n * Hq) if wide else table
    buf = rand((3, n, 2 * Hq + 3, 128), 652).to(dev())
    q = buf[:, :, :2 * Hq]
    rest = (cache, on(table), on(np.array(lens, np.int32)), on(random_parents(3, n, 653)))
    want = r9q.r9q_kv4_tree_attention(q.contiguous(), *rest)
    size = r9q.r9q_workspace_bytes(r9q.R9Q_OP_KV4_TREE_ATTENTION, n * Hq, 128, 3 * 2)
    ws = torch.zeros(size, dtype=torch.uint8, device=dev())
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o = r9q.r9q_kv4_tree_attention(q, *rest, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(o, want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = r9q.r9q_kv4_tree_attention(q, *rest)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for _, out in graphs:
            out.zero_()
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out in graphs)
    assert int(ws[:65536].count_nonzero()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq,D", [(32, 8, 128), (24, 6, 64), (64, 24, 128)])
def test_lengths_that_change_under_a_graph(r9q, n, Hq, D):  # noqa: F811
    """Many rows, one workspace: batches whose lengths differ between replays, places that are empty, fewer tokens than
    nodes, one long sequence alone; what an earlier replay split or left whole does not show."""
    most = [2500, 700, 40, 3, 90, 1300]
    cache, table, _ = make_cache(r9q, most, 2, D, 32, 671)
    wide = widened(table, 32, 2, n * Hq // 2)
    parents = random_parents(len(most), n, 672)
    parents[1, n // 2:] = -2
    q = rand((len(most), n, Hq, D), 673).to(dev())
    lens = on(np.array(most, np.int32))
    args = (q, cache, on(wide), lens, on(parents))
    r9q.r9q_kv4_tree_attention(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = r9q.r9q_kv4_tree_attention(*args, return_lse=True)
    for now in (most, [0, 0, 0, 0, 0, 0], [2500, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 1300], [1, 2, 3, 3, 64, 128], [700, 700, 40, 0, 0, 129],
                [0, 16, 0, 0, 0, 0], most):
        lens.copy_(on(np.array(now, np.int32)))
        o.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert r9q.r9q_last_device_error() == 0
        check(r9q, cache, table, now, parents, q, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("n,G,D", [(13, 5, 128), (19, 5, 64), (43, 3, 128), (33, 7, 128), (37, 7, 64)])
@pytest.mark.parametrize("B", [2, 120])
def test_rows_that_end_inside_a_warp(r9q, n, G, D, B):  # noqa: F811
    """Many rows, the last warp of a tile partly without: as parts that are joined, and items of a CTA's own."""
    lens = [n + (i * 53) % 190 for i in range(B)]
    cache, table, _ = make_cache(r9q, lens, 1, D, 16, 681)
    table = widened(table, 16, 1, n * G)
    parents = random_parents(B, n, 682)
    parents[1, n - 2:] = -2
    q = rand((B, n, G, D), 683).to(dev())
    lens = np.array(lens, np.int32)
    o, lse = r9q.r9q_kv4_tree_attention(q, cache, on(table), on(lens), on(parents), return_lse=True)
    assert r9q.r9q_last_device_error() == 0
    some = [0, 1, B // 2, B - 1][:B]
    check(r9q, cache, table[some], lens[some], parents[some], q[some], o[some], lse[some])
    assert bool(torch.isfinite(o).all())


# ------------------------------------------------------------------ moves --

@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,Hk,D,page", [(1, 1, 1, 128, 16), (3, 5, 2, 64, 16), (7, 64, 1, 128, 48), (40, 8, 8, 128, 64),
                                              (5, 33, 3, 64, 32)])
def test_moves(r9q, rows, n, Hk, D, page):  # noqa: F811
    """Any places to any others of the same row's own, over one another; what is not named stays."""
    r = np.random.default_rng(661)
    span = -(-2 * n // page) + 1                              # pages of a row's own
    total = rows * span * page
    cache = r9q.r9q_kv4_cache(rows * span, Hk, page, D)
    x = rand((total, 2 * Hk, D), 662).to(dev())
    r9q.r9q_kv4_append(x[:, :Hk], x[:, Hk:], cache, torch.arange(total, device=dev()))
    src = np.stack([i * span * page + r.permutation(span * page)[:n] for i in range(rows)])
    dst = np.stack([i * span * page + r.permutation(span * page)[:n] for i in range(rows)])
    src[0, n // 2], dst[-1, n // 3] = -1, -5                  # passed over
    if n > 4:
        dst[1, 3] = dst[1, 1]                                 # the later one stays
    tokens = lambda: r9q.r9q_kv4_gather(cache, torch.arange(total, device=dev()))  # noqa: E731
    k, v = (t.clone() for t in tokens())
    before = [t.clone() for t in cache]
    ek, ev = k.clone(), v.clone()
    for i in range(rows):
        for a, b in zip(src[i], dst[i]):
            if a >= 0 and b >= 0:
                ek[b], ev[b] = k[a], v[a]
    r9q.r9q_kv4_move(cache, on(src), on(dst))
    assert r9q.r9q_last_device_error() == 0
    gk, gv = tokens()
    assert torch.equal(gk, ek) and torch.equal(gv, ev)
    for t, old in zip(cache, before):
        t.copy_(old)
    dst[0, 0], src[-1, n - 1] = total, 1 << 40                # outside the cache: an error, and passed over
    src[0, 0] = max(0, src[0, 0])
    r9q.r9q_kv4_move(cache, on(src), on(dst))
    assert r9q.r9q_last_device_error() == -8
    ek, ev = k.clone(), v.clone()
    for i in range(rows):
        for a, b in zip(src[i], dst[i]):
            if 0 <= a < total and 0 <= b < total:
                ek[b], ev[b] = k[a], v[a]
    gk, gv = tokens()
    assert torch.equal(gk, ek) and torch.equal(gv, ev)


# --------------------------------------------------------------- refusals --

def test_refusals():
    """Argument checks, on the host and before any CUDA call (the pointers are not addresses)."""
    import __graft_entry__
    __graft_entry__._builder().build()
    import block_scaled_fp8_x128_gb300 as lib
    c, M = lib._lib, 1 << 24
    DIM, NULL, ALIGN, ARG, WS = -2, -1, -3, -8, -4

    def attn(q=M, o=2 * M, B=2, Lq=3, Hq=4, Hk=2, D=128, parents=11 * M, ws=12 * M, wsb=1 << 26, scale=0.1, window=0):
        return c.r9q_kv4_tree_attention(q, 2048, 512, 128, 5 * M, 6 * M, 7 * M, 8 * M, 4 * M, 9 * M, parents, o, None, B, Lq,
                                        Hq, Hk, D, 4, 16, 3, window, scale, ws, wsb, None)
    assert attn(Lq=65) == DIM and attn(Hq=5) == DIM and attn(D=32) == DIM and attn(window=-1) == DIM
    assert attn(parents=None) == NULL and attn(q=None) == NULL and attn(parents=11 * M + 2) == ALIGN
    assert attn(o=11 * M) == ARG and attn(scale=0.0) == ARG and attn(ws=None) == WS and attn(wsb=1000) == WS
    assert attn(B=0) == 0 and attn(Lq=0) == 0 and attn(B=0, parents=None) == 0

    def move(kc=5 * M, src=M, dst=2 * M, rows=2, n=3, Hk=2, D=128, pages=4, page=16):
        return c.r9q_kv4_move(kc, 6 * M, 7 * M, 8 * M, src, dst, rows, n, Hk, D, pages, page, None)
    assert move(n=65) == DIM and move(rows=-1) == DIM and move(D=96) == DIM and move(page=8) == DIM and move(pages=0) == DIM
    assert move(src=None) == NULL and move(kc=None) == NULL and move(dst=2 * M + 4) == ALIGN and move(kc=5 * M + 8) == ALIGN
    assert move(src=5 * M) == ARG and move(kc=7 * M) == ARG and move(rows=0) == 0 and move(n=0) == 0
