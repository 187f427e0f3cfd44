"""Trees of many rows seen through a window: the kernel for many rows, which takes a call by sequences, heads and rows
as well as by the window's length."""
import numpy as np
import pytest
import torch

from _helpers import dev
from test_attention_block import U, codes_of, make_cache, np64, on, r9q, rand  # noqa: F401
from test_gated_delta import random_parents
from test_tree_attention import check, way_to


def takes_many(B, Hk, rows, room, window, n):
    """Which kernel a call takes: more than 64 rows, and sequences x heads x groups of 16 keys x groups of 16 rows over 36000,
    with the keys that pages can hold or that a window reaches."""
    groups = min(room, window + n - 1 if window else room) // 16 + 1
    return rows > 64 and B * Hk * groups * -(-rows // 16) > 36000


# (sequences, nodes, Hq, Hk, D, page, window, the longest): 125 and 96 rows are one tile, the others two and more
WINDOWS = [(32, 20, 16, 2, 64, 16, 1000, 2600), (32, 20, 16, 2, 128, 32, 1000, 2600), (40, 33, 64, 8, 128, 64, 100, 900),
           (60, 64, 32, 4, 64, 16, 1, 400), (60, 64, 32, 4, 128, 16, 7, 400), (7, 48, 8, 1, 128, 48, 4000, 5000),
           (34, 12, 16, 2, 128, 16, 1500, 2000), (34, 25, 10, 2, 64, 16, 1200, 3000)]

# few rows, and many keys for each warp of the kernel that takes them
FEW = [(96, 16, 8, 2, 128, 16, 1500, 2600), (96, 12, 8, 2, 64, 32, 900, 2600), (200, 7, 4, 4, 128, 16, 600, 2600)]


def windowed(r9q, B, n, Hq, Hk, D, page, window, longest, kind, seed, q_scale=1.0):  # noqa: F811
    """Lengths about the window's edges and any; pages that no node sees any more are given back."""
    lens = [longest, 0, n - 1, n, n + window, n + window + 1, 1]
    lens += [1 + (i * 397) % longest for i in range(len(lens), B)]
    lens = np.minimum(np.array(lens[:B]), longest)
    cache, table, slots = make_cache(r9q, lens.tolist(), Hk, D, page, seed)
    whole = table.copy()
    for b, length in enumerate(lens):
        table[b, :max(0, length - n - window + 1) // page] = -1
    parents = {"random": random_parents(B, n, seed + 3), "chain": np.tile(np.arange(n) - 1, (B, 1))}[kind].astype(np.int32)
    parents[-1, n - 3:] = -2
    q = rand((B, n, Hq, D), seed + 4, q_scale).to(dev())
    assert takes_many(B, Hk, n * Hq // Hk, table.shape[1] * page, window, n) == (n * Hq // Hk > 64)
    return cache, whole, table, lens.astype(np.int32), parents, q, slots


@pytest.mark.gpu
@pytest.mark.parametrize("case", WINDOWS)
@pytest.mark.parametrize("kind", ["random", "chain"])
def test_windows_of_many_rows(r9q, case, kind):  # noqa: F811
    """Some sequences against the definition; all against the kernel for few rows, which takes them one by one: two results
    within the bounds of test_attention_block.py."""
    B, n, Hq, Hk, D, page, window, _ = case
    cache, _, table, lens, parents, q, _ = windowed(r9q, *case, kind, 801)
    o, lse = r9q.r9q_kv4_tree_attention(q, cache, on(table), on(lens), on(parents), window=window, return_lse=True)
    assert r9q.r9q_last_device_error() == 0
    some = [0, 1, 2, 3, 4, 5, 6, B - 1]
    check(r9q, cache, table[some], lens[some], parents[some], q[some], o[some], lse[some], window)
    codes, _, kp, vp = codes_of(cache)
    kp, vp = np.nan_to_num(kp), np.nan_to_num(vp)             # (places without a token)
    spread, most = 15 * vp[..., 0].max(), np.abs(vp).max() * 16
    reach = np.abs(kp[..., 1]).max() + 15 * kp[..., 0].max()  # the largest key's element
    S = max(1.0, np.abs(np64(q)).sum(-1).max() * reach * D ** -0.5)
    near = 2 * (2.0 ** -11 * spread + 2.0 ** -17 * S * most)
    for b in range(B):
        assert not takes_many(1, Hk, n * Hq // Hk, table.shape[1] * page, window, n)
        few, few_lse = r9q.r9q_kv4_tree_attention(q[b:b + 1], cache, on(table[b:b + 1]), on(lens[b:b + 1]), on(parents[b:b + 1]),
                                                  window=window, return_lse=True)
        d, seen = (o[b].float() - few[0].float()).abs(), torch.isfinite(few_lse[0])
        assert bool((d <= 2.02 * U * few[0].float().abs() + near).all()), b
        assert torch.equal(seen, torch.isfinite(lse[b]))
        assert bool(((lse[b] - few_lse[0])[seen].abs() <= 2.0 ** -16 * S).all()), b
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", [WINDOWS[1], WINDOWS[2], WINDOWS[4], WINDOWS[6], WINDOWS[7], *FEW])
@pytest.mark.parametrize("q_scale", [1.0, 12.0])
def test_what_is_before_a_window(r9q, case, q_scale):  # noqa: F811
    """A key before the window reaches no node, and one at its edge only the nodes that are not deep: the others' results stay,
    bit for bit, whatever it holds.  Scores of about one, and large ones, against which references move."""
    B, n, Hq, Hk, D, page, window, _ = case
    cache, whole, _, lens, parents, q, _ = windowed(r9q, *case, "random", 811, q_scale)
    args = (q, cache, on(whole), on(lens), on(parents))
    base = r9q.r9q_kv4_tree_attention(*args, window=window, return_lse=True)
    depth = np.array([[len(way_to(p, i) or []) - 1 for i in range(n)] for p in parents])
    node = parents != -2
    first = lens - n - window + 1                             # a node of depth d sees keys from first + d on
    for edge in (-1, 0, 2):
        at = first + edge
        which = np.nonzero((at >= 0) & (at < lens - n))[0]
        if not len(which):                                    # (a window of one has no such key)
            assert edge >= window - 1
            continue
        slots = whole[which, at[which] // page].astype(np.int64) * page + at[which] % page
        kept = r9q.r9q_kv4_gather(cache, on(slots))
        before = [t.clone() for t in cache]
        sees = np.zeros((B, n), bool)
        sees[which] = (depth[which] <= edge) & node[which]
        for x in (-3.3895313892515355e38, 1e30, float("inf"), float("nan")):
            k, v = kept[0].clone(), kept[1].clone()
            k[:, :, 3], v[:, :, 5] = x, x
            r9q.r9q_kv4_append(k, v, cache, on(slots))
            o, lse = r9q.r9q_kv4_tree_attention(*args, window=window, return_lse=True)
            keep = on(~sees)
            assert torch.equal(o[keep], base[0][keep]) and torch.equal(lse[keep], base[1][keep]), (edge, x)
            if not np.isfinite(x):
                assert bool(torch.isnan(o[~keep]).all()), (edge, x)
            for t, old in zip(cache, before):
                t.copy_(old)
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", [WINDOWS[0], WINDOWS[2]])
def test_windows_under_a_graph(r9q, case):  # noqa: F811
    """Lengths, trees and tables that change between replays."""
    B, n, Hq, Hk, D, page, window, _ = case
    cache, whole, table, lens, parents, q, _ = windowed(r9q, *case, "random", 821)
    t, le, pa = on(whole), on(lens), on(parents)
    r9q.r9q_kv4_tree_attention(q, cache, t, le, pa, window=window)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = r9q.r9q_kv4_tree_attention(q, cache, t, le, pa, window=window, return_lse=True)
    for shift in (0, 3, 11):
        now = np.maximum(0, lens - 37 * shift).astype(np.int32)
        tree = np.roll(parents, shift, 0)
        le.copy_(on(now))
        pa.copy_(on(tree))
        o.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert r9q.r9q_last_device_error() == 0
        some = [0, 1, 4, B - 1]
        check(r9q, cache, whole[some], now[some], tree[some], q[some], o[some], lse[some], window)
        want = r9q.r9q_kv4_tree_attention(q, cache, t, le, pa, window=window, return_lse=True)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("n,G,D", [(40, 1, 128), (24, 2, 64), (64, 1, 128), (36, 8, 128)])
@pytest.mark.parametrize("v_scale", [0.0, 1e-25])
def test_low_scores_behind_a_window(r9q, n, G, D, v_scale):  # noqa: F811
    """Tokens of which only the first see something of the first keys that a warp takes; then keys whose values are nearly nothing
    and whose scores are far under zero (2^score is 0 in fp32).  All of them count, for newest tokens and for a chain of nodes."""
    B, window, page = 160, 1500, 16
    lens = np.array([n + window + i % 64 for i in range(B)], np.int32)        # (every place of the window's edge in a step)
    cache, table, slots = make_cache(r9q, lens.tolist(), 1, D, page, 831)
    k = torch.full((len(slots), 1, D), -5.0, dtype=torch.bfloat16)
    r9q.r9q_kv4_append(k.to(dev()), rand((len(slots), 1, D), 832, v_scale).to(dev()), cache, on(slots))
    q = torch.full((B, n, G, D), 0.5, dtype=torch.bfloat16, device=dev())
    args = (q, cache, on(table), on(lens))
    chain = np.tile(np.arange(n) - 1, (B, 1)).astype(np.int32)
    # every key has the same score: lse is that and the logarithm of the window's tokens
    want = -5.0 * 0.5 * D + np.log(window)
    for o, lse in (r9q.r9q_kv4_attention(*args, scale=1.0, window=window, return_lse=True),
                   r9q.r9q_kv4_tree_attention(*args, on(chain), scale=1.0, window=window, return_lse=True)):
        off = np.abs(np64(lse) - want).max()
        assert off <= 2.0 ** -17 * (5.0 * 0.5 * D), off
        assert bool(torch.isfinite(o).all())
    assert r9q.r9q_last_device_error() == 0
