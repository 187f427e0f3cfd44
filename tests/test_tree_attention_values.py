"""Attention of a tree over values that are not of one size: a token's values far from zero with little between them, or far
larger than all others while the token is seen with next to no weight.  Both kernels, within the bounds of
test_attention_block.py: what weights and values lose to fp16 counts with the codes' range, not with the values' size.

Below a range the bound grows.  A weight times its step, against the largest weight and the largest step's exponent E as 2^8, is
an fp16 number: under 2^-14 it is rounded by up to 2^-25, which moves a value 7.5 steps from the codes' middle, or 8, by
2^-25 2^-8 8 2^E / (N p) with p the keys' mean weight and N p_max = p_max / p: 2^-30 N p_max 2^E."""
import numpy as np
import pytest
import torch

import _attention_ref as ref
from _helpers import dev
from test_attention_block import U, codes_of, make_cache, np64, on, r9q, rand  # noqa: F401
from test_gated_delta import random_parents
from test_tree_attention import check, way_to, widened

# (nodes, query heads of the one key-value head, D, many rows' kernel)
KERNELS = [(9, 2, 128, False), (40, 8, 128, False), (40, 8, 128, True), (33, 6, 64, True), (12, 8, 128, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq,D,wide", KERNELS)
@pytest.mark.parametrize("signs", ["one sign", "alternating", "any"])
@pytest.mark.parametrize("size", [50.0, 3e4])
def test_values_far_from_zero(r9q, n, Hq, D, wide, signs, size):  # noqa: F811
    lens = [n + 30, 150]
    cache, table, slots = make_cache(r9q, lens, 1, D, 16, 701)
    table = widened(table, 16, 1, n * Hq) if wide else table
    r = np.random.default_rng(702)
    off = size * r.uniform(0.5, 2, len(slots))
    if signs == "alternating":
        off[1::2] *= -1
    if signs == "any":
        off *= r.choice((-1, 1), len(slots))
    v = torch.from_numpy(off[:, None, None] * (1 + r.normal(0, 0.01, (len(slots), 1, D)))).to(torch.bfloat16)
    r9q.r9q_kv4_append(rand((len(slots), 1, D), 703).to(dev()), v.to(dev()), cache, on(slots))
    parents = random_parents(2, n, 704)
    q = rand((2, n, Hq, D), 705, 0.14).to(dev())              # (scores of about one: weights that fp16 rounds)
    o, lse = r9q.r9q_kv4_tree_attention(q, cache, on(table), on(np.array(lens, np.int32)), on(parents), return_lse=True)
    assert r9q.r9q_last_device_error() == 0
    check(r9q, cache, table, lens, parents, q, o, lse)


def one_large(r9q, n, Hq, D, wide, size, where, seed):  # noqa: F811
    """One sequence whose token `where` (of what is before the tree; -1: a node) has values `size` times the others' and a key
    that every query is far from."""
    length = 400
    cache, table, slots = make_cache(r9q, [length], 1, D, 16, seed)
    table = widened(table, 16, 1, n * Hq) if wide else table
    k, v = rand((length, 1, D), seed + 1), rand((length, 1, D), seed + 2)
    at = length - n if where < 0 else where                   # (the tree's first node, that most come from)
    v[at] *= size
    k[at, :, 0] = -400.0
    r9q.r9q_kv4_append(k.to(dev()), v.to(dev()), cache, on(slots))
    parents = np.maximum(random_parents(1, n, seed + 3), np.minimum(np.arange(n) - 1, 0)[None]).astype(np.int32)
    q = rand((1, n, Hq, D), seed + 4)
    q[..., 0] = 4.0 + q[..., 0].abs()
    q = q.to(dev())
    o, lse = r9q.r9q_kv4_tree_attention(q, cache, on(table), on(np.array([length], np.int32)), on(parents), return_lse=True)
    assert r9q.r9q_last_device_error() == 0
    return cache, table, length, parents, q, o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq,D,wide", KERNELS)
@pytest.mark.parametrize("where", [0, 130, -1])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 14, 2.0 ** 18])
def test_a_large_value_with_no_weight(r9q, n, Hq, D, wide, where, size):  # noqa: F811
    cache, table, length, parents, q, o, lse = one_large(r9q, n, Hq, D, wide, size, where, 711)
    check(r9q, cache, table, [length], parents, q, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq,D,wide", KERNELS)
@pytest.mark.parametrize("where", [0, -1])
@pytest.mark.parametrize("size", [2.0 ** 21, 2.0 ** 24, 2.0 ** 60])
def test_a_value_too_large_for_the_others(r9q, n, Hq, D, wide, where, size):  # noqa: F811
    """The range's end: what is lost is bounded by the largest step seen, and weights' sums stay."""
    cache, table, length, parents, q, o, lse = one_large(r9q, n, Hq, D, wide, size, where, 721)
    kc, vc, kp, vp = codes_of(cache)
    t = np.arange(length)
    p, at = table[0, t // 16], t % 16
    k = kp[p, :, at, 1:] + kp[p, :, at, :1] * kc[p, :, at]
    v = vp[p, :, at, 1:] + vp[p, :, at, :1] * vc[p, :, at]
    step = vp[p, :, at, 0]
    q, o, lse = np64(q), np64(o), np64(lse)
    for i in range(n):
        keys = list(range(length - n)) + [length - n + x for x in way_to(parents[0], i)]
        eo, el, wide_, mass, top = ref.attention(q[0, i:i + 1], k[keys], v[keys], 15 * step[keys], D ** -0.5, 0)
        S = np.maximum(1, top)
        assert (np.abs(lse[0, i] - el[0]) <= 2.0 ** -17 * S[0]).all()
        s = k[keys][:, 0] @ q[0, i].T * D ** -0.5
        most = np.exp(s.max(0) - el[0]) * len(keys)           # N p_max of every head
        lost = 2.0 ** -30 * most * step[keys].max()
        bound = U * np.abs(eo) * 1.01 + 2.0 ** -11 * wide_[..., None] + 2.0 ** -17 * S[..., None] * mass + lost[:, None]
        assert (np.abs(o[0, i] - eo[0]) <= bound[0]).all(), (i, (np.abs(o[0, i] - eo[0]) - bound[0]).max())
