"""Prompts, trees of drafted tokens, accepted paths and single tokens together, as a server runs them: the 4-bit
cache and the states of gated delta layers have to be what the accepted tokens alone make of them.  Every call is held
to its definition in 64 bits from what the cache and the states held before it (bounds: _delta_ref.py and
test_attention_block.py), and the end to the whole sequence token by token."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _delta_ref as ref
from _helpers import dev
from test_attention_block import check_attention, np64, on, r9q, rand  # noqa: F401
from test_gated_delta import check_state, inputs, some_state
from test_tree_attention import check

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu
HQ, HK, D, PAGE = 8, 2, 128, 16              # of the attention
KH, VH = 2, 4                                # of the delta rule
SCALE = D ** -0.5


class Run:
    """Sequences with a cache and states; a round is one call of each operator on buffers that stay."""

    def __init__(self, r9q, B, n, P, room):  # noqa: F811
        self.r9q, self.B, self.n, self.P = r9q, B, n, P
        per = -(-room // PAGE)
        self.cache = r9q.r9q_kv4_cache(B * per + 1, HK, PAGE, D)
        self.table = np.random.default_rng(5).permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
        self.dtable = on(self.table)
        self.state = some_state(B + 1, VH, D, 6).to(dev())
        self.slots = on(np.roll(np.arange(B, dtype=np.int32), 1))
        self.lens = np.zeros(B, np.int32)
        new = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=dev())  # noqa: E731
        self.q, self.k, self.v = new(B, n, HQ, D), new(B, n, HK, D), new(B, n, HK, D)
        self.dq, self.dk, self.dv = new(B, n, KH, D), new(B, n, KH, D), new(B, n, VH, D)
        self.g, self.beta = new(B, n, VH, t=torch.float32), new(B, n, VH, t=torch.float32)
        self.parents, self.path = new(B, n, t=torch.int32), new(B, P, t=torch.int32)
        self.places = new(B, n, t=torch.int64)
        self.src, self.dst = new(B, P, t=torch.int64), new(B, P, t=torch.int64)
        self.dlens = new(B, t=torch.int32)
        self.o, self.do = new(B, n, HQ, D), new(B, n, VH, D)
        self.lse = new(B, n, HQ, t=torch.float32)
        self.graph = None

    def slot(self, b, t):
        t = np.asarray(t)
        return self.table[b, t // PAGE].astype(np.int64) * PAGE + t % PAGE

    def prompt(self, lens, x, seed):
        """Packed prompts of these lengths: into the cache and the states."""
        q, k, v, g, beta = x
        kk, vv = (rand((sum(lens), HK, D), seed + i).to(dev()) for i in range(2))
        self.r9q.r9q_kv4_append(kk, vv, self.cache, on(np.concatenate([self.slot(b, np.arange(n)) for b, n in
                                                                        enumerate(lens)])))
        cu = np.cumsum([0, *lens]).astype(np.int32)
        self.r9q.r9q_gated_delta(q, k, v, on(g), on(beta), self.state, self.slots, on(cu), from_zero=True)
        self.lens[:] = lens
        return kk, vv

    def verify(self):
        r = self.r9q
        r.r9q_kv4_append(self.k.flatten(0, 1), self.v.flatten(0, 1), self.cache, self.places.view(-1))
        r.r9q_kv4_tree_attention(self.q, self.cache, self.dtable, self.dlens, self.parents, out=self.o, lse=self.lse)
        r.r9q_gated_delta_tree(self.dq, self.dk, self.dv, self.g, self.beta, self.state, self.slots, self.parents,
                               out=self.do)

    def accept(self):
        r = self.r9q
        r.r9q_kv4_move(self.cache, self.src, self.dst)
        r.r9q_gated_delta_commit(self.dk, self.dv, self.g, self.beta, self.state, self.slots, self.path)

    def launch(self, graphs):
        """Both halves of a round, between them what the caller looks at."""
        if not graphs:
            self.verify()
            yield
            self.accept()
            yield
            return
        if self.graph is None:
            kept = [t.clone() for t in (*self.cache, self.state)]
            self.verify()                                     # (a first call sets up what is not part of a graph)
            self.accept()
            for t, old in zip((*self.cache, self.state), kept):
                t.copy_(old)
            torch.cuda.synchronize()
            self.graph = []
            for f in (self.verify, self.accept):
                self.graph.append(torch.cuda.CUDAGraph())
                with torch.cuda.graph(self.graph[-1]):
                    f()
        for graph in self.graph:
            graph.replay()
            yield


def rounds_of(r9q, B, n, P, prompt, rounds, graphs, ends):  # noqa: F811
    """Everything that a run gave, for a comparison; `ends`: the drafts of a round that are no nodes."""
    rnd = np.random.default_rng(71)
    run = Run(r9q, B, n, P, max(prompt) + rounds * P + n + 2)
    x = inputs((sum(prompt),), KH, VH, D, 72)
    kk, vv = run.prompt(prompt, x, 73)
    cu = np.cumsum([0, *prompt])
    # what was accepted, of each sequence
    seq = [[np64(t[cu[b]:cu[b + 1]]) if torch.is_tensor(t) else t[cu[b]:cu[b + 1]].astype(np.float64) for t in x]
           for b in range(B)]
    kv = [[t[cu[b]:cu[b + 1]] for t in (kk, vv)] for b in range(B)]
    outs = []
    for i in range(rounds):
        # a tree: a chain of drafts, and others after any of it
        parents = np.full((B, n), -2, np.int32)
        path = np.full((B, P), -1, np.int32)
        for b in range(B):
            nodes = n - ends * ((i + b) % 3)
            for j in range(nodes):
                parents[b, j] = j - 1 if rnd.random() < 0.5 else rnd.integers(-1, j)
            j = int(rnd.integers(0, nodes))                   # the last accepted one; of some sequences none
            way = []
            while j != -1:
                way.append(j)
                j = parents[b, j]
            way = way[::-1][:P] if (i + b) % 4 else []
            path[b, :len(way)] = way
        y = inputs((B, n), KH, VH, D, 80 + 10 * i)
        for t, val in zip((run.dq, run.dk, run.dv, run.g, run.beta), y):
            t.copy_(val if torch.is_tensor(val) else on(val))
        for t, seed in ((run.q, 1), (run.k, 2), (run.v, 3)):
            t.copy_(rand(t.shape, 1000 + 10 * i + seed))
        run.parents.copy_(on(parents))
        run.path.copy_(on(path))
        run.dlens.copy_(on(run.lens + n))
        run.places.copy_(on(np.stack([run.slot(b, run.lens[b] + np.arange(n)) for b in range(B)])))
        run.src.copy_(on(np.stack([np.where(path[b] >= 0, run.slot(b, run.lens[b] + np.maximum(path[b], 0)), -1)
                                   for b in range(B)])))
        run.dst.copy_(on(np.stack([run.slot(b, run.lens[b] + np.arange(P)) for b in range(B)])))
        before = np64(run.state)
        halves = run.launch(graphs)
        next(halves)
        assert r9q.r9q_last_device_error() == 0
        assert np.array_equal(np64(run.state), before)        # a tree leaves the states alone
        check(r9q, run.cache, run.table, run.lens + n, parents, run.q, run.o, run.lse)
        do, z = np64(run.do), [np64(t) for t in (run.dq, run.dk, run.dv, run.g, run.beta)]
        slots = run.slots.cpu().numpy()
        for b in range(B):
            o, w = ref.tree(before[slots[b]], *(t[b] for t in z), parents[b], SCALE)
            assert (np.abs(do[b] - o) <= w).all()
        next(halves)
        assert r9q.r9q_last_device_error() == 0
        for b in range(B):
            way = path[b][path[b] >= 0]
            S, E, _, _ = ref.chain(before[slots[b]], *(t[b][way] for t in z), SCALE)
            check_state(run.state[int(slots[b])], S, E)
            seq[b] = [np.concatenate((s, t[b][way])) for s, t in zip(seq[b], z)]
            kv[b] = [torch.cat((s, t[b, on(way.astype(np.int64))])) for s, t in zip(kv[b], (run.k, run.v))]
            run.lens[b] += len(way)
        assert np.array_equal(np64(run.state[B]), before[B])            # nobody's state
        outs += [run.o.clone(), run.lse.clone(), run.do.clone(), run.state.clone()]
    # the cache: what the accepted tokens alone would have left
    plain = r9q.r9q_kv4_cache(*(run.cache.k.shape[i] for i in range(3)), D)
    for b in range(B):
        where = on(run.slot(b, np.arange(run.lens[b])))
        r9q.r9q_kv4_append(*kv[b], plain, where)
        assert all(torch.equal(s, t) for s, t in zip(r9q.r9q_kv4_gather(run.cache, where), r9q.r9q_kv4_gather(plain, where)))
    # and one more token of each, after all of its own
    one = inputs((B, 1), KH, VH, D, 999)
    q, k, v = (rand((B, 1, h, D), 990 + i).to(dev()) for i, h in enumerate((HQ, HK, HK)))
    r9q.r9q_kv4_append(k[:, 0], v[:, 0], run.cache, on(np.array([run.slot(b, run.lens[b]) for b in range(B)])))
    o, lse = r9q.r9q_kv4_attention(q, run.cache, run.dtable, on(run.lens + 1), return_lse=True)
    check_attention(r9q, run.cache, run.table, list(run.lens + 1), q, o, lse)
    do = np64(r9q.r9q_gated_delta_step(*(on(t) if isinstance(t, np.ndarray) else t for t in one), run.state, run.slots))
    for b in range(B):
        z = [np.concatenate((s, (np64(t) if torch.is_tensor(t) else t.astype(np.float64))[b])) for s, t in zip(seq[b], one)]
        S, E, eo, w = ref.chain(np.zeros((VH, D, D)), *z, SCALE)
        check_state(run.state[int(slots[b])], S, E)
        assert (np.abs(do[b, 0] - eo[-1]) <= w[-1]).all()
    return [*outs, o, lse, on(do)]


@pytest.mark.parametrize("B,n,P,prompt,ends", [(3, 7, 4, [50, 3, 17], 1), (2, 24, 9, [130, 64], 5), (1, 1, 1, [1], 0),
                                               (2, 64, 40, [20, 90], 11)])
def test_rounds(r9q, B, n, P, prompt, ends):  # noqa: F811
    """Call by call, and each half of a round captured once and replayed with other trees, paths and lengths: the same bits."""
    a = rounds_of(r9q, B, n, P, prompt, 5, False, ends)
    b = rounds_of(r9q, B, n, P, prompt, 5, True, ends)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "drafted_decoding.py"), "--prompt", "70", "--tokens",
                        "30", "--batch", "3", "--depth", "3"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens written" in r.stdout


# ------------------------------------------------- streams, devices, sizes --

def calls_of(r9q):  # noqa: F811
    """Each operator that allocates its outputs, on inputs large enough for their blocks to be seen."""
    B, n = 64, 40
    per = 4
    cache = r9q.r9q_kv4_cache(B * per, HK, PAGE, D)
    every = torch.arange(B * per * PAGE, device=dev())
    kv = rand((len(every), 2 * HK, D), 31).to(dev())
    r9q.r9q_kv4_append(kv[:, :HK], kv[:, HK:], cache, every)
    q = rand((B, n, HQ, D), 32).to(dev())
    table = torch.arange(B * per, dtype=torch.int32, device=dev()).view(B, per)
    lens = torch.full((B,), 60, dtype=torch.int32, device=dev())
    parents = torch.arange(-1, n - 1, dtype=torch.int32, device=dev()).repeat(B, 1)
    x = [on(t) if isinstance(t, np.ndarray) else t for t in inputs((B, n), KH, VH, D, 33)]
    flat = [t.flatten(0, 1) for t in x]
    state = torch.zeros((B, VH, D, D), device=dev())
    slots = torch.arange(B, dtype=torch.int32, device=dev())
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev()) * n
    return {"attention": lambda **k: r9q.r9q_kv4_tree_attention(q, cache, table, lens, parents, return_lse=True, **k),
            "prompt": lambda **k: r9q.r9q_gated_delta(*flat, state, slots, cu, from_zero=True, **k),
            "step": lambda **k: r9q.r9q_gated_delta_step(*x, state, slots, from_zero=True, **k),
            "tree": lambda **k: r9q.r9q_gated_delta_tree(*x, state, slots, parents, **k)}


@pytest.mark.parametrize("name", ["attention", "prompt", "step", "tree"])
def test_outputs_belong_to_the_stream_of_the_call(r9q, name):  # noqa: F811
    """The current stream still has work on a block that it has let go; outputs of a call on another stream are not
    made of that block."""
    call = calls_of(r9q)[name]
    st = torch.cuda.Stream()
    want = call()
    with torch.cuda.stream(st):
        call()                                                # (workspaces, and blocks that the stream can have again)
    torch.cuda.synchronize()
    want = want if isinstance(want, tuple) else (want,)
    block = torch.empty(want[0].untyped_storage().nbytes(), dtype=torch.uint8, device=dev())
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    block.fill_(7)
    del block
    got = call(stream=st)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_calls_run_on_the_device_of_their_tensors(r9q, monkeypatch):  # noqa: F811
    """With another device current (as the binding sees it), a call makes the tensors' own current; a stream of another
    device is refused."""
    calls = calls_of(r9q)
    wants = {name: f() for name, f in calls.items()}
    entered, now = [], [1]

    class Device(torch.cuda.device):
        def __enter__(self):
            entered.append(self.idx)
            now.append(self.idx)
            return super().__enter__()

        def __exit__(self, *error):
            now.pop()
            return super().__exit__(*error)

    class Other:
        device = torch.device("cuda", 1)
        cuda_stream = 12345
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(r9q, "_current_device", lambda: now[-1])
    for i, (name, f) in enumerate(calls.items()):
        got, want = f(), wants[name]
        assert entered == [0] * (i + 1) and now == [1]
        assert all(torch.equal(a, b) for a, b in zip(*(t if isinstance(t, tuple) else (t,) for t in (got, want))))
        with pytest.raises(ValueError):
            f(stream=Other())


def test_out_of_memory_is_torch_s(r9q):  # noqa: F811
    """Outputs that do not fit (of a small share of the memory that the process may have): the error that torch raises."""
    x = rand((1, 1, 2, 128), 35).to(dev()).expand(1, 20_000_000, 2, 128)
    g = torch.zeros((1, 1, 2), device=dev())
    args = (torch.zeros((1, 2, 128, 128), device=dev()), torch.zeros(1, dtype=torch.int32, device=dev()))
    rates = torch.zeros((1, 20_000_000, 2), device=dev())
    torch.cuda.empty_cache()                                  # (blocks that earlier tests left)
    torch.cuda.set_per_process_memory_fraction(0.01)
    try:
        with pytest.raises(torch.cuda.OutOfMemoryError):
            r9q.r9q_gated_delta_step(x, x, x, rates, rates, *args)       # 10 GB
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    o = r9q.r9q_gated_delta_step(x[:, :1], x[:, :1], x[:, :1], g, g, *args)
    assert o.shape == (1, 1, 2, 128) and r9q.r9q_last_device_error() == 0


@pytest.mark.parametrize("n,heads", [(8, 8), (40, 32)])
def test_cache_past_32_bits(r9q, n, heads):  # noqa: F811
    """Pages at the end of a cache of more than 2^32 bytes of keys, for few rows and for many; tokens moved between
    them."""
    Hk, page, pages = 8, 256, 34000                           # 4.5 GB of keys
    cache = r9q.r9q_kv4_cache(pages, Hk, page, D)
    table = np.full((1, 72), -1, np.int32)                    # (so wide that many rows take their own kernel)
    table[0, :3] = [pages - 1, 5, pages - 2]
    length = 600
    t = np.arange(length)
    slots = table[0, t // page].astype(np.int64) * page + t % page
    kv = rand((length, 2 * Hk, D), 41).to(dev())
    r9q.r9q_kv4_append(kv[:, :Hk], kv[:, Hk:], cache, on(slots))
    q = rand((1, n, heads, D), 42).to(dev())
    parents = torch.arange(-1, n - 1, dtype=torch.int32, device=dev())[None]
    o, lse = r9q.r9q_kv4_tree_attention(q, cache, on(table), on(np.array([length], np.int32)), parents, return_lse=True)
    small = r9q.r9q_kv4_cache(72, Hk, page, D)                # the same tokens in a small one
    low = np.full((1, 72), -1, np.int32)
    low[0, :3] = [2, 0, 1]
    there = low[0, t // page].astype(np.int64) * page + t % page
    r9q.r9q_kv4_append(kv[:, :Hk], kv[:, Hk:], small, on(there))
    e, elow = r9q.r9q_kv4_tree_attention(q, small, on(low), on(np.array([length], np.int32)), parents, return_lse=True)
    assert torch.equal(o, e) and torch.equal(lse, elow)
    r9q.r9q_kv4_move(cache, on(slots[None, 550:600]), on(slots[None, 10:60]))
    a, b = (r9q.r9q_kv4_gather(cache, on(slots[s])) for s in (slice(550, 600), slice(10, 60)))
    c = r9q.r9q_kv4_gather(small, on(there[550:600]))
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))
    assert r9q.r9q_last_device_error() == 0


@pytest.mark.parametrize("Lq", [1, 5, 70])
def test_states_past_32_bits(r9q, Lq):  # noqa: F811
    """A slot behind 2^32 elements of states."""
    n = (1 << 32) // (VH * D * D) + 3
    state = torch.empty((n, VH, D, D), device=dev())          # 17 GB
    state[n - 1] = 0.25
    z = [on(t) if isinstance(t, np.ndarray) else t for t in inputs((1, Lq), KH, VH, D, 51)]
    small = torch.full((1, VH, D, D), 0.25, device=dev())
    slot = torch.tensor([n - 1], dtype=torch.int32, device=dev())
    zero = torch.zeros_like(slot)
    parents = torch.arange(-1, Lq - 1, dtype=torch.int32, device=dev())[None]
    if Lq <= 64:
        assert torch.equal(r9q.r9q_gated_delta_tree(*z, state, slot, parents), r9q.r9q_gated_delta_tree(*z, small, zero, parents))
        path = parents + 1
        r9q.r9q_gated_delta_commit(*z[1:], state, slot, path)
        r9q.r9q_gated_delta_commit(*z[1:], small, zero, path)
        assert torch.equal(state[n - 1:], small)
    a, b = r9q.r9q_gated_delta_step(*z, state, slot), r9q.r9q_gated_delta_step(*z, small, zero)
    assert torch.equal(a, b) and torch.equal(state[n - 1:], small)
    assert r9q.r9q_last_device_error() == 0
