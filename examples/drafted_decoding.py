"""A hybrid decoder that verifies drafted tokens: a gated delta layer, then the attention layer of decode_layer.py.

    python examples/drafted_decoding.py [--batch 4] [--prompt 300] [--tokens 200] [--depth 4]

Each round, for every sequence, the newest token and `depth` levels of two drafts each form a tree (the second of a
level ends there).  Both layers run over its nodes at once, the delta rule from a state that they do not change:

    state layer       r9q_gated_delta (the prompt), r9q_gated_delta_tree (drafts)
    attention layer   nodes written behind the sequence's tokens in the 4-bit cache, r9q_kv4_tree_attention
    what is accepted  the longest path of nodes that are what the model says after their parents:
                      r9q_gated_delta_commit takes the state along it, r9q_kv4_move closes up its tokens in the cache

Drafts are what followed a token the last time and the time before, so that a model which repeats itself is
fast.  Weights are random and decoding is greedy.  A round is captured once as a CUDA graph and replayed: lengths, paths
and drafts are all on the device.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import block_scaled_fp8_x128_gb300 as r9q  # noqa: E402
from decode_layer import Layer, norm  # noqa: E402


class Decoder:
    def __init__(self, vocab=64, batch=4, depth=4, k_heads=4, v_heads=8, dim=128, max_tokens=2048, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.attention = Layer(batch=batch, max_tokens=max_tokens, seed=seed)
        hidden = self.attention.hidden
        self.vocab, self.batch, self.k_heads, self.v_heads, self.dim = vocab, batch, k_heads, v_heads, dim

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")
        self.embed = randn(vocab, hidden).to(torch.bfloat16)
        self.w_in = r9q.r9q_quant_weight_block128(randn((2 * k_heads + v_heads) * dim, hidden) * hidden ** -0.5)
        self.w_rates = (randn(hidden, 2 * v_heads) * hidden ** -0.5).to(torch.bfloat16)
        self.w_out = r9q.r9q_quant_weight_block128(randn(hidden, v_heads * dim) * (v_heads * dim) ** -0.5)
        self.state = torch.zeros((batch, v_heads, dim, dim), device="cuda")
        self.slots = torch.arange(batch, dtype=torch.int32, device="cuda")
        # the tree: node 0 the newest token, 2 l + 1 and 2 l + 2 the drafts after 2 l - 1
        parents = [-1] + [max(0, 2 * (i // 2) - 1) for i in range(2 * depth)]
        ways = []
        for i, up in enumerate(parents):
            ways.append((ways[up] if up >= 0 else []) + [i])
        self.nodes, self.longest = len(parents), depth + 1
        self.parents = torch.tensor(parents, dtype=torch.int32, device="cuda").repeat(batch, 1)
        self.depth = torch.tensor([len(w) - 1 for w in ways], device="cuda")
        self.way = torch.tensor([w + [-1] * (self.longest - len(w)) for w in ways], device="cuda")
        self.not_above = torch.tensor([[j not in w for j in range(len(ways))] for w in ways], device="cuda")
        self.up = torch.tensor(parents[1:], device="cuda")
        self.after = torch.randint(0, vocab, (batch, vocab, 2), generator=g, device="cuda")     # drafts of a token
        self.newest = torch.zeros(batch, dtype=torch.int64, device="cuda")
        self.written = torch.zeros((batch, max_tokens), dtype=torch.int64, device="cuda")
        self.count = torch.zeros(batch, dtype=torch.int64, device="cuda")

    def forward(self, tokens, tree):
        """int64 [batch][n] -> what the model says after each, and what a commit of the state takes."""
        n = tokens.shape[1]
        x = self.embed[tokens].view(self.batch * n, -1)
        h = norm(x)
        parts = r9q.r9q_gemm_fp8_block_qa(h, *self.w_in).view(self.batch, n, -1, self.dim)
        q, k, v = parts.split((self.k_heads, self.k_heads, self.v_heads), 2)
        g, beta = (h @ self.w_rates).float().view(self.batch, n, 2, self.v_heads).unbind(2)
        g, beta = -torch.nn.functional.softplus(g - 2), beta.sigmoid()
        if tree:
            o = r9q.r9q_gated_delta_tree(q, k, v, g, beta, self.state, self.slots, self.parents)
        else:
            starts = torch.arange(self.batch + 1, dtype=torch.int32, device="cuda") * n
            o = r9q.r9q_gated_delta(*(t.flatten(0, 1) for t in (q, k, v, g, beta)), self.state, self.slots, starts,
                                    from_zero=True)
        x = (x + r9q.r9q_gemm_fp8_block_qa(o.view(self.batch * n, -1), *self.w_out)).view(self.batch, n, -1)
        y = self.attention.step(x, self.parents, self.depth) if tree else self.attention.step(x)
        return (norm(y) @ self.embed.T).argmax(-1), (k, v, g, beta)

    def prompt(self, tokens):
        said, _ = self.forward(tokens, False)
        self.newest.copy_(said[:, -1])

    def round(self):
        nodes, t = [self.newest], self.newest
        for _ in range(self.longest - 1):
            draft = self.after.gather(1, t[:, None, None].expand(-1, 1, 2))[:, 0]
            nodes += [draft[:, 0], draft[:, 1]]
            t = draft[:, 0]
        nodes = torch.stack(nodes, 1)
        said, rates = self.forward(nodes, True)
        right = torch.cat((torch.ones_like(nodes[:, :1], dtype=torch.bool), nodes[:, 1:] == said[:, self.up]), 1)
        right = (right[:, None, :] | self.not_above).all(-1)
        last = torch.where(right, self.depth, -1).argmax(-1)
        path, length = self.way[last], self.depth[last] + 1
        # the caches follow
        r9q.r9q_gated_delta_commit(*rates, self.state, self.slots, path.int())
        layer = self.attention
        layer.lens -= self.nodes
        start = layer.lens.long()[:, None]
        taken = path >= 0
        to = torch.arange(self.longest, device="cuda")[None]
        src, dst = layer.places(start + path.clamp(min=0)), layer.places(start + to)
        r9q.r9q_kv4_move(layer.cache, torch.where(taken, src, -1), torch.where(taken, dst, -1))
        layer.lens += length.int()
        # what was written, and what followed what
        for i in range(self.longest):
            at, live = path[:, i].clamp(min=0)[:, None], taken[:, i]
            token, then = nodes.gather(1, at)[:, 0], said.gather(1, at)[:, 0]
            place = (self.count + i)[:, None]
            self.written.scatter_(1, place, torch.where(live, token, self.written.gather(1, place)[:, 0])[:, None])
            index = token[:, None, None].expand(-1, 1, 2)
            was = self.after.gather(1, index)[:, 0]
            new = torch.stack((then, torch.where(was[:, 0] == then, was[:, 1], was[:, 0])), 1)
            self.after.scatter_(1, index, torch.where(live[:, None], new, was)[:, None])
        self.count += length
        self.newest.copy_(said.gather(1, last[:, None])[:, 0])


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--depth", type=int, default=4)
    a = ap.parse_args()
    if not 1 <= a.depth <= 31:
        raise SystemExit("a tree has at most 64 nodes: --depth from 1 to 31")
    dec = Decoder(batch=a.batch, depth=a.depth, max_tokens=a.prompt + (a.tokens + 2) * (a.depth + 2) + 64)
    dec.prompt(torch.randint(0, dec.vocab, (a.batch, a.prompt), device="cuda"))
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        dec.round()                                      # what a first call sets up once is not part of the graph
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=warm):
            dec.round()
    torch.cuda.current_stream().wait_stream(warm)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    first, rounds = dec.count.clone(), 0
    start.record()
    while int(dec.count.min()) < a.tokens:               # (a round writes a token of every sequence at least)
        graph.replay()
        rounds += 1
    end.record()
    torch.cuda.synchronize()
    if r9q.r9q_last_device_error():
        raise SystemExit("a kernel reported an error")
    if not bool(torch.isfinite(dec.state).all()):
        raise SystemExit("a state is not finite")
    if rounds:
        tokens = float((dec.count - first).float().mean())
        print(f"{a.batch} sequences, {a.prompt} prompt tokens: {rounds} rounds, {start.elapsed_time(end) / rounds * 1e3:.1f} "
              f"us each, {tokens / rounds:.2f} tokens a round")
    print(f"at least {int(dec.count.min())} tokens written")


if __name__ == "__main__":
    main()
