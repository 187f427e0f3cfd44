"""The operators of a hybrid decoder with drafted tokens, as cases to be timed and compared.

A hybrid decoder has attention layers over the paged 4-bit cache and layers whose
memory is a matrix a head, the gated delta rule.  A drafter proposes a tree of
tokens after each sequence; the tree is verified in one step and the accepted path
is kept.  Five operators:

  attention  r9q_kv4_tree_attention: attention of a tree's nodes over the cached
             sequence and their ancestors;
  prompt     r9q_gated_delta: the gated delta rule over packed sequences;
  step       r9q_gated_delta_step: over the newest tokens of every sequence;
  tree       r9q_gated_delta_tree: along every path of a tree;
  accept     r9q_kv4_move and r9q_gated_delta_commit: an accepted path becomes the
             sequence's newest tokens, in the cache and in the state.

The gated delta rule, for a value head with the state S [D values][D keys]:

  S_t = a S + u k^T,  u = beta (v - a S k),  a = exp(g),  o = scale S_t q

with q and k of unit length (x / sqrt(sum x^2 + eps)).  In a tree S comes from the
node's parent.  A node's parent comes before it; -1 is the sequence before the
tree, -2 marks a place of the batch without a node.

The cache's layout is that of include/r9q.h: K codes [page][D/2], V codes in groups
of 16 tokens [page/16][D/64][8 r][4 j][4 m][4 b], one bf16 pair (step, lowest value)
for each token, K and V; a code c stands for lowest + step*c.

`own` selects the library's calls; otherwise `run` computes the plain forms.
"""
import math
import types

import torch

own = False

EPS = 1e-6
CHUNK = 64


def listed():
    return [
        # one sequence just begun and a tree of eight nodes, as many key-value heads as query heads: latency
        {"name": "attention_1x8_77", "op": "attention", "batch": 1, "nodes": 8, "context": 77, "q_heads": 32,
         "kv_heads": 32, "dim": 128, "page": 16, "window": 0, "ragged": False},
        # small heads, seven query heads to a key-value head, an odd tree after a long sequence seen through a window
        {"name": "attention_6x21_window", "op": "attention", "batch": 6, "nodes": 21, "context": 5000, "q_heads": 14,
         "kv_heads": 2, "dim": 64, "page": 16, "window": 1024, "ragged": True},
        # a small serving batch of mixed lengths, one place of it empty; 64 rows for each key-value head
        {"name": "attention_8x16_4096", "op": "attention", "batch": 8, "nodes": 16, "context": 4096, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "ragged": True},
        # the largest: trees of 32 nodes after sixteen long sequences, 256 rows for each key-value head
        {"name": "attention_16x32_8191", "op": "attention", "batch": 16, "nodes": 32, "context": 8191, "q_heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "ragged": False},
        # one prompt of one sequence: no more than a chain of chunks for each head
        {"name": "prompt_1x8192", "op": "prompt", "batch": 1, "tokens": 8192, "k_heads": 16, "v_heads": 32,
         "dim": 128, "ragged": False},
        # the prompts that a server has waiting, of mixed lengths, continued from earlier parts
        {"name": "prompt_16x2000", "op": "prompt", "batch": 16, "tokens": 2000, "k_heads": 16, "v_heads": 32,
         "dim": 128, "ragged": True},
        # a decode step of one sequence: latency
        {"name": "step_1", "op": "step", "batch": 1, "tokens": 1, "k_heads": 16, "v_heads": 32, "dim": 128},
        # a decode step of a full serving batch, one place of it padding: every state is read and written
        {"name": "step_128", "op": "step", "batch": 128, "tokens": 1, "k_heads": 16, "v_heads": 32, "dim": 128},
        # four drafted tokens a sequence, in small heads
        {"name": "tree_5x4", "op": "tree", "batch": 5, "nodes": 4, "k_heads": 4, "v_heads": 12, "dim": 64},
        # trees of sixteen nodes of sixteen sequences
        {"name": "tree_16x16", "op": "tree", "batch": 16, "nodes": 16, "k_heads": 16, "v_heads": 32, "dim": 128},
        # up to three of eight nodes accepted, of two sequences: latency
        {"name": "accept_2x8", "op": "accept", "batch": 2, "nodes": 8, "path": 3, "kv_heads": 8, "k_heads": 16,
         "v_heads": 32, "dim": 128, "page": 64},
        # up to five of sixteen nodes, of a full serving batch
        {"name": "accept_64x16", "op": "accept", "batch": 64, "nodes": 16, "path": 5, "kv_heads": 8, "k_heads": 16,
         "v_heads": 32, "dim": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "prompt", "prompt", "step", "tree", "accept"])
    dim = rng.choice([64, 128, 128])
    if op == "attention":
        context, nodes, kv = _log(rng, 1, 65536), _log(rng, 1, 64), rng.choice([1, 2, 4, 8, 8])
        group = rng.choice([1, 4, 5, 7, 8])
        # at most the work of the largest listed case
        batch = _log(rng, 1, max(1, min(64, 16 * 32 * 64 * 8191 // (context * nodes * kv * group),
                                        16 * 8 * 8191 // (context * kv))))
        return {"op": op, "batch": batch, "nodes": nodes, "context": context, "q_heads": kv * group, "kv_heads": kv,
                "dim": dim, "page": 16 * rng.choice([1, 2, 3, 4, 8]),
                "window": _log(rng, 16, 4096) if rng.random() < 0.2 else 0, "ragged": rng.random() < 0.6}
    k_heads = rng.choice([1, 2, 4, 8, 16])
    v_heads = min(32, k_heads * rng.choice([1, 2, 2, 3, 4]))
    v_heads -= v_heads % k_heads
    case = {"op": op, "k_heads": k_heads, "v_heads": v_heads, "dim": dim}
    if op == "prompt":
        case.update(tokens=_log(rng, 1, 8192), ragged=rng.random() < 0.6)
        case["batch"] = _log(rng, 1, max(1, min(32, 16 * 2000 * 32 // (case["tokens"] * v_heads), 24000 // case["tokens"])))
    elif op == "step":
        case.update(batch=_log(rng, 1, 128), tokens=rng.choice([1, 1, 1, 1, 2, 3, 5]))
    elif op == "tree":
        case.update(batch=_log(rng, 1, 16), nodes=_log(rng, 1, 64))
        case["batch"] = min(case["batch"], max(1, 256 // case["nodes"]))
    else:
        case.update(batch=_log(rng, 1, 64), nodes=_log(rng, 2, 32), kv_heads=rng.choice([1, 2, 4, 8]),
                    page=16 * rng.choice([1, 2, 3, 4, 8]))
        case["path"] = rng.randint(1, min(8, case["nodes"]))
    return case


# ------------------------------------------------------------------ inputs --

def _lengths(case, most, empty):
    """Tokens of each sequence.  Ragged: spread evenly up to `most`, and of four or more sequences one has none if `empty`."""
    n = case["batch"]
    if not case.get("ragged", False):
        return [most] * n
    lens = [max(1, most * (1 + (i * 7919) % n) // n) for i in range(n)]
    lens[0] = most
    if n >= 4 and empty:
        lens[2] = 0
    return lens


def _tree(batch, nodes, gen, dev):
    """Parents [batch][nodes] on the host: every node at one before it, more often a late one; the last places of every
    third tree of at least three nodes are without a node."""
    pick = torch.rand((batch, nodes), generator=gen, device=dev).cpu()
    at = torch.arange(nodes)
    parents = torch.clamp((at + 1) * pick.sqrt() - 1e-3, min=0).floor().long() - 1      # -1 .. i - 1
    if nodes >= 3:
        parents[2::3, nodes - nodes // 3:] = -2
    return parents


def _path(parents, most, gen, dev):
    """For every tree up to `most` nodes from its beginning on, at least none: [batch][most], -1 behind the last."""
    batch, nodes = parents.shape
    pick = torch.rand((batch,), generator=gen, device=dev).cpu()
    path = torch.full((batch, most), -1, dtype=torch.int64)
    for b in range(batch):
        real = [i for i in range(nodes) if parents[b, i] >= -1]
        at, way = real[int(pick[b] * len(real))], []
        while at >= 0:
            way.append(at)
            at = int(parents[b, at])
        way = way[::-1][:most]
        path[b, :len(way)] = torch.tensor(way)
    return path


def _quantise(x):
    """(codes, step, lowest) of the last dimension in 4 bits; step and lowest as bf16 holds them."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    low, step = lo.to(torch.bfloat16).to(x.dtype), ((hi - lo) / 15).to(torch.bfloat16).to(x.dtype)
    codes = torch.where(step > 0, ((x - low) / step).round().clamp(0, 15), torch.zeros_like(x))
    return codes, step, low


def _group_v(c):
    """V codes [..., page * D/2] -> [..., page/16 g, D/64 c, 8 r, 4 j, 4 m, 4 b] (a view)."""
    return c.v.view(c.v.shape[0], c.v.shape[1], -1, c.dim // 64, 8, 4, 4, 4)


def _cache(pages, heads, page, dim, gen, dev):
    """A cache of normal keys (a few strong channels) and values (of a size that differs by token)."""
    c = types.SimpleNamespace(
        dim=dim, page=page,
        k=torch.empty((pages, heads, page, dim // 2), dtype=torch.uint8, device=dev),
        v=torch.empty((pages, heads, page, dim // 2), dtype=torch.uint8, device=dev),
        kp=torch.empty((pages, heads, page, 2), dtype=torch.bfloat16, device=dev),
        vp=torch.empty((pages, heads, page, 2), dtype=torch.bfloat16, device=dev))
    channel = 1 + 3 * (torch.rand(dim, generator=gen, device=dev) < 0.05).float()
    codes, step, low = _quantise(torch.randn((pages, heads, page, dim), generator=gen, device=dev) * channel)
    codes = codes.to(torch.uint8).unflatten(-1, (-1, 2))
    c.k.copy_(codes[..., 0] | (codes[..., 1] << 4))
    c.kp.copy_(torch.cat((step, low), -1))
    size = torch.exp(0.5 * torch.randn((pages, heads, page, 1), generator=gen, device=dev))
    codes, step, low = _quantise(torch.randn((pages, heads, page, dim), generator=gen, device=dev) * size)
    codes = codes.to(torch.uint8).unflatten(-1, (-1, 4, 2, 8))
    b = (codes[..., 0, :] | (codes[..., 1, :] << 4)).transpose(-1, -2)                  # [..., token, c, r, m]
    b = b.unflatten(2, (-1, 2, 4, 2))                                                  # [n, heads, g, t/8, j, t%2, c, r, m]
    _group_v(c).copy_(b.permute(0, 1, 2, 6, 7, 4, 8, 5, 3).flatten(-2))
    c.vp.copy_(torch.cat((step, low), -1))
    return c


def _table(lens, page, gen, dev):
    """Pages of every sequence in any order, -1 behind the last: int32 [batch][most pages]."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(max(1, sum(need)), generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=dev)
    table[torch.arange(table.shape[1], device=dev) < torch.tensor(need, device=dev)[:, None]] = order[:sum(need)]
    return table, max(1, sum(need))


def _delta_inputs(s, n, case, gen, dev):
    """q, k, v as slices of one buffer, what a short convolution with a smooth gate leaves; decays from heads that forget at
    once to heads that hardly do; update rates between 0 and 1."""
    hk, hv, dim = case["k_heads"], case["v_heads"], case["dim"]
    x = torch.randn((n, 2 * hk + hv, dim), generator=gen, device=dev)
    x = x * (1 + 3 * (torch.rand(dim, generator=gen, device=dev) < 0.05).float()) + 0.3
    x = (x * torch.sigmoid(x)).to(torch.bfloat16)
    s.q, s.k, s.v = x[:, :hk], x[:, hk:2 * hk], x[:, 2 * hk:]
    rate = torch.exp(torch.empty(hv, device=dev).uniform_(math.log(0.02), math.log(8.0), generator=gen))
    s.g = -rate * torch.nn.functional.softplus(torch.randn((n, hv), generator=gen, device=dev) - 2)
    s.beta = torch.sigmoid(torch.randn((n, hv), generator=gen, device=dev))


def _states(s, batch, case, gen, dev, padded):
    """States that earlier tokens left, in any order, and one that no sequence has; a padded place where there are four."""
    n = batch + 1
    s.state = 0.2 * torch.randn((n, case["v_heads"], case["dim"], case["dim"]), generator=gen, device=dev)
    s.slots = torch.randperm(n, generator=gen, device=dev)[:batch].to(torch.int32)
    if padded and batch >= 4:
        s.slots[1] = -1


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, batch = case["op"], case["batch"]
    s = types.SimpleNamespace(case=case, op=op)
    if op == "attention":
        nodes = case["nodes"]
        lens = [n + nodes if n else 0 for n in _lengths(case, case["context"], True)]  # the tree's own tokens are cached
        s.table, pages = _table(lens, case["page"], gen, dev)
        s.cache = _cache(pages, case["kv_heads"], case["page"], case["dim"], gen, dev)
        s.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        s.parents = _tree(batch, nodes, gen, dev).to(torch.int32).to(dev)
        s.q = torch.randn((batch, nodes, case["q_heads"], case["dim"]), generator=gen, device=dev).to(torch.bfloat16)
        return s
    if op == "prompt":
        s.host_lens = _lengths(case, case["tokens"], True)
        s.cu = torch.tensor([0] + s.host_lens, device=dev).cumsum(0).to(torch.int32)
        _delta_inputs(s, sum(s.host_lens), case, gen, dev)
        _states(s, batch, case, gen, dev, False)
        return s
    n = case["tokens"] if op == "step" else case["nodes"]
    _delta_inputs(s, batch * n, case, gen, dev)
    s.q, s.k, s.v, s.g, s.beta = (x.unflatten(0, (batch, n)) for x in (s.q, s.k, s.v, s.g, s.beta))
    _states(s, batch, case, gen, dev, True)
    if op == "step":
        return s
    parents = _tree(batch, n, gen, dev)
    s.parents = parents.to(torch.int32).to(dev)
    if op == "accept":
        path = _path(parents, case["path"], gen, dev)
        s.path = path.to(torch.int32).to(dev)
        page = case["page"]
        before = [37 + 11 * b for b in range(batch)]                                   # tokens before the tree
        table, pages = _table([x + n for x in before], page, gen, dev)
        s.cache = _cache(pages, case["kv_heads"], page, case["dim"], gen, dev)
        first = torch.tensor(before, device=dev)[:, None]
        path = path.to(dev)

        def slots(at):
            return table.gather(1, at // page).long() * page + at % page
        s.src = torch.where(path >= 0, slots(first + path.clamp(min=0)), -1)
        s.dst = torch.where(path >= 0, slots(first + torch.arange(case["path"], device=dev)), -1)
    return s


# ------------------------------------------------------------- plain forms --

def _ancestors(parents):
    """[batch][n][n]: node j is node i or one of those that it comes from; nothing for a place without a node."""
    n = parents.shape[1]
    at = torch.arange(n, device=parents.device)
    reach = ((parents[..., None] == at) | (at[:, None] == at)) & (parents[..., None] >= -1)
    for _ in range((n - 1).bit_length()):
        reach = (reach.float() @ reach.float()) > 0
    return reach


def _unpack(cache, table):
    """Keys and values [B, heads, tokens, D] in 32 bits of the pages in `table`."""
    at = table.clamp(min=0).long()
    x, p = cache.k[at], cache.kp[at].float()
    k = p[..., 1:] + p[..., :1] * torch.stack((x & 15, x >> 4), -1).flatten(-2).float()
    x, p = _group_v(cache)[at].unflatten(-1, (2, 2)), cache.vp[at].float()   # [B, P, heads, g, c, r, j, m, t%2, t/8]
    x = torch.stack((x & 15, x >> 4), -1).permute(0, 1, 2, 3, 9, 6, 8, 4, 7, 10, 5)
    v = p[..., 1:] + p[..., :1] * x.flatten(-4).flatten(3, 6).float()
    return k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    case = s.case
    batch, n, heads, dim = s.q.shape
    kv = case["kv_heads"]
    k, v = _unpack(s.cache, s.table)
    first = s.lens.long()[:, None] - n                                             # the tree's first token
    above = _ancestors(s.parents)
    depth = above.sum(-1) - 1
    key = torch.arange(k.shape[2], device=k.device)
    node = key - first                                                             # [B, keys]
    real = (s.parents >= -1) & (s.lens > 0)[:, None]
    seen = (node < 0)[:, None]
    inside = above.gather(2, node.clamp(0, n - 1)[:, None].expand(batch, n, -1))
    if case["window"]:
        seen = seen & (node[:, None] > depth[..., None] - case["window"])
        near = depth[..., None] - depth[:, None] < case["window"]
        inside = inside & near.gather(2, node.clamp(0, n - 1)[:, None].expand(batch, n, -1))
    seen = (seen | (inside & ((node >= 0) & (node < n))[:, None])) & real[..., None]
    q = s.q.float().unflatten(2, (kv, heads // kv)).permute(0, 2, 1, 3, 4).flatten(2, 3)     # [B, kv, n*G, D]
    scores = q @ k.transpose(-1, -2) / math.sqrt(dim)
    seen = seen.repeat_interleave(heads // kv, 1)[:, None]
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    o = p @ v / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + total.log()
    o, lse = (x.unflatten(2, (n, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3) for x in (o, lse))
    return {"o": o.to(torch.bfloat16), "lse": lse[..., 0].contiguous()}


def _unit(x):
    x = x.float()
    return x / (x.square().sum(-1, keepdim=True) + EPS).sqrt()


def _inverse(a):
    """(1 + a)^-1 of strictly lower a [..., n, n], n a power of two: of blocks of one, two, four ... rows."""
    n = a.shape[-1]
    x = torch.ones_like(a[..., :1]).unsqueeze(-1)                                  # [..., blocks, size, size]
    size = 1
    while size < n:
        lower = a.unflatten(-2, (-1, 2, size)).unflatten(-1, (-1, 2, size))        # [..., b, 2, size, b, 2, size]
        lower = lower.diagonal(dim1=-6, dim2=-3)[..., 1, :, 0, :, :].movedim(-1, -3)
        first, second = x.unflatten(-3, (-1, 2)).unbind(-3)
        low = -(second @ lower @ first)
        x = torch.cat((torch.cat((first, torch.zeros_like(first)), -1), torch.cat((low, second), -1)), -2)
        size *= 2
    return x[..., 0, :, :]


class _Blocks:
    """Blocks of tokens [..., C, D] (C a power of two) in which token i comes after those that `above` [..., C, C] names,
    itself among them: all that does not need the state before them."""

    def __init__(self, q, k, v, g, beta, above):
        self.q, self.k, self.v, self.beta = q, k, v, beta[..., None]
        total = (above.double() @ g.double()[..., None])[..., 0]                   # of the decays up to a token
        fade = torch.where(above, (total[..., :, None] - total[..., None, :]).exp().float(), 0.0)
        self.decay = total.exp().float()[..., None]
        self.left = (total[..., -1:] - total).exp().float()[..., None]             # (for a chain: until its end)
        strict = fade * (1 - torch.eye(fade.shape[-1], device=fade.device))
        self.solve = _inverse(self.beta * strict * (k @ k.mT))
        self.weigh = None if q is None else fade * (q @ k.mT)

    def at(self, i):
        b = object.__new__(_Blocks)
        for name, x in vars(self).items():
            setattr(b, name, None if x is None else x[:, :, i])
        return b

    def updates(self, state):
        return self.solve @ (self.beta * (self.v - self.decay * (self.k @ state.mT)))

    def outputs(self, state, u):
        return (self.decay * (self.q @ state.mT) + self.weigh @ u) / math.sqrt(self.q.shape[-1])

    def end(self, state, u):
        return self.decay[..., -1:, :] * state + (self.left * u).mT @ self.k


def _heads_first(x, case):
    """[B, n, heads, D] -> [B, value heads, n, D]"""
    x = x.transpose(1, 2)
    return x.repeat_interleave(case["v_heads"] // x.shape[1], 1)


def _padded(x, n):
    """More tokens (dimension 1) of zeros, to n: zeros change no state."""
    return torch.cat((x, x.new_zeros((x.shape[0], n - x.shape[1], *x.shape[2:]))), 1) if n > x.shape[1] else x


def _power_of_two(n):
    return 1 << (n - 1).bit_length()


def _plain_chain(s, q, k, v, g, beta, slots, outputs=True):
    """The rule over [B][n] tokens in blocks, with the states of `slots` (a padded one: outputs of zero)."""
    case, n = s.case, k.shape[1]
    size = min(CHUNK, _power_of_two(n))
    most = -(-n // size) * size
    q, k = (None if x is None else _heads_first(_padded(_unit(x), most), case).unflatten(2, (-1, size)) for x in (q, k))
    v = _padded(v.float(), most).transpose(1, 2).unflatten(2, (-1, size))
    g, beta = (_padded(x, most).transpose(1, 2).unflatten(2, (-1, size)) for x in (g, beta))
    above = torch.ones((size, size), dtype=torch.bool, device=k.device).tril()
    blocks = _Blocks(q, k, v, g, beta, above)
    kept = (slots >= 0)
    state = s.state[slots.clamp(min=0).long()]
    out = []
    for i in range(most // size):
        b = blocks.at(i)
        u = b.updates(state)
        if outputs:
            out.append(b.outputs(state, u))
        state = b.end(state, u)
    s.state[slots[kept].long()] = state[kept]
    if outputs:
        return torch.where(kept[:, None, None, None], torch.cat(out, 2)[:, :, :n].transpose(1, 2), 0.0).to(torch.bfloat16)


def _plain_prompt(s):
    lens, most = s.host_lens, max(s.host_lens)
    start = s.cu[:-1].long()[:, None]
    at = torch.arange(most, device=s.k.device)
    inside = at < (s.cu[1:] - s.cu[:-1])[:, None]
    index = torch.where(inside, start + at, 0)
    q, k, v = (torch.where(inside[..., None, None], x[index], 0) for x in (s.q, s.k, s.v))
    g, beta = (torch.where(inside[..., None], x[index], 0) for x in (s.g, s.beta))
    o = _plain_chain(s, q, k, v, g, beta, s.slots)
    return {"o": o[inside], "state": s.state}


def _plain_tree(s):
    case, n = s.case, s.case["nodes"]
    size = _power_of_two(n)
    above = torch.zeros((case["batch"], 1, size, size), dtype=torch.bool, device=s.k.device)
    above[:, 0, :n, :n] = _ancestors(s.parents)
    q, k = (_heads_first(_padded(_unit(x), size), case) for x in (s.q, s.k))
    v, g, beta = (_padded(x.float(), size).transpose(1, 2) for x in (s.v, s.g, s.beta))
    b = _Blocks(q, k, v, g, beta, above)
    state = s.state[s.slots.clamp(min=0).long()]
    o = b.outputs(state, b.updates(state))[:, :, :n].transpose(1, 2)
    real = ((s.parents >= -1) & (s.slots >= 0)[:, None])[..., None, None]
    return {"o": torch.where(real, o, 0.0).to(torch.bfloat16)}


def _plain_accept(s):
    c = s.cache
    kept = s.src >= 0
    src, dst = s.src[kept], s.dst[kept]

    def place(slots):
        page, off = slots // c.page, slots % c.page
        g, t = off // 16, off % 16
        return page, off, g, (t % 8) // 2, 2 * (t % 2) + t // 8
    page, off, g, j, b = place(src)
    k, kp, vp, v = c.k[page, :, off], c.kp[page, :, off], c.vp[page, :, off], _group_v(c)[page, :, g, :, :, j, :, b]
    page, off, g, j, b = place(dst)
    c.k[page, :, off], c.kp[page, :, off], c.vp[page, :, off] = k, kp, vp
    _group_v(c)[page, :, g, :, :, j, :, b] = v
    # what the first places after each sequence hold now
    page, off, g, j, b = place(s.dst.clamp(min=0).flatten())
    x, p = c.k[page, :, off], c.kp[page, :, off].float()
    k = p[..., 1:] + p[..., :1] * torch.stack((x & 15, x >> 4), -1).flatten(-2).float()
    x, p = _group_v(c)[page, :, g, :, :, j, :, b].transpose(-1, -2), c.vp[page, :, off].float()
    v = p[..., 1:] + p[..., :1] * torch.stack((x & 15, x >> 4), -2).flatten(-4).float()
    k, v = (torch.where(kept.flatten()[:, None, None], x, 0.0).to(torch.bfloat16) for x in (k, v))
    way = s.path.clamp(min=0).long()
    real = s.path >= 0
    at = torch.arange(way.shape[0], device=way.device)[:, None]
    key, value = (torch.where(real[..., None, None], x[at, way], 0) for x in (s.k, s.v))
    fade, beta = (torch.where(real[..., None], x[at, way], 0) for x in (s.g, s.beta))
    _plain_chain(s, None, key, value, fade, beta, s.slots, outputs=False)
    return {"k": k, "v": v, "state": s.state}


def _plain(s):
    if s.op == "attention":
        return _plain_attention(s)
    if s.op == "prompt":
        return _plain_prompt(s)
    if s.op == "step":
        return {"o": _plain_chain(s, s.q, s.k, s.v, s.g, s.beta, s.slots), "state": s.state}
    return _plain_tree(s) if s.op == "tree" else _plain_accept(s)


# ------------------------------------------------------------------- calls --

def _library(s):
    import block_scaled_fp8_x128_gb300 as r9q
    if s.op == "attention":
        o, lse = r9q.r9q_kv4_tree_attention(s.q, r9q.KV4Cache(s.cache.k, s.cache.kp, s.cache.v, s.cache.vp), s.table,
                                            s.lens, s.parents, window=s.case["window"], return_lse=True)
        return {"o": o, "lse": lse}
    if s.op == "prompt":
        return {"o": r9q.r9q_gated_delta(s.q, s.k, s.v, s.g, s.beta, s.state, s.slots, s.cu, eps=EPS), "state": s.state}
    if s.op == "step":
        return {"o": r9q.r9q_gated_delta_step(s.q, s.k, s.v, s.g, s.beta, s.state, s.slots, eps=EPS), "state": s.state}
    if s.op == "tree":
        return {"o": r9q.r9q_gated_delta_tree(s.q, s.k, s.v, s.g, s.beta, s.state, s.slots, s.parents, eps=EPS)}
    cache = r9q.KV4Cache(s.cache.k, s.cache.kp, s.cache.v, s.cache.vp)
    r9q.r9q_kv4_move(cache, s.src, s.dst)
    r9q.r9q_gated_delta_commit(s.k, s.v, s.g, s.beta, s.state, s.slots, s.path, eps=EPS)
    k, v = r9q.r9q_kv4_gather(cache, s.dst.view(-1))
    return {"k": k, "v": v, "state": s.state}


def run(s):
    return _library(s) if own else _plain(s)


# -------------------------------------------------------------------- work --

def work(case):
    dim = case["dim"]
    token4 = 2 * (dim // 2 + 4)                                  # a token's key and value, one head, in the cache
    if case["op"] == "attention":
        n, heads, kv, w = case["nodes"], case["q_heads"], case["kv_heads"], case["window"]
        # a tree's depth is not known here: the keys before it that its first node sees, and its nodes
        seen = sum((min(x, w) if w else x) + n for x in _lengths(case, case["context"], True) if x)
        pairs = sum((min(x, w) if w else x) + (n + 1) // 2 for x in _lengths(case, case["context"], True) if x)
        rows = case["batch"] * n * heads
        return {"bytes": kv * seen * token4 + rows * (4 * dim + 4), "flops": 4 * n * heads * dim * pairs}
    hk, hv, batch = case["k_heads"], case["v_heads"], case["batch"]
    state = batch * hv * dim * dim * 4
    if case["op"] == "prompt":
        n = sum(_lengths(case, case["tokens"], True))
    else:
        n = batch * {"step": case.get("tokens"), "tree": case.get("nodes"), "accept": case.get("path")}[case["op"]]
    token = 2 * (2 * hk + hv) * dim + 8 * hv
    if case["op"] == "accept":
        return {"bytes": n * (token - 2 * hk * dim) + 2 * state + n * case["kv_heads"] * (3 * token4 + 4 * dim),
                "flops": 4 * n * hv * dim * dim}
    states = 1 if case["op"] == "tree" else 2
    return {"bytes": n * (token + 2 * hv * dim) + states * state, "flops": (4 if case["op"] == "tree" else 6) * n * hv * dim * dim}


# ------------------------------------------------------------------- exact --

def _way(parents, i):
    """The nodes from the tree's beginning to node i; none where there is no node."""
    way = []
    while i >= 0 and parents[i] >= -1:
        way.append(i)
        i = parents[i]
    return way[::-1]


def _exact_codes(c, slots):
    """Keys and values [tokens][heads][D] in 64 bits that the cache holds at `slots`."""
    page, off = slots // c.page, slots % c.page
    heads, dim = c.k.shape[1], c.dim
    d = torch.arange(dim, device=slots.device)
    k = (c.k[page, :, off].long()[..., d // 2] >> (4 * (d % 2))) & 15
    t = off % 16
    at = (off // 16 * 8 * dim)[:, None] + (d // 64 * 512 + d % 8 * 64 + d % 64 // 16 * 4) + (
        t % 8 // 2 * 16 + 2 * (t % 2) + t // 8)[:, None]
    b = c.v.flatten(2)[page[:, None, None], torch.arange(heads, device=at.device)[:, None], at[:, None]].long()
    v = (b >> (4 * (d % 16 // 8))) & 15
    kp, vp = c.kp[page, :, off].double(), c.vp[page, :, off].double()
    return kp[..., 1:] + kp[..., :1] * k, vp[..., 1:] + vp[..., :1] * v


def _exact_attention(s):
    case = s.case
    batch, n, heads, dim = s.q.shape
    kv, dev = case["kv_heads"], s.q.device
    o = torch.zeros((batch, n, heads, dim), dtype=torch.float64, device=dev)
    lse = torch.full((batch, n, heads), -math.inf, dtype=torch.float64, device=dev)
    for b, (length, parents) in enumerate(zip(s.lens.tolist(), s.parents.tolist())):
        if length == 0:
            continue
        token = torch.arange(length, device=dev)
        k, v = _exact_codes(s.cache, s.table[b].long()[token // s.cache.page] * s.cache.page + token % s.cache.page)
        for i in range(n):
            way = _way(parents, i)
            if not way:
                continue
            at = list(range(length - n)) + [length - n + x for x in way]
            if case["window"]:
                at = at[-case["window"]:]
            tail = torch.tensor(at[len(at) - min(len(at), len(way)):], device=dev)
            head = len(at) - len(tail)                            # keys before the tree: one run of them
            first = at[0] if head else 0
            kk, vv = (torch.cat((x[first:first + head], x[tail])) for x in (k, v))
            x = torch.einsum("hgd,thd->hgt", s.q[b, i].double().view(kv, heads // kv, dim), kk) / math.sqrt(dim)
            lse[b, i] = torch.logsumexp(x, -1).flatten()
            o[b, i] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), vv).flatten(0, 1)
    return {"o": o, "lse": lse}


def _token(state, q, k, v, g, beta):
    """One token: states [..., Hv, D, D] with the heads' q, k [..., Hk, D], v [..., Hv, D], g, beta [..., Hv]."""
    ratio = v.shape[-2] // k.shape[-2]
    k = k.double().repeat_interleave(ratio, -2)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS)
    state = torch.exp(g.double())[..., None, None] * state
    error = v.double() - torch.einsum("...vk,...k->...v", state, k)
    state = state + torch.einsum("...v,...k->...vk", beta.double()[..., None] * error, k)
    if q is None:
        return state, None
    q = q.double().repeat_interleave(ratio, -2)
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS)
    return state, torch.einsum("...vk,...k->...v", state, q) / math.sqrt(q.shape[-1])


def exact(case, seed):
    s = prepare(case, seed)
    if s.op == "attention":
        return _exact_attention(s)
    all_states = s.state.double()
    slots = s.slots.tolist()
    if s.op == "prompt":
        lens = s.host_lens
        states = all_states[s.slots.long()]
        o = torch.zeros(s.v.shape, dtype=torch.float64, device=s.v.device)
        order = sorted(range(len(lens)), key=lambda b: -lens[b])
        start = s.cu.long()[torch.tensor(order, device=o.device)]
        for t in range(max(lens)):
            live = sum(n > t for n in lens)
            who, at = torch.tensor(order[:live], device=o.device), start[:live] + t
            states[who], o[at] = _token(states[who], s.q[at], s.k[at], s.v[at], s.g[at], s.beta[at])
        all_states[s.slots.long()] = states
        return {"o": o, "state": all_states}
    o = torch.zeros(s.v.shape, dtype=torch.float64, device=s.v.device)
    for b, slot in enumerate(slots):
        if slot < 0:
            continue
        if s.op == "step":
            for t in range(case["tokens"]):
                all_states[slot], o[b, t] = _token(all_states[slot], s.q[b, t], s.k[b, t], s.v[b, t], s.g[b, t], s.beta[b, t])
        elif s.op == "accept":
            for i in s.path[b].tolist():
                if i >= 0:
                    all_states[slot], _ = _token(all_states[slot], None, s.k[b, i], s.v[b, i], s.g[b, i], s.beta[b, i])
        else:
            parents, after = s.parents[b].tolist(), {-1: all_states[slot]}
            for i, parent in enumerate(parents):
                if parent >= -1:
                    after[i], o[b, i] = _token(after[parent], s.q[b, i], s.k[b, i], s.v[b, i], s.g[b, i], s.beta[b, i])
    if s.op == "accept":
        k, v = _exact_codes(s.cache, s.src.clamp(min=0).flatten())  # what the accepted nodes' own places hold
        kept = (s.src >= 0).flatten()[:, None, None]
        return {"k": torch.where(kept, k, 0.0), "v": torch.where(kept, v, 0.0), "state": all_states}
    return {"o": o} if s.op == "tree" else {"o": o, "state": all_states}
