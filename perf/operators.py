"""The attention operators of a decode layer, as cases to be timed and compared.

Between the QKV GEMM and the output GEMM a decoder layer normalises and rotates
its queries and keys, writes the new keys and values to a cache held in 4 bits
and attends over that cache.  Four operators:

  rope       r9q_qk_norm_rope: RMS norm of every query and key head and the
             position rotation, in one pass;
  rope_grad  r9q_qk_norm_rope_bwd: its gradient (inputs and both norm weights);
  write      r9q_qk_norm_rope_kv4: the same pass with the keys and values written
             to the paged 4-bit cache, and r9q_kv4_gather, which reads them back;
  attention  r9q_kv4_attention: attention over the paged 4-bit cache, one new
             token or a few for every sequence.

The cache, per page and key-value head: K codes [page][D/2], byte i of a token
holding elements 2i (low nibble) and 2i+1; V codes in groups of 16 tokens,
[page/16][D/64][8 r][4 j][4 m][4 b], where token t of the group has j = (t%8)/2,
b = 2*(t%2) + t/8 and element d = 16*(4*c + m) + 8*nibble + r; and one bf16 pair
(step, lowest value) for each token, K and V.  A code c stands for lowest + step*c.

`own` selects the library's calls; otherwise `run` computes the plain forms.
"""
import math
import types

import torch

own = False

EPS = 1e-6
THETA = 10000.0


def listed():
    return [
        # one decode step of eight sequences: the 12288-wide QKV GEMM's output (32 + 2*32 heads of 128); latency
        {"name": "rope_decode_8", "op": "rope", "tokens": 8, "q_heads": 32, "kv_heads": 32, "dim": 128, "rot": 128,
         "interleaved": False},
        # one 8192-token prefill chunk of the same layer; bandwidth
        {"name": "rope_prefill_8192", "op": "rope", "tokens": 8192, "q_heads": 32, "kv_heads": 32, "dim": 128,
         "rot": 128, "interleaved": False},
        # a training micro-batch of odd length, small heads, half of each rotated in adjacent pairs
        {"name": "rope_grad_777", "op": "rope_grad", "tokens": 777, "q_heads": 14, "kv_heads": 2, "dim": 64, "rot": 32,
         "interleaved": True},
        # a training batch of 4096 tokens with grouped heads
        {"name": "rope_grad_4096", "op": "rope_grad", "tokens": 4096, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False},
        # a decode step of sixteen sequences (one of them padding) writing its new tokens to their pages
        {"name": "write_decode_16", "op": "write", "tokens": 16, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "page": 64, "scattered": True},
        # a prefill chunk written to consecutive places
        {"name": "write_prefill_8192", "op": "write", "tokens": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "page": 64, "scattered": False},
        # one sequence just begun, as many key-value heads as query heads: latency
        {"name": "attention_1x77", "op": "attention", "batch": 1, "q_len": 1, "context": 77, "q_heads": 32,
         "kv_heads": 32, "dim": 128, "page": 16, "window": 0, "ragged": False},
        # a small serving batch of mixed lengths, an empty slot among them
        {"name": "attention_8x4096", "op": "attention", "batch": 8, "q_len": 1, "context": 4096, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "ragged": True},
        # one long document
        {"name": "attention_1x131072", "op": "attention", "batch": 1, "q_len": 1, "context": 131072, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 128, "window": 0, "ragged": False},
        # the largest: a full serving batch
        {"name": "attention_64x16384", "op": "attention", "batch": 64, "q_len": 1, "context": 16384, "q_heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "ragged": True},
        # four drafted tokens of sixteen sequences verified at once: 32 query rows for each key-value head
        {"name": "attention_16x4_8191", "op": "attention", "batch": 16, "q_len": 4, "context": 8191, "q_heads": 64,
         "kv_heads": 8, "dim": 128, "page": 32, "window": 0, "ragged": False},
        # a sliding window over a longer cache, small heads, seven query heads to a key-value head
        {"name": "attention_32_window", "op": "attention", "batch": 32, "q_len": 1, "context": 5000, "q_heads": 14,
         "kv_heads": 2, "dim": 64, "page": 16, "window": 1024, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "write", "attention", "attention"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 8])
    if op != "attention":
        heads = kv * rng.choice([1, 4, 5, 7, 8])
        case = {"op": op, "tokens": _log(rng, 1, min(8192, 8192 * 64 // (heads + kv))), "q_heads": heads,
                "kv_heads": kv, "dim": dim, "rot": rng.choice([dim, dim, dim // 2]),
                "interleaved": rng.random() < 0.3}
        if op == "write":
            case.update(page=16 * rng.choice([1, 2, 3, 4, 8]), scattered=rng.random() < 0.5)
        return case
    context = _log(rng, 1, 131072)
    q_len = rng.choice([1, 1, 1, 2, 3, 5])
    # at most the work of the largest listed case, whose lengths come to about half of 64 * 16384
    batch = _log(rng, 1, max(1, min(256, 32 * 16384 * 8 // (context * kv * q_len))))
    return {"op": op, "batch": batch, "q_len": q_len, "context": context,
            "q_heads": kv * rng.choice([1, 4, 5, 7, 8]), "kv_heads": kv, "dim": dim,
            "page": 16 * rng.choice([1, 2, 3, 4, 8]), "window": _log(rng, 16, 4096) if rng.random() < 0.25 else 0,
            "ragged": rng.random() < 0.6}


# ------------------------------------------------------------------ inputs --

def _lengths(case):
    """Tokens of each sequence.  Ragged: spread evenly up to the context, and of four or more sequences one has none."""
    n, top = case["batch"], case["context"]
    if not case["ragged"]:
        return [top] * n
    lens = [max(1, top * (1 + (i * 7919) % n) // n) for i in range(n)]
    lens[0] = top
    if n >= 4:
        lens[2] = 0
    return lens


def _visible(case):
    """Keys that at least one new token of each sequence sees."""
    n, w = case["q_len"], case["window"]
    return [min(length, w + min(n, length) - 1) if w else length for length in _lengths(case)]


def _quantise(x):
    """(codes, step, lowest) of the last dimension in 4 bits; step and lowest as bf16 holds them."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    low, step = lo.to(torch.bfloat16).to(x.dtype), ((hi - lo) / 15).to(torch.bfloat16).to(x.dtype)
    codes = torch.where(step > 0, ((x - low) / step).round().clamp(0, 15), torch.zeros_like(x))
    return codes, step, low


def _pack_k(codes):
    """[..., D] codes -> [..., D/2] bytes."""
    c = codes.to(torch.uint8).unflatten(-1, (-1, 2))
    return c[..., 0] | (c[..., 1] << 4)


def _pack_v(codes):
    """[..., D] codes of one token -> its bytes [..., D/64 c, 8 r, 4 m]."""
    c = codes.to(torch.uint8).unflatten(-1, (-1, 4, 2, 8))
    return (c[..., 0, :] | (c[..., 1, :] << 4)).transpose(-1, -2)


def _pack_params(step, low):
    return torch.cat((step, low), -1).to(torch.bfloat16)


def _group_v(v):
    """V codes [..., page * D/2] -> [..., page/16 g, D/64 c, 8 r, 4 j, 4 m, 4 b] (a view)."""
    return v.v.view(v.v.shape[0], v.v.shape[1], -1, v.dim // 64, 8, 4, 4, 4)


def _cache(pages, heads, page, dim, device):
    return types.SimpleNamespace(
        dim=dim, page=page,
        k=torch.zeros((pages, heads, page, dim // 2), dtype=torch.uint8, device=device),
        v=torch.zeros((pages, heads, page, dim // 2), dtype=torch.uint8, device=device),
        kp=torch.zeros((pages, heads, page, 2), dtype=torch.bfloat16, device=device),
        vp=torch.zeros((pages, heads, page, 2), dtype=torch.bfloat16, device=device))


def _fill(cache, gen):
    """Every token of the cache from normal keys (a few strong channels) and values (of a size that differs by token)."""
    n, heads, page, _ = cache.k.shape
    dev = cache.k.device
    channel = 1 + 3 * (torch.rand(cache.dim, generator=gen, device=dev) < 0.05).float()
    codes, step, low = _quantise(torch.randn((n, heads, page, cache.dim), generator=gen, device=dev) * channel)
    cache.k.copy_(_pack_k(codes))
    cache.kp.copy_(_pack_params(step, low))
    size = torch.exp(0.5 * torch.randn((n, heads, page, 1), generator=gen, device=dev))
    codes, step, low = _quantise(torch.randn((n, heads, page, cache.dim), generator=gen, device=dev) * size)
    b = _pack_v(codes).unflatten(2, (-1, 2, 4, 2))              # [n, heads, g, t/8, j, t%2, c, r, m]
    _group_v(cache).copy_(b.permute(0, 1, 2, 6, 7, 4, 8, 5, 3).flatten(-2))
    cache.vp.copy_(_pack_params(step, low))


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = types.SimpleNamespace(case=case, op=case["op"], workspace=None)
    heads, kv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "attention":
        lens, page = _lengths(case), case["page"]
        need = [-(-n // page) for n in lens]
        s.cache = _cache(max(1, sum(need)), kv, page, dim, dev)
        _fill(s.cache, gen)
        order = torch.randperm(sum(need), generator=gen, device=dev).to(torch.int32)
        s.table = torch.full((case["batch"], max(1, max(need))), -1, dtype=torch.int32, device=dev)
        s.table[torch.arange(s.table.shape[1], device=dev) < torch.tensor(need, device=dev)[:, None]] = order
        s.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        s.q = torch.randn((case["batch"], case["q_len"], heads, dim), generator=gen, device=dev).to(torch.bfloat16)
        return s
    n, rot = case["tokens"], case["rot"]
    qkv = torch.randn((n, heads + 2 * kv, dim), generator=gen, device=dev)
    qkv = (qkv * (1 + 3 * (torch.rand(dim, generator=gen, device=dev) < 0.05).float())).to(torch.bfloat16)
    s.q, s.k, s.v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]      # slices of one GEMM's output
    s.wq = 1 + 0.2 * torch.randn(dim, generator=gen, device=dev)
    s.wk = 1 + 0.2 * torch.randn(dim, generator=gen, device=dev)
    first = 5 + seed % 1000
    angle = torch.arange(first + n, dtype=torch.float64, device=dev)[:, None] * THETA ** (
        -torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    s.cos, s.sin = angle.cos().float(), angle.sin().float()
    s.pos = torch.arange(first, first + n, device=dev)
    if case["op"] == "rope_grad":
        s.dq = torch.randn((n, heads, dim), generator=gen, device=dev).to(torch.bfloat16)
        s.dk = torch.randn((n, kv, dim), generator=gen, device=dev).to(torch.bfloat16)
    if case["op"] == "write":
        page = case["page"]
        # scattered: every token in a page of its own; else page after page, in any order of the pages
        pages = n if case["scattered"] else -(-n // page)
        s.cache = _cache(pages + 1, kv, page, dim, dev)          # one page that no token is given
        order = torch.randperm(pages, generator=gen, device=dev)
        if case["scattered"]:
            s.slots = order * page + torch.randint(0, page, (n,), generator=gen, device=dev)
            if n >= 4:
                s.slots[1] = -1                                  # a padded place of the batch
        else:
            at = torch.arange(n, device=dev)
            s.slots = order[at // page] * page + at % page
    return s


# ------------------------------------------------------------- plain forms --

def _rotate(x, cos, sin, interleaved, back=False):
    """Rotation of the first 2*cos.shape[-1] elements of each head; `back`: by the opposite angle."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], -sin[:, None] if back else sin[:, None]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, rest), -1)


def _norm(x):
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r, r


def _norm_rope(s):
    cos, sin, inter = s.cos[s.pos], s.sin[s.pos], s.case["interleaved"]
    return _rotate(_norm(s.q)[0] * s.wq, cos, sin, inter), _rotate(_norm(s.k)[0] * s.wk, cos, sin, inter)


def _norm_rope_grad(x, dy, w, s):
    g = _rotate(dy.float(), s.cos[s.pos], s.sin[s.pos], s.case["interleaved"], back=True)
    xn, r = _norm(x)
    dx = r * (g * w - xn * (g * w * xn).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (g * xn).sum((0, 1))


def _plain_write(s):
    q, k = _norm_rope(s)
    kept = (s.slots >= 0)[:, None, None]
    c = s.cache
    slots = torch.where(s.slots >= 0, s.slots, c.k.shape[0] * c.page - 1)        # padding goes to the spare page
    page, off = slots // c.page, slots % c.page
    g, t = off // 16, off % 16
    j, b = (t % 8) // 2, 2 * (t % 2) + t // 8
    codes, step, low = _quantise(k)
    c.k[page, :, off] = _pack_k(codes)
    c.kp[page, :, off] = _pack_params(step, low)
    codes, step, low = _quantise(s.v.float())
    _group_v(c)[page, :, g, :, :, j, :, b] = _pack_v(codes)
    c.vp[page, :, off] = _pack_params(step, low)
    # and back
    x, p = c.k[page, :, off], c.kp[page, :, off].float()
    kc = torch.stack((x & 15, x >> 4), -1).flatten(-2)
    x, r = _group_v(c)[page, :, g, :, :, j, :, b].transpose(-1, -2), c.vp[page, :, off].float()
    vc = torch.stack((x & 15, x >> 4), -2).flatten(-4)
    k, v = (torch.where(kept, p[..., 1:] + p[..., :1] * codes.float(), torch.zeros_like(k))
            for codes, p in ((kc, p), (vc, r)))
    return {"q": q.to(torch.bfloat16), "k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


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
    q = s.q.float().unflatten(2, (kv, heads // kv)).permute(0, 2, 1, 3, 4).flatten(2, 3)     # [B, kv, n*G, D]
    scores = q @ k.transpose(-1, -2) / math.sqrt(dim)
    last = s.lens.long()[:, None] - n + torch.arange(n, device=q.device)                     # a new token's own place
    key = torch.arange(k.shape[2], device=q.device)
    seen = key <= last[..., None]
    if case["window"]:
        seen = seen & (key > last[..., None] - case["window"])
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


def _plain(s):
    if s.op == "rope":
        q, k = _norm_rope(s)
        return {"q": q.to(torch.bfloat16), "k": k.to(torch.bfloat16)}
    if s.op == "rope_grad":
        dq, dwq = _norm_rope_grad(s.q, s.dq, s.wq, s)
        dk, dwk = _norm_rope_grad(s.k, s.dk, s.wk, s)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    return _plain_write(s) if s.op == "write" else _plain_attention(s)


# ------------------------------------------------------------------- calls --

def _library(s):
    import block_scaled_fp8_x128_gb300 as r9q
    if s.op == "attention":
        o, lse = r9q.r9q_kv4_attention(s.q, r9q.KV4Cache(s.cache.k, s.cache.kp, s.cache.v, s.cache.vp), s.table,
                                       s.lens, window=s.case["window"], return_lse=True)
        return {"o": o, "lse": lse}
    inter = s.case["interleaved"]
    if s.op == "rope":
        q, k = r9q.r9q_qk_norm_rope(s.q, s.k, s.wq, s.wk, s.cos, s.sin, s.pos, eps=EPS, interleaved=inter)
        return {"q": q, "k": k}
    if s.op == "rope_grad":
        dq, dk, dwq, dwk = r9q.r9q_qk_norm_rope_bwd(s.dq, s.dk, s.q, s.k, s.wq, s.wk, s.cos, s.sin, s.pos, eps=EPS,
                                                    interleaved=inter)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    cache = r9q.KV4Cache(s.cache.k, s.cache.kp, s.cache.v, s.cache.vp)
    q = r9q.r9q_qk_norm_rope_kv4(s.q, s.k, s.v, s.wq, s.wk, s.cos, s.sin, s.pos, cache, s.slots, eps=EPS,
                                 interleaved=inter)
    k, v = r9q.r9q_kv4_gather(cache, s.slots)
    return {"q": q, "k": k, "v": v}


def run(s):
    return _library(s) if own else _plain(s)


# -------------------------------------------------------------------- work --

def work(case):
    heads, kv, dim = case["q_heads"], case["kv_heads"], case["dim"]
    token4 = 2 * (dim // 2 + 4)                                  # a token's key and value, one head, in the cache
    if case["op"] == "attention":
        rows, seen = case["batch"] * case["q_len"] * heads, sum(_visible(case))
        return {"bytes": kv * seen * token4 + rows * (4 * dim + 4), "flops": 4 * case["q_len"] * heads * dim * seen}
    n, vec = case["tokens"], 2 * dim
    table = n * (8 + 4 * case["rot"])
    if case["op"] == "rope":
        return {"bytes": 2 * n * (heads + kv) * vec + table, "flops": 8 * n * (heads + kv) * dim}
    if case["op"] == "rope_grad":
        return {"bytes": 3 * n * (heads + kv) * vec + table + 16 * dim, "flops": 16 * n * (heads + kv) * dim}
    return {"bytes": 2 * n * heads * vec + 2 * n * kv * vec + table + 2 * n * kv * token4 + 8 * n + 2 * n * kv * vec,
            "flops": 8 * n * (heads + kv) * dim + 8 * n * kv * dim}


# ------------------------------------------------------------------- exact --

def _exact_norm_rope(x, w, cos, sin, interleaved):
    """Norm and rotation in 64 bits, as a product of each pair with a complex number of absolute value one."""
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    half = cos.shape[-1]
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(cos.double(), sin.double())[:, None]
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_four_bits(x):
    """What 4 bits hold of the last dimension, in 64 bits."""
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    low = lo.float().to(torch.bfloat16).double()
    step = ((hi - lo) / 15).float().to(torch.bfloat16).double()
    return low + step * torch.clamp(torch.round((x - low) / torch.where(step > 0, step, torch.ones_like(step))), 0, 15)


def _exact_sequence(s, b):
    """(o, lse) of sequence b in 64 bits, or zeros where it holds nothing."""
    case, cache = s.case, s.cache
    length, n, kv, dim = int(s.lens[b]), case["q_len"], case["kv_heads"], case["dim"]
    heads = case["q_heads"]
    o = torch.zeros((n, heads, dim), dtype=torch.float64, device=s.q.device)
    lse = torch.full((n, heads), -math.inf, dtype=torch.float64, device=s.q.device)
    if length == 0:
        return o, lse
    token = torch.arange(length, device=s.q.device)
    page, off = s.table[b].long()[token // cache.page], token % cache.page
    d = torch.arange(dim, device=s.q.device)
    kb = cache.k[page, :, off].long()                                            # [length, kv, D/2]
    k = (kb[..., d // 2] >> (4 * (d % 2))) & 15
    t = off % 16
    at = (off // 16 * 8 * dim)[:, None] + (d // 64 * 512 + d % 8 * 64 + d % 64 // 16 * 4) + (
        t % 8 // 2 * 16 + 2 * (t % 2) + t // 8)[:, None]                         # [length, D] bytes of V
    vb = cache.v.flatten(2)[page[:, None, None], torch.arange(kv, device=at.device)[:, None], at[:, None]].long()
    v = (vb >> (4 * (d % 16 // 8))) & 15
    kp, vp = cache.kp[page, :, off].double(), cache.vp[page, :, off].double()
    k, v = kp[..., 1:] + kp[..., :1] * k, vp[..., 1:] + vp[..., :1] * v
    for i in range(n):
        last = length - n + i
        first = max(0, last - case["window"] + 1) if case["window"] else 0
        if last < 0:
            continue
        q = s.q[b, i].double().view(kv, heads // kv, dim)
        x = torch.einsum("hgd,thd->hgt", q, k[first:last + 1]) / math.sqrt(dim)
        lse[i] = torch.logsumexp(x, -1).flatten()
        o[i] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v[first:last + 1]).flatten(0, 1)
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        both = [_exact_sequence(s, b) for b in range(case["batch"])]
        return {"o": torch.stack([o for o, _ in both]), "lse": torch.stack([x for _, x in both])}
    cos, sin, inter = s.cos[s.pos], s.sin[s.pos], case["interleaved"]
    if case["op"] == "rope_grad":
        # the gradient of sum(dy * y), by the chain rule through y = R (w * x / rms(x)) with R orthogonal
        out = {}
        for name, x, dy, w in (("q", s.q, s.dq, s.wq), ("k", s.k, s.dk, s.wk)):
            x = x.double().requires_grad_()
            w = w.double().requires_grad_()
            y = _exact_norm_rope(x, w, cos, sin, inter)
            out["d" + name], out["dw" + name] = torch.autograd.grad((y * dy.double()).sum(), (x, w))
        return out
    q = _exact_norm_rope(s.q, s.wq, cos, sin, inter)
    k = _exact_norm_rope(s.k, s.wk, cos, sin, inter)
    if case["op"] == "rope":
        return {"q": q, "k": k}
    kept = (s.slots >= 0)[:, None, None]
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    return {"q": q, "k": torch.where(kept, _exact_four_bits(k), zero),
            "v": torch.where(kept, _exact_four_bits(s.v.double()), zero)}
