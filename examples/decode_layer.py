"""One decoder layer on the library: a prompt, then decode steps replayed as a CUDA graph.

    python examples/decode_layer.py [--batch 8] [--prompt 500] [--steps 16]

The layer, for every sequence of the batch:

    qkv  = norm(x) Wqkv                            fp8 block GEMM, activations quantised inside
    q, k = rotate(norm(q)), rotate(norm(k))        one pass, which writes k and v to the
    cache <- k, v                                  paged 4-bit cache
    o    = attention(q, cache)
    x    = x + o Wo                                fp8 block GEMM
    x    = x + down(silu(gate) * up)               fused expert MLP, of norm(x)

Weights are random.  `Layer.step` takes the new tokens of every sequence, one (decode) or
many (a prompt); everything that depends on the lengths is read on the device, so that one
captured graph serves every decode step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_x128_gb300 as r9q  # noqa: E402


def norm(x):
    return (x.float() * (x.float().square().mean(-1, keepdim=True) + 1e-6).rsqrt()).to(torch.bfloat16)


class Layer:
    def __init__(self, hidden=1024, heads=8, kv_heads=2, dim=128, inner=1024, page=64, max_tokens=4096, batch=8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv, self.dim, self.page = hidden, heads, kv_heads, dim, page

        def weight(n, k):
            return r9q.r9q_quant_weight_block128(torch.randn((n, k), generator=g, device="cuda") * k ** -0.5)
        self.w_qkv = weight((heads + 2 * kv_heads) * dim, hidden)
        self.w_o = weight(hidden, heads * dim)
        self.w_gu, self.w_dn = weight(2 * inner, hidden), weight(hidden, inner)
        self.wq, self.wk = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda") for _ in range(2))
        angle = torch.arange(max_tokens, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, dim, 2, device="cuda") / dim)
        self.cos, self.sin = angle.cos(), angle.sin()
        per_seq = -(-max_tokens // page)
        self.cache = r9q.r9q_kv4_cache(batch * per_seq, kv_heads, page, dim)
        # which page holds what is up to the caller; here a fixed share for every sequence
        self.table = torch.arange(batch * per_seq, dtype=torch.int32, device="cuda").view(batch, per_seq)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")     # tokens in the cache

    def step(self, x):
        """x bf16 [batch][n][hidden], the n new tokens of every sequence -> the layer's output for them."""
        batch, n, hidden = x.shape
        rows = x.reshape(batch * n, hidden)
        pos = (self.lens[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")).long()
        slots = (self.table.gather(1, pos // self.page) * self.page + pos % self.page).view(-1)
        qkv = r9q.r9q_gemm_fp8_block_qa(norm(rows), *self.w_qkv).view(batch * n, -1, self.dim)
        q, k, v = qkv.split((self.heads, self.kv, self.kv), 1)
        q = r9q.r9q_qk_norm_rope_kv4(q, k, v, self.wq, self.wk, self.cos, self.sin, pos.view(-1), self.cache, slots)
        self.lens += n
        o = r9q.r9q_kv4_attention(q.view(batch, n, self.heads, self.dim), self.cache, self.table, self.lens)
        h = rows + r9q.r9q_gemm_fp8_block_qa(o.view(batch * n, -1), *self.w_o)
        y = h + r9q.r9q_gate_up_swiglu_down(norm(h), *self.w_gu, *self.w_dn)
        return y.view(batch, n, hidden)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    layer = Layer(batch=a.batch, max_tokens=a.prompt + a.steps + 64)
    prompt = torch.randn((a.batch, a.prompt, layer.hidden), device="cuda").to(torch.bfloat16)
    x = layer.step(prompt)[:, -1:].contiguous()

    # decode: one step captured, then replayed with its output as the next input
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        before = layer.lens.clone()
        layer.step(x)                                    # what a first call sets up once is not part of the graph
        layer.lens.copy_(before)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=warm):
            y = layer.step(x)
            x.copy_(y)
    torch.cuda.current_stream().wait_stream(warm)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if r9q.r9q_last_device_error():
        raise SystemExit("a kernel reported an error")
    if not bool(torch.isfinite(x).all()):
        raise SystemExit("the output is not finite")
    print(f"{a.batch} sequences, {a.prompt} prompt tokens, {a.steps} decode steps: "
          f"{start.elapsed_time(end) / a.steps * 1e3:.1f} us a step, {int(layer.lens[0])} tokens in the cache")


if __name__ == "__main__":
    main()
