"""The decode layer of examples/decode_layer.py: the attention block's operators between the library's GEMMs."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layers():
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_layer
    return decode_layer


def plain_step(layer, x, keys, values):
    """The layer in 32 bits: dequantised weights, and keys and values that are kept as they are."""
    def dense(w):
        q, s = w
        return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)

    def norm(t, w=1.0):
        return t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    batch, n, _ = x.shape
    x, start = x.float(), keys.shape[1]
    qkv = (norm(x) @ dense(layer.w_qkv).T).view(batch, n, -1, layer.dim)
    q, k, v = qkv.split((layer.heads, layer.kv, layer.kv), 2)
    c, s = (t[start:start + n, None] for t in (layer.cos, layer.sin))
    half = layer.dim // 2

    def turn(t):
        a, b = t[..., :half], t[..., half:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)
    q, k = turn(norm(q, layer.wq)), turn(norm(k, layer.wk))
    keys, values = torch.cat((keys, k), 1), torch.cat((values, v), 1)
    kk, vv = (t.repeat_interleave(layer.heads // layer.kv, 2).permute(0, 2, 1, 3) for t in (keys, values))
    score = q.permute(0, 2, 1, 3) @ kk.transpose(-1, -2) * layer.dim ** -0.5
    seen = torch.arange(start + n, device=x.device) <= torch.arange(start, start + n, device=x.device)[:, None]
    p = torch.where(seen, score, float("-inf")).softmax(-1)
    o = (p @ vv).permute(0, 2, 1, 3).reshape(batch, n, -1)
    h = x + o @ dense(layer.w_o).T
    gu = norm(h) @ dense(layer.w_gu).T
    gate, up = gu.view(batch, n, -1, 2, 128).unbind(-2)
    return h + (torch.nn.functional.silu(gate) * up).flatten(2) @ dense(layer.w_dn).T, keys, values


def test_layer_against_the_same_in_32_bits(layers):
    """Prompt, then single tokens and a pair.  The layer's own roundings set the distance: fp8 activations (2^-4 each,
    at random) in four products and 4-bit keys and values (a sixth of a standard deviation each): a relative error of a
    few hundredths of what attention and MLP add to x; 0.1 of the whole is far under what a wrong place, angle or mask
    makes of it (those turn the added parts, which are as large as x, into others)."""
    batch = 3
    layer = layers.Layer(batch=batch, max_tokens=512, page=32)
    g = torch.Generator(device="cuda").manual_seed(3)
    keys = values = torch.zeros((batch, 0, layer.kv, layer.dim), device="cuda")
    for n in (70, 1, 1, 2, 1, 40, 1):
        x = torch.randn((batch, n, layer.hidden), generator=g, device="cuda").to(torch.bfloat16)
        y = layer.step(x)
        ref, keys, values = plain_step(layer, x, keys, values)
        assert ((y.float() - ref).norm() / ref.norm()).item() < 0.1
    assert layer.lens.tolist() == [116] * batch


def test_decode_steps_chained_and_in_a_graph(layers):
    """With programmatic launch of the GEMMs on, and as a captured graph: the same tokens, bit for bit, as one by one."""
    import block_scaled_fp8_x128_gb300 as r9q
    outs = []
    for mode in ("plain", "pdl", "graph"):
        layer = layers.Layer(batch=4, max_tokens=512)
        x = torch.randn((4, 100, layer.hidden), generator=torch.Generator(device="cuda").manual_seed(5),
                        device="cuda").to(torch.bfloat16)
        x = layer.step(x)[:, -1:].contiguous()
        torch.cuda.synchronize()
        before = r9q.r9q_set_pdl(mode != "plain")
        try:
            if mode == "graph":
                st = torch.cuda.Stream()
                with torch.cuda.stream(st):
                    kept = layer.lens.clone()
                    layer.step(x)
                    layer.lens.copy_(kept)
                    st.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=st):
                        x.copy_(layer.step(x))
                torch.cuda.synchronize()
            for _ in range(12):
                if mode == "graph":
                    graph.replay()
                else:
                    x = layer.step(x)
            torch.cuda.synchronize()
        finally:
            r9q.r9q_set_pdl(before)
        assert r9q.r9q_last_device_error() == 0
        outs.append(x.clone())
    assert bool(torch.isfinite(outs[0]).all())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decode_layer.py"), "--prompt", "200", "--steps",
                        "5", "--batch", "4"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "205 tokens in the cache" in r.stdout
