"""Calls with stream=: what they allocate belongs to that stream."""
import pytest
import torch

from _helpers import dev


@pytest.fixture(scope="module")
def r9q():
    import __graft_entry__
    __graft_entry__.build()
    import block_scaled_fp8_x128_gb300 as lib
    return lib


class Inputs:
    def __init__(self, r9q, M=64, N=2048, K=1024):
        g = torch.Generator().manual_seed(7)
        self.a = torch.randn((M, K), generator=g).to(torch.bfloat16).to(dev())
        self.few = self.a[:16].contiguous()
        self.f32 = (torch.randn((N, K), generator=g) / 32).to(dev())
        self.w = r9q.r9q_quant_weight_block128(self.f32)
        self.down = r9q.r9q_quant_weight_block128((torch.randn((K, N // 2), generator=g) / 32).to(dev()))
        self.experts = [t[None] for t in self.w]


CALLS = {
    "e4m3": lambda r, x, **k: r.r9q_e4m3_from_f32(x.f32, **k),
    "quant": lambda r, x, **k: r.r9q_quant_group128(x.a, **k),
    "swiglu": lambda r, x, **k: r.r9q_swiglu_interleaved(x.a, **k),
    "weight": lambda r, x, **k: r.r9q_quant_weight_block128(x.f32, **k),
    "w8a8": lambda r, x, **k: r.r9q_gemm_fp8_block_qa(x.few, *x.w, **k),
    "w8bf16": lambda r, x, **k: r.r9q_gemm_fp8w_bf16a(x.few, *x.w, **k),
    "mlp": lambda r, x, **k: r.r9q_gate_up_swiglu_down(x.few, *x.w, *x.down, **k),
    "mlp_noalloc": lambda r, x, **k: r.r9q_gate_up_swiglu_down_noalloc(x.few, *x.w, *x.down, **k),
    "grouped": lambda r, x, **k: r.r9q_grouped_gemm_fp8(x.few, [0, 16], *x.experts, **k),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_outputs_belong_to_the_stream_of_the_call(r9q, name):
    """The current stream still has work on blocks that it has let go; outputs of a call on another stream are not made
    of them."""
    x, call = Inputs(r9q), CALLS[name]
    want = call(r9q, x)
    want = want if isinstance(want, tuple) else (want,)
    st = torch.cuda.Stream()
    sizes = sorted({t.numel() * t.element_size() for t in want} | {2 ** k for k in range(12, 24)})
    torch.cuda.synchronize()
    blocks = [torch.empty(n, dtype=torch.uint8, device=dev()) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    for b in blocks:
        b.fill_(7)
    del blocks, b
    got = call(r9q, x, stream=st)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


@pytest.mark.gpu
def test_a_call_s_own_workspace_is_not_reused_while_it_runs(r9q):
    """The expert MLP makes a workspace for each call: on a stream that is busy, the current one's next tensors must not
    be made of it."""
    x = Inputs(r9q)
    want = r9q.r9q_gate_up_swiglu_down(x.a, *x.w, *x.down)
    st = torch.cuda.Stream()
    y = torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
    r9q.r9q_gate_up_swiglu_down(x.a, *x.w, *x.down, y=y, stream=st)
    kept = [torch.full((2 ** k,), -1, dtype=torch.int8, device=dev()) for k in range(12, 24) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(want, y) and all(bool((t == -1).all()) for t in kept)
