"""Python binding of libr9q.so, the GB300 (sm_103a) block-scaled fp8 GEMM library.

Argument marshalling only: each function takes torch tensors, checks dtype,
shape and device, and calls the C entry point of the same name in
``include/r9q.h`` on the current CUDA stream, through ctypes or, for the
sequence operators' calls, through ``_calls.so``.  Every step of the computation
runs in the library's CUDA kernels; there is no fallback.  Importing this
package raises if ``libr9q.so`` has not been built (``build.py``), and the
attention block's calls if ``_calls.so`` has not been, for this torch.
"""
from __future__ import annotations

import ctypes
import importlib
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libr9q.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libr9q.so not built at {LIB_PATH}; run block_scaled_fp8_x128_gb300/build.py")

_lib = ctypes.CDLL(LIB_PATH)


class _Unloaded:
    """Stands for the module _calls, and loads it when an attention call first needs it: the rest does without it."""

    def __getattr__(self, name):
        module = importlib.import_module("._calls", __name__)    # (takes this object's place)
        if module.torch_version != torch.__version__:
            globals()["_calls"] = self
            raise ImportError(f"_calls.so was built for torch {module.torch_version}, this is {torch.__version__}: "
                              "run build.py")
        return getattr(module, name)


_calls = _Unloaded()

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t

_SIGS = {
    "r9q_version": ([], ctypes.c_int),
    "r9q_strerror": ([ctypes.c_int], ctypes.c_char_p),
    "r9q_last_device_error": ([_P], ctypes.c_int),
    "r9q_stream_capture_id": ([_P, ctypes.POINTER(ctypes.c_ulonglong)], ctypes.c_int),
    "r9q_set_pdl": ([ctypes.c_int], ctypes.c_int),
    "r9q_selftest_wait_timeout": ([ctypes.c_int, _P], ctypes.c_int),
    "r9q_grouped_gemm_fp8": ([_P, ctypes.POINTER(_I64), _I64, _P, _P, _P, _I64, _I64, ctypes.c_int, _P],
                             ctypes.c_int),
    "r9q_e4m3_from_f32": ([_P, _I64, _P, _P], ctypes.c_int),
    "r9q_quant_group128": ([_P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "r9q_quant_weight_block128": ([_P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "r9q_swiglu_interleaved": ([_P, _I64, _I64, _P, _P], ctypes.c_int),
    "r9q_gemm_fp8_block_qa": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "r9q_gemm_fp8w_bf16a": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "r9q_gate_up_swiglu_down": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, ctypes.c_int,
                                 _P, _SZ, _P], ctypes.c_int),
    "r9q_workspace_bytes": ([ctypes.c_int, _I64, _I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(_SZ)],
                            ctypes.c_int),
    "r9q_gate_up_swiglu_down_noalloc": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, ctypes.c_int, _P],
                                        ctypes.c_int),
    "r9q_qk_norm_rope": ([_P, _I64, _I64] * 2 + [_P] * 5 + [_P, _I64, _I64] * 2 + [_I64] * 6 +
                         [ctypes.c_float, ctypes.c_int, _P], ctypes.c_int),
    "r9q_qk_norm_rope_bwd": ([_P, _I64, _I64] * 4 + [_P] * 5 + [_P, _I64, _I64] * 2 + [_P] * 2 + [_I64] * 6 +
                             [ctypes.c_float, ctypes.c_int, _P, _SZ, _P], ctypes.c_int),
    "r9q_qk_norm_rope_kv4": ([_P, _I64, _I64] * 3 + [_P] * 5 + [_P, _I64, _I64] + [_P] * 5 + [_I64] * 8 +
                             [ctypes.c_float, ctypes.c_int, _P], ctypes.c_int),
    "r9q_kv4_append": ([_P, _I64, _I64] * 2 + [_P] * 5 + [_I64] * 5 + [_P], ctypes.c_int),
    "r9q_kv4_gather": ([_P] * 5 + [_I64] * 5 + [_P] * 3, ctypes.c_int),
    "r9q_kv4_attention": ([_P] + [_I64] * 3 + [_P] * 8 + [_I64] * 9 + [ctypes.c_float, _P, _SZ, _P], ctypes.c_int),
    "r9q_kv4_tree_attention": ([_P] + [_I64] * 3 + [_P] * 9 + [_I64] * 9 + [ctypes.c_float, _P, _SZ, _P], ctypes.c_int),
    "r9q_kv4_move": ([_P] * 6 + [_I64] * 6 + [_P], ctypes.c_int),
    "r9q_gated_delta": ([_P, _I64, _I64] * 3 + [_P] * 6 + [_I64] * 6 + [ctypes.c_float] * 2 + [ctypes.c_int, _P],
                        ctypes.c_int),
    "r9q_gated_delta_step": ([_P, _I64, _I64, _I64] * 3 + [_P] * 5 + [_I64] * 6 + [ctypes.c_float] * 2 +
                             [ctypes.c_int, _P], ctypes.c_int),
    "r9q_gated_delta_tree": ([_P, _I64, _I64, _I64] * 3 + [_P] * 6 + [_I64] * 6 + [ctypes.c_float] * 2 + [_P],
                             ctypes.c_int),
    "r9q_gated_delta_commit": ([_P, _I64, _I64, _I64] * 2 + [_P] * 5 + [_I64] * 7 + [ctypes.c_float, _P], ctypes.c_int),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = tuple(_SIGS)

R9Q_ERR_WORKSPACE = -4
R9Q_ERR_TIMEOUT = -6
R9Q_GROUPED_WEIGHT_ONLY = 1
R9Q_GROUPED_SWIGLU = 2
R9Q_MLP_WEIGHT_ONLY = 1
R9Q_MLP_UNFUSED = 2
R9Q_OP_GEMM_W8A8 = 1
R9Q_OP_GEMM_W8BF16 = 2
R9Q_OP_GATE_UP_SWIGLU_DOWN = 3
R9Q_OP_QK_NORM_ROPE_BWD = 4
R9Q_OP_KV4_ATTENTION = 5
R9Q_OP_KV4_TREE_ATTENTION = 6
R9Q_ROPE_INTERLEAVED = 1
R9Q_DELTA_FROM_ZERO = 1


class R9QError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {code} ({_lib.r9q_strerror(code).decode()})")


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise R9QError(rc, where)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _empty(shape, dtype, device, stream):
    """A new tensor of the stream that the call runs on: what the current one still does with a block that it has let go,
    or does next with one that this call lets go, does not meet the kernel."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _expect(t, dtype, shape, name):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def r9q_version() -> int:
    return int(_lib.r9q_version())


def r9q_strerror(code: int) -> str:
    return _lib.r9q_strerror(int(code)).decode()


def r9q_grouped_gemm_fp8(a: torch.Tensor, offsets, w: torch.Tensor, ws: torch.Tensor, y: torch.Tensor | None = None,
                         flags: int = 0, stream=None) -> torch.Tensor:
    """Several experts in one launch: a bf16 [offsets[-1]][K] (tokens sorted by
    expert), offsets host ints [E + 1], w e4m3 [E][N][K], ws fp32
    [E][N/128][K/128]; y bf16 [offsets[-1]][N] (N/2 with R9Q_GROUPED_SWIGLU)."""
    off = [int(v) for v in offsets]
    E = len(off) - 1
    Mtot, K = a.shape
    _expect(a, torch.bfloat16, (off[-1], K), "a")
    if w.dim() != 3 or w.shape[0] != E or w.shape[2] != K:
        raise ValueError("w must be [E][N][K]")
    N = w.shape[1]
    _expect(w, torch.uint8, (E, N, K), "w")
    _expect(ws, torch.float32, (E, N // 128, K // 128), "ws")
    ncols = N // 2 if flags & R9Q_GROUPED_SWIGLU else N
    if y is None:
        y = _empty((Mtot, ncols), torch.bfloat16, a.device, stream)
    _expect(y, torch.bfloat16, (Mtot, ncols), "y")
    arr = (_I64 * (E + 1))(*off)
    _check(_lib.r9q_grouped_gemm_fp8(_ptr(a), arr, E, _ptr(w), _ptr(ws), _ptr(y), N, K, int(flags), _stream(stream)),
           "r9q_grouped_gemm_fp8")
    return y


def r9q_selftest_wait_timeout(which: int, stream=None) -> None:
    """Launch the failure-detection self-test kernel (its bounded waits run
    out and record R9Q_ERR_TIMEOUT; read it with r9q_last_device_error)."""
    _check(_lib.r9q_selftest_wait_timeout(int(which), _stream(stream)), "r9q_selftest_wait_timeout")


def r9q_set_pdl(enable: bool) -> bool:
    """Programmatic dependent launch for the GEMMs (see include/r9q.h); returns the previous setting."""
    return bool(_lib.r9q_set_pdl(int(bool(enable))))


def r9q_last_device_error(stream=None) -> int:
    rc = int(_lib.r9q_last_device_error(_stream(stream)))
    if rc != 0:
        # a kernel may have given up mid-call and left its workspace's counters non-zero (graphs zero their own)
        _WORKSPACES.clear()
    return rc


# One zero-filled workspace per (device, stream) for calls that pass none.  Every call
# that completes leaves the workspace's counter header at zero again, so the same tensor
# serves every later call on that stream (calls on one stream are ordered); it grows when
# a larger call needs more.
_WORKSPACES: dict = {}
# A graph keeps the addresses of what it captured, and may be replayed at any time and on
# any stream, so the calls of a capture have a workspace of their own: from the graph's
# memory, its header zeroed by a node of the graph.  Here the last one of each stream,
# {(device, stream): (capture, workspace)}; the graph itself holds the memory.
_CAPTURED: dict = {}
_HEADER = 64 * 1024                                           # the counters, zero between calls
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def r9q_stream_capture_id(stream=None) -> int:
    """The id of the capture that the stream is part of, 0 if none."""
    out = ctypes.c_ulonglong(0)
    _check(_lib.r9q_stream_capture_id(_stream(stream), ctypes.byref(out)), "r9q_stream_capture_id")
    return int(out.value)


def _stream_workspace(need: int, device: torch.device, stream=None) -> torch.Tensor:
    """The workspace of the stream, or of the capture that it is part of, made or grown to `need` bytes."""
    s = stream if stream is not None else torch.cuda.current_stream(device)
    key = (device.index, s.cuda_stream)
    capture = r9q_stream_capture_id(s) if stream is not None or _capturing() else 0
    if capture:
        of, ws = _CAPTURED.get(key, (0, None))
        if of != capture or ws.numel() < need:
            with torch.cuda.stream(s):
                ws = torch.empty(need, dtype=torch.uint8, device=device)
                ws[:_HEADER].zero_()
            _CAPTURED[key] = (capture, ws)
        return ws
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < need:
        with torch.cuda.stream(s):                            # zeroed on the stream that uses it
            ws = torch.zeros(need, dtype=torch.uint8, device=device)
        _WORKSPACES[key] = ws
    return ws


def r9q_e4m3_from_f32(x: torch.Tensor, q: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _expect(x, torch.float32, x.shape, "x")
    if q is None:
        q = _empty(x.shape, torch.uint8, x.device, stream)
    _expect(q, torch.uint8, x.shape, "q")
    _check(_lib.r9q_e4m3_from_f32(_ptr(x), x.numel(), _ptr(q), _stream(stream)), "r9q_e4m3_from_f32")
    return q


def r9q_quant_group128(x: torch.Tensor, xq: torch.Tensor | None = None, xs: torch.Tensor | None = None,
                       stream=None):
    M, K = x.shape
    _expect(x, torch.bfloat16, (M, K), "x")
    if xq is None:
        xq = _empty((M, K), torch.uint8, x.device, stream)
    if xs is None:
        xs = _empty((M, K // 128), torch.float32, x.device, stream)
    _expect(xq, torch.uint8, (M, K), "xq")
    _expect(xs, torch.float32, (M, K // 128), "xs")
    _check(_lib.r9q_quant_group128(_ptr(x), M, K, _ptr(xq), _ptr(xs), _stream(stream)), "r9q_quant_group128")
    return xq, xs


def r9q_swiglu_interleaved(gu: torch.Tensor, h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gu bf16 [M][2I] (gate/up interleaved per 128 columns) -> h bf16 [M][I]."""
    M, I2 = gu.shape
    I = I2 // 2
    _expect(gu, torch.bfloat16, (M, 2 * I), "gu")
    if h is None:
        h = _empty((M, I), torch.bfloat16, gu.device, stream)
    _expect(h, torch.bfloat16, (M, I), "h")
    _check(_lib.r9q_swiglu_interleaved(_ptr(gu), M, I, _ptr(h), _stream(stream)), "r9q_swiglu_interleaved")
    return h


def r9q_quant_weight_block128(w: torch.Tensor, wq: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                              stream=None):
    N, K = w.shape
    _expect(w, torch.float32, (N, K), "w")
    if wq is None:
        wq = _empty((N, K), torch.uint8, w.device, stream)
    if ws is None:
        ws = _empty((N // 128, K // 128), torch.float32, w.device, stream)
    _expect(wq, torch.uint8, (N, K), "wq")
    _expect(ws, torch.float32, (N // 128, K // 128), "ws")
    _check(_lib.r9q_quant_weight_block128(_ptr(w), N, K, _ptr(wq), _ptr(ws), _stream(stream)),
           "r9q_quant_weight_block128")
    return wq, ws


def r9q_workspace_bytes(op: int, M: int, N: int, K: int, N2: int = 0, flags: int = 0) -> int:
    out = _SZ(0)
    _check(_lib.r9q_workspace_bytes(int(op), M, N, K, N2, int(flags), ctypes.byref(out)), "r9q_workspace_bytes")
    return int(out.value)


def r9q_gemm_fp8_block_qa(a: torch.Tensor | None, w: torch.Tensor, ws: torch.Tensor,
                          y: torch.Tensor | None = None, aq: torch.Tensor | None = None,
                          as_: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                          M: int | None = None, stream=None) -> torch.Tensor:
    """W8A8.  a (bf16 [M][K]) given: fused quant, aq/as_ optional outputs.
    a None: aq (uint8 [M][K]) / as_ (fp32 [M][K/128]) are the inputs.
    workspace: uint8 device tensor of at least r9q_workspace_bytes(R9Q_OP_GEMM_W8A8, M, N, K)
    bytes, zero-filled before its first use (e.g. torch.zeros); the calls keep its counter
    header at zero, so one workspace serves any sequence of calls on one stream.  When omitted,
    the binding reuses one zeroed workspace per (device, stream), allocated (and zero-filled)
    on the first call that needs it or needs more; the calls of a graph capture have one of the
    graph's own, which the graph zeroes whenever it is replayed.  Pass your own to save that node and to
    control the allocation."""
    N, K = w.shape
    src = a if a is not None else aq
    if src is None:
        raise ValueError("need a or aq/as_")
    M = src.shape[0]
    _expect(a, torch.bfloat16, (M, K), "a")
    _expect(aq, torch.uint8, (M, K), "aq")
    _expect(as_, torch.float32, (M, K // 128), "as")
    _expect(w, torch.uint8, (N, K), "w")
    _expect(ws, torch.float32, (N // 128, K // 128), "ws")
    if y is None:
        y = _empty((M, N), torch.bfloat16, w.device, stream)
    _expect(y, torch.bfloat16, (M, N), "y")
    if workspace is None:
        need = r9q_workspace_bytes(R9Q_OP_GEMM_W8A8, M, N, K)
        if need:
            workspace = _stream_workspace(need, w.device, stream)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.r9q_gemm_fp8_block_qa(_ptr(a), _ptr(aq), _ptr(as_), _ptr(w), _ptr(ws), _ptr(y), M, N, K,
                                      _ptr(workspace), wsb, _stream(stream)), "r9q_gemm_fp8_block_qa")
    return y


def r9q_gemm_fp8w_bf16a(a: torch.Tensor, w: torch.Tensor, ws: torch.Tensor, y: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M, K = a.shape
    N = w.shape[0]
    _expect(a, torch.bfloat16, (M, K), "a")
    _expect(w, torch.uint8, (N, K), "w")
    _expect(ws, torch.float32, (N // 128, K // 128), "ws")
    if y is None:
        y = _empty((M, N), torch.bfloat16, w.device, stream)
    _expect(y, torch.bfloat16, (M, N), "y")
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.r9q_gemm_fp8w_bf16a(_ptr(a), _ptr(w), _ptr(ws), _ptr(y), M, N, K, _ptr(workspace), wsb,
                                    _stream(stream)), "r9q_gemm_fp8w_bf16a")
    return y


def r9q_gate_up_swiglu_down(x: torch.Tensor, w_gu: torch.Tensor, s_gu: torch.Tensor, w_dn: torch.Tensor,
                            s_dn: torch.Tensor, y: torch.Tensor | None = None, h: torch.Tensor | None = None,
                            hq: torch.Tensor | None = None, hs: torch.Tensor | None = None, flags: int = 0,
                            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M, H = x.shape
    I = w_gu.shape[0] // 2
    H_out = w_dn.shape[0]
    _expect(x, torch.bfloat16, (M, H), "x")
    _expect(w_gu, torch.uint8, (2 * I, H), "w_gu")
    _expect(s_gu, torch.float32, (2 * I // 128, H // 128), "s_gu")
    _expect(w_dn, torch.uint8, (H_out, I), "w_dn")
    _expect(s_dn, torch.float32, (H_out // 128, I // 128), "s_dn")
    _expect(h, torch.bfloat16, (M, I), "h")
    _expect(hq, torch.uint8, (M, I), "hq")
    _expect(hs, torch.float32, (M, I // 128), "hs")
    if y is None:
        y = _empty((M, H_out), torch.bfloat16, x.device, stream)
    _expect(y, torch.bfloat16, (M, H_out), "y")
    if workspace is None:
        need = r9q_workspace_bytes(R9Q_OP_GATE_UP_SWIGLU_DOWN, M, I, H, H_out, flags)
        if need:
            workspace = _empty(need, torch.uint8, x.device, stream)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.r9q_gate_up_swiglu_down(_ptr(x), _ptr(w_gu), _ptr(s_gu), _ptr(w_dn), _ptr(s_dn), _ptr(y),
                                        M, H, I, H_out, _ptr(h), _ptr(hq), _ptr(hs), int(flags),
                                        _ptr(workspace), wsb, _stream(stream)), "r9q_gate_up_swiglu_down")
    return y


def r9q_gate_up_swiglu_down_noalloc(x: torch.Tensor, w_gu: torch.Tensor, s_gu: torch.Tensor, w_dn: torch.Tensor,
                                    s_dn: torch.Tensor, y: torch.Tensor | None = None,
                                    hq: torch.Tensor | None = None, hs: torch.Tensor | None = None,
                                    flags: int = 0, stream=None) -> torch.Tensor:
    """The fused expert MLP without workspace (h lives in the library's fixed
    scratch; see include/r9q.h for the size limit and the sharing rules)."""
    M, H = x.shape
    I = w_gu.shape[0] // 2
    H_out = w_dn.shape[0]
    _expect(x, torch.bfloat16, (M, H), "x")
    _expect(w_gu, torch.uint8, (2 * I, H), "w_gu")
    _expect(s_gu, torch.float32, (2 * I // 128, H // 128), "s_gu")
    _expect(w_dn, torch.uint8, (H_out, I), "w_dn")
    _expect(s_dn, torch.float32, (H_out // 128, I // 128), "s_dn")
    _expect(hq, torch.uint8, (M, I), "hq")
    _expect(hs, torch.float32, (M, I // 128), "hs")
    if y is None:
        y = _empty((M, H_out), torch.bfloat16, x.device, stream)
    _expect(y, torch.bfloat16, (M, H_out), "y")
    _check(_lib.r9q_gate_up_swiglu_down_noalloc(_ptr(x), _ptr(w_gu), _ptr(s_gu), _ptr(w_dn), _ptr(s_dn), _ptr(y),
                                                M, H, I, H_out, _ptr(hq), _ptr(hs), int(flags), _stream(stream)),
           "r9q_gate_up_swiglu_down_noalloc")
    return y


# ---- the attention block of a decode layer ----
# Of these calls r9q_qk_norm_rope is recorded by autograd; the others' outputs carry no gradient.

class KV4Cache(NamedTuple):
    """The paged 4-bit key-value cache (layout: include/r9q.h).  k uint8 [pages][Hk][page][D/2], v uint8 of the
    same shape (its bytes in groups of 16 tokens), kp and vp bf16 [pages][Hk][page][2]; r9q_kv4_cache makes one."""
    k: torch.Tensor
    kp: torch.Tensor
    v: torch.Tensor
    vp: torch.Tensor


def r9q_kv4_cache(pages: int, heads: int, page: int, dim: int, device=None) -> KV4Cache:
    """An empty cache of `pages` pages of `page` tokens (a multiple of 16) for `heads` key-value heads of `dim`."""
    if page < 16 or page % 16 or dim not in (64, 128) or pages < 1 or heads < 1:
        raise ValueError("page must be a multiple of 16, dim 64 or 128, pages and heads positive")
    device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    k = torch.zeros((pages, heads, page, dim // 2), dtype=torch.uint8, device=device)
    kp = torch.zeros((pages, heads, page, 2), dtype=torch.bfloat16, device=device)
    return KV4Cache(k, kp, torch.zeros_like(k), torch.zeros_like(kp))


# These calls last microseconds on the GPU: _calls (csrc/r9q_calls.cpp) checks their tensors and makes the C call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere(device, stream, call, *args):
    """call(*args, stream=None) with the tensors' device and the given stream current: the C call launches on the current
    device, and new outputs belong to the current stream."""
    index = device.index
    if index is None:
        raise ValueError("tensor must be on a CUDA device")
    if stream is None:
        with torch.cuda.device(index):
            return call(*args, stream=None)
    if stream.device.index != index:
        raise ValueError("stream is of another device than the tensors")
    with torch.cuda.stream(stream):
        return call(*args, stream=None)


def _checked(r, where):
    """The outputs of a call, or its code raised."""
    if r.__class__ is int:
        _check(r, where)
    return r


def _with_workspace(where, op, size, call, args, workspace, device, stream):
    """A call that needs a workspace: the caller's, or the stream's own, made or grown where that does not do.
    size(): the M, N and K that r9q_workspace_bytes takes."""
    index = device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(device, stream, _with_workspace, where, op, size, call, args, workspace, device)
    handle = _raw_stream(index)
    theirs = workspace is not None
    r = call(*args, workspace if theirs else _WORKSPACES.get((index, handle)), theirs, handle)
    if not theirs and r.__class__ is int and r in (_calls.CAPTURED, R9Q_ERR_WORKSPACE):
        own = _stream_workspace(r9q_workspace_bytes(op, *size()), device)
        r = call(*args, own, True, handle)
    return _checked(r, where)


def _readable(t):
    """t as the kernels read head tensors: contiguous vectors on 16-byte boundaries."""
    ok = t.stride(2) == 1 and t.stride(0) % 8 == 0 and t.stride(1) % 8 == 0 and t.data_ptr() % 16 == 0
    return t if ok else t.contiguous()


class _NormRope(torch.autograd.Function):
    """r9q_qk_norm_rope with r9q_qk_norm_rope_bwd as its gradient (to q, k, wq and wk)."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, positions, eps, interleaved):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        ctx.how = (eps, interleaved)
        return _checked(_calls.qk_norm_rope(q, k, wq, wk, cos, sin, positions, eps, interleaved, None, None,
                                            _raw_stream(q.device.index)), "r9q_qk_norm_rope")

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        return (*r9q_qk_norm_rope_bwd(_readable(dq_out), _readable(dk_out), *ctx.saved_tensors, *ctx.how),
                None, None, None, None, None)


def r9q_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, wq: torch.Tensor, wk: torch.Tensor,
                     cos: torch.Tensor | None = None, sin: torch.Tensor | None = None,
                     positions: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """RMS norm of the heads of q bf16 [T][Hq][D] and k bf16 [T][Hk][D] (any token and head strides) and the
    rotation by cos, sin fp32 [npos][rot/2] at positions int64 [T] (None: norm only); returns (q_out, k_out), which
    are parts of one allocation where neither was given.  Then they carry the gradient to q, k, wq and wk where one of
    these requires it; a call that is given an output is not recorded."""
    index = q.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(q.device, stream, r9q_qk_norm_rope, q, k, wq, wk, cos, sin, positions, eps, interleaved, q_out,
                          k_out)
    r = _calls.qk_norm_rope(q, k, wq, wk, cos, sin, positions, eps, interleaved, q_out, k_out, _raw_stream(index))
    if r.__class__ is int and r == _calls.RECORDED:
        return _NormRope.apply(q, k, wq, wk, cos, sin, positions, eps, interleaved)
    return _checked(r, "r9q_qk_norm_rope")


def r9q_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                         wq: torch.Tensor, wk: torch.Tensor, cos: torch.Tensor | None = None,
                         sin: torch.Tensor | None = None, positions: torch.Tensor | None = None, eps: float = 1e-6,
                         interleaved: bool = False, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                         dwq: torch.Tensor | None = None, dwk: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None):
    """The gradient of r9q_qk_norm_rope; returns (dq, dk, dwq, dwk), of two allocations (dq and dk, dwq and dwk)
    where they were not given.  workspace: as for r9q_gemm_fp8_block_qa
    (zero-filled before its first use; omitted: the stream's own)."""
    return _with_workspace("r9q_qk_norm_rope_bwd", R9Q_OP_QK_NORM_ROPE_BWD, lambda: (1, q.shape[-1], 0),
                           _calls.qk_norm_rope_bwd,
                           (dq_out, dk_out, q, k, wq, wk, cos, sin, positions, eps, interleaved, dq, dk, dwq, dwk),
                           workspace, q.device, stream)


def r9q_qk_norm_rope_kv4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, wq: torch.Tensor, wk: torch.Tensor,
                         cos: torch.Tensor | None, sin: torch.Tensor | None, positions: torch.Tensor | None,
                         cache: KV4Cache, slots: torch.Tensor, eps: float = 1e-6, interleaved: bool = False,
                         q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """r9q_qk_norm_rope with the keys, and v bf16 [T][Hk][D] as it is, written to the cache at slots int64 [T]
    (page * tokens of a page + place; negative: padding); returns q_out."""
    index = q.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(q.device, stream, r9q_qk_norm_rope_kv4, q, k, v, wq, wk, cos, sin, positions, cache, slots, eps,
                          interleaved, q_out)
    return _checked(_calls.qk_norm_rope_kv4(q, k, v, wq, wk, cos, sin, positions, *cache, slots, eps, interleaved, q_out,
                                            _raw_stream(index)), "r9q_qk_norm_rope_kv4")


def r9q_kv4_append(k: torch.Tensor, v: torch.Tensor, cache: KV4Cache, slots: torch.Tensor, stream=None) -> None:
    """Writes k and v bf16 [T][Hk][D] to the cache at slots int64 [T] (negative: padding)."""
    index = k.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(k.device, stream, r9q_kv4_append, k, v, cache, slots)
    _checked(_calls.kv4_append(k, v, *cache, slots, _raw_stream(index)), "r9q_kv4_append")


def r9q_kv4_gather(cache: KV4Cache, slots: torch.Tensor, k: torch.Tensor | None = None,
                   v: torch.Tensor | None = None, stream=None):
    """The tokens at slots int64 [T] as bf16 (k, v) [T][Hk][D] (parts of one allocation where neither was given);
    zeros for padding."""
    index = slots.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(slots.device, stream, r9q_kv4_gather, cache, slots, k, v)
    return _checked(_calls.kv4_gather(*cache, slots, k, v, _raw_stream(index)), "r9q_kv4_gather")


def r9q_kv4_attention(q: torch.Tensor, cache: KV4Cache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                      scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                      lse: torch.Tensor | None = None, return_lse: bool = False,
                      workspace: torch.Tensor | None = None, stream=None):
    """Attention of the last Lq tokens of each sequence, q bf16 [B][Lq][Hq][D] (any batch, token and head strides),
    over the cache: block_table int32 [B][max_pages], seq_lens int32 [B] (new tokens included).  scale: 1/sqrt(D) by
    default.  Returns o bf16 [B][Lq][Hq][D], or with return_lse (o, lse fp32 [B][Lq][Hq]), parts of one allocation where
    neither was given.  workspace: as for r9q_gemm_fp8_block_qa (zero-filled before its first use; omitted: the stream's
    own)."""
    return _with_workspace("r9q_kv4_attention", R9Q_OP_KV4_ATTENTION,
                           lambda: (max(1, q.shape[1] * q.shape[2] // cache.k.shape[1]), q.shape[3], 0),
                           _calls.kv4_attention,
                           (q, *cache, block_table, seq_lens, scale, window, out, lse, return_lse), workspace, q.device,
                           stream)


def r9q_kv4_tree_attention(q: torch.Tensor, cache: KV4Cache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                           parents: torch.Tensor, scale: float | None = None, window: int = 0,
                           out: torch.Tensor | None = None, lse: torch.Tensor | None = None, return_lse: bool = False,
                           workspace: torch.Tensor | None = None, stream=None):
    """r9q_kv4_attention with the last Lq (at most 64) tokens of each sequence as the nodes of a tree: parents int32
    [B][Lq], each node's parent before it (0 .. i - 1), -1 the sequence's token before the tree, -2 no node.  A node sees
    what is before the tree, its ancestors and itself.  Workspace, outputs and the rest as there."""
    return _with_workspace("r9q_kv4_tree_attention", R9Q_OP_KV4_TREE_ATTENTION,
                           lambda: (max(1, q.shape[1] * q.shape[2] // cache.k.shape[1]), q.shape[3],
                                    max(1, q.shape[0] * cache.k.shape[1])),
                           _calls.kv4_tree_attention,
                           (q, *cache, block_table, seq_lens, parents, scale, window, out, lse, return_lse), workspace,
                           q.device, stream)


def r9q_kv4_move(cache: KV4Cache, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Copies tokens of the cache from slots src to slots dst, int64 [rows][n] (n at most 64; negative: passed over).  All
    of a row is read before any of it is written; rows may not write what another row reads or writes."""
    index = src.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(src.device, stream, r9q_kv4_move, cache, src, dst)
    _checked(_calls.kv4_move(*cache, src, dst, _raw_stream(index)), "r9q_kv4_move")


# ---- the gated delta rule ----
# state fp32 [n_states][Hv][D][D] (values, keys) is read and written in place; the outputs carry no gradient.

def r9q_gated_delta(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                    state: torch.Tensor, slots: torch.Tensor, cu_seqlens: torch.Tensor, scale: float | None = None,
                    eps: float = 1e-6, from_zero: bool = False, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """The gated delta rule over packed sequences: q, k bf16 [T][Hk][D], v bf16 [T][Hv][D] (any token and head strides),
    g (log of the decay), beta fp32 [T][Hv]; sequence b has the tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32
    [B + 1]) and the state slots[b] (int32 [B]; negative: no sequence), which begins at zero with from_zero.  Keys and
    queries are brought to unit length.  scale: 1/sqrt(D) by default.  Returns o bf16 [T][Hv][D]; rows of no sequence
    are left as they are."""
    index = k.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(k.device, stream, r9q_gated_delta, q, k, v, g, beta, state, slots, cu_seqlens, scale, eps,
                          from_zero, out)
    return _checked(_calls.gated_delta(q, k, v, g, beta, state, slots, cu_seqlens, scale, eps, from_zero, out,
                                       _raw_stream(index)), "r9q_gated_delta")


def r9q_gated_delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                         state: torch.Tensor, slots: torch.Tensor, scale: float | None = None, eps: float = 1e-6,
                         from_zero: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The newest tokens of B sequences: r9q_gated_delta with q, k bf16 [B][Lq][Hk][D], v [B][Lq][Hv][D] (any batch, token
    and head strides), g, beta fp32 [B][Lq][Hv]; returns o bf16 [B][Lq][Hv][D]."""
    index = k.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(k.device, stream, r9q_gated_delta_step, q, k, v, g, beta, state, slots, scale, eps, from_zero, out)
    return _checked(_calls.gated_delta_step(q, k, v, g, beta, state, slots, None, scale, eps, from_zero, out,
                                            _raw_stream(index)), "r9q_gated_delta_step")


def r9q_gated_delta_tree(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                         state: torch.Tensor, slots: torch.Tensor, parents: torch.Tensor, scale: float | None = None,
                         eps: float = 1e-6, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Drafted tokens: r9q_gated_delta_step along every path of a tree of Lq (at most 64) nodes, parents int32 [B][Lq] as
    for r9q_kv4_tree_attention.  The states are not written; r9q_gated_delta_commit does that."""
    index = k.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(k.device, stream, r9q_gated_delta_tree, q, k, v, g, beta, state, slots, parents, scale, eps, out)
    return _checked(_calls.gated_delta_tree(q, k, v, g, beta, state, slots, parents, scale, eps, False, out,
                                            _raw_stream(index)), "r9q_gated_delta_tree")


def r9q_gated_delta_commit(k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, state: torch.Tensor,
                           slots: torch.Tensor, path: torch.Tensor, eps: float = 1e-6, stream=None) -> None:
    """Takes the states on along an accepted path of the tree that k, v, g and beta are of: path int32 [B][P] (P at most
    64), nodes from the tree's beginning on, until the first negative one."""
    index = k.device.index
    if stream is not None or index is None or index != _current_device():
        return _elsewhere(k.device, stream, r9q_gated_delta_commit, k, v, g, beta, state, slots, path, eps)
    _checked(_calls.gated_delta_commit(k, v, g, beta, state, slots, path, eps, _raw_stream(index)),
             "r9q_gated_delta_commit")
