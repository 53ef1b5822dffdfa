"""Python binding of the B200 4-bit MoE expert FFN library (libmoe_q4.so).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels (sm_100a).  PyTorch provides device memory and streams.  The function
names are the C ABI's (include/moe_q4.h).  Importing this module fails loudly
if the CUDA library has not been built; there is no fallback.

A call runs on `stream`, or on the current stream.  What it allocates (outputs
and workspaces that are not given) belongs to that stream; an output it returns
is marked as used by the current stream too.  Tensors that are given have to
live, and to be ordered, as with any other work on a stream.

The layer is the MoE expert FFN of "A 35B Hybrid-Attention Mixture-of-Experts
Model on a 6GB 2011 GPU: Hand-Written 4-bit CUDA Inference for Fermi" (Dutch
technical summary, Methodologie 1 and 2): top-k routing, Q8_0 activations,
grouped W4A8 gate/up and down projections over Q4_0 expert weights, SwiGLU,
and the router-weighted combine.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_q4.so")

QK = 32
Q4_BYTES = 18

MOE_Q4_OK = 0
ERRORS = {
    -1: "MOE_Q4_ERR_INVALID_ARG", -2: "MOE_Q4_ERR_SHAPE", -3: "MOE_Q4_ERR_ALIGN",
    -4: "MOE_Q4_ERR_WORKSPACE", -5: "MOE_Q4_ERR_ARCH", -6: "MOE_Q4_ERR_CUDA", -7: "MOE_Q4_ERR_OVERLAP",
}
STATUS_SCALE_OVERFLOW = 0x1
STATUS_SPIN_TIMEOUT = 0x2
STATUS_NONFINITE_LOGIT = 0x4
STATUS_BAD_EXPERT_INDEX = 0x8
STATUS_BAD_ADAPTER_INDEX = 0x10
STATUS_BAD_MASK_INDEX = 0x20
STATUS_NAN_LOGIT = 0x40

PATH_AUTO, PATH_GROUPED_DP4A, PATH_DECODE, PATH_TENSOR_CORE = 0, 1, 2, 3
PATH_TENSOR_CORE_N32, PATH_TENSOR_CORE_N128, PATH_TENSOR_CORE_N64 = 4, 5, 6

WS_NAMES = ["status", "logits", "topk_idx", "topk_w", "qa", "da", "cnt", "off", "tile_off",
            "chunk_cnt", "chunk_base", "sorted", "pos", "hq", "dh", "total"]

# Every extern "C" symbol of include/moe_q4.h.
EXPORTS = ["moe_q4_quantize_act", "moe_q4_route", "moe_q4_ffn_workspace_bytes", "moe_q4_ffn_forward",
           "moe_q4_ffn_host_workspace_bytes", "moe_q4_ffn_forward_host", "moe_q4_status_string",
           "moe_q4_workspace_layout", "moe_q4_ffn_forward_debug", "moe_q4_block_dots",
           "moe_q4_ffn_forward_noalloc", "moe_q4_last_cuda_error", "moe_q4_residual_rmsnorm",
           "moe_q4_stack_workspace_bytes", "moe_q4_stack_forward", "moe_q4_gemv_workspace_bytes", "moe_q4_gemv",
           "moe_q4_staging_bytes", "moe_q4_ffn_forward_streamed", "moe_q4_test_override_device",
           "moe_q4_rescale_ceiling", "moe_q4_adapters_workspace_bytes", "moe_q4_adapters_apply",
           "moe_q4_logits_apply"]


class MoeQ4Error(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        detail = moe_q4_status_string(code)
        if code == -6:
            detail += ": " + moe_q4_last_cuda_error()
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({detail})")


class _Layer(ctypes.Structure):
    _fields_ = [
        ("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32), ("n_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32), ("has_shared", ctypes.c_int32),
        ("w_router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
        ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
        ("sh_gate", ctypes.c_void_p), ("sh_up", ctypes.c_void_p), ("sh_down", ctypes.c_void_p),
    ]


class _Debug(ctypes.Structure):
    _fields_ = [("h_out", ctypes.c_void_p), ("path", ctypes.c_int32),
                ("ev_start", ctypes.c_void_p), ("ev_stop", ctypes.c_void_p), ("force_spin_timeout", ctypes.c_int32),
                ("block_dots_out", ctypes.c_void_p), ("block_dots_down", ctypes.c_int32),
                ("block_dots_group", ctypes.c_int32), ("block_dots_rb", ctypes.c_int32),
                ("decode_kernel_ns", ctypes.c_void_p)]


class _Adapters(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("rank", ctypes.c_int32), ("n_out", ctypes.c_int64),
                ("n_adapters", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


# moe_q4_logit_rules: fifteen fields of 8 bytes (a step makes one, and packing is
# quicker than a ctypes structure)
_pack_rules = struct.Struct("15q").pack


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the CUDA library first "
            "(python quantized_moe_q4_b200/build.py, or __graft_entry__.build()). There is no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    sigs = {
        "moe_q4_quantize_act": ([P, i64, i32, P, P, P, P], ctypes.c_int),
        "moe_q4_route": ([P, P, i64, P, P, P, P], ctypes.c_int),
        "moe_q4_ffn_workspace_bytes": ([P, i64], sz),
        "moe_q4_ffn_forward": ([P, P, i64, P, P, sz, P], ctypes.c_int),
        "moe_q4_ffn_host_workspace_bytes": ([P, i64], sz),
        "moe_q4_ffn_forward_host": ([P, P, i64, P, P, sz, P], ctypes.c_int),
        "moe_q4_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "moe_q4_workspace_layout": ([P, i64, P, ctypes.c_int], ctypes.c_int),
        "moe_q4_ffn_forward_debug": ([P, P, i64, P, P, sz, P, P], ctypes.c_int),
        "moe_q4_block_dots": ([P, P, i64, P, P], ctypes.c_int),
        "moe_q4_ffn_forward_noalloc": ([P, P, i64, P, P], ctypes.c_int),
        "moe_q4_last_cuda_error": ([], ctypes.c_char_p),
        "moe_q4_residual_rmsnorm": ([P, P, i64, i32, ctypes.c_float, P, P], ctypes.c_int),
        "moe_q4_stack_workspace_bytes": ([P, i64], sz),
        "moe_q4_stack_forward": ([P, i32, P, i64, ctypes.c_float, P, sz, P], ctypes.c_int),
        "moe_q4_gemv_workspace_bytes": ([i64, i32], sz),
        "moe_q4_gemv": ([P, i64, i32, P, i64, P, P, sz, P], ctypes.c_int),
        "moe_q4_staging_bytes": ([P], sz),
        "moe_q4_ffn_forward_streamed": ([P, P, i64, P, P, sz, P, sz, P], ctypes.c_int),
        "moe_q4_test_override_device": ([i32, i32, i32], ctypes.c_int),
        "moe_q4_rescale_ceiling": ([i32, i32, P, P, P], ctypes.c_int),
        "moe_q4_adapters_workspace_bytes": ([P, i64], sz),
        "moe_q4_adapters_apply": ([P, P, i64, P, i64, P, i64, P, i64, P, sz, P], ctypes.c_int),
        "moe_q4_logits_apply": ([P, P, i64, i64, P, i64, P, P, P, P], ctypes.c_int),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, what: str):
    if rc != MOE_Q4_OK:
        raise MoeQ4Error(rc, what)


def _scratch(stream, make, *args, **kw) -> torch.Tensor:
    """make(*args, **kw) on the stream of the call.  (A block of the caching
    allocator that is freed is handed out again in the order of the stream that
    it was allocated on: one of the current stream, freed on return, could be
    somebody else's before the call's kernels on `stream` have run.)"""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _result(stream, make, *args, **kw) -> torch.Tensor:
    """The same for what the call returns: the caller may use it, and let go of
    it, on the current stream."""
    t = _scratch(stream, make, *args, **kw)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def moe_q4_status_string(code: int) -> str:
    return _lib.moe_q4_status_string(int(code)).decode()


def moe_q4_last_cuda_error() -> str:
    return _lib.moe_q4_last_cuda_error().decode()


class Layer:
    """One MoE layer's weights on the device and its C descriptor.

    w_router [E,H] fp32, router_bias [E] fp32 or None, w_gate/w_up [E,F,H/32,18]
    uint8, w_down [E,H,F/32,18] uint8, sh_* the shared expert or None."""

    def __init__(self, hidden, ffn, n_experts, top_k, w_router, router_bias, w_gate, w_up, w_down,
                 sh_gate=None, sh_up=None, sh_down=None):
        self.hidden, self.ffn, self.n_experts, self.top_k = int(hidden), int(ffn), int(n_experts), int(top_k)
        self.tensors = dict(w_router=w_router, router_bias=router_bias, w_gate=w_gate, w_up=w_up,
                            w_down=w_down, sh_gate=sh_gate, sh_up=sh_up, sh_down=sh_down)
        for k, v in self.tensors.items():
            if v is not None and not v.is_contiguous():
                raise ValueError(f"{k} must be contiguous")
        self.has_shared = sh_gate is not None
        self.struct = _Layer(self.hidden, self.ffn, self.n_experts, self.top_k, int(self.has_shared),
                             *(None if v is None else v.data_ptr() for v in self.tensors.values()))

    @property
    def ref(self):
        return ctypes.byref(self.struct)

    @classmethod
    def from_host(cls, w, device="cuda"):
        """From an object with numpy attributes (hidden, ffn, n_experts, top_k,
        w_router, router_bias, w_gate, w_up, w_down, sh_gate, sh_up, sh_down)."""
        def dev(a):
            return None if a is None else torch.from_numpy(a).to(device).contiguous()
        return cls(w.hidden, w.ffn, w.n_experts, w.top_k, dev(w.w_router), dev(w.router_bias),
                   dev(w.w_gate), dev(w.w_up), dev(w.w_down), dev(w.sh_gate), dev(w.sh_up), dev(w.sh_down))

    @classmethod
    def from_host_pinned(cls, w, device="cuda"):
        """Router weights on the device, expert matrices in page-locked host
        memory (for moe_q4_ffn_forward_streamed)."""
        def dev(a):
            return None if a is None else torch.from_numpy(a).to(device).contiguous()

        def pinned(a):
            return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).pin_memory()
        return cls(w.hidden, w.ffn, w.n_experts, w.top_k, dev(w.w_router), dev(w.router_bias),
                   pinned(w.w_gate), pinned(w.w_up), pinned(w.w_down), pinned(w.sh_gate), pinned(w.sh_up),
                   pinned(w.sh_down))

    def replica(self):
        """A copy of every weight tensor at new device addresses."""
        t = {k: (None if v is None else v.clone()) for k, v in self.tensors.items()}
        return Layer(self.hidden, self.ffn, self.n_experts, self.top_k, **t)


def moe_q4_quantize_act(x: torch.Tensor, q=None, d=None, status=None, stream=None):
    T, H = x.shape
    q = _result(stream, torch.empty, (T, H), dtype=torch.int8, device=x.device) if q is None else q
    d = _result(stream, torch.empty, (T, H // QK), dtype=torch.int16, device=x.device) if d is None else d
    _check(_lib.moe_q4_quantize_act(_p(x), T, H, _p(q), _p(d), _p(status), _stream(stream)), "moe_q4_quantize_act")
    return q, d


def moe_q4_route(layer: Layer, x: torch.Tensor, topk_idx=None, topk_w=None, logits=None, stream=None):
    T = x.shape[0]
    k, E = layer.top_k, layer.n_experts
    topk_idx = _result(stream, torch.empty, (T, k), dtype=torch.int32, device=x.device) if topk_idx is None else topk_idx
    topk_w = _result(stream, torch.empty, (T, k), dtype=torch.float32, device=x.device) if topk_w is None else topk_w
    logits = _result(stream, torch.empty, (T, E), dtype=torch.float32, device=x.device) if logits is None else logits
    _check(_lib.moe_q4_route(layer.ref, _p(x), T, _p(topk_idx), _p(topk_w), _p(logits), _stream(stream)),
           "moe_q4_route")
    return topk_idx, topk_w, logits


def moe_q4_ffn_workspace_bytes(layer: Layer, T_max: int) -> int:
    return int(_lib.moe_q4_ffn_workspace_bytes(layer.ref, int(T_max)))


def moe_q4_ffn_host_workspace_bytes(layer: Layer, T_max: int) -> int:
    return int(_lib.moe_q4_ffn_host_workspace_bytes(layer.ref, int(T_max)))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte aligned uint8 device buffer (torch's allocator aligns to 512)."""
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def moe_q4_ffn_forward(layer: Layer, x: torch.Tensor, y=None, workspace=None, stream=None):
    T = x.shape[0]
    y = _result(stream, torch.empty_like, x) if y is None else y
    if workspace is None:
        workspace = _scratch(stream, alloc_workspace, moe_q4_ffn_workspace_bytes(layer, T), x.device)
    _check(_lib.moe_q4_ffn_forward(layer.ref, _p(x), T, _p(y), _p(workspace), workspace.numel(),
                                   _stream(stream)), "moe_q4_ffn_forward")
    return y


def moe_q4_ffn_forward_debug(layer: Layer, x: torch.Tensor, y, workspace, h_out=None, path=PATH_AUTO,
                             ev_start=None, ev_stop=None, stream=None, force_spin_timeout=False,
                             block_dots=None, decode_kernel_ns=None):
    """block_dots: None or (out int32 tensor, down (bool), group, row block):
    capture the per-block integer dot products of that row block (see
    moe_q4_debug in include/moe_q4.h for the layout)."""
    T = x.shape[0]
    bd_out, bd_down, bd_group, bd_rb = (None, 0, 0, 0) if block_dots is None else block_dots
    dbg = _Debug(None if h_out is None else h_out.data_ptr(), int(path),
                 None if ev_start is None else ev_start.cuda_event,
                 None if ev_stop is None else ev_stop.cuda_event, int(bool(force_spin_timeout)),
                 None if bd_out is None else bd_out.data_ptr(), int(bool(bd_down)), int(bd_group), int(bd_rb),
                 None if decode_kernel_ns is None else decode_kernel_ns.data_ptr())
    _check(_lib.moe_q4_ffn_forward_debug(layer.ref, _p(x), T, _p(y), _p(workspace), workspace.numel(),
                                         ctypes.byref(dbg), _stream(stream)), "moe_q4_ffn_forward_debug")
    return y


def moe_q4_ffn_forward_host(layer: Layer, x_host: torch.Tensor, y_host: torch.Tensor, workspace, stream=None):
    """x_host/y_host: CPU tensors (pinned for asynchronous copies)."""
    T = x_host.shape[0]
    _check(_lib.moe_q4_ffn_forward_host(layer.ref, _p(x_host), T, _p(y_host), _p(workspace), workspace.numel(),
                                        _stream(stream)), "moe_q4_ffn_forward_host")
    return y_host


def moe_q4_workspace_layout(layer: Layer, T: int) -> dict:
    arr = (ctypes.c_size_t * len(WS_NAMES))()
    _check(_lib.moe_q4_workspace_layout(layer.ref, int(T), arr, len(WS_NAMES)), "moe_q4_workspace_layout")
    return dict(zip(WS_NAMES, list(arr)))


def workspace_views(layer: Layer, T: int, ws: torch.Tensor) -> dict:
    """Typed views of the intermediates inside a forward workspace (for tests)."""
    off = moe_q4_workspace_layout(layer, T)
    E, k, H, F = layer.n_experts, layer.top_k, layer.hidden, layer.ffn
    P = T * k
    slots = P + (T if layer.has_shared else 0)

    def v(name, dtype, shape):
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return ws[off[name]:off[name] + nbytes].view(dtype).view(*shape)

    return dict(
        status=v("status", torch.int32, (4,)), logits=v("logits", torch.float32, (T, E)),
        topk_idx=v("topk_idx", torch.int32, (T, k)), topk_w=v("topk_w", torch.float32, (T, k)),
        qa=v("qa", torch.int8, (T, H)), da=v("da", torch.int16, (T, H // QK)),
        cnt=v("cnt", torch.int32, (E + 1,)), off=v("off", torch.int32, (E + 2,)),
        tile_off=v("tile_off", torch.int32, (E + 2,)), sorted=v("sorted", torch.int32, (P,)),
        pos=v("pos", torch.int32, (P,)), hq=v("hq", torch.int8, (slots, F)),
        dh=v("dh", torch.int16, (slots, F // QK)))


def moe_q4_block_dots(w_blocks: torch.Tensor, qa: torch.Tensor, out=None, stream=None):
    n = w_blocks.numel() // Q4_BYTES
    out = _result(stream, torch.empty, n, dtype=torch.int32, device=w_blocks.device) if out is None else out
    _check(_lib.moe_q4_block_dots(_p(w_blocks), _p(qa), n, _p(out), _stream(stream)), "moe_q4_block_dots")
    return out


def moe_q4_rescale_ceiling(int8_operands: bool, iters: int, sink: torch.Tensor, stream=None) -> int:
    """Launch the epilogue-rescale measurement kernel (include/moe_q4.h) on
    `stream`; returns the number of accumulator elements it rescales (each
    one 32 int8 multiply-adds).  sink: a device float32 tensor of >= 1."""
    n = ctypes.c_int64(0)
    _check(_lib.moe_q4_rescale_ceiling(int(bool(int8_operands)), int(iters), _p(sink), ctypes.byref(n),
                                       _stream(stream)), "moe_q4_rescale_ceiling")
    return n.value


def moe_q4_ffn_forward_noalloc(layer: Layer, x: torch.Tensor, y=None, stream=None):
    """The layer with the library's static device scratch instead of a
    caller workspace (for callers that cannot allocate device memory; see
    include/moe_q4.h).  Calls that overlap on the GPU race on the scratch."""
    T = x.shape[0]
    y = _result(stream, torch.empty_like, x) if y is None else y
    _check(_lib.moe_q4_ffn_forward_noalloc(layer.ref, _p(x), T, _p(y), _stream(stream)),
           "moe_q4_ffn_forward_noalloc")
    return y


# ---------------------------------------------------------------- stacks of layers

def moe_q4_residual_rmsnorm(x: torch.Tensor, y=None, eps: float = 1e-6, xn=None, stream=None):
    """x <- x + y (if y is given, in place), then returns xn = RMSNorm(x) (unit
    gain over the last dimension), written into `xn` if given."""
    T, H = x.shape
    xn = _result(stream, torch.empty_like, x) if xn is None else xn
    _check(_lib.moe_q4_residual_rmsnorm(_p(x), _p(y), T, H, float(eps), _p(xn), _stream(stream)),
           "moe_q4_residual_rmsnorm")
    return xn


def moe_q4_stack_workspace_bytes(layer: Layer, T_max: int) -> int:
    return int(_lib.moe_q4_stack_workspace_bytes(layer.ref, int(T_max)))


def moe_q4_stack_forward(layers, x: torch.Tensor, eps: float = 1e-6, workspace=None, stream=None):
    """x <- x + MoE_l(RMSNorm(x)) for every layer in order, in place on x."""
    T = x.shape[0]
    arr = (_Layer * len(layers))(*[l.struct for l in layers])
    if workspace is None:
        workspace = _scratch(stream, alloc_workspace, moe_q4_stack_workspace_bytes(layers[0], T), x.device)
    _check(_lib.moe_q4_stack_forward(arr, len(layers), _p(x), T, float(eps), _p(workspace), workspace.numel(),
                                     _stream(stream)), "moe_q4_stack_forward")
    return x


# ---------------------------------------------------------------- LM-head GEMV

def moe_q4_gemv_workspace_bytes(T: int, H: int) -> int:
    return int(_lib.moe_q4_gemv_workspace_bytes(int(T), int(H)))


def moe_q4_gemv(W: torch.Tensor, x: torch.Tensor, y=None, workspace=None, stream=None):
    """y [T, N] = W4A8 product of the Q4_0 matrix W [N, H/32, 18] (uint8) with
    the Q8_0 form of x [T, H] (T <= 8)."""
    T, H = x.shape
    N = W.shape[0]
    y = _result(stream, torch.empty, (T, N), dtype=torch.float32, device=x.device) if y is None else y
    if workspace is None:
        workspace = _scratch(stream, alloc_workspace, moe_q4_gemv_workspace_bytes(T, H), x.device)
    _check(_lib.moe_q4_gemv(_p(W), N, H, _p(x), T, _p(y), _p(workspace), workspace.numel(), _stream(stream)),
           "moe_q4_gemv")
    return y


# ---------------------------------------------------------------- per-request operators around the projections

def _rows(t: torch.Tensor, name: str, device: int, rows: int, cols: int) -> int:
    """The row pitch of a [rows, cols] fp32 tensor on a GPU with contiguous rows."""
    if t.dtype is not torch.float32 or t.get_device() != device or t.shape != (rows, cols):
        raise ValueError(f"{name} must be a ({rows}, {cols}) float32 tensor on GPU {device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return pitch if rows > 1 else cols  # (of a single row it does not matter)


def _vector(t, name: str, device: int, dtype, n=None):
    """The address of a contiguous 1D tensor (of n elements) on a GPU, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1D {dtype} tensor on GPU {device}")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    return t.data_ptr()


def _call(f, what: str, device: int, stream, *args):
    """f(*args, stream) with `device` current; stream None: its current one.
    (A tensor on it has initialised CUDA.)"""
    if torch._C._cuda_getDevice() != device:
        with torch.cuda.device(device):
            return _call(f, what, device, stream, *args)
    rc = f(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream)
    if rc != MOE_Q4_OK:
        raise MoeQ4Error(rc, what)


class Adapters:
    """Low-rank adapters on the device and their C descriptor.

    a [n, r, H] and b [n, N, r] (both float32, float16 or bfloat16,
    contiguous), scale [n] float32 or None (1).  Adapter i adds
    scale[i] * b[i] (a[i] x) to a projection of x."""

    _DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: Optional[torch.Tensor] = None):
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError("a must be [n, r, H] and b [n, N, r]")
        if a.dtype not in self._DTYPES or a.dtype != b.dtype or a.device != b.device:
            raise ValueError("a and b must be float32, float16 or bfloat16, alike, on one device")
        if not a.is_cuda or not a.is_contiguous() or not b.is_contiguous():
            raise ValueError("a and b must be contiguous, on a GPU")
        self.a, self.b, self.scale, self.device = a, b, scale, a.get_device()
        self.n_adapters, self.rank, self.hidden = a.shape
        self.n_out = b.shape[1]
        self.struct = _Adapters(self.hidden, self.rank, self.n_out, self.n_adapters, self._DTYPES[a.dtype],
                                a.data_ptr(), b.data_ptr(),
                                _vector(scale, "scale", self.device, torch.float32, self.n_adapters))

    @property
    def ref(self):
        return ctypes.byref(self.struct)


def moe_q4_adapters_workspace_bytes(adapters: Adapters, T_max: int) -> int:
    return int(_lib.moe_q4_adapters_workspace_bytes(adapters.ref, int(T_max)))


def moe_q4_adapters_apply(adapters: Adapters, x: torch.Tensor, adapter: torch.Tensor, base=None, y=None,
                          workspace=None, stream=None):
    """y[t] = base[t] + scale[e] * b[e] (a[e] x[t]) with e = adapter[t] (int32;
    -1: y[t] = base[t]).  base None: zeros; y may be base (in place).  x, base
    and y may be column slices of wider buffers (contiguous rows)."""
    dev = adapters.device
    T, N = x.shape[0], adapters.n_out
    ldx = _rows(x, "x", dev, T, adapters.hidden)
    ids = _vector(adapter, "adapter", dev, torch.int32, T)
    if y is None:
        y = _result(stream, torch.empty, (T, N), dtype=torch.float32, device=x.device)
    ldy = _rows(y, "y", dev, T, N)
    pbase, ldb = (None, 0) if base is None else (base.data_ptr(), _rows(base, "base", dev, T, N))
    if workspace is None:
        workspace = _scratch(stream, alloc_workspace, moe_q4_adapters_workspace_bytes(adapters, T), x.device)
    elif workspace.get_device() != dev or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on GPU {dev}")
    _call(_lib.moe_q4_adapters_apply, "moe_q4_adapters_apply", dev, stream, adapters.ref, x.data_ptr(), ldx, ids, T,
          pbase, ldb, y.data_ptr(), ldy, workspace.data_ptr(), workspace.numel())
    return y


class LogitRules:
    """What each row of a batch of logits is ruled by (see moe_q4_logit_rules
    in include/moe_q4.h); every part may be left out.

    tokens int32 [n], row_start int64 [T+1], generated_start int64 [T]: the
    rows' histories; repetition, presence, frequency float32 [T];
    bias_token int32 [m], bias_value float32 [m], bias_start int64 [T+1];
    mask int32 [n_masks, ceil(vocab/32)] (a bit per token, set: allowed),
    mask_row int32 [T] (-1: no mask) or None (mask t for row t)."""

    def __init__(self, tokens=None, row_start=None, generated_start=None, repetition=None, presence=None,
                 frequency=None, bias_token=None, bias_value=None, bias_start=None, mask=None, mask_row=None):
        if (tokens is None) != (row_start is None):
            raise ValueError("tokens and row_start belong together")
        if not (bias_token is None) == (bias_value is None) == (bias_start is None):
            raise ValueError("bias_token, bias_value and bias_start belong together")
        self.tokens, self.row_start, self.generated_start = tokens, row_start, generated_start
        self.repetition, self.presence, self.frequency = repetition, presence, frequency
        self.bias_token, self.bias_value, self.bias_start = bias_token, bias_value, bias_start
        self.mask, self.mask_row = mask, mask_row

    def struct(self, T: int, V: int, device: int) -> bytes:
        """The C descriptor for T rows of V logits on a GPU."""
        i32, i64, f32 = torch.int32, torch.int64, torch.float32
        tokens = row_start = generated = rep = pres = freq = n_tokens = 0
        bias_token = bias_value = bias_start = n_bias = masks = mask_row = n_masks = 0
        if self.tokens is not None:
            tokens = _vector(self.tokens, "tokens", device, i32)
            n_tokens = self.tokens.shape[0]
            row_start = _vector(self.row_start, "row_start", device, i64, T + 1)
        if self.generated_start is not None:
            generated = _vector(self.generated_start, "generated_start", device, i64, T)
        if self.repetition is not None:
            rep = _vector(self.repetition, "repetition", device, f32, T)
        if self.presence is not None:
            pres = _vector(self.presence, "presence", device, f32, T)
        if self.frequency is not None:
            freq = _vector(self.frequency, "frequency", device, f32, T)
        if self.bias_token is not None:
            bias_token = _vector(self.bias_token, "bias_token", device, i32)
            n_bias = self.bias_token.shape[0]
            bias_value = _vector(self.bias_value, "bias_value", device, f32, n_bias)
            bias_start = _vector(self.bias_start, "bias_start", device, i64, T + 1)
        mask = self.mask
        if mask is not None:
            if (mask.dtype is not i32 or mask.dim() != 2 or mask.shape[1] != (V + 31) // 32 or
                    mask.get_device() != device or not mask.is_contiguous()):
                raise ValueError(f"mask must be a contiguous [n_masks, {(V + 31) // 32}] int32 tensor on GPU {device}")
            masks, n_masks = mask.data_ptr(), mask.shape[0]
            if n_masks < 1 and T > 0:  # (an empty tensor has no address: it would count as no mask)
                raise ValueError("mask has no rows")
        if self.mask_row is not None:
            mask_row = _vector(self.mask_row, "mask_row", device, i32, T)
        return _pack_rules(V, tokens, n_tokens, row_start, generated, rep, pres, freq, bias_token, bias_value, n_bias,
                           bias_start, masks, n_masks, mask_row)


def moe_q4_logits_apply(rules: LogitRules, logits: torch.Tensor, out=None, token=None, lse=None, status=None,
                        stream=None):
    """Rules the logits [T, V] (fp32).  Writes the outputs that are given: out
    [T, V] fp32 (the processed logits; may be `logits`), token [T] int32 (the
    greedy token, -1 where nothing is left), lse [T] fp32 (log-sum-exp); with
    none given, a new out.  Returns (out, token, lse)."""
    if not logits.is_cuda or logits.dim() != 2:
        raise ValueError("logits must be a 2D tensor on a GPU")
    T, V = logits.shape
    dev = logits.get_device()
    ld = _rows(logits, "logits", dev, T, V)
    if out is None and token is None and lse is None:
        out = _result(stream, torch.empty, (T, V), dtype=torch.float32, device=logits.device)
    pout, ldo = (None, 0) if out is None else (out.data_ptr(), _rows(out, "out", dev, T, V))
    _call(_lib.moe_q4_logits_apply, "moe_q4_logits_apply", dev, stream, rules.struct(T, V, dev),
          logits.data_ptr(), ld, T, pout, ldo, _vector(token, "token", dev, torch.int32, T),
          _vector(lse, "lse", dev, torch.float32, T), _vector(status, "status", dev, torch.int32, 1))
    return out, token, lse


# ---------------------------------------------------------------- host-streamed experts

def moe_q4_staging_bytes(layer: Layer) -> int:
    return int(_lib.moe_q4_staging_bytes(layer.ref))


def moe_q4_ffn_forward_streamed(layer: Layer, x: torch.Tensor, y=None, workspace=None, staging=None, stream=None):
    """The layer with its expert matrices in page-locked host memory (see
    Layer.from_host_pinned): the experts the routing selects are copied into
    `staging` on the device, then the layer runs there."""
    T = x.shape[0]
    y = _result(stream, torch.empty_like, x) if y is None else y
    if workspace is None:
        workspace = _scratch(stream, alloc_workspace, moe_q4_ffn_workspace_bytes(layer, T), x.device)
    if staging is None:
        staging = _scratch(stream, alloc_workspace, moe_q4_staging_bytes(layer), x.device)
    _check(_lib.moe_q4_ffn_forward_streamed(layer.ref, _p(x), T, _p(y), _p(workspace), workspace.numel(),
                                            _p(staging), staging.numel(), _stream(stream)),
           "moe_q4_ffn_forward_streamed")
    return y


def moe_q4_test_override_device(enable: bool, major: int = 10, minor: int = 0) -> None:
    """Test hook: make every entry point see the current device as compute
    capability major.minor (enable=True) or query the driver again (False)."""
    _check(_lib.moe_q4_test_override_device(int(bool(enable)), int(major), int(minor)),
           "moe_q4_test_override_device")
