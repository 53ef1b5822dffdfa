"""What an entry point of the binding allocates belongs to the stream it runs on.

torch's allocator hands a freed block out again in the order of the stream it
was allocated on.  A workspace that a call makes for itself is freed when the
call returns, while its kernels may still be waiting on another stream; so with
`stream` given, everything that a call makes is made on that stream, and what
it returns is also marked as used by the caller's current one.  Host logic
only: the library and torch's CUDA calls are stand-ins here.
"""
import contextlib
import types

import pytest
import torch

import quantized_moe_q4_b200 as m


class OnGpu(torch.Tensor):
    """A host tensor that passes for one on a GPU and keeps what is done to it."""
    is_cuda = True

    def record_stream(self, s):
        self.used_by = getattr(self, "used_by", []) + [s]


@pytest.fixture
def calls(monkeypatch):
    """Stand-ins; `made` lists (stream current when it was made, tensor)."""
    state = types.SimpleNamespace(on="current", made=[])

    @contextlib.contextmanager
    def stream(s):
        before, state.on = state.on, state.on if s is None else s
        yield
        state.on = before

    def noted(f):
        def make(*a, **kw):
            t = f(*a, **{k: v for k, v in kw.items() if k != "device"}).as_subclass(OnGpu)
            state.made.append((state.on, t))
            return t
        return make

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 256 if name.endswith("_bytes") else 0

    def alloc(nbytes, device=None):
        return noted(torch.zeros)(int(nbytes), dtype=torch.uint8)

    zeros = torch.zeros
    monkeypatch.setattr(torch, "empty", noted(zeros))
    monkeypatch.setattr(torch, "empty_like", noted(torch.zeros_like))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.on)
    monkeypatch.setattr(m, "alloc_workspace", alloc)
    monkeypatch.setattr(m, "_lib", Lib())
    monkeypatch.setattr(m, "_stream", lambda s: s)
    monkeypatch.setattr(m, "_call", lambda f, what, device, s, *a: None)
    return state


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


class FakeLayer:
    hidden, ffn, n_experts, top_k, has_shared = 64, 32, 4, 2, False
    ref = None
    struct = m._Layer()


def adapters():
    A = object.__new__(m.Adapters)
    A.a = A.b = A.scale = None
    A.device, A.n_adapters, A.rank, A.hidden, A.n_out, A.struct = -1, 2, 8, 64, 10, m._Adapters()
    return A


ENTRIES = {
    "quantize_act": (2, lambda s: m.moe_q4_quantize_act(gpu(3, 64), stream=s)),
    "route": (3, lambda s: m.moe_q4_route(FakeLayer, gpu(3, 64), stream=s)),
    "ffn_forward": (2, lambda s: m.moe_q4_ffn_forward(FakeLayer, gpu(3, 64), stream=s)),
    "ffn_forward_noalloc": (1, lambda s: m.moe_q4_ffn_forward_noalloc(FakeLayer, gpu(3, 64), stream=s)),
    "ffn_forward_streamed": (3, lambda s: m.moe_q4_ffn_forward_streamed(FakeLayer, gpu(3, 64), stream=s)),
    "block_dots": (1, lambda s: m.moe_q4_block_dots(gpu(5, 18, dtype=torch.uint8), gpu(5, 32, dtype=torch.int8), stream=s)),
    "residual_rmsnorm": (1, lambda s: m.moe_q4_residual_rmsnorm(gpu(3, 64), stream=s)),
    "stack_forward": (1, lambda s: m.moe_q4_stack_forward([FakeLayer], gpu(3, 64), stream=s)),
    "gemv": (2, lambda s: m.moe_q4_gemv(gpu(7, 2, 18, dtype=torch.uint8), gpu(3, 64), stream=s)),
    "adapters_apply": (2, lambda s: m.moe_q4_adapters_apply(adapters(), gpu(3, 64), gpu(3, dtype=torch.int32), stream=s)),
    "logits_apply": (1, lambda s: m.moe_q4_logits_apply(m.LogitRules(), gpu(3, 50), stream=s)),
}


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_allocates_on_its_stream(calls, name):
    n, call = ENTRIES[name]
    got = call("s")
    assert len(calls.made) == n
    assert [on for on, _ in calls.made] == ["s"] * n and calls.on == "current"
    for t in got if isinstance(got, tuple) else (got,):
        if any(t is u for _, u in calls.made):   # returned: the caller's stream may use it as well
            assert t.used_by == ["current"]


@pytest.mark.parametrize("name", ENTRIES)
def test_without_a_stream_the_current_one_is_it(calls, name):
    n, call = ENTRIES[name]
    call(None)
    assert [on for on, _ in calls.made] == ["current"] * n
    assert not any(hasattr(t, "used_by") for _, t in calls.made)
