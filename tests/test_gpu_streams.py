"""Calls on a stream that is not the current one, with outputs and workspaces
that the calls make themselves: the stream is still busy when a call returns,
and the current stream allocates and fills memory meanwhile."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_moe_q4_b200 as m  # noqa: E402


def adapters(T):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    kw = dict(device="cuda", generator=g)
    A = m.Adapters(torch.randn(7, 16, 512, **kw).bfloat16(), torch.randn(7, 300, 16, **kw).bfloat16())
    x, ids = torch.randn(T, 512, **kw), torch.randint(-1, 7, (T,), **kw).int()
    return lambda s: m.moe_q4_adapters_apply(A, x, ids, stream=s)


def logits():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    l, rep = torch.randn(16, 5000, device="cuda", generator=g), torch.full((16,), 1.5, device="cuda")
    tokens = torch.randint(0, 5000, (16 * 40,), device="cuda", generator=g).int()
    R = m.LogitRules(tokens=tokens, row_start=torch.arange(17, device="cuda") * 40, repetition=rep)
    return lambda s: m.moe_q4_logits_apply(R, l, stream=s)[0]


def gemv():
    import numpy as np
    W = torch.from_numpy(synth._q4_0_matrix(np.random.Generator(np.random.PCG64(5)), 3001, 512 // 32)).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(8, 512, device="cuda", generator=g)
    return lambda s: m.moe_q4_gemv(W, x, stream=s)


def layer():
    x, lw = synth.random_layer(seed=9, H=512, F=256, E=16, k=4, shared=True, T=100)
    L, xd = m.Layer.from_host(lw), torch.from_numpy(x).cuda()
    return lambda s: m.moe_q4_ffn_forward(L, xd, stream=s)


CALLS = {"adapters-4": lambda: adapters(4), "adapters-300": lambda: adapters(300), "adapters-5000": lambda: adapters(5000),
         "logits": logits, "gemv": gemv, "layer": layer}


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_is_not_handed_out_while_its_stream_is_busy(name, monkeypatch):
    call = CALLS[name]()
    want = call(None)
    s = torch.cuda.Stream()
    call(s)                          # (both streams have had their first blocks)
    torch.cuda.synchronize()
    made = []
    alloc = m.alloc_workspace

    def noted(nbytes, device="cuda"):
        ws = alloc(nbytes, device)
        made.append((ws.data_ptr(), ws.numel()))
        return ws

    monkeypatch.setattr(m, "alloc_workspace", noted)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)   # about 10 ms
    y = call(s)
    made.append((y.data_ptr(), y.numel() * 4))
    # the current stream takes blocks of these sizes and fills them at once
    mine = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _, n in made for _ in range(8)]
    for p, n in made:
        assert all(t.data_ptr() + t.numel() <= p or p + n <= t.data_ptr() for t in mine)
    torch.cuda.current_stream().wait_stream(s)
    if name == "layer":
        # The layer adds its k + 1 = 5 expert outputs a row in no fixed order: two
        # orders are at most 2 * 4 * 2^-24 = 4.8e-7 of the sum of their magnitudes
        # apart, under 1e-5 of the row's scale for outputs of up to 20 times it.
        assert bool(((y - want).abs() <= 1e-5 * want.square().mean(1, keepdim=True).sqrt()).all())
    else:
        assert torch.equal(y, want)
    torch.cuda.synchronize()


def test_a_result_let_go_of_on_the_current_stream_is_not_overwritten_by_the_next_call():
    call = adapters(300)
    want = call(None)
    s = torch.cuda.Stream()
    call(s)
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    y = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)       # the current stream reads y late
    kept, at = y.clone(), y.data_ptr()
    del y
    z = call(s)
    assert z.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and torch.equal(z, want)


@pytest.mark.parametrize("T", [8, 300, 1500, 9000])
def test_calls_on_two_streams_at_once(T):
    """Two adapter calls and logit rules in flight together, each with a workspace of its own."""
    calls = [adapters(T), adapters(T + 1), logits()]
    want = [c(None) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for _ in range(10):
        for c, s, g in zip(calls, streams, got):
            g.append(c(s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(y, w) for y in g)
