"""Low-rank adapters of many requests (moe_q4_adapters_apply) against the
formula in binary64:  y[t] = base[t] + scale[e] * B_e (A_e x[t]).

Tolerance.  With u = 2^-24, a sum of products computed in binary32 is off by
at most c * u * (sum of the products' magnitudes), where c counts the
roundings a term passes through.  Rows kernel: a lane adds H/32 products, 5
shuffles join the lanes, up to 8 parts join, r products follow, then the
scale and the base: H/32 + r + 16.  Tile kernel: x, A x and binary32 weights as
two tf32 parts of 11 bits (2^-21 = 8 u, each once, so 24 u, and 4 u for the
product of two lo parts that is left out), H/8 accumulations of 8-wide steps
spread over the CTAs and accumulators, each truncated (2 u) -- at most 40 in a
row --, up to 16 accumulators and 8 parts joined, then r/8 accumulations again.
Both are under C = H/16 + 2 r + 64 times u S, with S = |base| + |scale| sum_k
|B_k| sum_h |A_kh x_h|.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_moe_q4_b200 as m  # noqa: E402

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def make(seed, T, H, N, r, n, kind, ids="mixed", pad=0, scale=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kw = dict(device="cuda", generator=g)
    x = torch.randn(T, H + pad, **kw)[:, :H]
    base = torch.randn(T, N + pad, **kw)[:, :N]
    a = (torch.randn(n, r, H, **kw) / H ** 0.5).to(TYPES[kind])
    b = (torch.randn(n, N, r, **kw) * 0.1).to(TYPES[kind])
    sc = torch.rand(n, **kw) * 4 - 2 if scale else None
    if isinstance(ids, str):
        if ids == "mixed":
            e = torch.randint(-1, n, (T,), **kw)
        elif ids == "one":
            e = torch.full((T,), n - 1, device="cuda")
        elif ids == "none":
            e = torch.full((T,), -1, device="cuda")
        else:  # runs
            e = torch.arange(T, device="cuda") * (n + 1) // T - 1
    else:
        e = torch.as_tensor(ids, device="cuda")
    return m.Adapters(a, b, sc), x, e.to(torch.int32), base


def expected(A, x, e, base):
    """(y, S) in binary64."""
    T, N = x.shape[0], A.n_out
    y = torch.zeros(T, N, dtype=torch.float64, device="cuda") if base is None else base.double().clone()
    S = y.abs()
    for i in range(A.n_adapters):
        at = torch.nonzero(e == i)[:, 0]
        if at.numel() == 0:
            continue
        a, b, xi = A.a[i].double(), A.b[i].double(), x[at].double()
        s = 1.0 if A.scale is None else float(A.scale[i])
        y[at] += s * ((xi @ a.t()) @ b.t())
        S[at] += abs(s) * ((xi.abs() @ a.abs().t()) @ b.abs().t())
    return y, S


def check(A, x, e, base, y):
    ref, S = expected(A, x, e, base)
    C = A.hidden / 16 + 2 * A.rank + 64
    bad = (y.double() - ref).abs() > C * U * S
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}"
    lone = torch.nonzero((e < 0) | (e >= A.n_adapters))[:, 0]   # rows without an adapter: the base, bit for bit
    assert torch.equal(y[lone], torch.zeros_like(y[lone]) if base is None else base[lone])


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,H,N,r,n,ids", [
    (1, 2048, 2048, 16, 4, "one"), (1, 256, 1, 8, 1, "one"), (1, 512, 33, 8, 3, "none"), (2, 768, 2049, 24, 2, "mixed"),
    (8, 2048, 5000, 128, 8, "mixed"), (9, 1024, 700, 40, 1, "one"), (63, 2048, 1001, 64, 5, "mixed"),
    (64, 512, 300, 56, 64, "mixed"), (65, 512, 300, 56, 64, "mixed"), (127, 1280, 257, 120, 2, "runs"),
    (129, 2560, 130, 96, 1, "one"), (255, 256, 40, 16, 300, "mixed"), (256, 768, 100, 8, 3, "mixed"), (257, 768, 100, 8, 3, "mixed"),
    (256, 512, 33, 24, 1, "one"), (257, 512, 33, 24, 200, "mixed"), (300, 2048, 1000, 32, 1000, "mixed"), (513, 256, 129, 8, 3, "runs"),
    (947, 2048, 2048, 64, 4, "runs"), (1100, 768, 1001, 128, 2, "mixed"), (2000, 1024, 640, 16, 1024, "mixed"),
    # tiles in clusters of 8, 4, 2 and 1, one adapter or several, ranks with one to four panels
    (1500, 512, 1500, 8, 2, "mixed"), (3000, 512, 300, 40, 2, "mixed"), (3000, 1024, 129, 128, 2, "runs"),
    (7000, 512, 130, 64, 3, "runs"), (7000, 256, 1000, 96, 1, "one"), (18000, 512, 260, 16, 4, "mixed"),
    (18000, 256, 64, 120, 1, "one"),
    # sums too long for the tensor core's accumulators: the rows kernel, however many rows
    (700, 16384, 100, 128, 1, "one"), (500, 16384, 100, 64, 2, "mixed")])
def test_adapters_match_the_formula(kind, T, H, N, r, n, ids):
    A, x, e, base = make(T + N, T, H, N, r, n, kind, ids)
    check(A, x, e, base, m.moe_q4_adapters_apply(A, x, e, base=base))


@pytest.mark.parametrize("T,n", [(2049, 3), (20000, 7), (40000, 1024), (131073, 5), (140000, 1023)])
def test_many_rows_in_several_grouping_chunks(T, n):
    A, x, e, base = make(T, T, 256, 24, 8, n, "bf16", "mixed")
    check(A, x, e, base, m.moe_q4_adapters_apply(A, x, e, base=base))


@pytest.mark.parametrize("T", [5, 100, 1500])
def test_pitches_in_place_no_base_no_scale(T):
    A, x, e, base = make(3, T, 512, 301, 16, 3, "bf16", "mixed", pad=8, scale=False)
    # outputs in a wider buffer: its other columns stay as they were
    buf = torch.full((T, 310), 7.0, device="cuda")
    y = m.moe_q4_adapters_apply(A, x, e, base=base, y=buf[:, 3:304])
    check(A, x, e, base, y)
    assert bool((buf[:, :3] == 7).all()) and bool((buf[:, 304:] == 7).all())
    # in place, in that buffer
    buf[:, 3:304] = base
    m.moe_q4_adapters_apply(A, x, e, base=buf[:, 3:304], y=buf[:, 3:304])
    assert torch.equal(buf[:, 3:304], y)
    assert bool((buf[:, :3] == 7).all()) and bool((buf[:, 304:] == 7).all())
    # no base
    check(A, x, e, None, m.moe_q4_adapters_apply(A, x, e))
    # x and y as column ranges of one buffer
    both = torch.zeros(T, 512 + 304, device="cuda")
    both[:, :512] = x
    m.moe_q4_adapters_apply(A, both[:, :512], e, base=base, y=both[:, 512:813])
    assert torch.equal(both[:, 512:813], y) and bool((both[:, 813:] == 0).all())


@pytest.mark.parametrize("T", [7, 64, 200, 1000, 5000, 140000])
def test_bad_indices_are_reported_and_count_as_none(T):
    A, x, e, base = make(5, T, 256, 100, 8, 3, "fp16", "mixed")
    ws = m.alloc_workspace(m.moe_q4_adapters_workspace_bytes(A, T))
    ws.fill_(255)
    m.moe_q4_adapters_apply(A, x, e, base=base, workspace=ws)
    assert int(ws[:4].view(torch.int32)) == 0
    bad = e.clone()
    bad[T // 2], bad[T - 1], bad[0] = 3, -2, 2 ** 31 - 1
    y = m.moe_q4_adapters_apply(A, x, bad, base=base, workspace=ws)
    assert int(ws[:4].view(torch.int32)) == m.STATUS_BAD_ADAPTER_INDEX
    check(A, x, bad, base, y)
    m.moe_q4_adapters_apply(A, x, e, base=base, workspace=ws)   # the next call starts from a clear word
    assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("T", [1, 40, 300, 2000])
def test_same_call_same_bits_and_rows_are_independent(T):
    A, x, e, base = make(11, T, 1024, 257, 32, 4, "bf16", "mixed")
    y = m.moe_q4_adapters_apply(A, x, e, base=base)
    for _ in range(3):
        assert torch.equal(m.moe_q4_adapters_apply(A, x, e, base=base), y)
    p = torch.randperm(T, device="cuda")   # the same rows in another order
    z = m.moe_q4_adapters_apply(A, x[p].contiguous(), e[p].contiguous(), base=base[p].contiguous())
    assert torch.equal(z, y[p])
    # a row that overflows stays alone with it
    x2 = x.clone()
    x2[T // 2] = 3e38
    z = m.moe_q4_adapters_apply(A, x2, e, base=base)
    keep = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("T", [3, 90, 1300])
def test_captured_and_on_another_stream(T):
    A, x, e, base = make(13, T, 512, 400, 16, 3, "fp16", "mixed")
    want = m.moe_q4_adapters_apply(A, x, e, base=base)
    ws = m.alloc_workspace(m.moe_q4_adapters_workspace_bytes(A, T))
    y1, y2 = torch.empty_like(want), torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.moe_q4_adapters_apply(A, x, e, base=base, y=y1, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(y1, want)
    # two graphs that share the workspace, replayed in turn on new ids
    graphs = []
    for y in (y1, y2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_q4_adapters_apply(A, x, e, base=base, y=y, workspace=ws)
        graphs.append(g)
    e.copy_(e.flip(0))
    want = m.moe_q4_adapters_apply(A, x, e, base=base)
    y1.zero_()
    y2.zero_()
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y1, want) and torch.equal(y2, want)


@pytest.mark.parametrize("T", [6, 260, 1200])
def test_rows_past_32_bit_offsets(T):
    """Pitches that put base's and y's rows more than 2^32 bytes from the first."""
    A, x, e, base = make(19, T, 512, 200, 16, 2, "bf16", "mixed")
    want = m.moe_q4_adapters_apply(A, x, e, base=base)
    ld = (6 << 30) // 4 // T // 4 * 4 + 8
    wide = torch.empty((T - 1) * ld + 200, device="cuda")   # 6 GB
    y = wide.as_strided((T, 200), (ld, 1))
    y.copy_(base)
    m.moe_q4_adapters_apply(A, x, e, base=y, y=y)
    assert torch.equal(y, want)
    xw = torch.empty((T - 1) * ld + 512, device="cuda").as_strided((T, 512), (ld, 1))
    xw.copy_(x)
    y.zero_()
    m.moe_q4_adapters_apply(A, xw, e, base=base, y=y)
    assert torch.equal(y, want)


def test_no_rows():
    A, x, e, base = make(1, 4, 256, 10, 8, 2, "bf16")
    y = m.moe_q4_adapters_apply(A, x[:0], e[:0], base=base[:0])
    assert y.shape == (0, 10)


def test_the_lm_head_shape():
    A, x, e, base = make(17, 8, 2048, 131072, 16, 8, "fp16", list(range(8)))
    check(A, x, e, base, m.moe_q4_adapters_apply(A, x, e, base=base))


@pytest.mark.parametrize("T,H,N,r,n,ids", [
    (257, 256, 300, 8, 1, "none"),         # no row has an adapter
    (300, 256, 300, 8, 255, "mixed"),      # the most adapters that a CTA finds its tile among
    (2048, 256, 300, 16, 255, "runs"),
    (2048, 256, 260, 64, 2, "mixed"),      # the most rows
    (1025, 512, 513, 24, 3, "one"),
    (640, 256, 40001, 16, 4, "runs"),      # several clusters a tile, a ragged last block
    (300, 256, 70000, 64, 2, "mixed"),
    (4000, 256, 9000, 32, 3, "runs"),
    (200, 256, 20000, 64, 1, "one"),       # tensor cores for a batch below the grouping kernels' sizes
    (250, 512, 30001, 128, 2, "runs"),
])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_tiles_found_by_their_own_ctas(kind, T, H, N, r, n, ids):
    A, x, e, base = make(T + N, T, H, N, r, n, kind, ids, pad=4)
    y = m.moe_q4_adapters_apply(A, x, e, base=base)
    check(A, x, e, base, y)
    z = base.clone()  # in place
    m.moe_q4_adapters_apply(A, x, e, base=z, y=z)
    assert torch.equal(z, y)
    check(A, x, e, None, m.moe_q4_adapters_apply(A, x, e))


@pytest.mark.parametrize("T,H,N,r,n", [
    (1, 256, 300, 8, 1), (128, 256, 4096, 128, 256), (256, 256, 4096, 128, 300), (256, 256, 20000, 64, 1),
    (257, 256, 300, 8, 300), (512, 256, 4096, 64, 64), (2048, 256, 300, 16, 256), (2049, 256, 300, 16, 1), (20000, 256, 260, 16, 5),
])
def test_nothing_past_the_workspace_is_written(T, H, N, r, n):
    A, x, e, base = make(T + n, T, H, N, r, n, "bf16")
    need = m.moe_q4_adapters_workspace_bytes(A, T)
    room = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    y = m.moe_q4_adapters_apply(A, x, e, base=base, workspace=room[:need])
    assert bool((room[need:] == 0x5A).all())
    check(A, x, e, base, y)
