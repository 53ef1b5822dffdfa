"""How precise the adapters' products are as a whole, and that a row's bits are
its own.

A bound for every element has to allow for roundings that all go the same way;
at large ranks and hidden sizes it is so wide that one dropped part of a split
value would pass.  Against the norm of the correction such a part is plain: a
value kept to the 11 bits of one tf32 is off by up to 2^-11 of itself, 2e-4 in
the mean square, and independent errors of the terms leave that ratio as it is
in their sums.

What the kernels may lose, in units of u = 2^-24 of the norm, each at its
largest: two-part values x, u and binary32 A and B 8 each (2^-21) and 4 for
either product of lo parts that is left out; truncated additions 2 each, at
most 40 in a row in step 1 (10 panels of 4), 24 in step 3 (8 steps of 8 with up
to 3 products on one of two accumulators); joins of 17 accumulators and 8 parts
1 each; scale and the accumulators of step 3 1 each:
    8 + 8 + 8 + 8 + 4 + 4 + 80 + 48 + 25 + 2 = 195  ->  195 u = 1.2e-5.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_moe_q4_b200 as m  # noqa: E402

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def make(T, H, N, r, n, kind, ids):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H + N + r)
    kw = dict(device="cuda", generator=g)
    x = torch.randn(T, H, **kw)
    A = m.Adapters((torch.randn(n, r, H, **kw) / H ** 0.5).to(TYPES[kind]), (torch.randn(n, N, r, **kw) * 0.1).to(TYPES[kind]),
                   torch.rand(n, **kw) * 2 + 0.5)
    e = torch.randint(0, n, (T,), **kw) if ids == "mixed" else torch.arange(T, device="cuda") * (n + 1) // T - 1
    return A, x, e.int()


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,H,N,r,n,ids", [
    (8, 2048, 2048, 16, 8, "mixed"), (64, 2048, 2048, 64, 5, "mixed"),
    # clusters of 8 CTAs: prompts, several clusters a tile, ten panels an accumulator
    (947, 2048, 2048, 64, 4, "runs"), (1100, 768, 1001, 128, 2, "mixed"), (1500, 512, 1500, 8, 2, "mixed"),
    (250, 512, 30001, 128, 2, "runs"), (700, 16384, 100, 64, 2, "mixed"), (1400, 7680, 300, 128, 2, "runs"),
    # of 4 and of 2
    (3000, 1024, 129, 128, 2, "runs"), (7000, 512, 130, 64, 3, "runs"), (9000, 2048, 520, 64, 3, "mixed"),
    (16384, 1024, 520, 128, 4, "mixed"),
    # one CTA: 64 panels on 7 accumulators in turn (up to 10 each), 40 on 4, 24 on 3, 8 on 2
    (16384, 2048, 300, 64, 8, "runs"), (16384, 2048, 2048, 64, 8, "runs"), (16384, 1280, 300, 96, 2, "mixed"),
    (20000, 768, 300, 128, 2, "runs"), (18000, 256, 64, 120, 1, "mixed"),
])
def test_norm_of_the_error(kind, T, H, N, r, n, ids):
    A, x, e = make(T, H, N, r, n, kind, ids)
    y = m.moe_q4_adapters_apply(A, x, e)
    for i in range(n):
        at = torch.nonzero(e == i)[:, 0]
        if at.numel() == 0:
            continue
        s = float(A.scale[i])
        want = s * ((x[at].double() @ A.a[i].double().t()) @ A.b[i].double().t())
        off = float((y[at].double() - want).norm() / want.norm())
        assert off <= 195 * U, (i, off)
        # and no row is far worse than the whole
        rows = (y[at].double() - want).norm(dim=1)
        S = abs(s) * ((x[at].double().abs() @ A.a[i].double().abs().t()) @ A.b[i].double().abs().t())
        assert bool((rows <= (H / 16 + 2 * r + 64) * U * S.norm(dim=1)).all())


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("T,H,N,r", [(40, 512, 300, 16), (256, 2048, 257, 64), (280, 768, 100, 8), (1200, 512, 400, 40),
                                     (3000, 512, 200, 24), (20000, 256, 100, 16)])
def test_a_rows_bits_do_not_depend_on_how_many_share_its_adapter(kind, T, H, N, r):
    """Rows of a tile are computed one, two, four or eight at a time."""
    n, row = 9, T // 2
    A, x, _ = make(T, H, N, r, n, kind, "mixed")
    others = torch.tensor([t for t in range(T) if t != row], device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    want = None
    for share in (0, 1, 2, 3, 4, 6, 7, 8, 15, T - 1):
        e = torch.randint(-1, n - 1, (T,), device="cuda", generator=g).int()   # (nobody else has the last one)
        mates = others[torch.randperm(T - 1, device="cuda", generator=g)[:share]]
        e[mates] = n - 1
        e[row] = n - 1
        y = m.moe_q4_adapters_apply(A, x, e)
        if want is None:
            want = y[row].clone()
            ref = float(A.scale[n - 1]) * ((x[row].double() @ A.a[n - 1].double().t()) @ A.b[n - 1].double().t())
            assert float((want.double() - ref).norm() / ref.norm()) <= 195 * U
        assert torch.equal(y[row], want), share
