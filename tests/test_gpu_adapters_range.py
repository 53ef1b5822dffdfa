"""Low-rank adapters at the top of binary32's range: finite values that a tf32
rounding would carry to infinity.

Products are in range (each large value meets a small one), so the result is
the formula's within the bound of roundings that either kernel makes: C u S
with u = 2^-24, C = H / 16 + 2 r + 64 and S the sum of the products'
magnitudes (H / 8 accumulations and 28 u of split values in the tensor-core
kernel, H / 32 in the other; r products and the joins after them).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_moe_q4_b200 as m  # noqa: E402

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
TOP = torch.finfo(torch.float32).max


def check(x, a, b, ids):
    T, H, N, r = x.shape[0], x.shape[1], b.shape[1], a.shape[1]
    y = m.moe_q4_adapters_apply(m.Adapters(a, b), x, ids)
    ref, S = torch.zeros(T, N, dtype=torch.float64, device="cuda"), torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for e in range(a.shape[0]):
        at = torch.nonzero(ids == e)[:, 0]
        ref[at] = (x[at].double() @ a[e].double().t()) @ b[e].double().t()
        S[at] = (x[at].double().abs() @ a[e].double().abs().t()) @ b[e].double().abs().t()
    assert bool((S < TOP).all())
    bad = ~((y.double() - ref).abs() <= (H / 16 + 2 * r + 64) * 2.0 ** -24 * S)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}: " \
                          f"{float(y[bad][0])} for {float(ref[bad][0])}"


def inputs(T, kind, H=512, N=300, r=16, n=2):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    kw = dict(device="cuda", generator=g)
    x = torch.randn(T, H, **kw)
    a = (torch.randn(n, r, H, **kw) / H ** 0.5).to(TYPES[kind])
    b = (torch.randn(n, N, r, **kw) * 0.1).to(TYPES[kind])
    return x, a, b, torch.randint(-1, n, (T,), **kw).int()


# (1 and 200 rows: FMAs; 1500 and 20000: tensor cores)
@pytest.mark.parametrize("T", [1, 200, 1500, 20000])
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
def test_activations_at_the_top(kind, T):
    x, a, b, ids = inputs(T, kind)
    ids[0] = 0
    small = 2.0 ** -24 if kind == "fp16" else 2.0 ** -120
    a[:, :, 7] = small
    a[:, ::2, 7] = -small
    x[::3, 7] = TOP
    x[1::3, 7] = -TOP
    x[2::3, 7] = 3.4025e38   # rounds to the type's next power of two as well
    check(x, a, b, ids)


@pytest.mark.parametrize("T", [1, 200, 1500, 20000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_middle_vector_at_the_top(kind, T):
    x, a, b, ids = inputs(T, kind)
    ids[0] = 0
    a[:, 3, :] = 0           # row 3 of A x is one element of x
    a[:, 3, 7] = 1
    a[:, :3, 7] = 0
    a[:, 4:, 7] = 0
    x[::2, 7] = TOP
    x[1::2, 7] = -TOP
    b[:, :, 3] = 2.0 ** -120
    check(x, a, b, ids)


@pytest.mark.parametrize("T", [1, 200, 1500, 20000])
def test_binary32_weights_at_the_top(T):
    x, a, b, ids = inputs(T, "fp32")
    ids[0] = 0
    a[:, :, 7] = TOP
    a[:, ::2, 7] = -TOP
    x[:, 7] = 2.0 ** -100
    check(x, a, b, ids)
    x, a, b, ids = inputs(T, "fp32")
    b[:, ::5, 3] = -TOP
    a[:, 3, :] *= 2.0 ** -100
    check(x, a, b, ids)
