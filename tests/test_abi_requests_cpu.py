"""Host-side refusals of the per-request entry points (low-rank adapters and
logit rules), no GPU needed: every bad argument is turned away with its code
before any CUDA call."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


@pytest.fixture(scope="module")
def lib():
    import importlib.util
    spec = importlib.util.spec_from_file_location(
        "moe_q4_cuda_build", os.path.join(ROOT, "quantized_moe_q4_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    lib = ctypes.CDLL(build.build())
    lib.moe_q4_adapters_workspace_bytes.argtypes = [P, i64]
    lib.moe_q4_adapters_workspace_bytes.restype = sz
    lib.moe_q4_adapters_apply.argtypes = [P, P, i64, P, i64, P, i64, P, i64, P, sz, P]
    lib.moe_q4_logits_apply.argtypes = [P, P, i64, i64, P, i64, P, P, P, P]
    return lib


class _A(ctypes.Structure):
    _fields_ = [("hidden", i32), ("rank", i32), ("n_out", i64), ("n_adapters", i32), ("dtype", i32),
                ("a", P), ("b", P), ("scale", P)]


class _R(ctypes.Structure):
    _fields_ = [("vocab", i64), ("tokens", P), ("n_tokens", i64), ("row_start", P), ("generated_start", P),
                ("repetition", P), ("presence", P), ("frequency", P), ("bias_token", P), ("bias_value", P),
                ("n_bias", i64), ("bias_start", P), ("mask", P), ("n_masks", i64), ("mask_row", P)]


FAKE = 0x7F0000000000  # a 256-byte aligned address that is never dereferenced
G = 1 << 30


def adapters(**kw):
    d = dict(hidden=512, rank=16, n_out=1000, n_adapters=4, dtype=2, a=FAKE, b=FAKE + G, scale=FAKE + 2 * G)
    d.update(kw)
    return _A(**d)


def apply(lib, A, x=FAKE + 3 * G, ldx=512, ids=FAKE + 4 * G, T=10, base=FAKE + 5 * G, ldb=1000, y=FAKE + 6 * G, ldy=1000,
          ws=FAKE + 7 * G, nbytes=1 << 20):
    return lib.moe_q4_adapters_apply(None if A is None else ctypes.byref(A), x, ldx, ids, T, base, ldb, y, ldy, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), -1), (dict(b=None), -1), (dict(n_out=0), -1), (dict(n_out=(1 << 30) + 1), -1),
    (dict(n_adapters=0), -1), (dict(n_adapters=1025), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1),
    (dict(hidden=0), -2), (dict(hidden=500), -2), (dict(hidden=16640), -2), (dict(rank=0), -2), (dict(rank=12), -2),
    (dict(rank=136), -2), (dict(rank=-8), -2), (dict(a=FAKE + 8), -3), (dict(b=FAKE + G + 2), -3),
    (dict(scale=FAKE + 2), -3)])
def test_adapters_refuse_bad_descriptors(lib, kw, code):
    A = adapters(**kw)
    assert apply(lib, A) == code
    assert lib.moe_q4_adapters_workspace_bytes(ctypes.byref(A), 10) == 0


X, IDS, BASE, Y, WS = (FAKE + k * G for k in (3, 4, 5, 6, 7))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(T=(1 << 24) + 1), -1), (dict(x=None), -1), (dict(ids=None), -1), (dict(y=None), -1),
    (dict(ws=None), -1), (dict(ldx=508), -1), (dict(ldy=999), -1), (dict(ldb=999), -1), (dict(ldx=1 << 33), -1),
    (dict(ldy=1 << 33), -1), (dict(ldb=-1000), -1), (dict(x=X + 4), -3), (dict(ldx=514), -3), (dict(ids=IDS + 2), -3),
    (dict(base=BASE + 2), -3), (dict(y=Y + 1), -3), (dict(ws=WS + 16), -3), (dict(nbytes=255), -4),
    (dict(y=X), -7), (dict(y=X + 4 * 512 * 9), -7),              # y over x's rows
    (dict(y=IDS - 4 * 1000), -7), (dict(y=WS), -7), (dict(y=FAKE + 16), -7), (dict(y=FAKE + G), -7),
    (dict(y=FAKE + 2 * G), -7),                                  # y over the ids, workspace, a, b, scale
    (dict(y=BASE + 4), -7), (dict(y=BASE, ldy=1001), -7), (dict(y=BASE + 4000), -7),   # y over base, not in place
    (dict(y=BASE, ldy=4000, ldb=4000 - 1), -7),
    (dict(x=X, ldx=1512, y=X + 4 * 511, ldy=1512), -7),          # one buffer, columns that share one
    (dict(x=X, ldx=1508, y=X + 4 * 512, ldy=1508), -7)])         # ... that wrap into the next row's x
def test_adapters_refuse_bad_calls(lib, kw, code):
    assert apply(lib, adapters(), **kw) == code


def test_adapters_calls_that_pass_the_checks(lib):
    """With the device overridden to another one, ARCH is what comes after all
    argument checks; T == 0 is a no-op before."""
    assert apply(lib, None) == -1
    assert apply(lib, adapters(), T=0, x=None, ids=None, y=None, ws=None) == 0
    lib.moe_q4_test_override_device(1, 9, 0)
    try:
        for kw in (dict(), dict(base=None, ldb=0), dict(base=Y), dict(x=X, ldx=1512, y=X + 4 * 512, ldy=1512),
                   dict(x=X + 4 * 1000, ldx=1512, y=X, ldy=1512), dict(ldy=1001, ldb=1003),
                   dict(base=BASE, ldb=2000, y=BASE + 4 * 1000, ldy=2000), dict(T=1, ldx=512, ldy=1000)):
            assert apply(lib, adapters(), **kw) == -5, kw
        assert apply(lib, adapters(scale=None)) == -5
    finally:
        lib.moe_q4_test_override_device(0, 0, 0)


def test_adapters_workspace_grows_with_the_rows(lib):
    A = adapters()
    got = [lib.moe_q4_adapters_workspace_bytes(ctypes.byref(A), T) for T in (0, 1, 256, 257, 1000, 16384, 16385, 1 << 24)]
    assert got[0] == got[1] == got[2] == 256 and all(b >= a for a, b in zip(got, got[1:])) and got[3] > 257 * 4
    assert lib.moe_q4_adapters_workspace_bytes(ctypes.byref(A), -1) == 0
    assert lib.moe_q4_adapters_workspace_bytes(ctypes.byref(A), (1 << 24) + 1) == 0
    assert apply(lib, A, T=257, nbytes=got[3] - 1) == -4


L, OUT, TOK, LSE, ST = (FAKE + k * G for k in (0, 1, 2, 3, 4))
H = FAKE + 8 * G


def rules(**kw):
    d = dict(vocab=1000, tokens=H, n_tokens=50, row_start=H + G, generated_start=H + 2 * G, repetition=H + 3 * G,
             presence=H + 4 * G, frequency=H + 5 * G, bias_token=H + 6 * G, bias_value=H + 7 * G, n_bias=9,
             bias_start=H + 8 * G, mask=H + 9 * G, n_masks=3, mask_row=H + 10 * G)
    d.update(kw)
    return _R(**d)


def logits(lib, R, l=L, ld=1000, T=4, out=OUT, ldo=1000, token=TOK, lse=LSE, status=ST):
    return lib.moe_q4_logits_apply(None if R is None else ctypes.byref(R), l, ld, T, out, ldo, token, lse, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(vocab=0), -1), (dict(vocab=(1 << 30) + 1), -1), (dict(n_tokens=-1), -1), (dict(tokens=None), -1),
    (dict(n_bias=-1), -1), (dict(bias_token=None), -1), (dict(bias_value=None), -1), (dict(n_masks=0), -1),
    (dict(mask_row=None), -1), (dict(tokens=H + 4), -3), (dict(row_start=H + G + 4), -3),
    (dict(generated_start=H + 2 * G + 4), -3), (dict(repetition=H + 3 * G + 1), -3), (dict(presence=H + 4 * G + 2), -3),
    (dict(frequency=H + 5 * G + 2), -3), (dict(bias_token=H + 6 * G + 2), -3), (dict(bias_value=H + 7 * G + 2), -3),
    (dict(bias_start=H + 8 * G + 4), -3), (dict(mask=H + 9 * G + 2), -3), (dict(mask_row=H + 10 * G + 2), -3),
    (dict(tokens=OUT + 16), -7), (dict(row_start=OUT), -7), (dict(generated_start=TOK - 24), -7), (dict(repetition=LSE), -7),
    (dict(presence=TOK), -7), (dict(frequency=OUT + 400), -7), (dict(bias_token=LSE - 32), -7), (dict(bias_value=ST), -7),
    (dict(bias_start=OUT), -7), (dict(mask=OUT + 15600), -7), (dict(mask_row=TOK + 12), -7)])
def test_logits_refuse_bad_rules(lib, kw, code):
    assert logits(lib, rules(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(T=(1 << 24) + 1), -1), (dict(l=None), -1), (dict(out=None, token=None, lse=None), -1),
    (dict(ld=999), -1), (dict(ldo=999), -1), (dict(ld=1 << 33), -1), (dict(ldo=1 << 33), -1), (dict(l=L + 2), -3),
    (dict(out=OUT + 1), -3), (dict(token=TOK + 2), -3), (dict(lse=LSE + 3), -3), (dict(status=ST + 1), -3),
    (dict(out=L + 4), -7), (dict(out=L, ldo=1001), -7), (dict(out=L + 4000), -7), (dict(token=L + 400), -7),
    (dict(lse=OUT + 8), -7), (dict(token=LSE - 12), -7), (dict(status=TOK), -7)])
def test_logits_refuse_bad_calls(lib, kw, code):
    assert logits(lib, rules(), **kw) == code


def test_logits_calls_that_pass_the_checks(lib):
    assert logits(lib, None) == -1
    assert logits(lib, rules(), T=0, l=None, out=None, token=None, lse=None) == 0
    lib.moe_q4_test_override_device(1, 10, 3)
    try:
        for kw in (dict(), dict(out=L), dict(out=None), dict(token=None, lse=None), dict(status=None),
                   dict(ld=2000, out=L + 4000, ldo=2000)):
            assert logits(lib, rules(), **kw) == -5, kw
        empty = {n: None for n in ("tokens", "row_start", "generated_start", "repetition", "presence", "frequency",
                                   "bias_token", "bias_value", "bias_start", "mask", "mask_row")}
        assert logits(lib, rules(**empty, n_tokens=0, n_bias=0, n_masks=0)) == -5
        assert logits(lib, rules(mask_row=None, n_masks=4)) == -5
        assert logits(lib, rules(tokens=None, n_tokens=0)) == -5
    finally:
        lib.moe_q4_test_override_device(0, 0, 0)


def test_binding_refuses_host_tensors():
    import torch
    import quantized_moe_q4_b200 as m
    with pytest.raises(ValueError):
        m.Adapters(torch.zeros(1, 8, 256), torch.zeros(1, 5, 8))
    with pytest.raises(ValueError):
        m.Adapters(torch.zeros(1, 8, 256), torch.zeros(2, 5, 8))
    with pytest.raises(ValueError):
        m.Adapters(torch.zeros(1, 8, 256), torch.zeros(1, 5, 8).half())
    with pytest.raises(ValueError):
        m.LogitRules(tokens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        m.LogitRules(bias_token=torch.zeros(3, dtype=torch.int32), bias_value=torch.zeros(3))
    with pytest.raises(ValueError):
        m.moe_q4_logits_apply(m.LogitRules(), torch.zeros(2, 10))
